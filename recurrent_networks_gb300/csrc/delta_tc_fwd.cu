// Gated delta rule, bf16 storage, forward (delta_tc.cuh has the formulas).
//   prep   every chunk by itself: TP and the per-step factors
//   chain  per head and tile of BV columns of v, the chunks one after the other:
//          o and the state, and what a backward needs
#include "delta.h"
#include "delta_tc.cuh"

namespace rnn {
namespace {

// ---- prep --------------------------------------------------------------------------
constexpr int PREP_LD = TC_C + 4;
// K and Q, then L (and PT in its place) and P; beside them Tm and the steps' factors
__host__ __device__ constexpr size_t prep_kq(int KP) {
  const size_t kq = (size_t)2 * TC_C * (KP + 8) * 2, lp = (size_t)2 * TC_C * PREP_LD * 4;
  return kq > lp ? kq : lp;
}
__host__ __device__ constexpr size_t prep_smem(int KP) { return prep_kq(KP) + (size_t)TC_C * PREP_LD * 4 + REC_N * TC_C * 4; }

// start + the dot product of N (a multiple of 4) values in shared memory and in
// registers, by packed pairs
template <int N> __device__ __forceinline__ float dot_pairs(const float* p, const float* x, float start) {
  FV<2> s[2] = {{{start, 0.0f}}, {{0.0f, 0.0f}}};
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const float4 l = *(const float4*)(p + k);
    s[0] = fma(FV<2>{{l.x, l.y}}, FV<2>{{x[k], x[k + 1]}}, s[0]);
    s[1] = fma(FV<2>{{l.z, l.w}}, FV<2>{{x[k + 2], x[k + 3]}}, s[1]);
  }
  return (s[0].v[0] + s[1].v[0]) + (s[0].v[1] + s[1].v[1]);
}

// K K^T and Q K^T by mma.sync, 16 rows a warp and the columns up to its last row;
// the rest in fp32 on the plain cores. Tm: its two diagonal blocks of 32 by forward
// substitution, a column to a thread, then T21 = -T22 (L21 T11); PT a column and
// every other row to a thread. Bound by instructions, about 3500 a warp (issue slots
// 42 % busy, barriers between the parts); four CTAs an SM (Dk <= 128). 133 us for
// the 4096 chunks of the chain's size below.
__global__ void __launch_bounds__(128, 4) delta_tc_prep_kernel(DeltaTcArgs a) {
  constexpr int C = TC_C, NT = C / 8, LD = PREP_LD, H = C / 2;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  const int LDK = a.KP + 8, kplane = C * LDK;
  bf16* Ks = (bf16*)sm_raw;
  bf16* Qs = Ks + kplane;
  float* Lf = (float*)sm_raw;  // [C][LD]; L21's place takes L21 T11, then all of it PT
  float* Pf = Lf + C * LD;     // [C][LD]
  float* Tf = (float*)(sm_raw + prep_kq(a.KP));  // [C][LD]
  float* rec = Tf + C * LD;                      // [REC_N][C]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long item = blockIdx.x;
  if (item == 0 && tid == 0) *a.status = 0;  // the kernels behind this one report there
  const int ch = (int)(item % a.nc), bn = (int)(item / a.nc), n = bn % a.N, b = bn / a.N;
  const int live = tc_live(a, b, ch);
  if (live == 0) return;
  const size_t stride = (size_t)a.Nk * a.Dk;
  const size_t at = ((size_t)b * a.T + (size_t)ch * C) * stride + (size_t)(n / (a.N / a.Nk)) * a.Dk;
  load_rows<bf16, C>(Ks, LDK, kplane, (const bf16*)a.k + at, stride, live, a.Dk, 0, a.KP);
  load_rows<bf16, C>(Qs, LDK, kplane, (const bf16*)a.q + at, stride, live, a.Dk, 0, a.KP);
  cp_commit();
  if (warp == 0) {  // the running sum of g (to the base 2), in 64 bits, and the documents
    double run = 0.0, cs[2];
    int seg = 0, sg[2];
    bool near[2];
    float be[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = h * 32 + lane;
      float g = 0.0f;
      bool mark = false;
      be[h] = 0.0f;
      if (i < live) {
        const size_t row = (size_t)b * a.T + (size_t)ch * C + i;
        g = a.g[row * a.N + n];
        be[h] = a.beta[row * a.N + n];
        if (a.Sh && fabsf(be[h]) < BETA_MIN) be[h] = copysignf(BETA_MIN, be[h]);  // a backward comes
        mark = a.reset && a.reset[row];
        if (g < -104.0f) mark = true;  // exp(g) is 0
        if (mark) g = 0.0f;
      }
      near[h] = g < GATE_NEAR;
      double c = (double)g * 1.4426950408889634;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += v;
      }
      c += run;
      run = __shfl_sync(0xffffffffu, c, 31);
      const unsigned m = __ballot_sync(0xffffffffu, mark);
      sg[h] = seg + __popc(m & (0xffffffffu >> (31 - lane)));
      seg += __popc(m);
      cs[h] = c;
      const float chi = (float)c;
      rec[REC_CHI * C + i] = chi;
      rec[REC_CLO * C + i] = (float)(c - (double)chi);
      rec[REC_SEG * C + i] = __int_as_float(sg[h]);
      rec[REC_GAM * C + i] = sg[h] == 0 ? keep_part(exp2f((float)c)) : 0.0f;
      rec[REC_BETA * C + i] = be[h];
    }
    const bool some = __any_sync(0xffffffffu, near[0] || near[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = h * 32 + lane;
      rec[REC_BR * C + i] = sg[h] == seg ? keep_part(be[h] * exp2f((float)(run - cs[h]))) : 0.0f;
      rec[REC_NEAR * C + i] = near[h] ? 2.0f : some ? 1.0f : 0.0f;
    }
  }
  cp_wait<0>();
  __syncthreads();
  for (int i = tid; i < REC_N * C; i += 128) a.rec[(size_t)item * REC_N * C + i] = rec[i];
  const int m0 = warp * 16;
  float kk[NT][4], qk[NT][4];
  zero(kk);
  zero(qk);
  {
    const int id = lane >> 3, r = lane & 7;
    uint32_t ka = smem_u32(Ks) + 2u * ((m0 + (id & 1) * 8 + r) * LDK + (id >> 1) * 8), qa = ka + 2u * kplane;
    uint32_t kb = smem_u32(Ks) + 2u * (((id >> 1) * 8 + r) * LDK + (id & 1) * 8);
#pragma unroll 2
    for (int k = 0; k < a.KP; k += 16, ka += 32, qa += 32, kb += 32) {
      uint32_t x[4], y[4];
      ldsm4<false>(ka, x);
      ldsm4<false>(qa, y);
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        if (j > warp) continue;
        uint32_t w[4];
        ldsm4<false>(kb + j * 32 * LDK, w);
        mma_bf16_16816(kk[2 * j], x, w[0], w[1]);
        mma_bf16_16816(kk[2 * j + 1], x, w[2], w[3]);
        mma_bf16_16816(qk[2 * j], y, w[0], w[1]);
        mma_bf16_16816(qk[2 * j + 1], y, w[2], w[3]);
      }
    }
  }
  __syncthreads();  // K and Q are read
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = m0 + (lane >> 2) + 8 * h;
    const float ci = rec[REC_CHI * C + i], li = rec[REC_CLO * C + i];
    const int si = __float_as_int(rec[REC_SEG * C + i]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t > 2 * warp + 1) continue;
      float p[2], l[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = t * 8 + (lane & 3) * 2 + e;
        const bool on = i >= j && si == __float_as_int(rec[REC_SEG * C + j]);
        const float gb = exp2_fast((ci - rec[REC_CHI * C + j]) + (li - rec[REC_CLO * C + j])) * rec[REC_BETA * C + j];
        p[e] = on ? a.scale * qk[t][2 * h + e] * gb : 0.0f;
        l[e] = on && i > j ? -kk[t][2 * h + e] * gb : 0.0f;
      }
      *(float2*)(Pf + i * LD + t * 8 + (lane & 3) * 2) = make_float2(p[0], p[1]);
      *(float2*)(Lf + i * LD + t * 8 + (lane & 3) * 2) = make_float2(l[0], l[1]);  // -L
    }
  }
  __syncthreads();
  if (warp < 2) {  // T11 and T22
    const int o = warp * H;
    float x[H];
#pragma unroll
    for (int i = 0; i < H; ++i) x[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float* l = Lf + (o + i) * LD + o;  // zero from column o + i on, as x is
      float s = i == lane ? 1.0f : 0.0f;
      FV<2> s0 = {{s, 0.0f}}, s1 = {{0.0f, 0.0f}};
#pragma unroll
      for (int k = 0; k < i; k += 4) {
        const float4 v = *(const float4*)(l + k);
        s0 = fma(FV<2>{{v.x, v.y}}, FV<2>{{x[k], x[k + 1]}}, s0);
        s1 = fma(FV<2>{{v.z, v.w}}, FV<2>{{x[k + 2], x[k + 3]}}, s1);
      }
      x[i] = (s0.v[0] + s1.v[0]) + (s0.v[1] + s1.v[1]);
    }
#pragma unroll
    for (int i = 0; i < H; ++i) Tf[(o + i) * LD + o + lane] = x[i];
  } else {  // T12 = 0
    for (int i = warp - 2; i < H; i += 2) Tf[i * LD + H + lane] = 0.0f;
  }
  __syncthreads();
  // two products of 32 x 32: 8 rows of column `lane` a thread
  auto small = [&](const float* A, const float* B, float (&s)[8]) {
    float col[H];
#pragma unroll
    for (int k = 0; k < H; ++k) col[k] = B[k * LD + lane];
#pragma unroll
    for (int r = 0; r < 8; ++r) s[r] = dot_pairs<H>(A + (warp * 8 + r) * LD, col, 0.0f);
  };
  float s8[8];
  small(Lf + H * LD, Tf, s8);  // -L21 T11
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 8; ++r) Lf[(H + warp * 8 + r) * LD + lane] = s8[r];
  __syncthreads();
  small(Tf + H * LD + H, Lf + H * LD, s8);
#pragma unroll
  for (int r = 0; r < 8; ++r) Tf[(H + warp * 8 + r) * LD + lane] = s8[r];
  __syncthreads();
  {  // PT = P Tm, in L's place; P's columns up to the next multiple of 4 are written (16 rows by 16 columns at once)
    const int j = tid & (C - 1), odd = tid >> 6;
    float x[C];
#pragma unroll
    for (int k = 0; k < C; ++k) x[k] = Tf[k * LD + j];
#pragma unroll
    for (int i = 0; i < C; i += 4) {
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const float* p = Pf + (i + r + odd) * LD;
        FV<2> s0 = {{0.0f, 0.0f}}, s1 = {{0.0f, 0.0f}};
#pragma unroll
        for (int k = 0; k < i + 4; k += 4) {
          const float4 v = *(const float4*)(p + k);
          s0 = fma(FV<2>{{v.x, v.y}}, FV<2>{{x[k], x[k + 1]}}, s0);
          s1 = fma(FV<2>{{v.z, v.w}}, FV<2>{{x[k + 2], x[k + 3]}}, s1);
        }
        Lf[(i + r + odd) * LD + j] = (s0.v[0] + s1.v[0]) + (s0.v[1] + s1.v[1]);
      }
    }
  }
  __syncthreads();
  unsigned char* tp = (unsigned char*)(a.tp + (size_t)item * 3 * 128 * C);
#pragma unroll 2
  for (int i = tid; i < 128 * 8; i += 128) {
    const int r = i >> 3, c = i & 7;
    const float* from = (r < C ? Tf + r * LD : Lf + (r - C) * LD) + c * 8;
    float x[8];
    *(float4*)x = *(const float4*)from;
    *(float4*)(x + 4) = *(const float4*)(from + 4);
    uint4 p[3];
    split8(x, p);
#pragma unroll
    for (int k = 0; k < 3; ++k) *(uint4*)(tp + k * TC_PANEL + img<128>(r, c)) = p[k];
  }
}

// ---- chain --------------------------------------------------------------------------
template <int BV, int MT> struct TcChain {
  static constexpr int RB = 2 * BV, KST = MT == 1 ? 2 : 1;  // bytes of a tile's row; stages of KQ
  static constexpr int KQ = 2 * MT * TC_PANEL, TP = 3 * TC_PANEL, SPLANE = MT * 128 * RB, YPLANE = 64 * RB;
  static constexpr int AT_TP = KST * KQ, AT_S = AT_TP + TP, AT_Y = AT_S + 3 * SPLANE, AT_V = AT_Y + 3 * YPLANE;
  static constexpr int AT_O = AT_V + YPLANE;  // o, on its way out
  static constexpr int AT_REC = AT_O + YPLANE, BYTES = AT_REC + 2 * 2 * 64 * 4 + 64 + 1024;
};

// Warps 0 .. 7 take values through registers: warp w has lanes 32 (w % 4) .. of
// the accumulators (rows 0 .. 63: K's steps, 64 .. 127: Q's; or rows of the state)
// and half of the tile's columns. Thread 256 issues the products and the bulk
// copies of images (an issuing thread waits while earlier products run: 150
// cycles a product) and of the tensors' rows; rows that are not whole 16-byte
// pieces are loaded and stored by warps 10 and 11. The third warpgroup gives
// registers to the other two: 256 * 200 + 128 * 104 = 384 * 168.
// MT: tiles of 128 state rows, whose fp32 values stay in registers. A chunk is
// three dependent products (2000 cycles for BV = 64, Dk = 128) and their ways
// through registers between barriers of the whole CTA, 4.7 us in all: 299 us for
// the 64 chunks of B = 8, T = 4096, N = 8, Dk = Dv = 128, where 557 MB pass in a
// training step (82 us). Tiles of 32 columns would double the CTAs and shorten a
// chunk to two thirds: 1.3 times the time where all SMs are taken.
template <int BV, int MT>
__global__ void __launch_bounds__(384, 1) delta_tc_chain_kernel(DeltaTcArgs a, const __grid_constant__ TcMaps maps) {
  using L = TcChain<BV, MT>;
  constexpr int RB = L::RB, NC = BV / 2, KST = L::KST, P = MT * 16;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)sm_raw + 1023) & ~(uintptr_t)1023);
  unsigned char *TP = sm + L::AT_TP, *SS = sm + L::AT_S, *YS = sm + L::AT_Y, *VS = sm + L::AT_V, *OS = sm + L::AT_O;
  float* recs = (float*)(sm + L::AT_REC);  // [2][gam, br][64]
  uint64_t* barp = (uint64_t*)(recs + 2 * 2 * 64);
  uint32_t* slot = (uint32_t*)(barp + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
  constexpr int KR = MT * 128;
  const int tiles = a.maps ? a.nvt + (a.KP + BV - 1) / BV : a.nvt;  // maps: and those of the identity
  const int vt = blockIdx.x % tiles, seg = blockIdx.x / tiles % a.segs, bn = blockIdx.x / tiles / a.segs;
  const int n = bn % a.N, b = bn / a.N, nk = n / (a.N / a.Nk);
  const bool ident = vt >= a.nvt;
  if (a.maps && seg == a.segs - 1 && !(ident && a.Sh)) return;  // nothing follows it; a backward wants its M
  const int nch = tc_chunks(a, b), ch0 = min(nch, seg * a.seglen), ch1 = min(nch, ch0 + a.seglen);
  const size_t vstride = (size_t)a.N * a.Dv, vat = (size_t)b * a.T * vstride + (size_t)n * a.Dv;
  const uint32_t bar = smem_u32(barp), bar_end = bar + 8, bar_tp = bar + 16, bar_in = bar + 24;
  if (tid == 0) {
    for (int k = 0; k < 4; ++k) mbar_init(bar + 8 * k, 1);
    fence_mbar_init_cluster();
  }
  if (warp == 0) tm_alloc<512>(slot);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *slot;
  // accumulators, three blocks of BV columns each: D1 (K S0, Q S0) and D3 (the state's change, by tile), D2 (Z, PT Y)
  constexpr int D1 = 0, D2 = 3 * BV * MT, D3 = 0;
  bool failed = false;
  auto wait = [&](uint32_t which, uint32_t par) { mbar_wait_bounded<false>(which, par, a.wait_limit_ns, a.status, failed); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8) {  // ---- products, bulk copies
      const unsigned char* tp = (const unsigned char*)a.tp + (size_t)bn * a.nc * L::TP;
      const bool one = lane == 0;
      // K, Q, V and the steps' factors of a chunk, counted by bar_in
      const int panels = (a.KP + 63) >> 6;
      const uint32_t bytes = panels * 16384 + (ident ? 0 : L::YPLANE) + 512;
      auto load_kq = [&](int ch) {
        unsigned char* d = sm + (ch % KST) * L::KQ;
        if (KST == 2) mbar_arrive_expect_tx(bar_in, bytes);
        for (int p = 0; p < panels; ++p) {
          tma_load_5d(smem_u32(d + p * TC_PANEL), &maps.k, bar_in, p * 64, nk, ch * TC_C, b, 0);
          tma_load_5d(smem_u32(d + p * TC_PANEL + 8192), &maps.q, bar_in, p * 64, nk, ch * TC_C, b, 0);
        }
      };
      auto load_v = [&](int ch) {
        if (KST == 1) mbar_arrive_expect_tx(bar_in, bytes);
        if (!ident) tma_load_5d(smem_u32(VS), &maps.v, bar_in, vt * BV, n, ch * TC_C, b, 0);
        const float* r = a.rec + ((size_t)bn * a.nc + ch) * REC_N * TC_C;
        const uint32_t d = smem_u32(recs + (ch & 1) * 2 * TC_C);
        bulk_load_global(d, r + REC_GAM * TC_C, 256, bar_in);
        bulk_load_global(d + 256, r + REC_BR * TC_C, 256, bar_in);
      };
      if (one && ch0 < ch1) {
        load_bulk(TP, tp + (size_t)ch0 * L::TP, L::TP, bar_tp);
        if (a.tma) {
          if (KST == 2) load_kq(ch0);
          load_v(ch0);
          if (KST == 1) load_kq(ch0);
        }
      }
      const uint64_t td = tc_desc(smem_u32(TP), 16), yd = tc_desc<RB>(smem_u32(YS), L::YPLANE);
      for (int ch = ch0; ch < ch1; ++ch) {
        unsigned char* kqs = sm + (ch % KST) * L::KQ;
        const uint32_t kq = smem_u32(kqs);
        const size_t tile = ((size_t)bn * a.nc + ch) * a.nvt + vt;
        if (a.tma) {
          wait(bar_in, (ch - ch0) & 1);
          const int live = tc_live(a, b, ch);
          if (live < TC_C && ch * TC_C + live < a.T) {  // steps of the tensor past the row's length
            for (int p = 0; p < panels; ++p) {
              clear_rows<128>(kqs + p * TC_PANEL, 0, live);
              clear_rows<128>(kqs + p * TC_PANEL, 64, live);
            }
            clear_rows<RB>(VS, 0, live);
            fence_proxy_async_smem();
          }
        }
        __syncthreads();  // 1
        if (one && !failed) {
          tm_fence_after();
          tc_wide<RB, MT>(panels, tm + D1, kq, smem_u32(SS), L::SPLANE, tc_idesc(3 * BV, false, true));
          tc_commit(bar);
          if (KST == 2 && a.tma && ch + 1 < ch1) load_kq(ch + 1);
          if (a.Sh && !a.maps) {  // the chunk's starting state: its first two planes
            for (int k = 0; k < 2; ++k) store_bulk(a.Sh + (tile * 2 + k) * a.KP * BV, SS + k * L::SPLANE, a.KP * RB);
            bulk_commit_group();
          }
        }
        if (one) bulk_wait_group_read<0>();  // the state's planes and o's image may be written again
        __syncthreads();  // 2
        if (one) {
          wait(bar_tp, (ch - ch0) & 1);
          if (!failed) {
            tm_fence_after();
#pragma unroll
            for (int p = 0; p < 3; ++p)  // plane p of TP, the first 3 - p of Y
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_mma(tm + D2 + p * BV, td + p * (TC_PANEL >> 4) + 2 * k, yd + k * RB, tc_idesc((3 - p) * BV, false, true), p || k);
            tc_commit(bar);
            if (a.tma && ch + 1 < ch1) load_v(ch + 1);
          }
        }
        __syncthreads();  // 3
        if (one && !failed) {
          tm_fence_after();
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma(tm + D3 + 3 * mt * BV, tc_desc(kq + 2 * mt * TC_PANEL + k * 2048, TC_PANEL), yd + k * RB,
                     tc_idesc(3 * BV, true, true), k);
          tc_commit(bar);
          if (ch + 1 < ch1) load_bulk(TP, tp + (size_t)(ch + 1) * L::TP, L::TP, bar_tp);  // the second products have read it
        }
        __syncthreads();  // 4
        if (one && !failed) {
          if (KST == 1 && a.tma && ch + 1 < ch1) load_kq(ch + 1);
          if (!a.maps && a.tma) {
            tma_store_5d(&maps.o, smem_u32(OS), vt * BV, n, ch * TC_C, b, 0);
            bulk_commit_group();
          }
        }
      }
      if (one) {
        bulk_wait_group_all();
        bool f = false;
        tc_commit(bar_end);
        mbar_wait_bounded<false>(bar_end, 0, a.wait_limit_ns, nullptr, f);
        if (failed)  // copies that nobody waited for land before the CTA ends
          for (int p = 0; p < 4; ++p) {
            f = false;
            mbar_wait_bounded<false>(p < 2 ? bar_tp : bar_in, p & 1, a.wait_limit_ns, nullptr, f);
          }
      }
    } else {  // ---- rows that TMA cannot take
      const int t = a.tma ? -1 : tid - 320;  // warps 10 and 11
      const size_t kstride = (size_t)a.Nk * a.Dk, kat = (size_t)b * a.T * kstride + (size_t)nk * a.Dk;
      auto load_kq = [&](int ch) {
        unsigned char* d = sm + (ch % KST) * L::KQ;
        const int live = tc_live(a, b, ch);
        const size_t at = kat + (size_t)ch * TC_C * kstride;
        load_img<128, P, 64>(t, d, 0, (const bf16*)a.k + at, kstride, live, a.Dk, 0, (a.KP + 63) & ~63, TC_PANEL);
        load_img<128, P, 64>(t, d, 64, (const bf16*)a.q + at, kstride, live, a.Dk, 0, (a.KP + 63) & ~63, TC_PANEL);
      };
      auto load_v = [&](int ch) {
        if (!ident)
          load_img<RB, BV / 8, 64>(t, VS, 0, (const bf16*)a.v + vat + (size_t)ch * TC_C * vstride, vstride, tc_live(a, b, ch), a.Dv,
                                   vt * BV, BV, 0);
        const float* r = a.rec + ((size_t)bn * a.nc + ch) * REC_N * TC_C;
        float* d = recs + (ch & 1) * 2 * TC_C;
        if (t < 32) cp16(smem_u32(d + t * 4), r + (t < 16 ? REC_GAM * TC_C + t * 4 : REC_BR * TC_C + (t - 16) * 4), true);
      };
      auto store_o = [&](int ch) {
        store_img<RB, 64>(t, OS, (bf16*)a.o + vat + (size_t)ch * TC_C * vstride, vstride, min(TC_C, a.T - ch * TC_C), a.Dv, vt * BV);
      };
      if (t >= 0 && ch0 < ch1) {
        load_kq(ch0);
        load_v(ch0);
        cp_wait_all();
        fence_proxy_async_smem();
      }
      for (int ch = ch0; ch < ch1; ++ch) {
        const bool more = ch + 1 < ch1 && t >= 0;
        __syncthreads();  // 1
        if (KST == 2 && more) load_kq(ch + 1);
        if (t >= 0 && ch > ch0 && !a.maps) store_o(ch - 1);
        __syncthreads();  // 2
        if (more) load_v(ch + 1);
        __syncthreads();  // 3
        __syncthreads();  // 4
        if (KST == 1 && more) load_kq(ch + 1);
        if (more) {
          cp_wait_all();
          fence_proxy_async_smem();
        }
      }
      if (t >= 0 && ch0 < ch1 && !a.maps) store_o(ch1 - 1);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const uint32_t row = tm + ((uint32_t)(quad * 32) << 16);
    float S[MT][NC];
    const int c0 = half * NC, v0 = vt * BV + c0;  // this thread's columns, in the tile and in v
    const int valid = a.Dv - v0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = mt * 128 + quad * 32 + lane;
      const float* s = a.s0 ? a.s0 + ((size_t)bn * a.Dk + r) * a.Dv + v0 : nullptr;
      const float* st = seg && !a.maps ? a.St + (((size_t)bn * a.segs + seg) * a.nvt * BV + v0) * KR + r : nullptr;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        S[mt][c] = ident ? (r == v0 - a.nvt * BV + c ? 1.0f : 0.0f)
                   : st ? st[(size_t)c * KR]
                        : s && !a.maps && r < a.Dk && c < valid ? s[c] : 0.0f;
    }
    auto put_state = [&]() {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) put_planes<RB, NC>(SS, L::SPLANE, mt * 128 + quad * 32 + lane, c0, S[mt]);
    };
    // S, as the threads hold it, to kept state e
    auto keep_state = [&](int e) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float4* f = (float4*)(a.sf + (((size_t)bn * a.ne + e) * a.nvt + vt) * MT * 128 * BV) +
                    (size_t)(half * MT + mt) * (NC / 4) * 128 + quad * 32 + lane;
#pragma unroll
        for (int c = 0; c < NC; c += 4) f[(c / 4) * 128] = make_float4(S[mt][c], S[mt][c + 1], S[mt][c + 2], S[mt][c + 3]);
      }
    };
    if (ch0 < ch1) put_state();
    else if (nch == 0 && seg == 0 && a.sf && !a.maps) keep_state(0);
    const int i = (quad & 1) * 32 + lane;  // this thread's step
    uint32_t parity = 0;
    auto take = [&]() {
      wait(bar, parity);
      parity ^= 1;
      tm_fence_after();
    };
    auto leave = [&]() {
      fence_proxy_async_smem();
      tm_fence_before();
      __syncthreads();
    };
    for (int ch = ch0; ch < ch1; ++ch) {
      const size_t tile = ((size_t)bn * a.nc + ch) * a.nvt + vt;
      const bool more = ch + 1 < ch1;
      leave();  // 1: KQ, V and S's planes are there
      const float *gam = recs + (ch & 1) * 2 * TC_C, *br = gam + TC_C;
      const float gi = gam[i];
      bool lost = false;  // whether a column's state is not finite and ends in this chunk
      float y[NC];
      if (ident)
#pragma unroll
        for (int c = 0; c < NC; ++c) y[c] = 0.0f;
      else if (quad < 2)
#pragma unroll
        for (int c = 0; c < NC; c += 8) widen8(*(const uint4*)(VS + img<RB>(i, (c0 + c) >> 3)), y + c);
      take();
      float x[NC];
      tm_sum<NC, BV>(x, row + D1 + c0);
      if (quad < 2) {
        if (has_part(gi)) {  // behind a reset the old state has no part, whatever it holds
#pragma unroll
          for (int c = 0; c < NC; ++c) y[c] = fmaf(-gi, x[c], y[c]);
          if (!has_part(gam[TC_C - 1]))  // the products with TP reach over the reset by zeros, which an infinity would pass
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (!isfinite(x[c])) y[c] = 0.0f, lost = true;
        }
        put_planes<RB, NC>(YS, L::YPLANE, i, c0, y);
      } else {
        const float f = gi * a.scale;
#pragma unroll
        for (int c = 0; c < NC; ++c) x[c] = has_part(gi) ? f * x[c] : 0.0f;
      }
      leave();  // 2: Y's planes are there, V is read
      const int live = tc_live(a, b, ch);
      const float bi = br[i];
      take();
      float z[NC];
      tm_sum<NC, BV>(z, row + D2 + c0);
      if (quad < 2) {
#pragma unroll
        for (int c = 0; c < NC; ++c) y[c] = bi * z[c];
        put_planes<RB, NC>(YS, L::YPLANE, i, c0, y);  // the products have read Y
      }
      leave();  // 3: beta rho Z's planes are there
      // what leaves for memory goes while the product runs
      if (a.maps) {
      } else if (quad < 2) {
        if (a.zf) {
          if (lost) z[0] = nanf("");  // for what is summed over z's columns: no more is made of this row's
          float4* f = (float4*)(a.zf + tile * 64 * BV) + (size_t)half * (NC / 4) * 64 + i;
#pragma unroll
          for (int c = 0; c < NC; c += 4) f[(c / 4) * 64] = make_float4(z[c], z[c + 1], z[c + 2], z[c + 3]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) z[c] = i < live ? z[c] + x[c] : 0.0f;
        if (a.of) {
          float4* f = (float4*)(a.of + tile * 64 * BV) + (size_t)half * (NC / 4) * 64 + i;
#pragma unroll
          for (int c = 0; c < NC; c += 4) f[(c / 4) * 64] = make_float4(z[c], z[c + 1], z[c + 2], z[c + 3]);
        }
#pragma unroll
        for (int c = 0; c < NC; c += 8) *(uint4*)(OS + img<RB>(i, (c0 + c) >> 3)) = round8(z + c);
      }
      const float gC = gam[TC_C - 1];
      take();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float d[NC];
        tm_sum<NC, BV>(d, row + D3 + 3 * mt * BV + c0);
#pragma unroll
        for (int c = 0; c < NC; ++c) S[mt][c] = has_part(gC) ? fmaf(gC, S[mt][c], d[c]) : d[c];
      }
      leave();  // 4: the products are over, o's image is there
      if (more) put_state();
      const int end = ch + 1 == nch ? 0 : (ch + 1) % TC_EDGE == 0 ? (ch + 1) / TC_EDGE : -1;
      if (a.sf && !a.maps && end >= 0) keep_state(end);
    }
    if (a.maps) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 128 + quad * 32 + lane, j = v0 - a.nvt * BV;
        float* s = ident ? a.Mt + (((size_t)bn * a.segs + seg) * KR + j) * KR + r
                         : a.Ht + (((size_t)bn * a.segs + seg) * a.nvt * BV + v0) * KR + r;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (!ident || j + c < KR) s[(size_t)c * KR] = r < a.KP ? S[mt][c] : 0.0f;
      }
    } else if (a.last && seg == a.segs - 1) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 128 + quad * 32 + lane;
        if (r < a.Dk) {
          float* s = a.last + ((size_t)bn * a.Dk + r) * a.Dv + v0;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < valid) s[c] = S[mt][c];
        }
      }
    }
  }
  // steps past the row's length
  if (!a.maps && seg == a.segs - 1) tc_zero_tail<BV>((bf16*)a.o + vat, vstride, nch * TC_C, a.T, vt * BV, a.Dv);
  tm_fence_before();
  __syncthreads();
  if (warp == 0) tm_free<512>(tm);
}

// ---- join ----------------------------------------------------------------------------
// The states between the segments, one after the other: forward S = M S + H from
// state0, backward dS = M^T dS + H from dlast. A CTA has CW columns of v of a head,
// S in shared memory, M by blocks of 64 KB, two of them; 4 x 2 values a thread.
// Rows and columns of M past KP are not looked at (the maps' pass writes whole tiles
// of columns, the rest of Mt is whatever the caller's memory held): the states are
// zero there, which the chain's whole panels count on. M is exactly zero where a reset
// stands in its segment: then nothing of S may pass, an infinity or a NaN neither,
// so where S holds one a reset is looked for and M left out.
template <int KR, bool BACK> __global__ void __launch_bounds__(256, 1) delta_tc_join_kernel(DeltaTcArgs a, int cols_total) {
  constexpr int CW = KR == 128 ? 16 : 8, LD = CW + 4, JB = 16384 / KR;  // rows of Mt in a block
  extern __shared__ __align__(16) unsigned char sm_raw[];
  float* M = (float*)sm_raw;  // [2][JB][KR]
  float* S = M + 2 * JB * KR; // [KR][LD]
  const int groups = cols_total / CW;
  const int tid = threadIdx.x, bn = blockIdx.x / groups, v0 = (blockIdx.x % groups) * CW, nch = tc_chunks(a, bn / a.N);
  const int cg = tid % (CW / 2) * 2, rg = tid / (CW / 2) * 4;
  const float* x0 = BACK ? a.dlast : a.s0;
  int odd = 0;
  for (int k = tid; k < KR * CW; k += 256) {
    const int r = k / CW, c = k % CW;
    const float x = x0 && r < a.Dk && v0 + c < a.Dv ? x0[((size_t)bn * a.Dk + r) * a.Dv + v0 + c] : 0.0f;
    S[r * LD + c] = x;
    odd |= !isfinite(x);
  }
  odd = __syncthreads_or(odd);
  const int blocks = (a.segs - 1) * (KR / JB);
  auto load = [&](int k) {  // block k of the matrices in the order of their use
    const int s = BACK ? a.segs - 1 - k / (KR / JB) : k / (KR / JB);
    const float* m = a.Mt + (((size_t)bn * a.segs + s) * KR + (k % (KR / JB)) * JB) * KR;
    const uint32_t to = smem_u32(M + (k & 1) * JB * KR);
    for (int i = tid; i < JB * KR / 4; i += 256) cp16(to + i * 16, m + i * 4, true);
    cp_commit();
  };
  load(0);
  float acc[4][2];
  int cut = 0;
  for (int k = 0; k < blocks; ++k) {
    const int s = BACK ? a.segs - 1 - k / (KR / JB) : k / (KR / JB), part = k % (KR / JB);
    if (k + 1 < blocks) load(k + 1);
    else cp_commit();
    cp_wait<1>();
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[r][c] = 0.0f;
      cut = 0;
      if (odd) {
        for (int ch = s * a.seglen + tid; ch < min(nch, (s + 1) * a.seglen); ch += 256)
          cut |= !has_part(a.rec[(((size_t)bn * a.nc + ch) * REC_N + REC_GAM) * TC_C + TC_C - 1]);
        cut = __syncthreads_or(cut);
      }
    }
    const float* m = M + (k & 1) * JB * KR;
    if (!cut) {
      if constexpr (!BACK) {  // column j of M times row j of S
#pragma unroll 4
        for (int j = 0; j < min(JB, a.KP - part * JB); ++j) {
          const float4 x = *(const float4*)(m + j * KR + rg);
          const float2 y = *(const float2*)(S + (part * JB + j) * LD + cg);
          const float xs[4] = {x.x, x.y, x.z, x.w}, ys[2] = {y.x, y.y};
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) acc[r][c] = fmaf(xs[r], ys[c], acc[r][c]);
        }
      } else if (rg >= part * JB && rg < min((part + 1) * JB, a.KP)) {  // this thread's columns of M, summed over its rows
#pragma unroll 2
        for (int j = 0; j < a.KP; j += 4) {
          float4 x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = *(const float4*)(m + (rg - part * JB + r) * KR + j);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 y = *(const float2*)(S + (j + q) * LD + cg);
            const float ys[2] = {y.x, y.y};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float xr = q == 0 ? x[r].x : q == 1 ? x[r].y : q == 2 ? x[r].z : x[r].w;
#pragma unroll
              for (int c = 0; c < 2; ++c) acc[r][c] = fmaf(xr, ys[c], acc[r][c]);
            }
          }
        }
      }
    }
    __syncthreads();
    if (part == KR / JB - 1) {
      odd = 0;
      const size_t from = (((size_t)bn * a.segs + s) * cols_total + v0 + cg) * KR + rg;
      const size_t to = (((size_t)bn * a.segs + (BACK ? s - 1 : s + 1)) * cols_total + v0 + cg) * KR + rg;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float4 h = *(const float4*)(a.Ht + from + (size_t)c * KR);
        const float4 x = make_float4(acc[0][c] + h.x, acc[1][c] + h.y, acc[2][c] + h.z, acc[3][c] + h.w);
        *(float4*)(a.St + to + (size_t)c * KR) = x;
        S[rg * LD + cg + c] = x.x;
        S[(rg + 1) * LD + cg + c] = x.y;
        S[(rg + 2) * LD + cg + c] = x.z;
        S[(rg + 3) * LD + cg + c] = x.w;
        odd |= !isfinite(x.x) | !isfinite(x.y) | !isfinite(x.z) | !isfinite(x.w);
      }
      odd = __syncthreads_or(odd);
    }
  }
}

template <int KR, bool BACK> cudaError_t join_run(const DeltaTcArgs& a, int BV, cudaStream_t st) {
  constexpr int CW = KR == 128 ? 16 : 8;
  constexpr size_t sm = 2 * 65536 + (size_t)KR * (CW + 4) * 4;
  cudaError_t e = set_smem_attr((const void*)delta_tc_join_kernel<KR, BACK>, sm);
  if (e != cudaSuccess) return e;
  const int cols = a.nvt * BV;
  delta_tc_join_kernel<KR, BACK><<<(unsigned)(a.B * a.N * (cols / CW)), 256, sm, st>>>(a, cols);
  note_launch();
  return cudaGetLastError();
}

template <int BV, int MT> cudaError_t chain(DeltaTcArgs a, const TcMaps& maps, cudaStream_t st) {
  constexpr int sm = TcChain<BV, MT>::BYTES;
  cudaError_t e = set_smem_attr((const void*)delta_tc_chain_kernel<BV, MT>, sm);
  if (e != cudaSuccess) return e;
  const unsigned lanes = (unsigned)(a.B * a.N * a.segs);
  if (a.segs > 1) {
    a.maps = 1;
    delta_tc_chain_kernel<BV, MT><<<lanes * (a.nvt + (a.KP + BV - 1) / BV), 384, sm, st>>>(a, maps);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = join_run<MT * 128, false>(a, BV, st)) != cudaSuccess) return e;
    a.maps = 0;
  }
  delta_tc_chain_kernel<BV, MT><<<lanes * a.nvt, 384, sm, st>>>(a, maps);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_tc_join_back(int BV, const DeltaTcArgs& a, cudaStream_t st) {
  return a.KP > 128 ? join_run<256, true>(a, BV, st) : join_run<128, true>(a, BV, st);
}

cudaError_t tc_map(CUtensorMap* m, const void* base, const DeltaTcArgs& a, int heads, int D, int cols) {
  const unsigned long long dims[5] = {(unsigned long long)D, (unsigned long long)heads, (unsigned long long)a.T, (unsigned long long)a.B, 1};
  const unsigned int box[5] = {(unsigned)cols, 1, TC_C, 1, 1};
  return encode_tensor_map_swizzled(m, base, 2, 5, dims, box, cols * 2);
}

cudaError_t delta_tc_fwd_launch(int BV, const DeltaTcArgs& a, cudaStream_t st) {
  const size_t sm = prep_smem(a.KP);
  cudaError_t e = set_smem_attr((const void*)delta_tc_prep_kernel, sm);
  if (e != cudaSuccess) return e;
  delta_tc_prep_kernel<<<(unsigned)((long long)a.B * a.N * a.nc), 128, sm, st>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  TcMaps maps;
  DeltaTcArgs x = a;
  x.tma = a.Dk % 8 == 0 && a.Dv % 8 == 0;
  if (x.tma && ((e = tc_map(&maps.k, a.k, a, a.Nk, a.Dk, 64)) != cudaSuccess || (e = tc_map(&maps.q, a.q, a, a.Nk, a.Dk, 64)) != cudaSuccess ||
                (e = tc_map(&maps.v, a.v, a, a.N, a.Dv, BV)) != cudaSuccess || (e = tc_map(&maps.o, a.o, a, a.N, a.Dv, BV)) != cudaSuccess))
    return e;
  if (a.KP > 128) return chain<32, 2>(x, maps, st);
  return BV == 64 ? chain<64, 1>(x, maps, st) : chain<32, 1>(x, maps, st);
}

}  // namespace rnn
