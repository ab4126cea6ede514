// Gated delta rule, bf16 storage, backward (delta_tc.cuh has the formulas), from
// what the forward left.
//   chain  per head and tile of BV columns of v, the chunks from the last to the
//          first: dV and the state's gradient
//   grad   every chunk by itself: dQ, dK
//   gates  dg and dbeta from the chain's row products
// and, where heads share q and k, the sums of dQ and dK over them.
#include "delta.h"
#include "delta_tc.cuh"

namespace rnn {
namespace {

// ---- chain --------------------------------------------------------------------------
template <int BV, int MT> struct TcBack {
  static constexpr int RB = 2 * BV, KST = MT == 1 ? 2 : 1;
  static constexpr int KQ = 2 * MT * TC_PANEL, TP = 3 * TC_PANEL, SPLANE = MT * 128 * RB, GPLANE = 128 * RB;
  static constexpr int AT_TP = KST * KQ, AT_S = AT_TP + TP, AT_G = AT_S + 3 * SPLANE, AT_O = AT_G + 3 * GPLANE;
  static constexpr int AT_V = AT_O + 64 * RB, AT_REC = AT_V + 64 * RB, BYTES = AT_REC + 2 * 2 * 64 * 4 + 64 + 1024;
};

// Warps as in the forward's chain. The image G holds, by planes, W in rows 0 .. 63
// until dY's products have read it, then -gam dY; rows 64 .. 127 scale gam dO,
// written by the threads of Q's steps while the first product runs. dY goes out
// through V's image, each value in the place of the v that its thread has read.
// Warps 9 to 11 take <S0, dS1> of the chunks with a step below GATE_NEAR.
// The products for dY take TP by columns, 64 of them; the other 64 rows of the
// accumulator come from whatever lies a panel further (inside this CTA's shared
// memory) and are not looked at. Bound as the forward's chain: 377 us at its size.
template <int BV, int MT>
__global__ void __launch_bounds__(384, 1) delta_tc_back_kernel(DeltaTcArgs a, const __grid_constant__ TcMaps maps) {
  using L = TcBack<BV, MT>;
  constexpr int RB = L::RB, NC = BV / 2, KST = L::KST, P = MT * 16;
  static_assert(3 * L::SPLANE >= TC_PANEL, "what TP's last plane is read past");
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)sm_raw + 1023) & ~(uintptr_t)1023);
  unsigned char *TP = sm + L::AT_TP, *SS = sm + L::AT_S, *GS = sm + L::AT_G, *OS = sm + L::AT_O, *VS = sm + L::AT_V;
  float* recs = (float*)(sm + L::AT_REC);  // [2][gam, br][64]
  uint64_t* barp = (uint64_t*)(recs + 2 * 2 * 64);
  uint32_t* slot = (uint32_t*)(barp + 5);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
  constexpr int KR = MT * 128;
  const int vt = blockIdx.x % a.nvt, seg = blockIdx.x / a.nvt % a.segs, bn = blockIdx.x / a.nvt / a.segs;
  const int n = bn % a.N, b = bn / a.N, nk = n / (a.N / a.Nk);
  if (a.maps && seg == 0) return;  // nothing comes before it
  const int nch = tc_chunks(a, b), ch0 = min(nch, seg * a.seglen), ch1 = min(nch, ch0 + a.seglen);
  const size_t vstride = (size_t)a.N * a.Dv, vat = (size_t)b * a.T * vstride + (size_t)n * a.Dv;
  const uint32_t bar = smem_u32(barp), bar_end = bar + 8, bar_tp = bar + 16, bar_in = bar + 24, bar_v = bar + 32;
  if (tid == 0) {
    for (int k = 0; k < 5; ++k) mbar_init(bar + 8 * k, 1);
    fence_mbar_init_cluster();
  }
  if (warp == 0) tm_alloc<512>(slot);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *slot;
  constexpr int D1 = 0, D2 = 3 * BV * MT, D3 = 0;  // as in the forward: K dS1; dY; the state's change
  bool failed = false;
  auto wait = [&](uint32_t which, uint32_t par) { mbar_wait_bounded<false>(which, par, a.wait_limit_ns, a.status, failed); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8) {  // ---- products, bulk copies
      const unsigned char* tp = (const unsigned char*)a.tp + (size_t)bn * a.nc * L::TP;
      const bool one = lane == 0;
      // K, Q, dO and the steps' factors of a chunk, counted by bar_in; V by bar_v
      const int panels = (a.KP + 63) >> 6;
      const uint32_t bytes = panels * 16384 + (a.dO ? 64 * RB : 0) + 512;
      auto load_kq = [&](int ch) {
        unsigned char* d = sm + (ch % KST) * L::KQ;
        if (KST == 2) mbar_arrive_expect_tx(bar_in, bytes);
        for (int p = 0; p < panels; ++p) {
          tma_load_5d(smem_u32(d + p * TC_PANEL), &maps.k, bar_in, p * 64, nk, ch * TC_C, b, 0);
          tma_load_5d(smem_u32(d + p * TC_PANEL + 8192), &maps.q, bar_in, p * 64, nk, ch * TC_C, b, 0);
        }
      };
      auto load_o = [&](int ch) {
        if (KST == 1) mbar_arrive_expect_tx(bar_in, bytes);
        if (a.dO) tma_load_5d(smem_u32(OS), &maps.dO, bar_in, vt * BV, n, ch * TC_C, b, 0);
        const float* r = a.rec + ((size_t)bn * a.nc + ch) * REC_N * TC_C;
        const uint32_t d = smem_u32(recs + (ch & 1) * 2 * TC_C);
        bulk_load_global(d, r + REC_GAM * TC_C, 256, bar_in);
        bulk_load_global(d + 256, r + REC_BR * TC_C, 256, bar_in);
      };
      if (a.tma && !a.dO) {
        clear_rows<RB>(OS, 0, 0);
        fence_proxy_async_smem();
      }
      if (one && ch0 < ch1) {
        load_bulk(TP, tp + (size_t)(ch1 - 1) * L::TP, L::TP, bar_tp);
        if (a.tma) {
          if (KST == 2) load_kq(ch1 - 1);
          load_o(ch1 - 1);
          if (KST == 1) load_kq(ch1 - 1);
        }
      }
      const uint64_t td = tc_desc(smem_u32(TP), TC_PANEL), gd = tc_desc<RB>(smem_u32(GS), L::GPLANE), od = tc_desc<RB>(smem_u32(OS), 16);
      for (int ch = ch1 - 1; ch >= ch0; --ch) {
        unsigned char* kqs = sm + (ch % KST) * L::KQ;
        const uint32_t kq = smem_u32(kqs);
        const size_t tile = ((size_t)bn * a.nc + ch) * a.nvt + vt;
        const int live = tc_live(a, b, ch);
        const bool cut = a.tma && live < TC_C && ch * TC_C + live < a.T;  // steps of the tensor past the row's length
        if (a.tma) {
          wait(bar_in, (ch1 - 1 - ch) & 1);
          if (cut) {
            for (int p = 0; p < panels; ++p) {
              clear_rows<128>(kqs + p * TC_PANEL, 0, live);
              clear_rows<128>(kqs + p * TC_PANEL, 64, live);
            }
            clear_rows<RB>(OS, 0, live);
            fence_proxy_async_smem();
          }
        }
        __syncthreads();  // 1
        if (one && !failed) {
          tm_fence_after();
          tc_wide<RB, MT>(panels, tm + D1, kq, smem_u32(SS), L::SPLANE, tc_idesc(3 * BV, false, true));
          tc_commit(bar);
          if (KST == 2 && a.tma && ch > ch0) load_kq(ch - 1);
          if (!a.maps) {
            // the gradient of the chunk's last state: its first two planes
            for (int k = 0; k < 2; ++k) store_bulk(a.dSh + (tile * 2 + k) * a.KP * BV, SS + k * L::SPLANE, a.KP * RB);
            bulk_commit_group();
            if (a.tma) {
              bulk_wait_group_read<1>();  // dY has left V's image
              mbar_arrive_expect_tx(bar_v, 64 * RB);
              tma_load_5d(smem_u32(VS), &maps.v, bar_v, vt * BV, n, ch * TC_C, b, 0);
            }
          }
          bulk_wait_group_read<0>();  // the state's planes may be written again
        }
        __syncthreads();  // 2
        if (one) {
          wait(bar_tp, (ch1 - 1 - ch) & 1);
          if (!failed) {
            tm_fence_after();
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // Tm's plane p with W's first 3 - p, PT's with dO
                tc_mma(tm + D2 + p * BV, td + p * (TC_PANEL >> 4) + k * 128, gd + k * RB, tc_idesc((3 - p) * BV, true, true), p || k);
                tc_mma(tm + D2 + p * BV, td + p * (TC_PANEL >> 4) + 512 + k * 128, od + k * RB, tc_idesc(BV, true, true), true);
              }
            tc_commit(bar);
          }
        }
        __syncwarp();
        if (a.tma && !a.maps) {
          wait(bar_v, (ch1 - 1 - ch) & 1);
          if (cut) clear_rows<RB>(VS, 0, live);
        }
        __syncthreads();  // 3
        if (one && !failed) {
          tm_fence_after();
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tc_mma(tm + D3 + 3 * mt * BV, tc_desc(kq + 2 * mt * TC_PANEL + k * 2048, TC_PANEL), gd + k * RB,
                     tc_idesc(3 * BV, true, true), k);
          tc_commit(bar);
          if (ch > ch0) {
            load_bulk(TP, tp + (size_t)(ch - 1) * L::TP, L::TP, bar_tp);  // the second products have read it
            if (a.tma) load_o(ch - 1);
          }
        }
        __syncthreads();  // 4
        if (one && !failed && a.tma) {
          if (KST == 1 && ch > ch0) load_kq(ch - 1);
          if (!a.maps) {
            tma_store_5d(&maps.dv, smem_u32(VS), vt * BV, n, ch * TC_C, b, 0);
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
          for (int p = 0; p < 6; ++p) {
            f = false;
            mbar_wait_bounded<false>(bar_tp + 8 * (p >> 1), p & 1, a.wait_limit_ns, nullptr, f);
          }
      }
    } else if (a.tma || warp == 9) {  // ---- <S0, dS1>
      // Of the chunks whose gates want it, from two planes of each, which are laid out
      // alike: a third between each two barriers, the pieces of S0 loaded between the
      // two before. A thread's pieces of both go to mma.sync as they are, in the same
      // places of A and B; the diagonal of the 8 x 8 products is theirs.
      const int cw = warp - 9, cws = a.tma ? 3 : 1;  // rows that TMA cannot take keep the other two warps busy
      const int bytes = a.KP * RB;
      constexpr int CU = 4;  // pieces of 16 bytes that a thread has of a third at once
      uint4 sx[CU][2];
      float dot[4];
      unsigned wanted = 0;  // of the 32 chunks around
      auto wants = [&](int ch) -> bool {
        if (ch < ch0 || a.maps) return false;
        if (ch == ch1 - 1 || (ch & 31) == 31) {
          const int k = (ch & ~31) + lane;
          wanted = __ballot_sync(0xffffffffu, k <= ch && a.rec[(((size_t)bn * a.nc + k) * REC_N + REC_NEAR) * TC_C] != 0.0f);
        }
        return wanted >> (ch & 31) & 1;
      };
      auto place = [&](int part, int u) { return (((u * 3 + part) * cws + cw) * 32 + lane) * 16; };
      auto fetch = [&](int ch, int part, int u0) {
        const unsigned char* s0 = (const unsigned char*)(a.Sh + (((size_t)bn * a.nc + ch) * a.nvt + vt) * 2 * a.KP * BV);
#pragma unroll
        for (int u = 0; u < CU; ++u) {
          const int o = place(part, u0 + u);
          sx[u][0] = sx[u][1] = make_uint4(0, 0, 0, 0);
          if (o < bytes) {
            sx[u][0] = __ldg((const uint4*)(s0 + o));
            sx[u][1] = __ldg((const uint4*)(s0 + bytes + o));
          }
        }
      };
      auto add = [&](const uint4& p, const uint4& q) {
        const uint32_t a0[4] = {p.x, 0, p.y, 0}, a1[4] = {p.z, 0, p.w, 0};
        mma_bf16_16816(dot, a0, q.x, q.y);
        mma_bf16_16816(dot, a1, q.z, q.w);
      };
      auto cross = [&](int ch, int part) {
        for (int u0 = 0;; u0 += CU) {
#pragma unroll
          for (int u = 0; u < CU; ++u) {
            const int o = place(part, u0 + u), at = o < bytes ? o : 0;  // past the end x is zero
            const uint4 y = *(const uint4*)(SS + at), yl = *(const uint4*)(SS + L::SPLANE + at);
            add(sx[u][1], y);
            add(sx[u][0], yl);
            add(sx[u][0], y);
          }
          if (place(part, u0 + CU) - lane * 16 >= bytes) break;
          fetch(ch, part, u0 + CU);
        }
      };
      bool want = wants(ch1 - 1);
      if (want) fetch(ch1 - 1, 0, 0);
      for (int ch = ch1 - 1; ch >= ch0; --ch) {
        dot[0] = dot[1] = dot[2] = dot[3] = 0.0f;
        __syncthreads();  // 1
        if (want) {
          cross(ch, 0);
          fetch(ch, 1, 0);
        }
        __syncthreads();  // 2
        if (want) {
          cross(ch, 1);
          fetch(ch, 2, 0);
        }
        __syncthreads();  // 3
        if (want) {
          cross(ch, 2);
          // of rows lane / 4 and columns lane % 4 * 2 and one on
          float d = lane >> 2 == (lane & 3) * 2 ? dot[0] : lane >> 2 == (lane & 3) * 2 + 1 ? dot[1] : 0.0f;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
          float* to = a.cross + (((size_t)bn * a.nc + ch) * a.nvt + vt) * 3;
          if (lane < 3 && (lane == cw || cws == 1)) to[lane] = lane == cw ? d : 0.0f;
        }
        want = wants(ch - 1);
        if (want) fetch(ch - 1, 0, 0);
        __syncthreads();  // 4
      }
    } else {  // ---- rows that TMA cannot take
      const int t = tid - 320;  // warps 10 and 11
      const size_t kstride = (size_t)a.Nk * a.Dk, kat = (size_t)b * a.T * kstride + (size_t)nk * a.Dk;
      auto load_kq = [&](int ch) {
        unsigned char* d = sm + (ch % KST) * L::KQ;
        const int live = tc_live(a, b, ch);
        const size_t at = kat + (size_t)ch * TC_C * kstride;
        load_img<128, P, 64>(t, d, 0, (const bf16*)a.k + at, kstride, live, a.Dk, 0, (a.KP + 63) & ~63, TC_PANEL);
        load_img<128, P, 64>(t, d, 64, (const bf16*)a.q + at, kstride, live, a.Dk, 0, (a.KP + 63) & ~63, TC_PANEL);
      };
      auto load_o = [&](int ch) {
        load_img<RB, BV / 8, 64>(t, OS, 0, (const bf16*)(a.dO ? a.dO : a.v) + vat + (size_t)ch * TC_C * vstride, vstride,
                                 a.dO ? tc_live(a, b, ch) : 0, a.Dv, vt * BV, BV, 0);
        const float* r = a.rec + ((size_t)bn * a.nc + ch) * REC_N * TC_C;
        float* d = recs + (ch & 1) * 2 * TC_C;
        if (t < 32) cp16(smem_u32(d + t * 4), r + (t < 16 ? REC_GAM * TC_C + t * 4 : REC_BR * TC_C + (t - 16) * 4), true);
      };
      auto store_dv = [&](int ch) {
        store_img<RB, 64>(t, VS, (bf16*)a.dv + vat + (size_t)ch * TC_C * vstride, vstride, min(TC_C, a.T - ch * TC_C), a.Dv, vt * BV);
      };
      if (ch0 < ch1) {
        load_kq(ch1 - 1);
        load_o(ch1 - 1);
        cp_wait_all();
        fence_proxy_async_smem();
      }
      for (int ch = ch1 - 1; ch >= ch0; --ch) {
        const bool more = ch > ch0;
        __syncthreads();  // 1
        if (!a.maps) {
          if (ch + 1 < ch1) store_dv(ch + 1);
          asm volatile("bar.sync 1, 64;" ::: "memory");  // the rows are read: V's may follow
          load_img<RB, BV / 8, 64>(t, VS, 0, (const bf16*)a.v + vat + (size_t)ch * TC_C * vstride, vstride, tc_live(a, b, ch), a.Dv,
                                   vt * BV, BV, 0);
          cp_commit();
        }
        if (KST == 2 && more) load_kq(ch - 1);
        cp_commit();
        __syncthreads();  // 2
        cp_wait<1>();     // V
        __syncthreads();  // 3
        if (more) load_o(ch - 1);
        __syncthreads();  // 4
        if (KST == 1 && more) load_kq(ch - 1);
        if (more) {
          cp_wait_all();
          fence_proxy_async_smem();
        }
      }
      if (ch0 < ch1 && !a.maps) store_dv(ch0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const uint32_t row = tm + ((uint32_t)(quad * 32) << 16);
    float S[MT][NC];  // dS
    const int c0 = half * NC, v0 = vt * BV + c0, valid = a.Dv - v0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = mt * 128 + quad * 32 + lane;
      const float* s = a.dlast ? a.dlast + ((size_t)bn * a.Dk + r) * a.Dv + v0 : nullptr;
      const float* st = seg < a.segs - 1 && !a.maps ? a.St + (((size_t)bn * a.segs + seg) * a.nvt * BV + v0) * KR + r : nullptr;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        S[mt][c] = st ? st[(size_t)c * KR] : s && !a.maps && r < a.Dk && c < valid ? s[c] : 0.0f;
    }
    auto put_state = [&]() {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) put_planes<RB, NC>(SS, L::SPLANE, mt * 128 + quad * 32 + lane, c0, S[mt]);
    };
    // <S, dS> at a kept state
    auto put_edge = [&](int e) {
      float s = 0.0f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float4* f = (const float4*)(a.sf + (((size_t)bn * a.ne + e) * a.nvt + vt) * MT * 128 * BV) +
                          (size_t)(half * MT + mt) * (NC / 4) * 128 + quad * 32 + lane;
        if (mt * 128 + quad * 32 + lane < a.Dk) {
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 x = f[(c / 4) * 128];
            s = fmaf(x.x, S[mt][c], s);
            s = fmaf(x.y, S[mt][c + 1], s);
            s = fmaf(x.z, S[mt][c + 2], s);
            s = fmaf(x.w, S[mt][c + 3], s);
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) a.edge[(((size_t)bn * a.ne + e) * a.nvt + vt) * 8 + warp] = s;
    };
    if (ch0 < ch1) {
      put_state();
      if (ch1 == nch && !a.maps) put_edge(0);
    }
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
    for (int ch = ch1 - 1; ch >= ch0; --ch) {
      const size_t tile = ((size_t)bn * a.nc + ch) * a.nvt + vt;
      const bool more = ch > ch0;
      leave();  // 1: KQ, dO and dS's planes are there
      const float *gam = recs + (ch & 1) * 2 * TC_C, *br = gam + TC_C;
      const float gi = gam[i], bi = br[i];
      unsigned lost = 0;  // columns where the state's gradient is not finite and ends in this chunk
      float kept[NC];  // z (K's steps) or o (Q's), in fp32
      if (!a.maps) {
        const float4* f = (const float4*)((quad < 2 ? a.zf : a.of) + tile * 64 * BV) + (size_t)half * (NC / 4) * 64 + i;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 x = __ldcs(f + (c / 4) * 64);
          kept[c] = x.x, kept[c + 1] = x.y, kept[c + 2] = x.z, kept[c + 3] = x.w;
        }
      }
      if (quad >= 2) {
        const float f = gi * a.scale;
        float d[NC], s[4] = {};
#pragma unroll
        for (int c = 0; c < NC; c += 8) widen8(*(const uint4*)(OS + img<RB>(i, (c0 + c) >> 3)), d + c);
        if (!a.maps)
#pragma unroll
          for (int c = 0; c < NC; ++c) s[c & 3] = fmaf(d[c], kept[c], s[c & 3]);
#pragma unroll
        for (int c = 0; c < NC; ++c) d[c] = gi != 0.0f ? f * d[c] : 0.0f;
        put_planes<RB, NC>(GS, L::GPLANE, 64 + i, c0, d);
        if (!a.maps) a.dots[((tile * 3 + 2) * 2 + half) * TC_C + i] = i < tc_live(a, b, ch) ? (s[0] + s[1]) + (s[2] + s[3]) : 0.0f;
      }
      take();
      if (quad < 2) {
        float x[NC];
        tm_sum<NC, BV>(x, row + D1 + c0);
#pragma unroll
        for (int c = 0; c < NC; ++c) x[c] = has_part(bi) ? bi * x[c] : 0.0f;  // no part of it before a later document
        if (!has_part(gam[TC_C - 1]))  // as the forward's Y
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (!isfinite(x[c])) {
              x[c] = 0.0f;
              lost |= 1u << c;
            }
        put_planes<RB, NC>(GS, L::GPLANE, i, c0, x);
      }
      leave();  // 2: W's planes are there
      take();
      float y[NC];
      if (quad < 2) {
        tm_sum<NC, BV>(y, row + D2 + c0);
        if (lost)  // its dY are no numbers
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (lost >> c & 1) y[c] = nanf("");
        float g[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) g[c] = has_part(gi) ? -gi * y[c] : 0.0f;
        put_planes<RB, NC>(GS, L::GPLANE, i, c0, g);
      }
      leave();  // 3: -gam dY's planes are there, dO is read, V is there
      if (quad < 2 && !a.maps) {  // what leaves for memory goes while the product runs
        float zy[4] = {}, vy[4] = {};
        if (i >= tc_live(a, b, ch))  // also where the state or its gradient is not finite
#pragma unroll
          for (int c = 0; c < NC; ++c) y[c] = 0.0f;
        uint4* low = (uint4*)(a.dYl + tile * 64 * BV) + (size_t)half * (NC / 8) * 64 + i;
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          uint4* at = (uint4*)(VS + img<RB>(i, (c0 + c) >> 3));
          uint4 p[3];
          float v[8];
          widen8(*at, v);
          split8(y + c, p);
          *at = p[0];
          low[(c / 8) * 64] = p[1];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            zy[e & 3] = fmaf(kept[c + e], y[c + e], zy[e & 3]);
            vy[e & 3] = fmaf(v[e], y[c + e], vy[e & 3]);
          }
        }
        a.dots[((tile * 3 + 0) * 2 + half) * TC_C + i] = (zy[0] + zy[1]) + (zy[2] + zy[3]);
        a.dots[((tile * 3 + 1) * 2 + half) * TC_C + i] = -((vy[0] + vy[1]) + (vy[2] + vy[3]));
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
      leave();  // 4: the products are over, dY's image is there
      if (more) put_state();
      if (ch > 0 && ch % TC_EDGE == 0 && !a.maps) put_edge(ch / TC_EDGE);
    }
    if (a.maps) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 128 + quad * 32 + lane;
        float* s = a.Ht + (((size_t)bn * a.segs + seg) * a.nvt * BV + v0) * KR + r;
#pragma unroll
        for (int c = 0; c < NC; ++c) s[(size_t)c * KR] = r < a.KP ? S[mt][c] : 0.0f;
      }
    } else if (a.ds0 && seg == 0) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = mt * 128 + quad * 32 + lane;
        if (r < a.Dk) {
          float* s = a.ds0 + ((size_t)bn * a.Dk + r) * a.Dv + v0;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < valid) s[c] = S[mt][c];
        }
      }
    }
  }
  if (!a.maps && seg == a.segs - 1) tc_zero_tail<BV>((bf16*)a.dv + vat, vstride, nch * TC_C, a.T, vt * BV, a.Dv);
  tm_fence_before();
  __syncthreads();
  if (warp == 0) tm_free<512>(tm);
}

// ---- grad ----------------------------------------------------------------------------
// TMEM: two accumulators of KT columns; the second one's hold N and F before.
template <int KT, int BV> struct TcGrad {  // KT: Dk rounded up to 128 or 256
  static constexpr int RB = 2 * BV;
  static constexpr int KQ = KT / 64 * TC_PANEL, SB = KT * RB;  // bytes of KQ and of a plane of a tile of S0
  // a tile of X = [dY; dO], of Z's two planes and of dY's second
  static constexpr int AT_Z = 128 * RB, AT_L = AT_Z + 128 * RB, XZ = AT_L + 64 * RB;
  // planes of tiles of S0 and dS1 at once; one where two CTAs an SM fit then
  static constexpr int STAGES = KT == 128 && BV == 64 ? 1 : 2;
  static constexpr int SD = STAGES * 2 * SB > 2 * TC_PANEL ? STAGES * 2 * SB : 2 * TC_PANEL;
  // what reaches over a step: E's columns by warps' rows, G and H by halves, E's rows
  static constexpr int NEAR_E = 0, NEAR_G = 4 * 64, NEAR_H = NEAR_G + 2 * 128, NEAR_T = NEAR_H + 2 * 64, NEAR = (NEAR_T + 2 * 32) * 4;
  static constexpr int LATE = KQ + 2 * TC_PANEL + NEAR;  // what X's and Z's place holds when they are done with
  static __host__ __device__ constexpr int at_sd(int nvt) { return nvt * XZ > LATE ? nvt * XZ : (LATE + 1023) & ~1023; }
  static __host__ __device__ constexpr size_t bytes(int nvt) { return (size_t)at_sd(nvt) + SD + 3 * TC_C * 4 + TC_C + 64; }
  static constexpr int COLS = KT == 128 ? 256 : 512;
};
static_assert(2 * (TcGrad<128, 64>::bytes(2) + 1024) <= 228 * 1024, "two CTAs an SM for heads of 128 channels");
static_assert(TcGrad<128, 64>::bytes(4) <= 227 * 1024 && TcGrad<128, 32>::bytes(8) <= 227 * 1024 && TcGrad<256, 32>::bytes(8) <= 227 * 1024, "fits");

// X and Z stay in shared memory, S0 and dS1 pass by planes of tiles of BV columns
// of v. N and F go to registers, M and R are made from them while the state's
// products run, and multiply KQ: their first planes from the buffers of S0 and
// dS1, their second from behind KQ, which has X's and Z's place. The products of
// 64 rows (Z's, dY's second plane) read as many rows behind them: Z's results
// there are not looked at, dY's are not written, since dO's stand there.
// Where a step is below GATE_NEAR, the rows of the state's parts times K's and Q's,
// and K K^T and Q K^T times M and R, give what reaches over each step of the chunk.
// Measured 273 us at the chain's size, where its 1.14 GB take 168: an item waits
// for its loads, two CTAs an SM cover half of it. Single buffers for the planes,
// two in flight, took 353 us (of 324 then: the issuing thread waits in turn).
template <int KT, int BV> __global__ void __launch_bounds__(256, KT == 128 ? 2 : 1) delta_tc_grad_kernel(DeltaTcArgs a) {
  using L = TcGrad<KT, BV>;
  constexpr int RB = L::RB;
  extern __shared__ __align__(1024) unsigned char sm_grad[];
  unsigned char *X = sm_grad, *KQ = sm_grad, *SD = sm_grad + L::at_sd(a.nvt), *ML = KQ + L::KQ;
  float* rec = (float*)(SD + L::SD);  // chi, clo, beta
  const float* beta = rec + 2 * TC_C;
  unsigned char* segs = (unsigned char*)(rec + 3 * TC_C);
  uint64_t* barp = (uint64_t*)(segs + TC_C);
  uint32_t* slot = (uint32_t*)(barp + 5);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
  const long long item = blockIdx.x;
  const int ch = (int)(item % a.nc), bn = (int)(item / a.nc), n = bn % a.N, b = bn / a.N, nk = n / (a.N / a.Nk);
  const int live = tc_live(a, b, ch), steps = min(TC_C, a.T - ch * TC_C);
  const size_t kstride = (size_t)a.Nk * a.Dk, vstride = (size_t)a.N * a.Dv, row0 = (size_t)b * a.T + (size_t)ch * TC_C;
  const size_t kat = row0 * kstride + (size_t)nk * a.Dk, vat = row0 * vstride + (size_t)n * a.Dv;
  const bool shared_heads = a.pq != nullptr;
  const size_t pstride = (size_t)a.N * a.Dk, pat = row0 * pstride + (size_t)n * a.Dk;
  if (live == 0) {  // nothing of the chunk exists
    for (int i = tid; i < steps * a.Dk; i += 256) {
      const int r = i / a.Dk, c = i % a.Dk;
      if (shared_heads) a.pq[pat + r * pstride + c] = a.pk[pat + r * pstride + c] = 0.0f;
      else ((bf16*)a.dq)[kat + r * kstride + c] = ((bf16*)a.dk)[kat + r * kstride + c] = __float2bfloat16_rn(0.0f);
    }
    return;
  }
  const uint32_t bar = smem_u32(barp), bar_end = bar + 8, bar_s = bar + 16, bar_m = bar + 32;  // bar_s: by stage
  if (tid == 0) {
    for (int k = 0; k < 5; ++k) mbar_init(bar + 8 * k, 1);
    fence_mbar_init_cluster();
  }
  auto load_sd = [&](int p) {  // plane p % 2 of tile p / 2; one thread
    const size_t at = ((size_t)item * a.nvt * 2 + p) * a.KP * BV;
    const uint32_t bytes = a.KP * RB, to = smem_u32(SD + (p % L::STAGES) * 2 * L::SB), br = bar_s + 8 * (p % L::STAGES);
    mbar_arrive_expect_tx(br, 2 * bytes);
    bulk_load_global(to, a.Sh + at, bytes, br);
    bulk_load_global(to + L::SB, a.dSh + at, bytes, br);
  };
  if (tid == 0) {
    load_sd(0);
    if (L::STAGES == 2) load_sd(1);
  }
  constexpr int UN = 64 * (BV / 8) / 256;  // pieces of 8 columns of a step that a thread has of a tile
  float4 z[UN][2];
  auto fetch = [&](int p) {
    const float4* f = (const float4*)(a.zf + ((size_t)item * a.nvt + p) * 64 * BV) + (tid >> 6) * 128 + (tid & 63);
#pragma unroll
    for (int u = 0; u < UN; ++u) z[u][0] = __ldcs(f + u * 512), z[u][1] = __ldcs(f + u * 512 + 64);
  };
  fetch(0);
  const float* own = a.rec + (size_t)item * REC_N * TC_C;
  const int i = (quad & 1) * 32 + lane, j0 = half * 32;  // this thread's step and columns of M and R
  const float gi = own[REC_GAM * TC_C + i], bri = own[REC_BR * TC_C + i];
  const bool near = own[REC_NEAR * TC_C] != 0.0f;  // the chunk's gates want what reaches over a step
  for (int p = 0; p < a.nvt; ++p) {
    unsigned char* x = X + p * L::XZ;
    load_img<RB, BV / 8, 256>(tid, x, 0, (const bf16*)a.dv + vat, vstride, live, a.Dv, p * BV, BV, 0);
    load_img<RB, BV / 8, 256>(tid, x, 64, (const bf16*)(a.dO ? a.dO : a.dv) + vat, vstride, a.dO ? live : 0, a.Dv, p * BV, BV, 0);
    const bf16* low = a.dYl + (((size_t)item * a.nvt + p) * 64 * (BV / 8) + tid) * 8;
#pragma unroll
    for (int u = 0; u < UN; ++u) cp16(smem_u32(x + L::AT_L) + img<RB>(tid & 63, (tid >> 6) + 4 * u), low + u * 2048, (tid & 63) < live);
    uint4 q[UN][3];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const float zs[8] = {z[u][0].x, z[u][0].y, z[u][0].z, z[u][0].w, z[u][1].x, z[u][1].y, z[u][1].z, z[u][1].w};
      split8(zs, q[u]);
    }
    if (p + 1 < a.nvt) fetch(p + 1);
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) *(uint4*)(x + L::AT_Z + k * 64 * RB + img<RB>(tid & 63, (tid >> 6) + 4 * u)) = q[u][k];
  }
  cp_commit();
  if (tid < TC_C) {
    rec[tid] = own[REC_CHI * TC_C + tid];
    rec[TC_C + tid] = own[REC_CLO * TC_C + tid];
    rec[2 * TC_C + tid] = own[REC_BETA * TC_C + tid];
    segs[tid] = (unsigned char)__float_as_int(own[REC_SEG * TC_C + tid]);  // 0 .. 64
  }
  {  // K and Q, which come last, on their way to the L2
    const bf16* s = (const bf16*)(tid < 128 ? a.k : a.q) + kat + (size_t)((tid & 127) >> 1) * kstride;
    if ((tid & 127) >> 1 < live)
      for (int c = (tid & 1) * 64; c < a.Dk; c += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(s + c));
  }
  if (warp == 0) tm_alloc<L::COLS>(slot);
  cp_wait_all();
  fence_proxy_async_smem();
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *slot, row = tm + ((uint32_t)(quad * 32) << 16);
  uint32_t parity = 0;
  bool failed = false;
  auto wait = [&](uint32_t which, uint32_t par) { mbar_wait_bounded<false>(which, par, a.wait_limit_ns, a.status, failed); };
  auto take = [&]() {
    wait(bar, parity);
    parity ^= 1;
    tm_fence_after();
  };
  constexpr uint64_t XZ = L::AT_Z >> 4, XL = L::AT_L >> 4, PZ = 64 * RB >> 4;  // in descriptors: Z, dY's second plane, from plane to plane of Z
  // the state's products with plane p % 2 of tile p / 2
  auto state = [&](int p) {
    wait(bar_s + 8 * (p % L::STAGES), (p / L::STAGES) & 1);
    if (failed) return;
    const uint32_t id = tc_idesc(a.KP, false, false);
    const uint64_t x = tc_desc<RB>(smem_u32(X) + (p >> 1) * L::XZ, 16), s = tc_desc<RB>(smem_u32(SD) + (p % L::STAGES) * 2 * L::SB, 16);
    const uint64_t ds = s + (L::SB >> 4);
#pragma unroll
    for (int k = 0; k < BV / 16; ++k) tc_mma(tm, x + 2 * k, s + 2 * k, id, p || k);  // [dY; dO] S0^T
#pragma unroll
    for (int k = 0; k < BV / 16; ++k) tc_mma(tm + KT, x + XZ + 2 * k, ds + 2 * k, id, p || k);  // Z dS1^T (rows 0 .. 63)
    if (!(p & 1)) {
#pragma unroll
      for (int k = 0; k < BV / 16; ++k) tc_mma_upper(tm, x + XL + 2 * k, s + 2 * k, id, true);
#pragma unroll
      for (int k = 0; k < BV / 16; ++k) tc_mma(tm + KT, x + XZ + PZ + 2 * k, ds + 2 * k, id, true);
    }
    tc_commit(p + 1 < 2 * a.nvt ? bar_m : bar);  // the CTA waits for the last tile's alone
  };
  if (tid == 0) {  // [N; F] = X Z^T, in the second accumulator's columns
    constexpr uint32_t id = tc_idesc(64, false, false);
    for (int p = 0; p < a.nvt; ++p) {
      const uint64_t x = tc_desc<RB>(smem_u32(X) + p * L::XZ, 16);
#pragma unroll
      for (int k = 0; k < BV / 16; ++k) tc_mma(tm + KT, x + 2 * k, x + XZ + 2 * k, id, p || k);
#pragma unroll
      for (int k = 0; k < BV / 16; ++k) tc_mma(tm + KT, x + 2 * k, x + XZ + PZ + 2 * k, id, true);
#pragma unroll
      for (int k = 0; k < BV / 16; ++k) tc_mma_upper(tm + KT, x + XL + 2 * k, x + XZ + 2 * k, id, true);
    }
    tc_commit(bar);
  }
  take();
  float nf[32];
  {
    uint32_t r[32];
    tm_ld16(r, row + KT + j0);
    tm_ld16(r + 16, row + KT + j0 + 16);
    tm_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; ++c) nf[c] = __uint_as_float(r[c]);
  }
  tm_fence_before();
  __syncthreads();
  if (tid == 0 && !failed) {
    tm_fence_after();
    state(0);
  }
  {  // R_ij (Q's steps) or M_ij (K's), i the thread's step
    const float ci = rec[i], li = rec[TC_C + i];
    const int si = segs[i];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const int j = j0 + c;
      const bool on = (quad < 2 ? i > j : i >= j) && si == segs[j];
      nf[c] = on ? (quad < 2 ? -nf[c] : a.scale * nf[c]) * exp2_fast((ci - rec[j]) + (li - rec[TC_C + j])) * beta[j] : 0.0f;
    }
  }
  if (tid == 0)
    for (int p = 1; p < 2 * a.nvt && !failed; ++p) {
      wait(bar_m, (p - 1) & 1);  // before the next commit: the barrier's parity tells two phases apart
      if (L::STAGES == 1) load_sd(p);
      else if (p + 1 < 2 * a.nvt) load_sd(p + 1);
      state(p);
    }
  take();
  // X and Z are done with
  load_img<128, KT / 8, 256>(tid, KQ, 0, (const bf16*)a.k + kat, kstride, live, a.Dk, 0, (a.KP + 63) & ~63, TC_PANEL);
  load_img<128, KT / 8, 256>(tid, KQ, 64, (const bf16*)a.q + kat, kstride, live, a.Dk, 0, (a.KP + 63) & ~63, TC_PANEL);
  cp_commit();
  // [M + M^T, R^T; R, 0], two panels of 128 rows: the first plane over the buffers
  // of S0 and dS1, the second behind KQ. Rows first (M's hold zeros past the
  // diagonal), then what is transposed: its 2-byte stores are of one row a warp.
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    uint4 p[3];
    split8(nf + c, p);
    const uint32_t at = img<128>(quad * 32 + lane, (j0 + c) >> 3);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      unsigned char* to = k ? ML : SD;
      *(uint4*)(to + at) = p[k];
      if (quad >= 2) *(uint4*)(to + TC_PANEL + at) = make_uint4(0, 0, 0, 0);
    }
  }
  if (quad < 2) asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const int j = j0 + c;
    const uint32_t at = (quad < 2 ? 0 : TC_PANEL) + img<128>(j, i >> 3) + (i & 7) * 2;
    const bf16 hi = __float2bfloat16_rn(nf[c]);
    if (quad >= 2 || j < i) {
      *(bf16*)(SD + at) = hi;
      *(bf16*)(ML + at) = __float2bfloat16_rn(nf[c] - __bfloat162float(hi));
    }
  }
  if (near) {  // K's and Q's rows are looked at
    cp_wait_all();
    __syncthreads();
  }
  // The state's parts, scaled by rows in fp32, back into the first accumulator; with
  // the row itself they make G and H
  const float f0 = quad < 2 ? -gi : a.scale * gi, f1 = quad < 2 ? bri : 0.0f;
  float gsum = 0.0f, hsum = 0.0f;
  for (int c = half * 16; c < a.KP; c += 32) {
    uint32_t x[16], h[16];
    tm_ld16(x, row + c);
    tm_ld16(h, row + KT + c);
    tm_wait_ld();
    if (near) {
      const unsigned char* im = KQ + (c >> 6) * TC_PANEL;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float k[8];
        widen8(*(const uint4*)(im + img<128>(quad * 32 + lane, ((c & 63) >> 3) + u)), k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (has_part(gi)) gsum = fmaf(k[e], f0 * __uint_as_float(x[u * 8 + e]), gsum);
          if (has_part(f1)) hsum = fmaf(k[e], f1 * __uint_as_float(h[u * 8 + e]), hsum);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float s = has_part(gi) ? f0 * __uint_as_float(x[e]) : 0.0f;
      if (has_part(f1)) s = fmaf(f1, __uint_as_float(h[e]), s);
      x[e] = __float_as_uint(s);
    }
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(row + c),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
        "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
        : "memory");
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
  cp_wait_all();
  fence_proxy_async_smem();
  tm_fence_before();
  __syncthreads();
  if (tid == 0 && !failed) {
    tm_fence_after();
    const uint32_t id = tc_idesc(a.KP, false, true);
    const uint64_t m = tc_desc(smem_u32(SD), 16), ml = tc_desc(smem_u32(ML), 16), k0 = tc_desc(smem_u32(KQ), TC_PANEL);
#pragma unroll
    for (int k = 0; k < 8; ++k) tc_mma(tm, m + (k >> 2) * (TC_PANEL >> 4) + (k & 3) * 2, k0 + k * 128, id, true);
#pragma unroll
    for (int k = 0; k < 8; ++k) tc_mma(tm, ml + (k >> 2) * (TC_PANEL >> 4) + (k & 3) * 2, k0 + k * 128, id, true);
    if (near) {  // [K K^T; Q K^T], in the second accumulator's columns
      const uint64_t kq = tc_desc(smem_u32(KQ), 16);
      for (int k = 0; k < (a.KP + 63) >> 6 << 2; ++k) {
        const uint64_t at = kq + (k >> 2) * (TC_PANEL >> 4) + (k & 3) * 2;
        tc_mma(tm + KT, at, at, tc_idesc(64, false, false), k);
      }
    }
    tc_commit(bar);
  }
  take();
  if (near) {
    // E_ij = M_ij k_i.k_j + R_ij q_i.k_j, j < i, from M's and R's planes; a thread has
    // 32 columns of a row. Summed along the row up to t - 1, then over the rows from t
    // on, it reaches over t.
    float* sums = (float*)(ML + 2 * TC_PANEL);
    float e[32];
    {
      uint32_t r[32];
      tm_ld16(r, row + KT + j0);
      tm_ld16(r + 16, row + KT + j0 + 16);
      tm_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        const uint32_t at = img<128>(quad * 32 + lane, (j0 + c) >> 3);
        float hi[8], lo[8];
        widen8(*(const uint4*)(SD + at), hi);
        widen8(*(const uint4*)(ML + at), lo);
#pragma unroll
        for (int k = 0; k < 8; ++k) e[c + k] = j0 + c + k < i ? (hi[k] + lo[k]) * __uint_as_float(r[c + k]) : 0.0f;
      }
    }
#pragma unroll
    for (int c = 1; c < 32; ++c) e[c] += e[c - 1];
    float rest = e[31];  // of the row's first half: reaches over all of the second's steps up to i
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (j0 + c + 1 > i) e[c] = 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)  // the warp's rows: lane l keeps column l
#pragma unroll
      for (int c = 0; c < o; ++c) {
        const bool up = lane & o;
        const float keep = up ? e[c + o] : e[c], give = up ? e[c] : e[c + o];
        e[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    sums[L::NEAR_E + quad * 64 + j0 + lane] = e[0];  // over t = j0 + lane + 1
    if (half == 0 && (quad & 1)) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, rest, o);
        if (lane + o < 32) rest += x;
      }
      sums[L::NEAR_T + (quad >> 1) * 32 + lane] = rest;
    }
    sums[L::NEAR_G + half * 128 + quad * 32 + lane] = gsum;
    if (quad < 2) sums[L::NEAR_H + half * 64 + i] = hsum;
    __syncthreads();
    if (warp == 0) {  // steps lane and 32 + lane
      const float *E = sums + L::NEAR_E + lane, *G = sums + L::NEAR_G + lane, *H = sums + L::NEAR_H + lane, *T = sums + L::NEAR_T + lane;
      float g[2], h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        g[u] = (G[32 * u] + G[128 + 32 * u]) + (G[64 + 32 * u] + G[192 + 32 * u]);
        h[u] = H[32 * u] + H[64 + 32 * u];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = __shfl_down_sync(0xffffffffu, g[u], o), y = __shfl_up_sync(0xffffffffu, h[u], o);
          if (lane + o < 32) g[u] += x;
          if (lane >= o) h[u] += y;
        }
      }
      g[0] += __shfl_sync(0xffffffffu, g[1], 0);
      const float h31 = __shfl_sync(0xffffffffu, h[0], 31);
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // of the steps before
        h[u] = __shfl_up_sync(0xffffffffu, h[u], 1);
        if (lane == 0) h[u] = 0.0f;
      }
      float* to = a.near + (size_t)item * TC_C + lane;
      to[0] = g[0] + h[0] + (lane ? (E[-1] + E[63]) + (E[127] + E[191]) : 0.0f);
      to[32] = g[1] + (h[1] + h31) + ((E[31] + E[95]) + (E[159] + E[223])) + (lane ? T[0] + T[32] : 0.0f);
    }
  }
  if (shared_heads) {
    for (int c = half * 16; c < a.KP; c += 32) {
      uint32_t r[16];
      tm_ld16(r, row + c);
      tm_wait_ld();
      if (i < steps) {
        float* p = (quad < 2 ? a.pk : a.pq) + pat + (size_t)i * pstride + c;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < a.Dk - c) p[e] = i < live ? __uint_as_float(r[e]) : 0.0f;
      }
      __syncwarp();
    }
  } else {  // dK and dQ by way of KQ's image, so that rows leave whole
    for (int c = half * 16; c < a.KP; c += 32) {
      uint32_t r[16];
      tm_ld16(r, row + c);
      tm_wait_ld();
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = i < live ? __uint_as_float(r[e]) : 0.0f;
      unsigned char* d = KQ + (c >> 6) * TC_PANEL;
      *(uint4*)(d + img<128>(quad * 32 + lane, (c & 63) >> 3)) = round8(x);
      *(uint4*)(d + img<128>(quad * 32 + lane, ((c & 63) >> 3) + 1)) = round8(x + 8);
    }
    __syncthreads();
    for (int c = 0; c < a.Dk; c += 64) {
      store_img<128, 256>(tid, KQ + (c >> 6) * TC_PANEL, (bf16*)a.dk + kat, kstride, steps, a.Dk, c);
      store_img<128, 256>(tid, KQ + (c >> 6) * TC_PANEL + 64 * 128, (bf16*)a.dq + kat, kstride, steps, a.Dk, c);
    }
  }
  if (tid == 0 && failed) {  // copies that nobody waited for land before the CTA ends
    for (int k = 0; k < L::STAGES; ++k)
      for (int q = 0; q < 2; ++q) {
        bool f = false;
        mbar_wait_bounded<false>(bar_s + 8 * k, q, a.wait_limit_ns, nullptr, f);
      }
  }
  tc_finish(bar_end, a.wait_limit_ns);
  if (warp == 0) tm_free<L::COLS>(tm);
}

// ---- gates ---------------------------------------------------------------------------
// dg and dbeta of TC_EDGE chunks: a thread has a step, sums its document's dc to
// the chunk's end (and no other's, which may not be finite), and what lies beyond
// comes from chunk to chunk after that. The sums run in 64 bits: dc's signs change,
// and where memories are short a sum of hundreds of them is small beside what it
// passes through (21 us at the chain's size, 12 in 32 bits, which are twice as far
// off). How far dc's own rounding carries is at GATE_NEAR; steps below it have their
// dg from the grad kernel and the back chain.
__global__ void __launch_bounds__(TC_EDGE * TC_C) delta_tc_gates_kernel(DeltaTcArgs a) {
  __shared__ double tail[TC_EDGE], from[TC_EDGE], after[TC_EDGE];
  __shared__ int tseg[TC_EDGE];
  __shared__ float es[32];
  __shared__ unsigned marks[TC_EDGE][2];
  const int groups = (a.nc + TC_EDGE - 1) / TC_EDGE, k = threadIdx.x / TC_C, i = threadIdx.x % TC_C, lane = threadIdx.x & 31;
  const int bn = blockIdx.x / groups, gr = blockIdx.x % groups, n = bn % a.N, b = bn / a.N;
  const int nch = tc_chunks(a, b), lo = gr * TC_EDGE, ch = lo + k;
  const int live = ch < a.nc ? tc_live(a, b, ch) : 0;
  const size_t item = (size_t)bn * a.nc + ch;
  const float* rec = a.rec + item * REC_N * TC_C;
  float zy = 0.0f, bt = 1.0f;
  bool near = false;
  int seg = 0;
  double c = 0.0;
  bool mark = false;  // the first step of a document
  if (live > 0) {
#pragma unroll 2
    for (int vt = 0; vt < a.nvt; ++vt) {
      const float* d = a.dots + (item * a.nvt + vt) * 6 * TC_C;
      zy += d[i] + d[TC_C + i];
      c += ((double)d[2 * TC_C + i] + d[3 * TC_C + i]) + ((double)d[4 * TC_C + i] + d[5 * TC_C + i]);
    }
    bt = rec[REC_BETA * TC_C + i];
    near = rec[REC_NEAR * TC_C + i] == 2.0f;
    seg = __float_as_int(rec[REC_SEG * TC_C + i]);
    mark = seg != (i ? __float_as_int(rec[REC_SEG * TC_C + i - 1]) : 0);
  }
  const unsigned m = __ballot_sync(0xffffffffu, mark);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_down_sync(0xffffffffu, c, o);
    const int sx = __shfl_down_sync(0xffffffffu, seg, o);
    if (lane + o < 32 && sx == seg) c += x;
  }
  if (i == 32) tail[k] = c, tseg[k] = seg;  // the second half's first document
  if (lane == 0) marks[k][i >> 5] = m;
  if (threadIdx.x < 32) {  // <S, dS> at the group's end: a lane has every 32nd part
    const int at = lo + TC_EDGE >= nch ? 0 : gr + 1;
    float e = 0.0f;
    if (lo < nch)
      for (int w = threadIdx.x; w < a.nvt * 8; w += 32) e += a.edge[((size_t)bn * a.ne + at) * a.nvt * 8 + w];
    es[threadIdx.x] = e;
  }
  __syncthreads();
  const unsigned long long starts = (unsigned long long)marks[k][1] << 32 | marks[k][0], later = starts >> i >> 1;
  double s = i < 32 && tseg[k] == seg ? c + tail[k] : c;  // the document's steps from here on
  if (i == 0) from[k] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double e = 0.0;
    for (int w = 0; w < 32; ++w) e += es[w];
    for (int q = min(TC_EDGE, nch - lo) - 1; q >= 0; --q) {
      after[q] = e;
      // a chunk that begins a document needs nothing before it
      e = marks[q][0] & 1 ? 0.0 : from[q] + (marks[q][0] | marks[q][1] ? 0.0 : e);
    }
  }
  __syncthreads();
  if (ch >= a.nc || ch * TC_C + i >= a.T) return;
  const size_t out = ((size_t)b * a.T + (size_t)ch * TC_C + i) * a.N + n;
  if (i < live && !later) s += after[k];
  if (near) {
    s = a.near[item * TC_C + i];
    const float gC = rec[REC_GAM * TC_C + TC_C - 1];
    if (has_part(gC))
      for (int w = 0; w < a.nvt * 3; ++w) s += gC * a.cross[item * a.nvt * 3 + w];
  }
  a.dg[out] = i < live && !mark ? (float)s : 0.0f;
  a.dbeta[out] = i < live ? zy / bt : 0.0f;
}

// dq, dk [rows, Nk, Dk] = sums of pq, pk [rows, Nk, share, Dk], in the heads' order
__global__ void __launch_bounds__(256) delta_tc_share_kernel(const float* pq, const float* pk, bf16* dq, bf16* dk, long long n,
                                                             int share, int Dk) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = i / Dk;
    const size_t at = (size_t)r * share * Dk + (size_t)(i - r * Dk);
    float x = 0.0f, y = 0.0f;
    for (int s = 0; s < share; ++s) {
      x += pq[at + (size_t)s * Dk];
      y += pk[at + (size_t)s * Dk];
    }
    dq[i] = __float2bfloat16_rn(x);
    dk[i] = __float2bfloat16_rn(y);
  }
}

template <int BV, int MT> cudaError_t back(DeltaTcArgs a, const TcMaps& maps, cudaStream_t st) {
  constexpr int sm = TcBack<BV, MT>::BYTES;
  cudaError_t e = set_smem_attr((const void*)delta_tc_back_kernel<BV, MT>, sm);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(a.B * a.N * a.segs * a.nvt);
  if (a.segs > 1) {
    a.maps = 1;
    delta_tc_back_kernel<BV, MT><<<grid, 384, sm, st>>>(a, maps);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = delta_tc_join_back(BV, a, st)) != cudaSuccess) return e;
    a.maps = 0;
  }
  delta_tc_back_kernel<BV, MT><<<grid, 384, sm, st>>>(a, maps);
  note_launch();
  return cudaGetLastError();
}
template <int KT, int BV> cudaError_t grad(const DeltaTcArgs& a, cudaStream_t st) {
  const size_t sm = TcGrad<KT, BV>::bytes(a.nvt);
  cudaError_t e = set_smem_attr((const void*)delta_tc_grad_kernel<KT, BV>, sm);
  if (e != cudaSuccess) return e;
  delta_tc_grad_kernel<KT, BV><<<(unsigned)((long long)a.B * a.N * a.nc), 256, sm, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_tc_bwd_launch(int BV, const DeltaTcArgs& a, cudaStream_t st) {
  TcMaps maps;
  DeltaTcArgs x = a;
  cudaError_t e;
  int dev = 0;  // a thread of autograd's makes its first call here, perhaps: the maps' encoding wants a context
  if ((e = cudaGetDevice(&dev)) != cudaSuccess || (e = cudaSetDevice(dev)) != cudaSuccess) return e;
  x.tma = a.Dk % 8 == 0 && a.Dv % 8 == 0;
  if (x.tma && ((e = tc_map(&maps.k, a.k, a, a.Nk, a.Dk, 64)) != cudaSuccess || (e = tc_map(&maps.q, a.q, a, a.Nk, a.Dk, 64)) != cudaSuccess ||
                (e = tc_map(&maps.v, a.v, a, a.N, a.Dv, BV)) != cudaSuccess || (e = tc_map(&maps.dv, a.dv, a, a.N, a.Dv, BV)) != cudaSuccess ||
                (a.dO && (e = tc_map(&maps.dO, a.dO, a, a.N, a.Dv, BV)) != cudaSuccess)))
    return e;
  e = a.KP > 128 ? back<32, 2>(x, maps, st) : BV == 64 ? back<64, 1>(x, maps, st) : back<32, 1>(x, maps, st);
  if (e != cudaSuccess) return e;
  if ((e = a.KP > 128 ? grad<256, 32>(a, st) : BV == 64 ? grad<128, 64>(a, st) : grad<128, 32>(a, st)) != cudaSuccess) return e;
  const int groups = (a.nc + TC_EDGE - 1) / TC_EDGE;
  delta_tc_gates_kernel<<<(unsigned)(a.B * a.N * groups), TC_EDGE * TC_C, 0, st>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess || !a.pq) return e;
  const long long n = (long long)a.B * a.T * a.Nk * a.Dk, blocks = (n + 255) / 256, most = 16LL * device_sms();
  delta_tc_share_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(a.pq, a.pk, (bf16*)a.dq, (bf16*)a.dk, n,
                                                                                a.N / a.Nk, a.Dk);
  note_launch();
  return cudaGetLastError();
}

}  // namespace rnn
