// Gated delta rule, forward: three kernels (the formulas are in delta.cuh).
//   prep   every chunk by itself: Tm, P and the per-step factors
//   chain  per head and tile of BV columns, the chunks one after the other:
//          Y, Z and the state; it leaves every chunk's starting state and Z
//   out    every chunk by itself: O
// Measured 13 + 56 + 10 us at B=3 T=515, 6 heads of 40 x 72: 54 CTAs walk 17 chunks
// of 3.3 us each; six products for one on mma.sync, loads that split into planes.
#include "delta.h"
#include "kernels.cuh"

namespace rnn {
namespace {

// ---- prep --------------------------------------------------------------------------
struct PrepSmem {
  static constexpr int C = F32_C, NP = F32_NP;
  static __host__ __device__ size_t bytes(int DKP) {
    return (size_t)2 * NP * C * (DKP + 8) * 2 + (size_t)C * (C + 4) * 4 + REC_N * C * 4;
  }
};

// A warp takes 16 rows of K K^T and Q K^T; Tm by forward substitution, a column
// to a thread with its values in registers.
__global__ void __launch_bounds__(2 * F32_C) delta_prep_kernel(DeltaArgs a) {
  constexpr int C = F32_C, NP = F32_NP, NT = C / 8;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  const int LDK = a.DKP + 8, kplane = C * LDK;
  bf16* Ks = (bf16*)sm_raw;
  bf16* Qs = Ks + NP * kplane;
  float* Lf = (float*)(Qs + NP * kplane);  // [C][C + 4]
  float* rec = Lf + C * (C + 4);           // [REC_N][C]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long item = blockIdx.x;
  if (item == 0 && tid == 0) *a.status = 0;  // no kernel of fp32 storage waits for another
  const int ch = (int)(item % a.nc), bn = (int)(item / a.nc), n = bn % a.N, b = bn / a.N;
  const int live = live_steps(a, b, ch, C);
  if (live == 0) return;
  const int nk = n / (a.N / a.Nk);
  const size_t stride = (size_t)a.Nk * a.Dk, at = ((size_t)b * a.T + (size_t)ch * C) * stride + (size_t)nk * a.Dk;
  load_rows<float, C>(Ks, LDK, kplane, (const float*)a.k + at, stride, live, a.Dk, 0, a.DKP);
  load_rows<float, C>(Qs, LDK, kplane, (const float*)a.q + at, stride, live, a.Dk, 0, a.DKP);
  cp_commit();
  if (warp == 0) {  // the running sum of g, in 64 bits, and the documents
    static_assert(C == 32, "a lane a step");
    float g = 0.0f, be = 0.0f;
    bool mark = false;
    if (lane < live) {
      const size_t s = ((size_t)b * a.T + (size_t)ch * C + lane) * a.N + n;
      g = a.g[s];
      be = a.beta[s];
      mark = a.reset && a.reset[(size_t)b * a.T + (size_t)ch * C + lane];
      if (g < -104.0f) mark = true;  // exp(g) is 0
      if (mark) g = 0.0f;
    }
    double c = (double)g;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += v;
    }
    const double all = __shfl_sync(0xffffffffu, c, 31);
    const unsigned m = __ballot_sync(0xffffffffu, mark);
    const int seg = __popc(m & (0xffffffffu >> (31 - lane)));
    const bool last = seg == __popc(m);
    const float chi = (float)c, rho = last ? keep_part(expf((float)(all - c))) : 0.0f;
    rec[REC_CHI * C + lane] = chi;
    rec[REC_CLO * C + lane] = (float)(c - (double)chi);
    rec[REC_SEG * C + lane] = __int_as_float(seg);
    rec[REC_GAM * C + lane] = seg == 0 ? keep_part(expf(chi)) : 0.0f;
    rec[REC_RHO * C + lane] = rho;
    rec[REC_BETA * C + lane] = be;
    rec[REC_BR * C + lane] = last ? keep_part(be * rho) : 0.0f;
  }
  cp_wait<0>();
  __syncthreads();
  for (int i = tid; i < REC_N * C; i += 2 * C) a.rec[(size_t)item * REC_N * C + i] = rec[i];
  const Opnd K = opnd(Ks, LDK, kplane), Q = opnd(Qs, LDK, kplane);
  const int m0 = warp * 16;
  float kk[NT][4], qk[NT][4];
  zero(kk);
  zero(qk);
  mma_acc<NT, false, true>(kk, K, m0, K, 0, a.DKP);
  mma_acc<NT, false, true>(qk, Q, m0, K, 0, a.DKP);
  bf16* pm = a.pm + (size_t)item * NP * C * C;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = m0 + (lane >> 2) + 8 * h;
    const float ci = rec[REC_CHI * C + i], li = rec[REC_CLO * C + i];
    const int si = __float_as_int(rec[REC_SEG * C + i]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float p[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = t * 8 + (lane & 3) * 2 + e;
        const bool on = i >= j && si == __float_as_int(rec[REC_SEG * C + j]);
        const float gb = on ? expf((ci - rec[REC_CHI * C + j]) + (li - rec[REC_CLO * C + j])) * rec[REC_BETA * C + j] : 0.0f;
        p[e] = on ? qk[t][2 * h + e] * gb : 0.0f;
        Lf[i * (C + 4) + j] = on && i > j ? kk[t][2 * h + e] * gb : 0.0f;
      }
      split_store(pm + i * C + t * 8 + (lane & 3) * 2, C * C, p[0], p[1]);
    }
  }
  __syncthreads();
  if (tid < C) {
    float x[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float s[4] = {i == tid ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < i; k += 4) {
        const float4 l = *(const float4*)(Lf + i * (C + 4) + k);
        s[0] -= l.x * x[k];
        if (k + 1 < i) s[1] -= l.y * x[k + 1];
        if (k + 2 < i) s[2] -= l.z * x[k + 2];
        if (k + 3 < i) s[3] -= l.w * x[k + 3];
      }
      x[i] = (s[0] + s[1]) + (s[2] + s[3]);
    }
    bf16* tm = a.tm + (size_t)item * NP * C * C;
#pragma unroll
    for (int i = 0; i < C; ++i) split_store1(tm + i * C + tid, C * C, x[i]);
  }
}

// ---- chain --------------------------------------------------------------------------
struct ChainSmem {
  static constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  static __host__ __device__ size_t bytes(int DKP) {
    return 2 * ((size_t)NP * C * (DKP + 8) + (size_t)NP * C * (C + 8) + (size_t)NP * C * (BV + 8) +
                (size_t)NP * DKP * (BV + 8) + (size_t)2 * NP * C * (BV + 8)) +
           2 * 2 * C * 4;
  }
};

// MT: tiles of 16 state rows a warp (1 for Dk <= 128, else 2), in registers.
template <int MT>
__global__ void __launch_bounds__(256, 1) delta_chain_kernel(DeltaArgs a) {
  constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  constexpr int WM = C / 16, WN = 8 / WM, NT = BV / WN / 8, NS = BV / 8, LDV = BV + 8, LDC = C + 8;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  const int DKP = a.DKP, LDK = DKP + 8, kplane = C * LDK;
  bf16* Ks = (bf16*)sm_raw;
  bf16* Ts = Ks + NP * kplane;
  bf16* Vs = Ts + NP * C * LDC;
  bf16* Ss = Vs + NP * C * LDV;
  bf16* Ys = Ss + NP * DKP * LDV;
  bf16* Zs = Ys + NP * C * LDV;
  float* recs = (float*)(Zs + NP * C * LDV);  // [2][gam, br][C]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int vt = blockIdx.x % a.nvt, bn = blockIdx.x / a.nvt, n = bn % a.N, b = bn / a.N, nk = n / (a.N / a.Nk);
  const int nch = live_chunks(a, b, C);
  const size_t kstride = (size_t)a.Nk * a.Dk, vstride = (size_t)a.N * a.Dv;
  const float* kb = (const float*)a.k + (size_t)b * a.T * kstride + (size_t)nk * a.Dk;
  const float* vb = (const float*)a.v + (size_t)b * a.T * vstride + (size_t)n * a.Dv;
  auto load_k = [&](int ch) {
    load_rows<float, C>(Ks, LDK, kplane, kb + (size_t)ch * C * kstride, kstride,
                    live_steps(a, b, ch, C), a.Dk, 0, DKP);
  };
  auto load_v = [&](int ch) {
    load_rows<float, C>(Vs, LDV, C * LDV, vb + (size_t)ch * C * vstride, vstride, live_steps(a, b, ch, C), a.Dv, vt * BV, BV);
    const float* r = a.rec + ((size_t)bn * a.nc + ch) * REC_N * C;
    float* d = recs + (ch & 1) * 2 * C;
    if (tid < C / 4) cp16(smem_u32(d + tid * 4), r + REC_GAM * C + tid * 4, true);
    else if (tid < C / 2) cp16(smem_u32(d + tid * 4), r + REC_BR * C + (tid - C / 4) * 4, true);
  };
  auto load_t = [&](int ch) {
    const bf16* t = a.tm + ((size_t)bn * a.nc + ch) * NP * C * C;
    cp_tile(Ts, LDC, t, C, NP * C, C);  // the planes' rows follow one another here and there
  };
  float S[MT][NS][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NS; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = (warp + 8 * mt) * 16 + (lane >> 2) + 8 * (e >> 1), c = vt * BV + t * 8 + (lane & 3) * 2 + (e & 1);
        S[mt][t][e] = a.s0 && r < a.Dk && c < a.Dv ? a.s0[((size_t)bn * a.Dk + r) * a.Dv + c] : 0.0f;
      }
  auto put_state = [&]() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = (warp + 8 * mt) * 16;
      if (r >= DKP) break;
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          split_store(Ss + (r + (lane >> 2) + 8 * h) * LDV + t * 8 + (lane & 3) * 2, DKP * LDV, S[mt][t][2 * h],
                          S[mt][t][2 * h + 1]);
    }
  };
  if (nch > 0) {
    load_k(0);
    load_v(0);
    load_t(0);
    cp_commit();
    put_state();
  }
  const int m0 = (warp % WM) * 16, n0 = (warp / WM) * (BV / WN);
  const Opnd Tm = opnd(Ts, LDC, C * LDC), So = opnd(Ss, LDV, DKP * LDV), Yo = opnd(Ys, LDV, C * LDV), Zo = opnd(Zs, LDV, C * LDV);
  for (int ch = 0; ch < nch; ++ch) {
    const size_t item = (size_t)bn * a.nc + ch, tile = item * a.nvt + vt;
    const bool more = ch + 1 < nch;
    cp_wait<0>();
    __syncthreads();
    const Opnd K = opnd(Ks, LDK, kplane);
    const float *gam = recs + (ch & 1) * 2 * C, *br = gam + C, gC = gam[C - 1];
    float acc[NT][4];
    zero(acc);
    mma_acc<NT, false, false>(acc, K, m0, So, n0, DKP);
    {  // the chunk's starting state, for the other kernels
      bf16* d = a.S + tile * NP * DKP * BV;
      for (int i = tid; i < NP * DKP * (BV / 8); i += 256) {
        const int r = i / (BV / 8), c = (i % (BV / 8)) * 8;
        *(uint4*)(d + (size_t)r * BV + c) = *(const uint4*)(Ss + r * LDV + c);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = m0 + (lane >> 2) + 8 * h;
      const float gi = gam[i];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = n0 + t * 8 + (lane & 3) * 2;
        float2 y = planes_sum(Vs + i * LDV + c, C * LDV);
        if (has_part(gi)) {  // behind a reset the old state has no part, whatever it holds
          y.x -= gi * acc[t][2 * h];
          y.y -= gi * acc[t][2 * h + 1];
          // The products with Tm and P reach over the reset by zeros, which an infinity
          // would pass. o and the gradients have it from S0.
          if (!has_part(gC)) {
            if (!isfinite(acc[t][2 * h])) y.x = 0.0f;
            if (!isfinite(acc[t][2 * h + 1])) y.y = 0.0f;
          }
        }
        split_store(Ys + i * LDV + c, C * LDV, y.x, y.y);
      }
    }
    __syncthreads();
    if (more) load_v(ch + 1);
    cp_commit();
    zero(acc);
    mma_acc<NT, false, false>(acc, Tm, m0, Yo, n0, C);
    {
      bf16* z = a.Z + tile * NP * C * BV;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m0 + (lane >> 2) + 8 * h;
        const float bi = br[i];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int c = n0 + t * 8 + (lane & 3) * 2;
          split_store(z + i * BV + c, C * BV, acc[t][2 * h], acc[t][2 * h + 1]);
          split_store(Zs + i * LDV + c, C * LDV, bi * acc[t][2 * h], bi * acc[t][2 * h + 1]);
        }
      }
    }
    __syncthreads();
    if (more) load_t(ch + 1);
    cp_commit();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = (warp + 8 * mt) * 16;
      if (r >= DKP) break;
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[mt][t][e] = has_part(gC) ? gC * S[mt][t][e] : 0.0f;
      mma_acc<NS, true, false>(S[mt], K, r, Zo, 0, C);
    }
    if (more) put_state();
    if (more) {
      __syncthreads();
      load_k(ch + 1);
      cp_commit();
    }
  }
  if (a.last) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = (warp + 8 * mt) * 16 + (lane >> 2) + 8 * (e >> 1), c = vt * BV + t * 8 + (lane & 3) * 2 + (e & 1);
          if (r < a.Dk && c < a.Dv) a.last[((size_t)bn * a.Dk + r) * a.Dv + c] = S[mt][t][e];
        }
  }
}

// ---- out -----------------------------------------------------------------------------
struct OutSmem {
  static constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  static __host__ __device__ size_t bytes(int DKP) {
    return 2 * ((size_t)NP * C * (DKP + 8) + (size_t)NP * C * (C + 8) + (size_t)NP * DKP * (BV + 8) +
                (size_t)NP * C * (BV + 8)) + C * 4;
  }
};

__global__ void __launch_bounds__(256) delta_out_kernel(DeltaArgs a) {
  constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  constexpr int WM = C / 16, WN = 8 / WM, NT = BV / WN / 8, LDV = BV + 8, LDC = C + 8;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  const int DKP = a.DKP, LDK = DKP + 8;
  bf16* Qs = (bf16*)sm_raw;
  bf16* Ps = Qs + NP * C * LDK;
  bf16* Ss = Ps + NP * C * LDC;
  bf16* Zs = Ss + NP * DKP * LDV;
  float* gam = (float*)(Zs + NP * C * LDV);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int vt = (int)(blockIdx.x % a.nvt);
  const long long item = blockIdx.x / a.nvt;
  const int ch = (int)(item % a.nc), bn = (int)(item / a.nc), n = bn % a.N, b = bn / a.N, nk = n / (a.N / a.Nk);
  const int live = live_steps(a, b, ch, C);
  const size_t ostride = (size_t)a.N * a.Dv;
  float* o = (float*)a.o + ((size_t)b * a.T + (size_t)ch * C) * ostride + (size_t)n * a.Dv + vt * BV;
  const int steps = min(C, a.T - ch * C), cols = min(BV, a.Dv - vt * BV);
  if (live == 0) {
    for (int i = tid; i < steps * BV; i += 256)
      if (i % BV < cols) o[(size_t)(i / BV) * ostride + i % BV] = 0.0f;
    return;
  }
  const size_t qstride = (size_t)a.Nk * a.Dk;
  load_rows<float, C>(Qs, LDK, C * LDK, (const float*)a.q + ((size_t)b * a.T + (size_t)ch * C) * qstride + (size_t)nk * a.Dk,
                  qstride, live, a.Dk, 0, DKP);
  cp_tile(Ss, LDV, a.S + ((size_t)item * a.nvt + vt) * NP * DKP * BV, BV, NP * DKP, BV);
  if (tid < C / 4) cp16(smem_u32(gam + tid * 4), a.rec + ((size_t)item * REC_N + REC_GAM) * C + tid * 4, true);
  cp_commit();
  cp_tile(Ps, LDC, a.pm + (size_t)item * NP * C * C, C, NP * C, C);
  cp_tile(Zs, LDV, a.Z + ((size_t)item * a.nvt + vt) * NP * C * BV, BV, NP * C, BV);
  cp_commit();
  cp_wait<1>();
  __syncthreads();
  const int m0 = (warp % WM) * 16, n0 = (warp / WM) * (BV / WN);
  float acc[NT][4];
  zero(acc);
  mma_acc<NT, false, false>(acc, opnd(Qs, LDK, C * LDK), m0, opnd(Ss, LDV, DKP * LDV), n0, DKP);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float gi = gam[m0 + (lane >> 2) + 8 * h];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) acc[t][2 * h + e] = has_part(gi) ? gi * acc[t][2 * h + e] : 0.0f;
  }
  cp_wait<0>();
  __syncthreads();
  mma_acc<NT, false, false>(acc, opnd(Ps, LDC, C * LDC), m0, opnd(Zs, LDV, C * LDV), n0, C);
  const bool pairs = a.Dv % 2 == 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = m0 + (lane >> 2) + 8 * h;
    if (i >= steps) continue;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = n0 + t * 8 + (lane & 3) * 2;
      const float x = i < live ? a.scale * acc[t][2 * h] : 0.0f, y = i < live ? a.scale * acc[t][2 * h + 1] : 0.0f;
      float* p = o + (size_t)i * ostride + c;
      if (pairs) {
        if (c < cols) *(float2*)p = make_float2(x, y);
      } else {
        if (c < cols) p[0] = x;
        if (c + 1 < cols) p[1] = y;
      }
    }
  }
}

cudaError_t run(const DeltaArgs& a, cudaStream_t st) {
  const long long items = (long long)a.B * a.N * a.nc;
  size_t sm = PrepSmem::bytes(a.DKP);
  cudaError_t e = set_smem_attr((const void*)delta_prep_kernel, sm);
  if (e != cudaSuccess) return e;
  delta_prep_kernel<<<(unsigned)items, 2 * F32_C, sm, st>>>(a);
  note_launch();
  void (*chain)(DeltaArgs) = a.DKP <= 128 ? delta_chain_kernel<1> : delta_chain_kernel<2>;
  sm = ChainSmem::bytes(a.DKP);
  if ((e = set_smem_attr((const void*)chain, sm)) != cudaSuccess) return e;
  chain<<<(unsigned)(a.B * a.N * a.nvt), 256, sm, st>>>(a);
  note_launch();
  sm = OutSmem::bytes(a.DKP);
  if ((e = set_smem_attr((const void*)delta_out_kernel, sm)) != cudaSuccess) return e;
  delta_out_kernel<<<(unsigned)(items * a.nvt), 256, sm, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_fwd_launch(const DeltaArgs& a, cudaStream_t st) { return run(a, st); }

}  // namespace rnn
