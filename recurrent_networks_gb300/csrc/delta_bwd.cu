// Gated delta rule, backward (the formulas are in delta.cuh), from what the
// forward left: Tm, P, Z and every chunk's starting state.
//   chain  per head and tile of BV columns, the chunks from the last to the
//          first: dY (= dV) and the state's gradient, left for every chunk
//   grad   every chunk by itself: dQ, dK, dg, dbeta
//   share  sums dQ and dK over the heads that share q and k
// Measured 83 + 49 + 3 us at B=3 T=515, 6 heads of 40 x 72 on 2 (54 CTAs walk 17
// chunks of 5 us each).
#include "delta.h"
#include "kernels.cuh"

namespace rnn {
namespace {

// ---- chain --------------------------------------------------------------------------
struct BwdChainSmem {
  static constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  static __host__ __device__ size_t bytes(int DKP) {
    return 2 * ((size_t)2 * NP * C * (DKP + 8) + (size_t)2 * NP * C * (C + 8) + (size_t)NP * C * (BV + 8) +
                (size_t)NP * DKP * (BV + 8) + (size_t)3 * NP * C * (BV + 8)) +
           2 * 2 * C * 4;
  }
};

template <int MT>
__global__ void __launch_bounds__(256, 1) delta_bwd_chain_kernel(DeltaArgs a) {
  constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  constexpr int WM = C / 16, WN = 8 / WM, NT = BV / WN / 8, NS = BV / 8, LDV = BV + 8, LDC = C + 8;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  const int DKP = a.DKP, LDK = DKP + 8, kplane = C * LDK;
  bf16* Ks = (bf16*)sm_raw;
  bf16* Qs = Ks + NP * kplane;
  bf16* Ts = Qs + NP * kplane;
  bf16* Ps = Ts + NP * C * LDC;
  bf16* Os = Ps + NP * C * LDC;          // dO
  bf16* Ss = Os + NP * C * LDV;          // dS1
  bf16* Zs = Ss + NP * DKP * LDV;        // dZ
  bf16* Ys = Zs + NP * C * LDV;          // -gam dY
  bf16* Gs = Ys + NP * C * LDV;          // gam scale dO
  float* recs = (float*)(Gs + NP * C * LDV);  // [2][gam, br][C]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int vt = blockIdx.x % a.nvt, bn = blockIdx.x / a.nvt, n = bn % a.N, b = bn / a.N, nk = n / (a.N / a.Nk);
  const int nch = live_chunks(a, b, C);
  const size_t kstride = (size_t)a.Nk * a.Dk, vstride = (size_t)a.N * a.Dv;
  const size_t kat = (size_t)b * a.T * kstride + (size_t)nk * a.Dk, vat = (size_t)b * a.T * vstride + (size_t)n * a.Dv;
  auto load_k = [&](int ch) {
    load_rows<float, C>(Ks, LDK, kplane, (const float*)a.k + kat + (size_t)ch * C * kstride, kstride,
                    live_steps(a, b, ch, C), a.Dk, 0, DKP);
  };
  auto load_q = [&](int ch) {
    load_rows<float, C>(Qs, LDK, kplane, (const float*)a.q + kat + (size_t)ch * C * kstride, kstride, live_steps(a, b, ch, C),
                    a.Dk, 0, DKP);
  };
  auto load_po = [&](int ch) {
    const size_t item = (size_t)bn * a.nc + ch;
    if (a.dO) {
      load_rows<float, C>(Os, LDV, C * LDV, (const float*)a.dO + vat + (size_t)ch * C * vstride, vstride, live_steps(a, b, ch, C),
                      a.Dv, vt * BV, BV);
    } else {
      for (int i = tid; i < NP * C * LDV; i += 256) Os[i] = __float2bfloat16_rn(0.0f);
    }
    cp_tile(Ps, LDC, a.pm + item * NP * C * C, C, NP * C, C);
    const float* r = a.rec + item * REC_N * C;
    float* d = recs + (ch & 1) * 2 * C;
    if (tid < C / 4) cp16(smem_u32(d + tid * 4), r + REC_GAM * C + tid * 4, true);
    else if (tid < C / 2) cp16(smem_u32(d + tid * 4), r + REC_BR * C + (tid - C / 4) * 4, true);
  };
  auto load_t = [&](int ch) { cp_tile(Ts, LDC, a.tm + ((size_t)bn * a.nc + ch) * NP * C * C, C, NP * C, C); };
  float S[MT][NS][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NS; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = (warp + 8 * mt) * 16 + (lane >> 2) + 8 * (e >> 1), c = vt * BV + t * 8 + (lane & 3) * 2 + (e & 1);
        S[mt][t][e] = a.dlast && r < a.Dk && c < a.Dv ? a.dlast[((size_t)bn * a.Dk + r) * a.Dv + c] : 0.0f;
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
    load_k(nch - 1);
    load_po(nch - 1);
    load_t(nch - 1);
    cp_commit();
    load_q(nch - 1);
    cp_commit();
    put_state();
  }
  const int m0 = (warp % WM) * 16, n0 = (warp / WM) * (BV / WN);
  const Opnd Q = opnd(Qs, LDK, kplane), Tm = opnd(Ts, LDC, C * LDC), P = opnd(Ps, LDC, C * LDC), O = opnd(Os, LDV, C * LDV);
  const Opnd So = opnd(Ss, LDV, DKP * LDV), Zo = opnd(Zs, LDV, C * LDV), Yo = opnd(Ys, LDV, C * LDV), Go = opnd(Gs, LDV, C * LDV);
  for (int ch = nch - 1; ch >= 0; --ch) {
    const size_t tile = ((size_t)bn * a.nc + ch) * a.nvt + vt;
    const bool more = ch > 0;
    cp_wait<1>();  // all but q
    __syncthreads();
    const Opnd K = opnd(Ks, LDK, kplane);
    const float *gam = recs + (ch & 1) * 2 * C, *br = gam + C, gC = gam[C - 1];
    bool lost[NT][4];  // where the state's gradient is not finite and ends in this chunk
    float acc[NT][4], acc2[NT][4];
    zero(acc);
    zero(acc2);
    mma_acc<NT, true, false>(acc, P, m0, O, n0, C);
    mma_acc<NT, false, false>(acc2, K, m0, So, n0, DKP);
    {
      bf16* d = a.dS + tile * NP * DKP * BV;
      for (int i = tid; i < NP * DKP * (BV / 8); i += 256) {
        const int r = i / (BV / 8), c = (i % (BV / 8)) * 8;
        *(uint4*)(d + (size_t)r * BV + c) = *(const uint4*)(Ss + r * LDV + c);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = m0 + (lane >> 2) + 8 * h;
      const float bi = br[i], gi = gam[i] * a.scale;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = n0 + t * 8 + (lane & 3) * 2;
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[e] = a.scale * acc[t][2 * h + e];
          // no part of the state's gradient before a later document; the products reach
          // there by zeros, which an infinity would pass
          const float w = has_part(bi) ? bi * acc2[t][2 * h + e] : 0.0f;
          lost[t][2 * h + e] = !has_part(gC) && !isfinite(w);
          if (!lost[t][2 * h + e]) x[e] += w;
        }
        split_store(Zs + i * LDV + c, C * LDV, x[0], x[1]);
        const float2 d = planes_sum(Os + i * LDV + c, C * LDV);
        split_store(Gs + i * LDV + c, C * LDV, gi * d.x, gi * d.y);
      }
    }
    __syncthreads();
    if (more) load_po(ch - 1);
    cp_commit();
    zero(acc);
    mma_acc<NT, true, false>(acc, Tm, m0, Zo, n0, C);
    {
      bf16* y = a.dY + tile * NP * C * BV;
      float* dv = a.dv ? (float*)a.dv + vat + (size_t)ch * C * vstride + vt * BV : nullptr;
      const int steps = min(C, a.T - ch * C), cols = a.Dv - vt * BV, live = live_steps(a, b, ch, C);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m0 + (lane >> 2) + 8 * h;
        const float gi = gam[i];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int c = n0 + t * 8 + (lane & 3) * 2;
          const float x0 = lost[t][2 * h] ? nanf("") : acc[t][2 * h], x1 = lost[t][2 * h + 1] ? nanf("") : acc[t][2 * h + 1];
          split_store(y + i * BV + c, C * BV, x0, x1);
          split_store(Ys + i * LDV + c, C * LDV, has_part(gi) ? -gi * x0 : 0.0f, has_part(gi) ? -gi * x1 : 0.0f);
          if (dv && i < steps) {
            float* p = dv + (size_t)i * vstride + c;
            const float v0 = i < live ? x0 : 0.0f, v1 = i < live ? x1 : 0.0f;
            if (a.Dv % 2 == 0) {
              if (c < cols) *(float2*)p = make_float2(v0, v1);
            } else {
              if (c < cols) p[0] = v0;
              if (c + 1 < cols) p[1] = v1;
            }
          }
        }
      }
    }
    cp_wait<1>();  // q
    __syncthreads();
    if (more) load_t(ch - 1);
    cp_commit();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = (warp + 8 * mt) * 16;
      if (r >= DKP) break;
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[mt][t][e] = has_part(gC) ? gC * S[mt][t][e] : 0.0f;
      mma_acc<NS, true, false>(S[mt], Q, r, Go, 0, C);
      mma_acc<NS, true, false>(S[mt], K, r, Yo, 0, C);
    }
    if (more) {
      put_state();
      __syncthreads();  // q and k are done with
      load_k(ch - 1);
      cp_commit();
      load_q(ch - 1);
      cp_commit();
    }
  }
  if (a.ds0) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = (warp + 8 * mt) * 16 + (lane >> 2) + 8 * (e >> 1), c = vt * BV + t * 8 + (lane & 3) * 2 + (e & 1);
          if (r < a.Dk && c < a.Dv) a.ds0[((size_t)bn * a.Dk + r) * a.Dv + c] = S[mt][t][e];
        }
  }
}

// ---- grad ----------------------------------------------------------------------------
constexpr int GRAD_BK = 64;  // columns of dQ and dK taken at once

struct GradSmem {
  static constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  static __host__ __device__ size_t bytes(int DKP) {
    return 2 * ((size_t)2 * NP * C * (DKP + 8) + (size_t)2 * NP * C * (C + 8) + (size_t)NP * C * (BV + 8) +
                (size_t)2 * NP * C * (BV + 8) + (size_t)2 * NP * GRAD_BK * (BV + 8)) +
           4 * (REC_N * C + C * (C + 1) + 4 * C + 3 * 4 * C + 2 * C + 16);
  }
};

__global__ void __launch_bounds__(256, 1) delta_grad_kernel(DeltaArgs a) {
  constexpr int C = F32_C, NP = F32_NP, BV = F32_BV;
  constexpr int WM = C / 16, WN = 8 / WM, NT = C / WN / 8, NK = GRAD_BK / WN / 8, LDV = BV + 8, LDC = C + 8;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  const int DKP = a.DKP, LDK = DKP + 8, kplane = C * LDK;
  bf16* Ks = (bf16*)sm_raw;
  bf16* Qs = Ks + NP * kplane;
  bf16* Rs = Qs + NP * kplane;
  bf16* Ms = Rs + NP * C * LDC;  // M + M^T
  bf16* Os = Ms + NP * C * LDC;  // dO
  bf16* Zs = Os + NP * C * LDV;
  bf16* Ys = Zs + NP * C * LDV;  // dY
  bf16* Ss = Ys + NP * C * LDV;  // GRAD_BK rows of S0
  bf16* Ds = Ss + NP * GRAD_BK * LDV;  // of dS1
  float* rec = (float*)(Ds + NP * GRAD_BK * LDV);
  float* Es = rec + REC_N * C;    // [C][C + 1]: E below the diagonal
  float* colB = Es + C * (C + 1); // [WM][C] partial sums
  float* dots = colB + 4 * C;     // [3][WN][C]: q.dq, k.dk1, k.H of the state's parts
  float* fin = dots + 12 * C;     // [2][C]
  float* wsum = fin + 2 * C;      // [8]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long item = blockIdx.x;
  const int ch = (int)(item % a.nc), bn = (int)(item / a.nc), n = bn % a.N, b = bn / a.N, nk = n / (a.N / a.Nk);
  const int live = live_steps(a, b, ch, C), steps = min(C, a.T - ch * C);
  const size_t kstride = (size_t)a.Nk * a.Dk, vstride = (size_t)a.N * a.Dv;
  const size_t row0 = (size_t)b * a.T + (size_t)ch * C;
  const size_t kat = row0 * kstride + (size_t)nk * a.Dk, vat = row0 * vstride + (size_t)n * a.Dv;
  const bool shared_heads = a.pq != nullptr;
  const size_t pstride = (size_t)a.N * a.Dk, pat = row0 * pstride + (size_t)n * a.Dk;
  if (live == 0) {  // nothing of the chunk exists
    for (int i = tid; i < steps; i += 256) {
      a.dg[(row0 + i) * a.N + n] = 0.0f;
      a.dbeta[(row0 + i) * a.N + n] = 0.0f;
    }
    for (int i = tid; i < steps * a.Dk; i += 256) {
      const int r = i / a.Dk, c = i % a.Dk;
      if (shared_heads) a.pq[pat + r * pstride + c] = a.pk[pat + r * pstride + c] = 0.0f;
      else ((float*)a.dq)[kat + r * kstride + c] = ((float*)a.dk)[kat + r * kstride + c] = 0.0f;
    }
    for (int i = tid; i < steps * a.Dv; i += 256)
      ((float*)a.dv)[vat + (size_t)(i / a.Dv) * vstride + i % a.Dv] = 0.0f;
    return;
  }
  auto load_v = [&](int vt) {
    if (a.dO) {
      load_rows<float, C>(Os, LDV, C * LDV, (const float*)a.dO + vat, vstride, live, a.Dv, vt * BV, BV);
    } else {
      for (int i = tid; i < NP * C * LDV; i += 256) Os[i] = __float2bfloat16_rn(0.0f);
    }
    const size_t t = ((size_t)item * a.nvt + vt) * NP * C * BV;
    cp_tile(Zs, LDV, a.Z + t, BV, NP * C, BV);
    cp_tile(Ys, LDV, a.dY + t, BV, NP * C, BV);
  };
  load_rows<float, C>(Ks, LDK, kplane, (const float*)a.k + kat, kstride, live, a.Dk, 0, DKP);
  load_rows<float, C>(Qs, LDK, kplane, (const float*)a.q + kat, kstride, live, a.Dk, 0, DKP);
  for (int i = tid; i < REC_N * C / 4; i += 256) cp16(smem_u32(rec + i * 4), a.rec + (size_t)item * REC_N * C + i * 4, true);
  load_v(0);
  cp_commit();
  cp_wait<0>();
  __syncthreads();
  const int m0 = (warp % WM) * 16, wn = warp / WM, n0 = wn * (C / WN);
  const Opnd K = opnd(Ks, LDK, kplane), Q = opnd(Qs, LDK, kplane), R = opnd(Rs, LDC, C * LDC), M = opnd(Ms, LDC, C * LDC);
  const Opnd O = opnd(Os, LDV, C * LDV), Z = opnd(Zs, LDV, C * LDV), Y = opnd(Ys, LDV, C * LDV);
  const Opnd S = opnd(Ss, LDV, GRAD_BK * LDV), D = opnd(Ds, LDV, GRAD_BK * LDV);
  const float *gam = rec + REC_GAM * C, *rho = rec + REC_RHO * C, *beta = rec + REC_BETA * C;
  {
    float kk[NT][4], qk[NT][4], f[NT][4], nn[NT][4];
    zero(kk);
    zero(qk);
    zero(f);
    zero(nn);
    mma_acc<NT, false, true>(kk, K, m0, K, n0, DKP);
    mma_acc<NT, false, true>(qk, Q, m0, K, n0, DKP);
    for (int vt = 0; vt < a.nvt; ++vt) {
      if (vt) {
        __syncthreads();
        load_v(vt);
        cp_commit();
        cp_wait<0>();
        __syncthreads();
      }
      mma_acc<NT, false, true>(f, O, m0, Z, n0, BV);
      mma_acc<NT, false, true>(nn, Y, m0, Z, n0, BV);
    }
    float csum[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) csum[t][0] = csum[t][1] = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = m0 + (lane >> 2) + 8 * h;
      const float ci = rec[REC_CHI * C + i], li = rec[REC_CLO * C + i];
      const int si = __float_as_int(rec[REC_SEG * C + i]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = n0 + t * 8 + (lane & 3) * 2 + e;
          const bool on = i >= j && si == __float_as_int(rec[REC_SEG * C + j]);
          const float ga = on ? expf((ci - rec[REC_CHI * C + j]) + (li - rec[REC_CLO * C + j])) : 0.0f, bj = beta[j];
          const float fx = on ? a.scale * f[t][2 * h + e] * ga : 0.0f;
          const float nx = on && i > j ? -nn[t][2 * h + e] * ga : 0.0f;
          r[e] = fx * bj;
          const float e0 = on ? fx * qk[t][2 * h + e] + nx * kk[t][2 * h + e] : 0.0f;
          Es[i * (C + 1) + j] = i > j ? bj * e0 : 0.0f;
          csum[t][e] += e0;
          if (i > j) {
            split_store1(Ms + i * LDC + j, C * LDC, nx * bj);
            split_store1(Ms + j * LDC + i, C * LDC, nx * bj);
          } else if (i == j) {
            split_store1(Ms + i * LDC + j, C * LDC, 0.0f);
          }
        }
        split_store(Rs + i * LDC + n0 + t * 8 + (lane & 3) * 2, C * LDC, r[0], r[1]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = csum[t][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (lane < 4) colB[(warp % WM) * C + n0 + t * 8 + lane * 2 + e] = s;
      }
  }
  float dot[3][2] = {}, ss = 0.0f;
  const int i0 = m0 + (lane >> 2);
  for (int k0 = 0; k0 < DKP; k0 += GRAD_BK) {
    const int rows = min(GRAD_BK, DKP - k0), nn0 = wn * (GRAD_BK / WN);
    float aq[NK][4], ak[NK][4], ah[NK][4];
    zero(aq);
    zero(ak);
    zero(ah);
    for (int vt = 0; vt < a.nvt; ++vt) {
      __syncthreads();
      const size_t t = (((size_t)item * a.nvt + vt) * NP * DKP + k0) * BV;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        cp_tile(Ss + p * GRAD_BK * LDV, LDV, a.S + t + (size_t)p * DKP * BV, BV, rows, BV);
        cp_tile(Ds + p * GRAD_BK * LDV, LDV, a.dS + t + (size_t)p * DKP * BV, BV, rows, BV);
      }
      if (a.nvt > 1) load_v(vt);
      cp_commit();
      cp_wait<0>();
      __syncthreads();
      if (nn0 < rows) {
        mma_acc<NK, false, true>(aq, O, m0, S, nn0, BV);
        mma_acc<NK, false, true>(ak, Y, m0, S, nn0, BV);
        mma_acc<NK, false, true>(ah, Z, m0, D, nn0, BV);
      }
      for (int i = tid; i < rows * (BV / 2); i += 256) {
        const int at = (i / (BV / 2)) * LDV + (i % (BV / 2)) * 2;
        const float2 x = planes_sum(Ss + at, GRAD_BK * LDV), y = planes_sum(Ds + at, GRAD_BK * LDV);
        ss += x.x * y.x + x.y * y.y;
      }
    }
    if (nn0 < rows) {
      float dk[NK][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = i0 + 8 * h;
        const float gi = gam[i], ri = rho[i], bi = beta[i];
#pragma unroll
        for (int t = 0; t < NK; ++t) {
          const int c = k0 + nn0 + t * 8 + (lane & 3) * 2;
          if (c >= DKP) {
#pragma unroll
            for (int e = 0; e < 2; ++e) aq[t][2 * h + e] = dk[t][2 * h + e] = 0.0f;
            continue;
          }
          const float2 q = planes_sum(Qs + i * LDK + c, kplane), k = planes_sum(Ks + i * LDK + c, kplane);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = has_part(gi) ? gi * a.scale * aq[t][2 * h + e] : 0.0f;
            const float k1 = has_part(gi) ? -gi * ak[t][2 * h + e] : 0.0f;
            const float hh = has_part(ri) ? ri * ah[t][2 * h + e] : 0.0f;
            const float qe = e ? q.y : q.x, ke = e ? k.y : k.x;
            dot[0][h] += qe * x;
            dot[1][h] += ke * k1;
            dot[2][h] += ke * hh;
            aq[t][2 * h + e] = x;
            dk[t][2 * h + e] = k1 + bi * hh;
          }
        }
      }
      mma_acc<NK, false, false>(aq, R, m0, K, k0 + nn0, C);
      mma_acc<NK, false, false>(dk, M, m0, K, k0 + nn0, C);
      mma_acc<NK, true, false>(dk, R, m0, Q, k0 + nn0, C);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = i0 + 8 * h;
        if (i >= steps) continue;
#pragma unroll
        for (int t = 0; t < NK; ++t) {
          const int c = k0 + nn0 + t * 8 + (lane & 3) * 2;
          if (c >= a.Dk) continue;
          const bool on = i < live;
          const float x0 = on ? aq[t][2 * h] : 0.0f, x1 = on ? aq[t][2 * h + 1] : 0.0f;
          const float y0 = on ? dk[t][2 * h] : 0.0f, y1 = on ? dk[t][2 * h + 1] : 0.0f;
          if (shared_heads) {
            float *p = a.pq + pat + i * pstride + c, *r = a.pk + pat + i * pstride + c;
            p[0] = x0;
            r[0] = y0;
            if (c + 1 < a.Dk) p[1] = x1, r[1] = y1;
          } else {
            float *p = (float*)a.dq + kat + i * kstride + c, *r = (float*)a.dk + kat + i * kstride + c;
            p[0] = x0;
            r[0] = y0;
            if (c + 1 < a.Dk) p[1] = x1, r[1] = y1;
          }
        }
      }
    }
  }
#pragma unroll
  for (int d = 0; d < 3; ++d)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s = dot[d][h];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if ((lane & 3) == 0) dots[(d * WN + wn) * C + i0 + 8 * h] = s;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) wsum[warp] = ss;
  __syncthreads();
  if (tid < C) {
    float cb = 0.0f, d[3] = {};
#pragma unroll
    for (int w = 0; w < WM; ++w) cb += colB[w * C + tid];
#pragma unroll
    for (int w = 0; w < WN; ++w)
#pragma unroll
      for (int k = 0; k < 3; ++k) d[k] += dots[(k * WN + w) * C + tid];
    fin[tid] = d[0] + d[1];
    fin[C + tid] = beta[tid] * d[2];
    // z is left finite where a reset follows a state that is not
    if (tid < steps) a.dbeta[(row0 + tid) * a.N + n] = tid < live ? cb + d[2] + 0.0f * d[1] : 0.0f;
  }
  __syncthreads();
  {  // dg: what reaches over a step, 8 threads a step
    static_assert(C * 8 == 256, "all threads");
    const int t = tid >> 3, k = tid & 7;
    const float* seg = rec + REC_SEG * C;
    const bool mark = __float_as_int(seg[t]) != (t ? __float_as_int(seg[t - 1]) : 0);
    float s = 0.0f;
    for (int i = t + k; i < C; i += 8) {
      float r = fin[i];
      for (int j = 0; j < t; ++j) r += Es[i * (C + 1) + j];
      s += r;
    }
    for (int j = k; j < t; j += 8) s += fin[C + j];
    if (has_part(gam[C - 1])) s = fmaf(gam[C - 1], wsum[k], s);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (k == 0 && t < steps) a.dg[(row0 + t) * a.N + n] = t < live && !mark ? s : 0.0f;
  }
}

// ---- share ---------------------------------------------------------------------------
// dq, dk [rows, Nk, Dk] = sums of pq, pk [rows, Nk, share, Dk], in the heads' order
__global__ void __launch_bounds__(256) delta_share_kernel(const float* pq, const float* pk, float* dq, float* dk, long long n, int share,
                                                          int Dk) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = i / Dk;
    const size_t at = (size_t)r * share * Dk + (size_t)(i - r * Dk);
    float x = 0.0f, y = 0.0f;
    for (int s = 0; s < share; ++s) {
      x += pq[at + (size_t)s * Dk];
      y += pk[at + (size_t)s * Dk];
    }
    dq[i] = x;
    dk[i] = y;
  }
}

cudaError_t run(const DeltaArgs& a, cudaStream_t st) {
  void (*chain)(DeltaArgs) = a.DKP <= 128 ? delta_bwd_chain_kernel<1> : delta_bwd_chain_kernel<2>;
  size_t sm = BwdChainSmem::bytes(a.DKP);
  cudaError_t e = set_smem_attr((const void*)chain, sm);
  if (e != cudaSuccess) return e;
  chain<<<(unsigned)(a.B * a.N * a.nvt), 256, sm, st>>>(a);
  note_launch();
  sm = GradSmem::bytes(a.DKP);
  if ((e = set_smem_attr((const void*)delta_grad_kernel, sm)) != cudaSuccess) return e;
  delta_grad_kernel<<<(unsigned)((long long)a.B * a.N * a.nc), 256, sm, st>>>(a);
  note_launch();
  if (a.pq) {
    const long long n = (long long)a.B * a.T * a.Nk * a.Dk;
    const long long blocks = (n + 255) / 256, most = 16LL * device_sms();
    delta_share_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(a.pq, a.pk, (float*)a.dq, (float*)a.dk, n,
                                                                                   a.N / a.Nk, a.Dk);
    note_launch();
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_bwd_launch(const DeltaArgs& a, cudaStream_t st) { return run(a, st); }

}  // namespace rnn
