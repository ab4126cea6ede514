// Gated delta rule: a scan whose state is a matrix S [Dk, Dv] per head,
//   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  S_t = a_t S_{t-1} + k_t u_t^T,
//   o_t = scale S_t^T q_t,                   a_t = exp(g_t), 0 at a reset.
// In chunks of C steps from the state S0 at the chunk's start, with c_i the sum
// of g up to step i of the chunk, Gam_ij = exp(c_i - c_j) for i >= j of the same
// document (0 otherwise), gam_i = exp(c_i) (0 behind a reset), rho_j = Gam_{C-1,j}:
//   L_ij = Gam_ij (k_i.k_j) beta_j (i > j),   Tm = (I + L)^-1,
//   P_ij = Gam_ij (q_i.k_j) beta_j (i >= j),  Y = V - gam K S0,  Z = Tm Y  (u = beta z)
//   O = scale (gam Q S0 + P Z),  S1 = gam_{C-1} S0 + K^T (beta rho Z).
// Backward, from dO' = scale dO and the gradient dS1 of S1:
//   dZ = P^T dO' + beta rho K dS1,  dY = Tm^T dZ = dV,
//   dS0 = gam_{C-1} dS1 + Q^T gam dO' - K^T gam dY,
//   F = dO' Z^T (i >= j), N = -dY Z^T (i > j), R = F Gam beta_j, M = N Gam beta_j,
//   dQ = gam dO' S0^T + R K,
//   dK = -gam dY S0^T + beta H + (M + M^T) K + R^T Q,  H = rho Z dS1^T,
//   dbeta_j = sum_i F_ij Gam_ij q_i.k_j + sum_i N_ij Gam_ij k_i.k_j + k_j.H_j,
//   G_i = q_i.(gam dO' S0^T)_i - k_i.(gam dY S0^T)_i,  E = F P + N L,
//   dg_t = what reaches over step t in its document:
//          sum_{i >= t > j} E_ij + sum_{i >= t} G_i + sum_{j < t} beta_j k_j.H_j + gam_{C-1} <S0, dS1>.
// (As a difference of sums of rows and columns of E, dg_t would have the error of
// terms that do not reach over t and are not small with a_t.)
//
// This file has what the kernels of fp32 storage need (delta_fwd.cu, delta_bwd.cu);
// those of bf16 storage are in delta_tc*.
//
// fp32: the products run on mma.sync with operands in NP = 3 bf16 planes: a value
// is the sum of its planes, each the rounding of what the planes before it left
// (2^-24 of the value remain), and a product takes the plane pairs (i, j) with
// i + j < NP: six products instead of one. Three planes of every operand leave
// shared memory for chunks of 32 steps and tiles of 32 columns of v.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gated.cuh"
#include "ptx.cuh"

namespace rnn {

typedef __nv_bfloat16 bf16;

constexpr int F32_NP = 3, F32_C = 32, F32_BV = 32;  // planes, steps of a chunk, columns of a tile of v

// per-step values of a chunk that delta_prep leaves for the other kernels
enum { REC_CHI = 0, REC_CLO, REC_SEG, REC_GAM, REC_RHO, REC_BETA, REC_BR, REC_N };

// gam is +0 for the steps behind a reset alone, and -0 where the decays' product is
// below the smallest number: the state before the reset has no part in the former,
// whatever it holds, and is multiplied by the latter as by any factor (an infinity
// stays no number). So rho and br = beta rho, for the steps before a later reset and
// the gradient of the state behind it.
__device__ __forceinline__ float keep_part(float f) { return f == 0.0f ? -0.0f : f; }
__device__ __forceinline__ bool has_part(float f) { return __float_as_uint(f) != 0u; }

struct DeltaArgs {
  int B, T, Nk, N, Dk, Dv;
  int DKP, nvt, nc;  // Dk rounded up to 16, tiles of BV columns of v, chunks
  const void *q, *k, *v;
  const float *g, *beta, *s0;
  const unsigned char* reset;
  const int* lengths;
  float scale;
  unsigned* status;
  void* o;
  float* last;
  float* rec;  // [items][REC_N][C], items = (b N + n) nc + chunk
  bf16 *tm, *pm;  // [items][NP][C][C]
  bf16* S;        // [items][nvt][NP][DKP][BV]
  bf16* Z;        // [items][nvt][NP][C][BV]
  const void* dO;
  const float* dlast;
  bf16 *dY, *dS;  // as Z, S
  void *dq, *dk, *dv;
  float *dg, *dbeta, *ds0;
  float *pq, *pk;  // dq, dk of every v head [B,T,N,Dk] where heads share q and k, else null
};

// ---- fragments -------------------------------------------------------------------
template <bool TRANS> __device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool TRANS> __device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t* r) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}

// An operand in shared memory: planes of rows of `ld` elements (columns + 8: the
// rows of an 8 x 8 matrix then start in different banks).
struct Opnd {
  uint32_t at;  // shared-memory address of plane 0
  int ld, plane;  // in elements
};
__device__ __forceinline__ Opnd opnd(const bf16* p, int ld, int plane) { return {smem_u32(p), ld, plane}; }

// acc[NT] (16 x 8 NT) += A(m0.., :) B(:, n0..) over K (a multiple of 16).
// A(m, k) is stored [m][k] (AT: [k][m]); B(k, n) is stored [k][n] (BK: [n][k]).
// The tensor cores cut an accumulator off at each addition, always towards zero
// (2^-23 of it), so the large products (0, 0) have an accumulator to themselves
// and the sum so far joins by a rounded addition: 24 additions of six products
// into the running state were 7e-6 off after a few chunks of fp32.
template <int NT, bool AT, bool BK>
__device__ __forceinline__ void mma_acc(float (&acc)[NT][4], const Opnd& A, int m0, const Opnd& B, int n0, int K) {
  constexpr int NP = F32_NP;
  const int lane = threadIdx.x & 31, id = lane >> 3, r = lane & 7;
  const int arow = AT ? (id >> 1) * 8 + r : (id & 1) * 8 + r, acol = AT ? (id & 1) * 8 : (id >> 1) * 8;
  uint32_t aat = A.at + 2u * (uint32_t)(AT ? arow * A.ld + m0 + acol : (m0 + arow) * A.ld + acol);
  const uint32_t astep = AT ? 32u * A.ld : 32u;
  const int kofs = (id & 1) * 8, nofs = (id >> 1) * 8;
  uint32_t bat = B.at + 2u * (uint32_t)(BK ? (n0 + nofs + r) * B.ld + kofs : (kofs + r) * B.ld + n0 + nofs);
  const uint32_t bstep = BK ? 32u : 32u * B.ld, bpair = BK ? 32u * B.ld : 32u;
  float hi[NT][4] = {}, lo[NT][4] = {};
#pragma unroll 2
  for (int k = 0; k < K; k += 16, aat += astep, bat += bstep) {
    uint32_t a[NP][4];
#pragma unroll
    for (int p = 0; p < NP; ++p) ldsm4<AT>(aat + 2u * p * A.plane, a[p]);
#pragma unroll
    for (int j = 0; j < (NT + 1) / 2; ++j) {
      uint32_t b[NP][4];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        if (2 * j + 1 < NT) ldsm4<!BK>(bat + j * bpair + 2u * p * B.plane, b[p]);
        else ldsm2<!BK>(bat + j * bpair + 2u * p * B.plane, b[p]);
      }
      // the small products first
#pragma unroll
      for (int s = NP - 1; s >= 0; --s)
#pragma unroll
        for (int pa = 0; pa <= s; ++pa) {
          const uint32_t* w = b[s - pa];
          mma_bf16_16816(s ? lo[2 * j] : hi[2 * j], a[pa], w[0], w[1]);
          if (2 * j + 1 < NT) mma_bf16_16816(s ? lo[2 * j + 1] : hi[2 * j + 1], a[pa], w[2], w[3]);
        }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] += hi[t][e] + lo[t][e];
}
template <int NT> __device__ __forceinline__ void zero(float (&acc)[NT][4]) {
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
}

// x0, x1 as planes, written to p (+ plane, ...) as pairs
__device__ __forceinline__ void split_store(bf16* p, int plane, float x0, float x1) {
#pragma unroll
  for (int i = 0; i < F32_NP; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    *(__nv_bfloat162*)(p + (size_t)i * plane) = h;
    if (i + 1 < F32_NP) {
      x0 -= __bfloat162float(h.x);
      x1 -= __bfloat162float(h.y);
    }
  }
}
// one value as planes
__device__ __forceinline__ void split_store1(bf16* p, int plane, float x) {
#pragma unroll
  for (int i = 0; i < F32_NP; ++i) {
    const bf16 h = __float2bfloat16_rn(x);
    p[(size_t)i * plane] = h;
    x -= __bfloat162float(h);
  }
}
__device__ __forceinline__ float2 planes_sum(const bf16* p, int plane) {
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = F32_NP - 1; i >= 0; --i) {
    const __nv_bfloat162 h = *(const __nv_bfloat162*)(p + (size_t)i * plane);
    s.x += __bfloat162float(h.x);
    s.y += __bfloat162float(h.y);
  }
  return s;
}

// ---- copies ------------------------------------------------------------------------
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// rows x cols (cols a multiple of 8) of a dense 16-byte-aligned matrix with
// rows of `src_ld`, into rows of ld elements
__device__ __forceinline__ void cp_tile(bf16* dst, int ld, const bf16* src, int src_ld, int rows, int cols) {
  const int v = cols >> 3;
  for (int i = threadIdx.x; i < rows * v; i += blockDim.x) {
    const int r = i / v, c = (i - r * v) * 8;
    cp16(smem_u32(dst + r * ld + c), src + (size_t)r * src_ld + c, true);
  }
}

// The C rows of a chunk of an input [.., D] (rows `stride` elements apart), the
// columns c0 .. c0 + cols, into planes (bf16: one); rows from `live` on and columns past D
// are zero and not read. bf16 rows of whole 16-byte vectors arrive by
// asynchronous copies, others and fp32 at once.
template <typename T, int C>
__device__ __forceinline__ void load_rows(bf16* dst, int ld, int plane, const T* src, size_t stride, int live, int D,
                                          int c0, int cols) {
  if constexpr (sizeof(T) == 2) {
    if (D % 8 == 0) {
      const int v = cols >> 3;
      for (int i = threadIdx.x; i < C * v; i += blockDim.x) {
        const int r = i / v, c = (i - r * v) * 8;
        const bool on = r < live && c0 + c < D;
        cp16(smem_u32(dst + r * ld + c), on ? src + (size_t)r * stride + c0 + c : src, on);
      }
    } else {
      const int v = cols >> 1;
      for (int i = threadIdx.x; i < C * v; i += blockDim.x) {
        const int r = i / v, c = (i - r * v) * 2;
        __nv_bfloat162 x = __floats2bfloat162_rn(0.0f, 0.0f);
        if (r < live) {
          const T* p = src + (size_t)r * stride + c0 + c;
          if (c0 + c < D) x.x = p[0];
          if (c0 + c + 1 < D) x.y = p[1];
        }
        *(__nv_bfloat162*)(dst + r * ld + c) = x;
      }
    }
  } else {
    const int v = cols >> 1;
#pragma unroll 4
    for (int i = threadIdx.x; i < C * v; i += blockDim.x) {
      const int r = i / v, c = (i - r * v) * 2;
      float x0 = 0.0f, x1 = 0.0f;
      if (r < live) {
        const float* p = (const float*)src + (size_t)r * stride + c0 + c;
        if (c0 + c < D) x0 = p[0];
        if (c0 + c + 1 < D) x1 = p[1];
      }
      split_store(dst + r * ld + c, plane, x0, x1);
    }
  }
}

// steps of chunk `ch` that exist for row b
__device__ __forceinline__ int live_steps(const DeltaArgs& a, int b, int ch, int C) {
  int len = a.T;
  if (a.lengths) len = max(0, min(a.T, __ldg(a.lengths + b)));
  const long long left = (long long)len - (long long)ch * C;
  return left < 0 ? 0 : (int)(left < C ? left : C);
}
__device__ __forceinline__ int live_chunks(const DeltaArgs& a, int b, int C) {
  int len = a.T;
  if (a.lengths) len = max(0, min(a.T, __ldg(a.lengths + b)));
  return (len + C - 1) / C;
}

}  // namespace rnn
