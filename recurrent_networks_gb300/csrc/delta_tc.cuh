// Gated delta rule, bf16 storage: the products on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory). The formulas are in delta.cuh;
// here
//   P carries the scale, PT = P Tm, and the stacked matrices are
//   KQ = [K; Q] (128 rows) and TP = [Tm; PT] (128 x 64).
// Forward, a chunk:
//   [K S0; Q S0] = KQ S0,  Y = V - gam K S0,
//   [Z; PT Y] = TP Y,      O = scale gam Q S0 + PT Y,
//   S1 = gam_63 S0 + K^T (beta rho Z).
// Backward:
//   W = beta rho (K dS1),  dY = Tm^T W + PT^T dO = dV,
//   dS0 = gam_63 dS1 + KQ^T [-gam dY; scale gam dO],
//   [dK; dQ] = rows of [-gam dY S0^T + beta rho Z dS1^T; scale gam dO S0^T] + [M + M^T, R^T; R, 0] KQ.
// With u = beta z, v's and o's own definitions give the scalars' gradients from
// row products alone (pairs of steps inside a chunk cancel in dc):
//   dbeta_j = z_j.dY_j / beta_j,   dc_i = dO_i.o_i - dY_i.v_i,
//   dg_t = the sum of dc_i over i >= t of t's document, to the chunk's end, +
//          <S1, dS1> where the document goes on.
// That sum's terms do not become small with a_t. Where g_t is below GATE_NEAR, dg_t
// is taken as what reaches over the step (delta.cuh), from the grad kernel's operands
// in two planes.
// dY_j carries the factor beta_j throughout, so the quotient keeps its digits as
// long as dY_j's planes do: where a backward comes, |beta_j| below 2^-60 counts as
// 2^-60 (a shut gate, down to 0; far below a rounding of anything else it enters).
//
// The states, o, dY and all that fp32 outputs follow from are held to fp32: the
// computed operands (S, Y, Z, TP, ...) in three bf16 planes, plane pairs (i, j)
// with i + j < 3 summed, those of equal i + j in an accumulator of their own
// (delta.cuh says why). An operand's planes are one operand of three times the
// columns: the other operand is read once for all three (a 128 x 64 x 16 product
// reads 6 KB of shared memory in the time it multiplies 4 KB). dQ and dK, bf16
// themselves, are taken from operands in two planes (dY, Z, S0, dS1, M, R: 2^-18 of
// a value remain), without the product of two second planes. One plane would put
// four more roundings beside the result's own: 3e-3 to 4.4e-3 off (2-norm) instead
// of 1.7e-3.
//
// Shared-memory images are rows of 128 bytes (64 columns; 64 bytes where a tile
// of v has 32), 16-byte pieces swizzled as the tensor cores read them, panels of
// 64 columns one after the other. The same image serves as an operand whose rows
// are the outer index (K-major) or the summed one (MN-major).
#pragma once
#include "delta.cuh"
#include "kernels.cuh"

namespace rnn {

constexpr int TC_C = 64;        // steps of a chunk
constexpr int TC_EDGE = 8;      // chunks between the states kept in fp32 for dg
constexpr int TC_PANEL = 16384; // bytes of a panel of 128 rows
constexpr float BETA_MIN = 0x1p-60f;
// Which of its two sums dg_t is taken from, the row products' or (below) what reaches
// over the step. Off by (L2, T = 512, heads of 64, all steps with this g)
//   g                       -0.01   -0.1    -0.5    -1      -5      -10     -20
//   row products            8.0e-7  8.5e-7  4.8e-6  6.3e-6  1.6e-4  5.6e-2  1e3
//   what reaches over       5.9e-6  3.6e-6  5.3e-6  2.9e-6  3.4e-6  3.4e-6  3.6e-6
// The second costs a chunk of it 11 % of the back chain and 12 % of the grad kernel
// (418 us for 377 and 306 for 273 at the chain's size with all chunks), and a chunk
// without such a step nothing but the question.
constexpr float GATE_NEAR = -0.75f;
// What bf16 storage has in rho's place in rec (its kernels need beta rho alone): 2
// for a step whose g is below GATE_NEAR, 1 for the others of a chunk with such a step,
// 0 in a chunk without one.
constexpr int REC_NEAR = REC_RHO;

struct DeltaTcArgs {
  int B, T, Nk, N, Dk, Dv;
  int KP, nvt, nc, ne;  // Dk rounded to 16, tiles of BV columns of v, chunks, kept states a head
  // The chunks in `segs` segments of `seglen` (a multiple of TC_EDGE), which run
  // side by side once the states between them are known: the chain kernels first
  // run with maps = 1, each segment from zeros (H) and, forward, from the identity
  // (M), and S at a segment's end is M S + H (the gradient at its start M^T dS + H).
  int segs, seglen, maps;
  float *Mt, *Ht, *St;  // [B N][segs][KR][KR] M by columns, [B N][segs][nvt BV][KR] H and S at the start (backward: end), by columns
  const void *q, *k, *v;
  const float *g, *beta, *s0;
  const unsigned char* reset;
  const int* lengths;
  float scale;
  bool tma;
  void* o;
  float* last;
  unsigned* status;
  unsigned long long wait_limit_ns;
  float* rec;  // [items][REC_N][64]
  bf16* tp;    // [items][3][128 x 64 image]
  // what a backward needs besides (null: none comes)
  bf16* Sh;            // [items][nvt][2][KP x BV image] two planes of S0
  float *zf, *of;      // [items][nvt][BV / 4][64][4] z and o in fp32, as the threads hold them
  float* sf;           // [B N][ne][nvt][...] S at the end (0) and at every TC_EDGE-th chunk's start
  // backward
  const void* dO;
  const float* dlast;
  bf16* dSh;           // as Sh, of dS1
  bf16* dYl;           // [items][nvt][BV / 8][64][8] the second plane of dY (the first is dv)
  float* dots;         // [items][nvt][3][2][64]: z.dY, -v.dY, o.dO of half a tile's columns
  float* edge;         // [B N][ne][nvt][8]: <S, dS> there, by warp
  float* near;         // [items][64] dg without the next, of chunks with a step that wants it
  float* cross;        // [items][nvt][3] <S0, dS1>, by warp
  void *dq, *dk, *dv;
  float *dg, *dbeta, *ds0;
  float *pq, *pk;
};

// Tensor maps of the rows' tensors [B, T, heads, D] where their rows are whole
// 16-byte pieces (a.tma), boxes of 64 steps of a head: k and q by 64 columns, the
// others by a tile's.
struct TcMaps {
  CUtensorMap k, q, v, o, dO, dv;
};

// ---- tensor memory -----------------------------------------------------------------
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
template <int COLS> __device__ __forceinline__ void tm_alloc(uint32_t* slot) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "n"(COLS) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS> __device__ __forceinline__ void tm_free(uint32_t at) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "n"(COLS) : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tm_ld16(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
// x[N] = the sum of N columns, from column at on, of the three accumulators, STEP
// columns apart, that an operand's planes have
template <int N, int STEP> __device__ __forceinline__ void tm_sum(float (&x)[N], uint32_t at) {
#pragma unroll
  for (int c = 0; c < N; c += 16) {
    uint32_t a[3][16];
#pragma unroll
    for (int p = 0; p < 3; ++p) tm_ld16(a[p], at + p * STEP + c);
    tm_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) x[c + e] = __uint_as_float(a[0][e]) + (__uint_as_float(a[1][e]) + __uint_as_float(a[2][e]));
  }
}

// Instruction of 128 x n products, bf16 operands, fp32 accumulator.
__device__ __forceinline__ constexpr uint32_t tc_idesc(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         (8u << 24);
}
// Operand at `at`. K-major (rows = outer index): lbo 16; MN-major (rows = summed
// index): lbo the distance of the panels, or of the planes that make one operand
// of three times the columns. RB: bytes of a row. An address moves on by adding
// its 16-byte pieces to the descriptor.
template <int RB = 128> __device__ __forceinline__ uint64_t tc_desc(uint32_t at, uint32_t lbo) {
  return (uint64_t)((at >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(8 * RB >> 4) << 32) | (1ull << 46) |
         ((RB == 128 ? 2ull : 4ull) << 61);
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// the same, lanes 64 .. 127 of the accumulator left as they are
__device__ __forceinline__ void tc_mma_upper(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %5, %6, %6}, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(0u), "r"(0xffffffffu)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The end of a kernel, whose thread 0 has issued all products: they are over (also
// after a wait ran out) when the CTA goes on. bar is used here alone.
__device__ __forceinline__ void tc_finish(uint32_t bar, unsigned long long limit_ns) {
  if (threadIdx.x == 0) {
    bool failed = false;
    tc_commit(bar);
    mbar_wait_bounded<false>(bar, 0, limit_ns, nullptr, failed);
  }
  tm_fence_before();
  __syncthreads();
}

// Byte offset of 16-byte piece c of row r of an image with rows of RB bytes.
template <int RB> __device__ __forceinline__ uint32_t img(int r, int c) {
  return RB == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// 8 values as three planes of one 16-byte piece each
__device__ __forceinline__ void split8(const float* x, uint4 (&p)[3]) {
  uint32_t w[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      w[k][i] = *(const uint32_t*)&h;
      if (k < 2) {
        a -= __uint_as_float(w[k][i] << 16);
        b -= __uint_as_float(w[k][i] & 0xffff0000u);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) p[k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}
__device__ __forceinline__ uint4 round8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *(const uint32_t*)&h;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void widen8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// N values of row r, from column c0 (a multiple of 8) on, into the planes of an
// image (plane bytes apart)
template <int RB, int N> __device__ __forceinline__ void put_planes(unsigned char* im, int plane, int r, int c0, const float (&x)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 8) {
    uint4 p[3];
    split8(x + c, p);
    const uint32_t at = img<RB>(r, (c0 + c) >> 3);
#pragma unroll
    for (int k = 0; k < 3; ++k) *(uint4*)(im + k * plane + at) = p[k];
  }
}

// 64 rows of an input (rows `stride` elements apart), its columns c0 .. c0 + cols
// (at most 8 P), into rows row0 .. of panels; rows from `live` on and columns past
// D are zero and not read. Thread t of NTH has piece t % P of every NTH / P-th row.
template <int RB, int P, int NTH>
__device__ __forceinline__ void load_img(int t, unsigned char* im, int row0, const bf16* src, size_t stride, int live, int D,
                                         int c0, int cols, int panel_bytes) {
  constexpr int PR = RB / 16, STEP = NTH / P, IT = 64 / STEP;  // pieces of a panel's row
  static_assert(STEP >= 1 && IT >= 1, "whole rows a step");
  const int c = t % P, r = t / P, col = c0 + c * 8;
  if (c * 8 >= cols) return;
  unsigned char* d = im + (c / PR) * panel_bytes;
  const bf16* s = src + (size_t)r * stride + col;
  if (D % 8 == 0) {
    const uint32_t to = smem_u32(d);
    const bool in = col < D;
#pragma unroll 4
    for (int k = 0; k < IT; ++k, s += (size_t)STEP * stride) {
      const bool on = in && r + k * STEP < live;
      cp16(to + img<RB>(row0 + r + k * STEP, c % PR), on ? s : src, on);
    }
  } else {
#pragma unroll 4
    for (int k = 0; k < IT; ++k, s += (size_t)STEP * stride) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (r + k * STEP < live) {
        const unsigned short* p = (const unsigned short*)s;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < D) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
      }
      *(uint4*)(d + img<RB>(row0 + r + k * STEP, c % PR)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}
// The first `rows` rows of an image of 64 rows to the columns c0 .. of a tensor
// whose rows have D columns: 128 bytes (64) of a row to 8 (4) threads.
template <int RB, int NTH>
__device__ __forceinline__ void store_img(int t, const unsigned char* im, bf16* dst, size_t stride, int rows, int D, int c0) {
  constexpr int P = RB / 16, STEP = NTH / P;
  const int c = t % P, col = c0 + c * 8;
#pragma unroll 4
  for (int r = t / P; r < rows; r += STEP) {
    const uint4 v = *(const uint4*)(im + img<RB>(r, c));
    bf16* p = dst + (size_t)r * stride + col;
    if (D % 8 == 0) {
      if (col < D) *(uint4*)p = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < D) ((unsigned short*)p)[e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}
// `bytes` of an image that global memory holds as it stands, by one thread, counted
// by the barrier; and an image to global memory (bulk_commit_group and
// bulk_wait_group_read follow)
__device__ __forceinline__ void load_bulk(unsigned char* im, const void* src, uint32_t bytes, uint32_t bar) {
  mbar_arrive_expect_tx(bar, bytes);
  bulk_load_global(smem_u32(im), src, bytes, bar);
}
__device__ __forceinline__ void store_bulk(void* dst, const unsigned char* im, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(im)), "r"(bytes) : "memory");
}

// The products of one operand's K-major image (panels of 64 columns, 128 rows) with
// the MN-major planes at b (rows of RB bytes, `plane` bytes apart). Whole panels:
// their columns past KP are zero, the states' rows past it finite.
template <int RB, int PANELS>
__device__ __forceinline__ void tc_panels(uint32_t d, uint32_t a, uint32_t b, int plane, uint32_t id) {
  const uint64_t ad = tc_desc(a, 16), bd = tc_desc<RB>(b, plane);
#pragma unroll
  for (int k = 0; k < 4 * PANELS; ++k) tc_mma(d, ad + (k >> 2) * (TC_PANEL >> 4) + (k & 3) * 2, bd + k * RB, id, k);
}
template <int RB, int MT>
__device__ __forceinline__ void tc_wide(int panels, uint32_t d, uint32_t a, uint32_t b, int plane, uint32_t id) {
  if (MT == 1) {
    if (panels == 1) tc_panels<RB, 1>(d, a, b, plane, id);
    else tc_panels<RB, 2>(d, a, b, plane, id);
  } else {
    if (panels == 3) tc_panels<RB, 3>(d, a, b, plane, id);
    else tc_panels<RB, 4>(d, a, b, plane, id);
  }
}

// Rows `live` .. 63 of an image (from row0 on) are zero; one warp.
template <int RB> __device__ __forceinline__ void clear_rows(unsigned char* im, int row0, int live) {
  for (int i = (threadIdx.x & 31) * 16; i < (64 - live) * RB; i += 512) *(uint4*)(im + (row0 + live) * RB + i) = make_uint4(0, 0, 0, 0);
}
// Rows from t0 to T of a tile's columns are zero; all threads of the CTA.
template <int BV>
__device__ __forceinline__ void tc_zero_tail(bf16* p, size_t stride, int t0, int T, int c0, int D) {
  constexpr int P = BV / 8;
  const int c = c0 + threadIdx.x % P * 8;
  if (c >= D) return;
  for (int t = t0 + threadIdx.x / P; t < T; t += blockDim.x / P) {
    bf16* d = p + (size_t)t * stride + c;
    if (D % 8 == 0) {
      *(uint4*)d = make_uint4(0, 0, 0, 0);
    } else {
      for (int e = 0; e < 8; ++e)
        if (c + e < D) d[e] = __float2bfloat16_rn(0.0f);
    }
  }
}

__device__ __forceinline__ int tc_live(const DeltaTcArgs& a, int b, int ch) {
  int len = a.T;
  if (a.lengths) len = max(0, min(a.T, __ldg(a.lengths + b)));
  const long long left = (long long)len - (long long)ch * TC_C;
  return left < 0 ? 0 : (int)(left < TC_C ? left : TC_C);
}
__device__ __forceinline__ int tc_chunks(const DeltaTcArgs& a, int b) {
  int len = a.T;
  if (a.lengths) len = max(0, min(a.T, __ldg(a.lengths + b)));
  return (len + TC_C - 1) / TC_C;
}

// A tensor's map (host).
cudaError_t tc_map(CUtensorMap* m, const void* base, const DeltaTcArgs& a, int heads, int D, int cols);

}  // namespace rnn
