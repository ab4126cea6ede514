// 8-bit activation checkpoints: int8 values with one power-of-two scale per
// block of 32 rows of a column (include/rnn.h).
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "rnn.h"

namespace rnn {
namespace {

// A thread packs one block of 32 rows of V columns, a warp 32 V neighbouring
// columns. All rows are loaded before the scale is known, so each value is read
// once: 32 loads in flight hide the memory's latency. V = 4 where the columns
// allow (8- or 16-byte loads, 4-byte stores of q), else 1.
template <typename T, int V> struct Cols;
template <> struct Cols<__nv_bfloat16, 4> {
  uint2 r;
  __device__ void load(const __nv_bfloat16* p) { r = __ldcs((const uint2*)p); }
  __device__ void clear() { r = make_uint2(0, 0); }
  __device__ float get(int v) const {
    const uint32_t w = v < 2 ? r.x : r.y;
    return __uint_as_float(v & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <> struct Cols<float, 4> {
  float4 r;
  __device__ void load(const float* p) { r = __ldcs((const float4*)p); }
  __device__ void clear() { r = make_float4(0, 0, 0, 0); }
  __device__ float get(int v) const { return v == 0 ? r.x : v == 1 ? r.y : v == 2 ? r.z : r.w; }
};
template <typename T> struct Cols<T, 1> {
  T r;
  __device__ void load(const T* p) { r = *p; }
  __device__ void clear() { r = from_f<T>(0.0f); }
  __device__ float get(int) const { return to_f(r); }
};
__device__ __forceinline__ void store_q(signed char* p, const int (&q)[4]) {
  *(uint32_t*)p = (q[0] & 255) | (q[1] & 255) << 8 | (q[2] & 255) << 16 | (uint32_t)q[3] << 24;
}
__device__ __forceinline__ void store_q(signed char* p, const int (&q)[1]) { *p = (signed char)q[0]; }

template <typename T, int V>
__global__ void __launch_bounds__(128) act_pack_kernel(long long rows, int cols, const T* x, signed char* q,
                                                       unsigned char* scales) {
  const long long blocks = (rows + ACT_BLOCK - 1) / ACT_BLOCK;
  const int groups = (cols + V - 1) / V;
  for (long long id = (long long)blockIdx.x * 128 + threadIdx.x; id < blocks * groups;
       id += (long long)gridDim.x * 128) {
    const long long k = id / groups;
    const int c = (int)(id % groups) * V;
    const int n = (int)(rows - k * ACT_BLOCK < ACT_BLOCK ? rows - k * ACT_BLOCK : ACT_BLOCK);
    const size_t at = (size_t)k * ACT_BLOCK * cols + c;
    Cols<T, V> w[ACT_BLOCK];
#pragma unroll
    for (int r = 0; r < ACT_BLOCK; ++r) {
      if (r < n) w[r].load(x + at + (size_t)r * cols);
      else w[r].clear();
    }
    float inv[V];
    bool fin[V];
    uint32_t bytes = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint32_t top = 0;  // magnitudes compared as bits: NaN and infinity are the largest
#pragma unroll
      for (int r = 0; r < ACT_BLOCK; ++r) top = max(top, __float_as_uint(fabsf(w[r].get(v))));
      const unsigned s = act_scale_byte(__uint_as_float(top));
      inv[v] = act_inv_scale(s);
      fin[v] = s != ACT_NONFINITE;
      bytes |= s << (8 * v);
    }
    unsigned char* sc = scales + (size_t)k * cols + c;
    if (V == 4) *(uint32_t*)sc = bytes;
    else *sc = (unsigned char)bytes;
#pragma unroll
    for (int r = 0; r < ACT_BLOCK; ++r) {
      if (r >= n) break;
      int b[V];
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] = fin[v] ? act_quant(w[r].get(v), inv[v]) : 0;
      store_q(q + at + (size_t)r * cols, b);
    }
  }
}

// A thread unpacks 8 rows of V columns of one block.
template <typename T> __device__ __forceinline__ void store_cols(T* p, const float (&x)[1]) { *p = from_f<T>(x[0]); }
__device__ __forceinline__ void store_cols(float* p, const float (&x)[4]) {
  *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_cols(__nv_bfloat16* p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *(uint2*)p = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
}
template <typename T, int V>
__global__ void __launch_bounds__(128) act_unpack_kernel(long long rows, int cols, const signed char* q,
                                                         const unsigned char* scales, T* x) {
  constexpr int ROWS = 8;
  const int groups = (cols + V - 1) / V;
  const long long parts = (rows + ROWS - 1) / ROWS;
  for (long long id = (long long)blockIdx.x * 128 + threadIdx.x; id < parts * groups;
       id += (long long)gridDim.x * 128) {
    const long long r0 = id / groups * ROWS;
    const int c = (int)(id % groups) * V;
    const int n = (int)(rows - r0 < ROWS ? rows - r0 : ROWS);
    const size_t at = (size_t)r0 * cols + c;
    const unsigned char* sc = scales + (size_t)(r0 / ACT_BLOCK) * cols + c;
    uint32_t w[ROWS], s;
    s = V == 4 ? __ldg((const uint32_t*)sc) : __ldg(sc);
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (r < n) w[r] = V == 4 ? __ldcs((const uint32_t*)(q + at + (size_t)r * cols)) : (uint32_t)(unsigned char)q[at + (size_t)r * cols];
    float scale[V];
#pragma unroll
    for (int v = 0; v < V; ++v) scale[v] = act_scale(s >> (8 * v) & 255);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r >= n) break;
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = (float)(signed char)(w[r] >> (8 * v)) * scale[v];
      store_cols(x + at + (size_t)r * cols, y);
    }
  }
}

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RNN_OK;
  fprintf(stderr, "librnn_gb300: CUDA error: %s\n", cudaGetErrorString(e));
  return RNN_ECUDA;
}
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool act_ok(long long rows, int cols, int dtype) {
  return rows >= 0 && rows < (1ll << 40) && cols >= 1 && (dtype == RNN_F32 || dtype == RNN_BF16);
}

unsigned act_blocks(long long threads) {
  const long long n = (threads + 127) / 128;
  return (unsigned)(n < (1ll << 30) ? n : (1ll << 30));
}
template <typename T, int V>
cudaError_t act_run(bool pack, long long rows, int cols, void* x, void* q, void* scales, cudaStream_t st) {
  const long long groups = (cols + V - 1) / V;
  if (pack)
    act_pack_kernel<T, V><<<act_blocks((rows + ACT_BLOCK - 1) / ACT_BLOCK * groups), 128, 0, st>>>(
        rows, cols, (const T*)x, (signed char*)q, (unsigned char*)scales);
  else
    act_unpack_kernel<T, V><<<act_blocks((rows + 7) / 8 * groups), 128, 0, st>>>(
        rows, cols, (const signed char*)q, (const unsigned char*)scales, (T*)x);
  note_launch();
  return cudaGetLastError();
}
int act_call(bool pack, long long rows, int cols, int dtype, void* x, void* q, void* scales, void* stream) {
  if (!act_ok(rows, cols, dtype)) return RNN_EINVAL;
  if (rows == 0) return RNN_OK;
  if (!x || !q || !scales || !al16(x) || !al16(q) || !al16(scales)) return RNN_EINVAL;
  cudaStream_t st = (cudaStream_t)stream;
  const bool four = cols % 4 == 0;
  if (dtype == RNN_BF16)
    return cuda_status(four ? act_run<__nv_bfloat16, 4>(pack, rows, cols, x, q, scales, st)
                            : act_run<__nv_bfloat16, 1>(pack, rows, cols, x, q, scales, st));
  return cuda_status(four ? act_run<float, 4>(pack, rows, cols, x, q, scales, st)
                          : act_run<float, 1>(pack, rows, cols, x, q, scales, st));
}

}  // namespace
}  // namespace rnn

using namespace rnn;

extern "C" {

size_t rnn_act_scale_bytes(long long rows, int cols) {
  return act_ok(rows, cols, RNN_F32) ? (size_t)((rows + ACT_BLOCK - 1) / ACT_BLOCK) * cols : 0;
}

int rnn_act_pack(long long rows, int cols, int dtype, const void* x, void* q, void* scales, void* stream) {
  return act_call(true, rows, cols, dtype, (void*)x, q, scales, stream);
}

int rnn_act_unpack(long long rows, int cols, int dtype, const void* q, const void* scales, void* x, void* stream) {
  return act_call(false, rows, cols, dtype, x, (void*)q, (void*)scales, stream);
}

}  // extern "C"
