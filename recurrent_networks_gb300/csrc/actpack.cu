// 8-bit activation checkpoints: int8 values with one power-of-two scale per
// block of 32 rows of a column (include/rnn.h).
#include <limits.h>
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "rnn.h"

namespace rnn {
namespace {

// Four threads pack a block of 32 rows of V columns, 8 rows each (lanes 8
// apart: a warp has 8 V neighbouring columns, 128 bytes of a row where V is 8
// bf16 or 4 fp32). Every value is read once; 8 loads of 16 bytes a thread and
// 64 registers keep 128 KB of an SM's loads in flight: 65521 x 1024 bf16 40 us,
// 5.1 TB/s (a thread with all 32 rows took 160 registers, 52 us).
template <typename T, int V> struct Cols;
template <> struct Cols<__nv_bfloat16, 8> {
  static constexpr int W = 4, N = 2;  // words, columns of a word
  uint32_t w[4];
  __device__ void load(const __nv_bfloat16* p) { *(uint4*)w = __ldcs((const uint4*)p); }
};
template <> struct Cols<float, 4> {
  static constexpr int W = 4, N = 1;
  uint32_t w[4];
  __device__ void load(const float* p) { *(uint4*)w = __ldcs((const uint4*)p); }
};
template <> struct Cols<__nv_bfloat16, 1> {
  static constexpr int W = 1, N = 1;
  uint32_t w[1];
  __device__ void load(const __nv_bfloat16* p) { w[0] = *(const unsigned short*)p; }
};
template <> struct Cols<float, 1> {
  static constexpr int W = 1, N = 1;
  uint32_t w[1];
  __device__ void load(const float* p) { w[0] = *(const uint32_t*)p; }
};
template <typename T> __device__ __forceinline__ FV<1> word_values(uint32_t w, FV<1>*) {
  return {{__uint_as_float(sizeof(T) == 4 ? w : w << 16)}};
}
template <typename T> __device__ __forceinline__ FV<2> word_values(uint32_t w, FV<2>*) {
  return {{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}};
}
// V bytes at p
template <int V> __device__ __forceinline__ void store_bytes(void* p, const uint32_t (&b)[2]) {
  if constexpr (V == 8) *(uint2*)p = make_uint2(b[0], b[1]);
  else if constexpr (V == 4) *(uint32_t*)p = b[0];
  else *(unsigned char*)p = (unsigned char)b[0];
}

template <typename T, int V>
__global__ void __launch_bounds__(256) act_pack_kernel(long long rows, int cols, const T* x, signed char* q,
                                                       unsigned char* scales) {
  using X = Cols<T, V>;
  constexpr int W = X::W, N = X::N, ROWS = 8;
  const long long blocks = (rows + ACT_BLOCK - 1) / ACT_BLOCK;
  const int lane = threadIdx.x & 31, part = lane >> 3;
  const int groups = (cols + 8 * V - 1) / (8 * V);  // of 8 V columns, a warp's
  for (long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); id < blocks * groups; id += (long long)gridDim.x * 8) {
    const long long k = id / groups;
    const int c = ((int)(id % groups) * 8 + (lane & 7)) * V;
    const bool on = c < cols;
    const long long r0 = k * ACT_BLOCK + part * ROWS;
    const int n = on ? (int)max(0ll, min((long long)ROWS, rows - r0)) : 0;
    const size_t at = (size_t)r0 * cols + c;
    X v[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r < n) v[r].load(x + at + (size_t)r * cols);
      else
#pragma unroll
        for (int i = 0; i < W; ++i) v[r].w[i] = 0;
    }
    FV<N> inv[W];
    uint32_t bytes[2] = {0, 0};
    bool huge = false, odd = false;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      uint32_t top = 0;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) top = mag_max<T>(top, v[r].w[i]);
      top = mag_max<T>(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = mag_max<T>(top, __shfl_xor_sync(0xffffffffu, top, 16));
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const unsigned s = act_scale_byte(__uint_as_float(mag_bits<T>(top, j)));
        inv[i].v[j] = act_inv_scale(s);
        huge |= s == 248;
        odd |= s == ACT_NONFINITE;
        bytes[(i * N + j) / 4] |= s << (8 * ((i * N + j) % 4));
      }
    }
    if (on && part == 0) store_bytes<V>(scales + (size_t)k * cols + c, bytes);
    huge = __any_sync(0xffffffffu, huge);
    odd = __any_sync(0xffffffffu, odd);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r >= n) break;
      FV<N> t[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        t[i] = quant(word_values<T>(v[r].w[i], (FV<N>*)nullptr), inv[i], huge);
        if (odd) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (inv[i].v[j] == 0.0f) t[i].v[j] = 0.0f;
        }
      }
      uint32_t b[2];
      if constexpr (V == 1) {
        b[0] = __float_as_uint(t[0].v[0]);
      } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          auto value = [&](int k) { return t[(i * 4 + k) / N].v[(i * 4 + k) % N]; };
          b[i] = __byte_perm(low_bytes(value(0), value(1)), low_bytes(value(2), value(3)), 0x5410);
        }
      }
      store_bytes<V>(q + at + (size_t)r * cols, b);
    }
  }
}

// A thread unpacks 8 rows of V columns of one block: 65521 x 1024 bf16 35 us,
// 5.7 TB/s.
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
  return rows >= 0 && rows < (1ll << 40) && cols >= 1 && cols <= INT_MAX - 64 && (dtype == RNN_F32 || dtype == RNN_BF16);
}

unsigned act_blocks(long long n) { return (unsigned)(n < (1ll << 30) ? n : (1ll << 30)); }
template <typename T, int V>
cudaError_t act_pack_run(long long rows, int cols, const void* x, void* q, void* scales, cudaStream_t st) {
  const long long warps = (rows + ACT_BLOCK - 1) / ACT_BLOCK * ((cols + 8 * V - 1) / (8 * V));
  act_pack_kernel<T, V><<<act_blocks((warps + 7) / 8), 256, 0, st>>>(rows, cols, (const T*)x, (signed char*)q,
                                                                     (unsigned char*)scales);
  note_launch();
  return cudaGetLastError();
}
template <typename T, int V>
cudaError_t act_unpack_run(long long rows, int cols, const void* q, const void* scales, void* x, cudaStream_t st) {
  const long long threads = (rows + 7) / 8 * ((cols + V - 1) / V);
  act_unpack_kernel<T, V><<<act_blocks((threads + 127) / 128), 128, 0, st>>>(rows, cols, (const signed char*)q,
                                                                             (const unsigned char*)scales, (T*)x);
  note_launch();
  return cudaGetLastError();
}
int act_call(bool pack, long long rows, int cols, int dtype, void* x, void* q, void* scales, void* stream) {
  if (!act_ok(rows, cols, dtype)) return RNN_EINVAL;
  if (rows == 0) return RNN_OK;
  if (!x || !q || !scales || !al16(x) || !al16(q) || !al16(scales)) return RNN_EINVAL;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = dtype == RNN_BF16;
  if (pack)
    return cuda_status(bf ? cols % 8 == 0 ? act_pack_run<__nv_bfloat16, 8>(rows, cols, x, q, scales, st)
                                          : act_pack_run<__nv_bfloat16, 1>(rows, cols, x, q, scales, st)
                       : cols % 4 == 0 ? act_pack_run<float, 4>(rows, cols, x, q, scales, st)
                                       : act_pack_run<float, 1>(rows, cols, x, q, scales, st));
  const bool four = cols % 4 == 0;
  return cuda_status(bf ? four ? act_unpack_run<__nv_bfloat16, 4>(rows, cols, q, scales, x, st)
                               : act_unpack_run<__nv_bfloat16, 1>(rows, cols, q, scales, x, st)
                     : four ? act_unpack_run<float, 4>(rows, cols, q, scales, x, st)
                            : act_unpack_run<float, 1>(rows, cols, q, scales, x, st));
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
