// 8-bit activation checkpoints: int8 values with one power-of-two scale per
// block of 32 rows of a column (include/rnn.h).
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "rnn.h"

namespace rnn {
namespace {

// One thread per (block of rows, column).
template <typename T>
__global__ void __launch_bounds__(128) act_pack_kernel(long long rows, int cols, const int* lengths, const T* x,
                                                       signed char* q, unsigned char* scales) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= cols) return;
  const long long blocks = (rows + ACT_BLOCK - 1) / ACT_BLOCK;
  for (long long k = blockIdx.y; k < blocks; k += gridDim.y) {
    const long long r0 = k * ACT_BLOCK, r1 = r0 + ACT_BLOCK < rows ? r0 + ACT_BLOCK : rows;
    const size_t base = (size_t)blockIdx.z * rows;
    const long long len = lengths ? lengths[blockIdx.z] : rows;
    unsigned top = 0;  // magnitudes compared as bits: NaN and infinity are the largest
    for (long long r = r0; r < r1; ++r)
      if (r < len) top = max(top, __float_as_uint(fabsf(to_f(x[(base + r) * cols + c]))));
    const unsigned s = act_scale_byte(__uint_as_float(top));
    const float inv = act_inv_scale(s);
    scales[((size_t)blockIdx.z * blocks + k) * cols + c] = (unsigned char)s;
    for (long long r = r0; r < r1; ++r)
      q[(base + r) * cols + c] =
          s != ACT_NONFINITE && r < len ? (signed char)act_quant(to_f(x[(base + r) * cols + c]), inv) : 0;
  }
}

template <typename T>
__global__ void __launch_bounds__(128) act_unpack_kernel(long long rows, int cols, const signed char* q,
                                                         const unsigned char* scales, T* x) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= cols) return;
  for (long long r = blockIdx.y; r < rows; r += gridDim.y)
    x[(size_t)r * cols + c] = from_f<T>((float)q[(size_t)r * cols + c] * act_scale(scales[(size_t)(r / ACT_BLOCK) * cols + c]));
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

}  // namespace

cudaError_t act_pack_run(int dtype, int batch, long long rows, int cols, const int* lengths, const void* x,
                         signed char* q, unsigned char* scales, cudaStream_t st) {
  const long long blocks = (rows + ACT_BLOCK - 1) / ACT_BLOCK;
  for (int b = 0; b < batch; b += 65535) {  // grid.z holds at most 65535
    const int n = batch - b < 65535 ? batch - b : 65535;
    const dim3 grid((cols + 127) / 128, (unsigned)(blocks < 65535 ? blocks : 65535), n);
    const size_t at = (size_t)b * rows * cols;
    const int* len = lengths ? lengths + b : nullptr;
    unsigned char* s = scales + (size_t)b * blocks * cols;
    if (dtype == RNN_BF16)
      act_pack_kernel<<<grid, 128, 0, st>>>(rows, cols, len, (const __nv_bfloat16*)x + at, q + at, s);
    else
      act_pack_kernel<<<grid, 128, 0, st>>>(rows, cols, len, (const float*)x + at, q + at, s);
    note_launch();
  }
  return cudaGetLastError();
}

}  // namespace rnn

using namespace rnn;

extern "C" {

size_t rnn_act_scale_bytes(long long rows, int cols) {
  return act_ok(rows, cols, RNN_F32) ? (size_t)((rows + ACT_BLOCK - 1) / ACT_BLOCK) * cols : 0;
}

int rnn_act_pack(long long rows, int cols, int dtype, const void* x, void* q, void* scales, void* stream) {
  if (!act_ok(rows, cols, dtype)) return RNN_EINVAL;
  if (rows == 0) return RNN_OK;
  if (!x || !q || !scales || !al16(x) || !al16(q) || !al16(scales)) return RNN_EINVAL;
  return cuda_status(act_pack_run(dtype, 1, rows, cols, nullptr, x, (signed char*)q, (unsigned char*)scales,
                                  (cudaStream_t)stream));
}

int rnn_act_unpack(long long rows, int cols, int dtype, const void* q, const void* scales, void* x, void* stream) {
  if (!act_ok(rows, cols, dtype)) return RNN_EINVAL;
  if (rows == 0) return RNN_OK;
  if (!x || !q || !scales || !al16(x) || !al16(q) || !al16(scales)) return RNN_EINVAL;
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((cols + 127) / 128, (unsigned)(rows < 65535 ? rows : 65535));
  if (dtype == RNN_BF16)
    act_unpack_kernel<<<grid, 128, 0, st>>>(rows, cols, (const signed char*)q, (const unsigned char*)scales, (__nv_bfloat16*)x);
  else
    act_unpack_kernel<<<grid, 128, 0, st>>>(rows, cols, (const signed char*)q, (const unsigned char*)scales, (float*)x);
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
