// Token embedding with scaling and its gradient (include/rnn.h).
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "rnn.h"

namespace rnn {
namespace {

template <typename T, typename I>
__global__ void __launch_bounds__(256) embed_fwd_kernel(long long n, int V, int E, const I* ids, const T* W, float scale,
                                                        T* out, unsigned* status) {
  for (long long i = blockIdx.x; i < n; i += gridDim.x) {
    const long long v = (long long)ids[i];
    const bool ok = v >= 0 && v < V;
    if (!ok && threadIdx.x == 0 && status) atomicOr(status, STATUS_RANGE);
    for (int e = threadIdx.x; e < E; e += 256)
      out[(size_t)i * E + e] = ok ? from_f<T>(to_f(W[(size_t)v * E + e]) * scale) : from_f<T>(0.0f);
  }
}

// One block per row of the table and 256 columns: every token in order.
template <typename T, typename I>
__global__ void __launch_bounds__(256) embed_bwd_kernel(long long n, int V, int E, const I* ids, long long pad,
                                                        const T* dout, float scale, T* dW, unsigned* status) {
  const int v = blockIdx.x, e = blockIdx.y * 256 + threadIdx.x;
  float s = 0.0f;
  for (long long i = 0; i < n; ++i) {
    const long long id = (long long)ids[i];
    if (id == v && v != pad && e < E) s += to_f(dout[(size_t)i * E + e]);
    if (v == 0 && (id < 0 || id >= V)) atomicOr(status, STATUS_RANGE);
  }
  if (e < E) dW[(size_t)v * E + e] = from_f<T>(s * scale);
}

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RNN_OK;
  fprintf(stderr, "librnn_gb300: CUDA error: %s\n", cudaGetErrorString(e));
  return RNN_ECUDA;
}
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool embed_ok(long long n, int V, int E, int dtype, int id_bytes) {
  return n >= 0 && n < (1ll << 31) && V >= 1 && E >= 1 && (dtype == RNN_F32 || dtype == RNN_BF16) &&
         (id_bytes == 4 || id_bytes == 8);
}

template <typename T, typename I>
void embed_fwd_launch(long long n, int V, int E, const void* ids, const void* W, float scale, void* out, unsigned* status,
                      cudaStream_t st) {
  embed_fwd_kernel<T, I><<<(unsigned)(n < 65535 ? n : 65535), 256, 0, st>>>(n, V, E, (const I*)ids, (const T*)W, scale,
                                                                            (T*)out, status);
}
template <typename T, typename I>
void embed_bwd_launch(long long n, int V, int E, const void* ids, long long pad, const void* dout, float scale, void* dW,
                      unsigned* status, cudaStream_t st) {
  embed_bwd_kernel<T, I><<<dim3(V, (E + 255) / 256), 256, 0, st>>>(n, V, E, (const I*)ids, pad, (const T*)dout, scale,
                                                                   (T*)dW, status);
}

}  // namespace
}  // namespace rnn

using namespace rnn;

extern "C" {

size_t rnn_embed_bwd_workspace_size(long long n, int V, int E) {
  return embed_ok(n, V, E, RNN_F32, 4) ? 256 : 0;
}

int rnn_embed_fwd(long long n, int V, int E, int dtype, int id_bytes, const void* ids, const void* W, float scale,
                  void* out, void* status_word, void* stream) {
  if (!embed_ok(n, V, E, dtype, id_bytes) || !W || (n > 0 && (!ids || !out))) return RNN_EINVAL;
  if (!al16(W) || !al16(out) || ((uintptr_t)status_word & 3u) || ((uintptr_t)ids & (id_bytes - 1))) return RNN_EINVAL;
  if (n == 0) return RNN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  unsigned* status = (unsigned*)status_word;
  if (dtype == RNN_BF16) {
    if (id_bytes == 4) embed_fwd_launch<__nv_bfloat16, int>(n, V, E, ids, W, scale, out, status, st);
    else embed_fwd_launch<__nv_bfloat16, long long>(n, V, E, ids, W, scale, out, status, st);
  } else {
    if (id_bytes == 4) embed_fwd_launch<float, int>(n, V, E, ids, W, scale, out, status, st);
    else embed_fwd_launch<float, long long>(n, V, E, ids, W, scale, out, status, st);
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

int rnn_embed_bwd(long long n, int V, int E, int dtype, int id_bytes, const void* ids, long long padding_idx,
                  const void* dout, float scale, void* dW, void* workspace, size_t ws_bytes, void* stream) {
  if (!embed_ok(n, V, E, dtype, id_bytes) || !dW || !workspace || (n > 0 && (!ids || !dout))) return RNN_EINVAL;
  if (!al16(dW) || !al16(dout) || !al16(workspace) || ((uintptr_t)ids & (id_bytes - 1))) return RNN_EINVAL;
  if (ws_bytes < rnn_embed_bwd_workspace_size(n, V, E)) return RNN_ENOSPC;
  cudaStream_t st = (cudaStream_t)stream;
  int rc = cuda_status(cudaMemsetAsync(workspace, 0, 256, st));
  if (rc) return rc;
  unsigned* status = (unsigned*)workspace;
  if (dtype == RNN_BF16) {
    if (id_bytes == 4) embed_bwd_launch<__nv_bfloat16, int>(n, V, E, ids, padding_idx, dout, scale, dW, status, st);
    else embed_bwd_launch<__nv_bfloat16, long long>(n, V, E, ids, padding_idx, dout, scale, dW, status, st);
  } else {
    if (id_bytes == 4) embed_bwd_launch<float, int>(n, V, E, ids, padding_idx, dout, scale, dW, status, st);
    else embed_bwd_launch<float, long long>(n, V, E, ids, padding_idx, dout, scale, dW, status, st);
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
