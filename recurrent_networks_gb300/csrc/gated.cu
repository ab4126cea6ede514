// The gated linear scan: forward, backward and the single-token step, and
// their C entry points (include/rnn.h).
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "rnn.h"

namespace rnn {
namespace {

struct GatedArgs {
  int B, T, C, chunks;  // C = N D channels
  const void* Wx;
  const void* bias;
  const float* s0;
  const unsigned char* reset;
  const int* lengths;
  void* h;
  float* last;
  float* carry;              // [B][chunks][C]: the state before every chunk
  const signed char* q;      // 8-bit pre-activations (backward)
  const unsigned char* qs;
  const void* dh;
  const float* dlast;
  void* dWx;
  float* ds0;
  float* dbp;                // [B][G][C]
};

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// One thread per channel, the steps in order.
template <typename T, int FN>
__global__ void __launch_bounds__(128) gated_fwd_kernel(GatedArgs p) {
  constexpr int G = gated_gates(FN);
  constexpr bool FAST = sizeof(T) == 2;
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  if (id >= (long long)p.B * p.C) return;
  const int b = (int)(id / p.C), ch = (int)(id % p.C);
  const int len = clamp_len(p.lengths, b, p.T);
  const T* x = (const T*)p.Wx + (size_t)b * p.T * G * p.C + ch;
  T* h = (T*)p.h + (size_t)b * p.T * p.C + ch;
  float bias[G];
#pragma unroll
  for (int g = 0; g < G; ++g) bias[g] = p.bias ? to_f(((const T*)p.bias)[(size_t)g * p.C + ch]) : 0.0f;
  float c = p.s0 ? p.s0[id] : 0.0f;
  for (int t = 0; t < p.T; ++t) {
    if (p.carry && t % GATED_CHUNK == 0) p.carry[((size_t)b * p.chunks + t / GATED_CHUNK) * p.C + ch] = c;
    float y = 0.0f;
    if (t < len) {
      float a[G], f, u;
#pragma unroll
      for (int g = 0; g < G; ++g) a[g] = to_f(x[((size_t)t * G + g) * p.C]) + bias[g];
      gated_coeff<FN, FAST>(a, f, u);
      const bool rst = p.reset && p.reset[(size_t)b * p.T + t];
      c = rst ? u : fmaf(f, c, u);
      y = gated_out<FN, FAST>(a, c);
    }
    h[(size_t)t * p.C] = from_f<T>(y);
  }
  if (p.last) p.last[id] = c;
}

template <typename T, int FN>
__global__ void __launch_bounds__(128) gated_bwd_kernel(GatedArgs p) {
  constexpr int G = gated_gates(FN);
  constexpr bool FAST = sizeof(T) == 2;
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  if (id >= (long long)p.B * p.C) return;
  const int b = (int)(id / p.C), ch = (int)(id % p.C);
  const int len = clamp_len(p.lengths, b, p.T);
  const int qblocks = (p.T + ACT_BLOCK - 1) / ACT_BLOCK;
  float bias[G], db[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    bias[g] = p.bias ? to_f(((const T*)p.bias)[(size_t)g * p.C + ch]) : 0.0f;
    db[g] = 0.0f;
  }
  auto load = [&](int t, float* a) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const size_t at = (((size_t)b * p.T + t) * G + g) * p.C + ch;
      if (p.q) {
        const unsigned s = p.qs[(((size_t)b * qblocks + t / ACT_BLOCK) * G + g) * p.C + ch];
        a[g] = (float)p.q[at] * act_scale(s) + bias[g];
      } else {
        a[g] = to_f(((const T*)p.Wx)[at]) + bias[g];
      }
    }
  };
  float carry = p.dlast ? p.dlast[id] : 0.0f;  // f_{t+1} delta_{t+1}
  float cs[GATED_CHUNK];
  for (int k = p.chunks - 1; k >= 0; --k) {
    const int t0 = k * GATED_CHUNK, t1 = min(p.T, t0 + GATED_CHUNK);
    const float start = p.carry[((size_t)b * p.chunks + k) * p.C + ch];
    float c = start;
    for (int t = t0; t < min(t1, len); ++t) {
      float a[G], f, u;
      load(t, a);
      gated_coeff<FN, FAST>(a, f, u);
      c = p.reset && p.reset[(size_t)b * p.T + t] ? u : fmaf(f, c, u);
      cs[t - t0] = c;
    }
    for (int t = t1 - 1; t >= t0; --t) {
      float da[G];
#pragma unroll
      for (int g = 0; g < G; ++g) da[g] = 0.0f;
      if (t < len) {
        float a[G], f, u;
        load(t, a);
        gated_coeff<FN, FAST>(a, f, u);
        const bool rst = p.reset && p.reset[(size_t)b * p.T + t];
        const float dh = p.dh ? to_f(((const T*)p.dh)[((size_t)b * p.T + t) * p.C + ch]) : 0.0f;
        const float delta = carry + gated_into<FN, FAST>(a, dh);
        const float cp = rst ? 0.0f : (t > t0 ? cs[t - t0 - 1] : start);
        gated_grad<FN, FAST>(a, cp, cs[t - t0], dh, delta, da);
        carry = rst ? 0.0f : f * delta;
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        db[g] += da[g];
        if (p.dWx) ((T*)p.dWx)[(((size_t)b * p.T + t) * G + g) * p.C + ch] = from_f<T>(da[g]);
      }
    }
  }
  if (p.ds0) p.ds0[id] = carry;
  if (p.dbp) {
#pragma unroll
    for (int g = 0; g < G; ++g) p.dbp[((size_t)b * G + g) * p.C + ch] = db[g];
  }
}

// db[j] = sum over `rows` of dbp[row][j], in row order within 8 interleaved
// lanes, then the lanes in order.
template <typename T>
__global__ void __launch_bounds__(256) gated_db_kernel(const float* dbp, T* db, int rows, int cols) {
  __shared__ float red[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + tx;
  float s = 0.0f;
  if (j < cols)
    for (int r = ty; r < rows; r += 8) s += dbp[(size_t)r * cols + j];
  red[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && j < cols) {
    for (int k = 1; k < 8; ++k) s += red[k][tx];
    db[j] = from_f<T>(s);
  }
}

struct StepArgs {
  int rows, C, slots;
  const void* Wx;
  const void* bias;
  const int* slot;
  const float* pool;
  float* pool_out;
  void* h;
  unsigned* status;
};

template <typename T, int FN>
__global__ void __launch_bounds__(128) gated_step_kernel(StepArgs p) {
  constexpr int G = gated_gates(FN);
  constexpr bool FAST = sizeof(T) == 2;
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  if (id >= (long long)p.rows * p.C) return;
  const int m = (int)(id / p.C), ch = (int)(id % p.C);
  const int slot = p.slot ? p.slot[m] : m;
  float y = 0.0f;
  if (slot >= 0 && slot < p.slots) {
    float a[G], f, u;
#pragma unroll
    for (int g = 0; g < G; ++g)
      a[g] = to_f(((const T*)p.Wx)[((size_t)m * G + g) * p.C + ch]) +
             (p.bias ? to_f(((const T*)p.bias)[(size_t)g * p.C + ch]) : 0.0f);
    gated_coeff<FN, FAST>(a, f, u);
    const size_t at = (size_t)slot * p.C + ch;
    const float c = fmaf(f, p.pool[at], u);
    p.pool_out[at] = c;
    y = gated_out<FN, FAST>(a, c);
  } else if (slot >= p.slots && ch == 0 && p.status) {
    atomicOr(p.status, STATUS_RANGE);
  }
  ((T*)p.h)[id] = from_f<T>(y);
}

// ---- host ----------------------------------------------------------------------
int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RNN_OK;
  fprintf(stderr, "librnn_gb300: CUDA error: %s\n", cudaGetErrorString(e));
  return RNN_ECUDA;
}
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

bool gated_dims_ok(const rnn_gated_dims_t* d) {
  return d && d->B >= 1 && d->T >= 0 && d->N >= 1 && d->D >= 1 && (d->function == RNN_LINEAR || d->function == RNN_LINEAR_COUPLED) &&
         (d->dtype == RNN_F32 || d->dtype == RNN_BF16) && (d->checkpoint == RNN_CKPT_NONE || d->checkpoint == RNN_CKPT_INT8) &&
         (long long)d->N * d->D <= (1 << 28) && (unsigned long long)d->B * d->N * d->D < (1ull << 37);
}

struct GatedSizes {
  int G, C, chunks, qblocks;
  size_t esize, carry, q, qs, tape, dbp;
};
GatedSizes gated_sizes(const rnn_gated_dims_t* d) {
  GatedSizes z;
  z.G = gated_gates(d->function);
  z.C = d->N * d->D;
  z.chunks = (d->T + GATED_CHUNK - 1) / GATED_CHUNK;
  z.qblocks = (d->T + ACT_BLOCK - 1) / ACT_BLOCK;
  z.esize = d->dtype == RNN_BF16 ? 2 : 4;
  z.carry = up256((size_t)d->B * z.chunks * z.C * sizeof(float));
  const bool q8 = d->checkpoint == RNN_CKPT_INT8;
  z.q = q8 ? up256((size_t)d->B * d->T * z.G * z.C) : 0;
  z.qs = q8 ? up256((size_t)d->B * z.qblocks * z.G * z.C) : 0;
  z.tape = z.carry + z.q + z.qs;
  z.dbp = up256((size_t)d->B * z.G * z.C * sizeof(float));
  return z;
}

template <typename T>
cudaError_t gated_launch(int fn, bool bwd, const GatedArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)(((long long)a.B * a.C + 127) / 128);
  if (fn == GATED_LINEAR) {
    if (bwd) gated_bwd_kernel<T, GATED_LINEAR><<<grid, 128, 0, st>>>(a);
    else gated_fwd_kernel<T, GATED_LINEAR><<<grid, 128, 0, st>>>(a);
  } else {
    if (bwd) gated_bwd_kernel<T, GATED_COUPLED><<<grid, 128, 0, st>>>(a);
    else gated_fwd_kernel<T, GATED_COUPLED><<<grid, 128, 0, st>>>(a);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace
}  // namespace rnn

using namespace rnn;

extern "C" {

int rnn_gated_num_gates(int function) {
  return function == RNN_LINEAR || function == RNN_LINEAR_COUPLED ? gated_gates(function) : -1;
}

size_t rnn_gated_tape_size(const rnn_gated_dims_t* d) { return gated_dims_ok(d) ? gated_sizes(d).tape : 0; }

size_t rnn_gated_workspace_size(const rnn_gated_dims_t* d, int kind) {
  if (!gated_dims_ok(d) || (kind != RNN_WS_FWD && kind != RNN_WS_BWD)) return 0;
  return 256 + (kind == RNN_WS_BWD ? gated_sizes(d).dbp : 0);
}

int rnn_gated_fwd(const rnn_gated_dims_t* d, const void* Wx, const void* b, const void* state0,
                  const unsigned char* reset, const int* lengths, void* h, void* last, void* tape,
                  void* workspace, size_t ws_bytes, void* stream) {
  if (!gated_dims_ok(d) || !workspace || (d->T > 0 && (!Wx || !h))) return RNN_EINVAL;
  const void* ptrs[] = {Wx, b, state0, h, last, tape, workspace};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (lengths && ((uintptr_t)lengths & 3u)) return RNN_EINVAL;
  if (ws_bytes < rnn_gated_workspace_size(d, RNN_WS_FWD)) return RNN_ENOSPC;
  cudaStream_t st = (cudaStream_t)stream;
  const GatedSizes z = gated_sizes(d);
  int rc = cuda_status(cudaMemsetAsync(workspace, 0, 256, st));
  if (rc) return rc;
  if (d->T == 0) {
    const size_t bytes = (size_t)d->B * z.C * sizeof(float);
    if (!last) return RNN_OK;
    return cuda_status(state0 ? cudaMemcpyAsync(last, state0, bytes, cudaMemcpyDeviceToDevice, st)
                              : cudaMemsetAsync(last, 0, bytes, st));
  }
  GatedArgs a{};
  a.B = d->B; a.T = d->T; a.C = z.C; a.chunks = z.chunks;
  a.Wx = Wx; a.bias = b; a.s0 = (const float*)state0; a.reset = reset; a.lengths = lengths;
  a.h = h; a.last = (float*)last; a.carry = (float*)tape;
  rc = cuda_status(d->dtype == RNN_BF16 ? gated_launch<__nv_bfloat16>(d->function, false, a, st)
                                        : gated_launch<float>(d->function, false, a, st));
  if (rc == RNN_OK && tape && d->checkpoint == RNN_CKPT_INT8)
    rc = cuda_status(act_pack_run(d->dtype, d->B, d->T, z.G * z.C, lengths, Wx, (signed char*)tape + z.carry,
                                  (unsigned char*)tape + z.carry + z.q, st));
  return rc;
}

int rnn_gated_bwd(const rnn_gated_dims_t* d, const void* Wx, const void* b, const unsigned char* reset,
                  const int* lengths, const void* tape, const void* dh, const void* dlast, void* dWx, void* db,
                  void* dstate0, void* workspace, size_t ws_bytes, void* stream) {
  if (!gated_dims_ok(d) || !workspace) return RNN_EINVAL;
  const bool q8 = d->checkpoint == RNN_CKPT_INT8;
  if (d->T > 0 && (!tape || (!q8 && !Wx))) return RNN_EINVAL;
  const void* ptrs[] = {Wx, b, tape, dh, dlast, dWx, db, dstate0, workspace};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (lengths && ((uintptr_t)lengths & 3u)) return RNN_EINVAL;
  if (ws_bytes < rnn_gated_workspace_size(d, RNN_WS_BWD)) return RNN_ENOSPC;
  cudaStream_t st = (cudaStream_t)stream;
  const GatedSizes z = gated_sizes(d);
  int rc = cuda_status(cudaMemsetAsync(workspace, 0, 256, st));
  if (rc) return rc;
  if (d->T == 0) {
    const size_t bytes = (size_t)d->B * z.C * sizeof(float);
    if (dstate0) {
      rc = cuda_status(dlast ? cudaMemcpyAsync(dstate0, dlast, bytes, cudaMemcpyDeviceToDevice, st)
                             : cudaMemsetAsync(dstate0, 0, bytes, st));
      if (rc) return rc;
    }
    return db ? cuda_status(cudaMemsetAsync(db, 0, (size_t)z.G * z.C * z.esize, st)) : RNN_OK;
  }
  GatedArgs a{};
  a.B = d->B; a.T = d->T; a.C = z.C; a.chunks = z.chunks;
  a.Wx = Wx; a.bias = b; a.reset = reset; a.lengths = lengths;
  a.carry = (float*)tape;
  if (q8) {
    a.q = (const signed char*)tape + z.carry;
    a.qs = (const unsigned char*)tape + z.carry + z.q;
  }
  a.dh = dh; a.dlast = (const float*)dlast; a.dWx = dWx; a.ds0 = (float*)dstate0;
  a.dbp = db ? (float*)((char*)workspace + 256) : nullptr;
  rc = cuda_status(d->dtype == RNN_BF16 ? gated_launch<__nv_bfloat16>(d->function, true, a, st)
                                        : gated_launch<float>(d->function, true, a, st));
  if (rc || !db) return rc;
  const int cols = z.G * z.C;
  if (d->dtype == RNN_BF16)
    gated_db_kernel<<<(cols + 31) / 32, 256, 0, st>>>(a.dbp, (__nv_bfloat16*)db, d->B, cols);
  else
    gated_db_kernel<<<(cols + 31) / 32, 256, 0, st>>>(a.dbp, (float*)db, d->B, cols);
  note_launch();
  return cuda_status(cudaGetLastError());
}

int rnn_gated_step(int rows, int slots, int N, int D, int function, int dtype, const void* Wx, const void* b,
                   const int* slot, const void* pool, void* pool_out, void* h, void* status, void* stream) {
  if (rows < 0 || slots < 1 || N < 1 || D < 1 || (long long)N * D > (1 << 28) || rnn_gated_num_gates(function) < 0 ||
      (dtype != RNN_F32 && dtype != RNN_BF16) || (!slot && rows > slots))
    return RNN_EINVAL;
  if (!pool || !pool_out || (rows > 0 && (!Wx || !h))) return RNN_EINVAL;
  const void* ptrs[] = {Wx, b, pool, pool_out, h};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (((uintptr_t)slot & 3u) || ((uintptr_t)status & 3u)) return RNN_EINVAL;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) return RNN_OK;
  StepArgs a{rows, N * D, slots, Wx, b, slot, (const float*)pool, (float*)pool_out, h, (unsigned*)status};
  const unsigned grid = (unsigned)(((long long)rows * a.C + 127) / 128);
  if (dtype == RNN_BF16) {
    if (function == RNN_LINEAR) gated_step_kernel<__nv_bfloat16, GATED_LINEAR><<<grid, 128, 0, st>>>(a);
    else gated_step_kernel<__nv_bfloat16, GATED_COUPLED><<<grid, 128, 0, st>>>(a);
  } else {
    if (function == RNN_LINEAR) gated_step_kernel<float, GATED_LINEAR><<<grid, 128, 0, st>>>(a);
    else gated_step_kernel<float, GATED_COUPLED><<<grid, 128, 0, st>>>(a);
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
