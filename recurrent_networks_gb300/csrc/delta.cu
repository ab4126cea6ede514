// Gated delta rule: C entry points, sizes, and the single-token step on a pool
// of states (include/rnn.h).
#include <limits.h>
#include <stdio.h>

#include "delta.h"
#include "delta_tc.cuh"
#include "kernels.cuh"
#include "rnn.h"

namespace rnn {
namespace {

// ---- one step -------------------------------------------------------------------
struct StepArgs {
  int rows, slots, Nk, N, Dk, Dv, tiles;
  const void *q, *k, *v;
  const float *g, *beta;
  const int* slot;
  const float* pool;
  float* out;
  float scale;
  void* o;
  unsigned* status;
};

// A CTA takes 32 columns of one row's and head's state: the state is read once
// into registers (8 rows of 4 columns a thread, or 32 rows of one where rows are
// not whole 16-byte vectors), k^T S and q^T S are summed over the CTA, and
// o = q^T S' = a q^T S + (q.k) u needs no second pass before the new state is
// written. Bound by memory, 8 bytes a state element: 51 us for 237 MB (256 rows of 8
// heads of 128 x 128, an eighth unused; 4.6 TB/s, 35 us at the copy's rate).
template <typename T, int VEC> __global__ void __launch_bounds__(256) delta_step_kernel(StepArgs p) {
  constexpr int CL = 32 / VEC, RG = 256 / CL, NR = 256 / RG;  // column lanes, row groups, rows a thread
  __shared__ float ks[256], qs[256], red[8][2][32], dot[8], us[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = (int)(blockIdx.x % p.tiles), mn = (int)(blockIdx.x / p.tiles), n = mn % p.N, m = mn / p.N;
  const int c0 = tile * 32, cols = min(32, p.Dv - c0);
  const int slot = p.slot ? __ldg(p.slot + m) : m;
  T* o = (T*)p.o + ((size_t)m * p.N + n) * p.Dv + c0;
  if (slot < 0 || slot >= p.slots) {
    if (tid < cols) o[tid] = from_f<T>(0.0f);
    if (slot >= p.slots && tile == 0 && n == 0 && tid == 0 && p.status) atomicOr(p.status, STATUS_RANGE);
    return;
  }
  const int cl = tid % CL, rg = tid / CL, c = cl * VEC;
  const size_t at = (((size_t)slot * p.N + n) * p.Dk) * p.Dv + c0 + c;
  float s[NR][VEC];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = rg + RG * i;
    const bool on = r < p.Dk && c < cols;
    if constexpr (VEC == 4) {
      const float4 x = on ? __ldcs((const float4*)(p.pool + at + (size_t)r * p.Dv)) : make_float4(0, 0, 0, 0);
      s[i][0] = x.x, s[i][1] = x.y, s[i][2] = x.z, s[i][3] = x.w;
    } else {
      s[i][0] = on ? __ldcs(p.pool + at + (size_t)r * p.Dv) : 0.0f;
    }
  }
  const size_t kat = ((size_t)m * p.Nk + n / (p.N / p.Nk)) * p.Dk;
  float kv = 0.0f, qv = 0.0f;
  if (tid < p.Dk) {
    kv = to_f(((const T*)p.k)[kat + tid]);
    qv = to_f(((const T*)p.q)[kat + tid]);
  }
  ks[tid] = kv;
  qs[tid] = qv;
  float d = kv * qv;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
  if (lane == 0) dot[warp] = d;
  const float decay = expf(p.g[(size_t)m * p.N + n]);
  __syncthreads();
  float sk[VEC] = {}, sq[VEC] = {};
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = rg + RG * i;
    const float kr = ks[r], qr = qs[r];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      s[i][e] = decay != 0.0f ? decay * s[i][e] : 0.0f;  // nothing is left of the state, whatever it holds
      sk[e] += kr * s[i][e];
      sq[e] += qr * s[i][e];
    }
  }
  if constexpr (CL < 32) {  // the warp's row groups
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
      for (int k = CL; k < 32; k <<= 1) {
        sk[e] += __shfl_xor_sync(0xffffffffu, sk[e], k);
        sq[e] += __shfl_xor_sync(0xffffffffu, sq[e], k);
      }
  }
  if (lane < CL) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      red[warp][0][c + e] = sk[e];
      red[warp][1][c + e] = sq[e];
    }
  }
  __syncthreads();
  if (tid < 32) {
    float x = 0.0f, y = 0.0f, qk = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      x += red[w][0][tid];
      y += red[w][1][tid];
      qk += dot[w];
    }
    float u = 0.0f;
    if (tid < cols) {
      u = p.beta[(size_t)m * p.N + n] * (to_f(((const T*)p.v)[((size_t)m * p.N + n) * p.Dv + c0 + tid]) - x);
      o[tid] = from_f<T>(p.scale * (y + qk * u));
    }
    us[tid] = u;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = rg + RG * i;
    if (r >= p.Dk || c >= cols) continue;
    const float kr = ks[r];
    float* w = p.out + at + (size_t)r * p.Dv;
    if constexpr (VEC == 4)
      __stcs((float4*)w, make_float4(s[i][0] + kr * us[c], s[i][1] + kr * us[c + 1], s[i][2] + kr * us[c + 2],
                                     s[i][3] + kr * us[c + 3]));
    else
      __stcs(w, s[i][0] + kr * us[c]);
  }
}

// ---- host ------------------------------------------------------------------------
int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RNN_OK;
  fprintf(stderr, "librnn_gb300: CUDA error: %s\n", cudaGetErrorString(e));
  return RNN_ECUDA;
}
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// What the calls lay out in the tape (behind the status word) and the workspace.
struct DeltaSizes {
  bool bf;
  int C, NP, BV, KP, nvt, segs, seglen;
  long long nc, items, ne;
  size_t rec, tri, S, Z, zf, sf;  // bytes
  size_t M, H;                    // of the segments' maps, of H and of the states between
  size_t tape;
  size_t dots, edge, near, cross, part, bwd;
};

bool delta_heads_ok(int Nk, int N, int Dk, int Dv, int dtype) {
  return Nk >= 1 && N >= Nk && N <= 65536 && N % Nk == 0 && Dk >= 1 && Dk <= RNN_DELTA_MAX_D && Dv >= 1 &&
         Dv <= RNN_DELTA_MAX_D && (dtype == RNN_F32 || dtype == RNN_BF16);
}

// keep: with what a backward needs
bool delta_sizes(const rnn_delta_dims_t* d, bool keep, DeltaSizes* z) {
  if (!d || d->B < 1 || d->T < 0 || d->T > INT_MAX - 64 || !delta_heads_ok(d->Nk, d->N, d->Dk, d->Dv, d->dtype)) return false;
  *z = DeltaSizes{};
  z->bf = d->dtype == RNN_BF16;
  z->C = z->bf ? TC_C : F32_C;
  z->NP = F32_NP;
  z->KP = (d->Dk + 15) / 16 * 16;
  z->nc = ((long long)d->T + z->C - 1) / z->C;
  z->items = z->nc * d->B * d->N;
  if ((long long)d->B * d->N * 64 > INT_MAX || z->items > INT_MAX / 16) return false;  // counted in 32 bits with their tiles
  DeltaLay lay{F32_BV, 1, 0};
  if (z->bf) lay = delta_lay((long long)d->B * d->N, d->Dv, z->KP, z->nc, device_sms(), keep);
  z->BV = lay.BV; z->segs = lay.segs; z->seglen = lay.seglen;
  z->nvt = (d->Dv + z->BV - 1) / z->BV;
  const size_t n = (size_t)z->items, heads = (size_t)d->B * d->N;
  z->rec = up256(n * REC_N * z->C * 4);
  if (z->bf) {
    z->ne = z->nc / TC_EDGE + 1;
    z->tri = up256(n * 3 * 128 * TC_C * 2);  // TP
    z->S = up256(n * z->nvt * 2 * z->KP * z->BV * 2);
    z->Z = up256(n * z->nvt * 64 * z->BV * 2);  // dY's second plane
    z->zf = up256(n * z->nvt * 64 * z->BV * 4);
    z->sf = up256(heads * z->ne * z->nvt * (z->KP > 128 ? 256 : 128) * z->BV * 4);
    if (z->segs > 1) {
      const size_t KR = z->KP > 128 ? 256 : 128;
      z->M = up256(heads * z->segs * KR * KR * 4);
      z->H = up256(heads * z->segs * z->nvt * z->BV * KR * 4);
    }
    z->tape = z->rec + z->tri + z->M + 2 * z->H;
    if (keep) z->tape += z->S + 2 * z->zf + z->sf;
    z->dots = up256(n * z->nvt * 6 * TC_C * 4);
    z->edge = up256(heads * z->ne * z->nvt * 8 * 4);
    z->near = up256(n * TC_C * 4);
    z->cross = up256(n * z->nvt * 3 * 4);
    z->bwd = z->S + z->Z + z->dots + z->edge + z->near + z->cross + 2 * z->H;
  } else {
    z->tri = up256(n * z->NP * z->C * z->C * 2);  // each of Tm and P
    z->S = up256(n * z->nvt * z->NP * z->KP * z->BV * 2);
    z->Z = up256(n * z->nvt * z->NP * z->C * z->BV * 2);
    z->tape = z->rec + 2 * z->tri + z->S + z->Z;
    z->bwd = z->S + z->Z;
  }
  z->part = d->N != d->Nk ? up256((size_t)d->B * d->T * d->N * d->Dk * 4) : 0;
  z->bwd += 2 * z->part;
  return true;
}

DeltaArgs delta_args(const rnn_delta_dims_t* d, const DeltaSizes& z, void* tape) {
  DeltaArgs a{};
  a.B = d->B; a.T = d->T; a.Nk = d->Nk; a.N = d->N; a.Dk = d->Dk; a.Dv = d->Dv;
  a.DKP = z.KP; a.nvt = z.nvt; a.nc = (int)z.nc;
  a.status = (unsigned*)tape;
  char* t = (char*)tape + 256;
  a.rec = (float*)t;
  a.tm = (bf16*)(t + z.rec);
  a.pm = (bf16*)(t + z.rec + z.tri);
  a.S = (bf16*)(t + z.rec + 2 * z.tri);
  a.Z = (bf16*)(t + z.rec + 2 * z.tri + z.S);
  return a;
}

DeltaTcArgs delta_tc_args(const rnn_delta_dims_t* d, const DeltaSizes& z, void* tape, bool keep) {
  DeltaTcArgs a{};
  a.B = d->B; a.T = d->T; a.Nk = d->Nk; a.N = d->N; a.Dk = d->Dk; a.Dv = d->Dv;
  a.KP = z.KP; a.nvt = z.nvt; a.nc = (int)z.nc; a.ne = (int)z.ne;
  a.status = (unsigned*)tape;
  a.wait_limit_ns = wait_limit_ns();
  a.segs = z.segs; a.seglen = z.seglen;
  char* t = (char*)tape + 256;
  a.rec = (float*)t;
  a.tp = (bf16*)(t += z.rec);
  a.Mt = (float*)(t += z.tri);
  a.Ht = (float*)(t += z.M);
  a.St = (float*)(t += z.H);
  t += z.H;
  if (!keep) return a;
  a.Sh = (bf16*)t;
  a.zf = (float*)(t += z.S);
  a.of = (float*)(t += z.zf);
  a.sf = (float*)(t += z.zf);
  return a;
}

}  // namespace
}  // namespace rnn

using namespace rnn;

extern "C" {

size_t rnn_delta_tape_size(const rnn_delta_dims_t* d, int keep) {
  DeltaSizes z;
  return delta_sizes(d, keep != 0, &z) ? 256 + z.tape : 0;
}

size_t rnn_delta_bwd_workspace_size(const rnn_delta_dims_t* d) {
  DeltaSizes z;
  return delta_sizes(d, true, &z) ? 256 + z.bwd : 0;
}

int rnn_delta_fwd(const rnn_delta_dims_t* d, const void* q, const void* k, const void* v, const void* g,
                  const void* beta, const void* state0, const unsigned char* reset, const int* lengths, float scale,
                  void* o, void* last, int keep, void* tape, size_t tape_bytes, void* stream) {
  DeltaSizes z;
  if (!delta_sizes(d, keep != 0, &z) || !tape || (d->T > 0 && (!q || !k || !v || !g || !beta || !o))) return RNN_EINVAL;
  const void* ptrs[] = {q, k, v, g, beta, state0, o, last, tape};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (!al4(lengths)) return RNN_EINVAL;
  if (tape_bytes < 256 + z.tape) return RNN_ENOSPC;
  cudaStream_t st = (cudaStream_t)stream;
  if (d->T == 0) {
    const size_t bytes = (size_t)d->B * d->N * d->Dk * d->Dv * sizeof(float);
    const int rc = cuda_status(cudaMemsetAsync(tape, 0, 256, st));
    if (rc || !last) return rc;
    return cuda_status(state0 ? cudaMemcpyAsync(last, state0, bytes, cudaMemcpyDeviceToDevice, st)
                              : cudaMemsetAsync(last, 0, bytes, st));
  }
  auto fill = [&](auto& a) {
    a.q = q; a.k = k; a.v = v; a.g = (const float*)g; a.beta = (const float*)beta; a.s0 = (const float*)state0;
    a.reset = reset; a.lengths = lengths; a.scale = scale; a.o = o; a.last = (float*)last;
  };
  if (z.bf) {
    DeltaTcArgs a = delta_tc_args(d, z, tape, keep != 0);
    fill(a);
    return cuda_status(delta_tc_fwd_launch(z.BV, a, st));
  }
  DeltaArgs a = delta_args(d, z, tape);
  fill(a);
  return cuda_status(delta_fwd_launch(a, st));
}

int rnn_delta_bwd(const rnn_delta_dims_t* d, const void* q, const void* k, const void* v, const int* lengths, float scale,
                  void* tape, size_t tape_bytes, const void* dO, const void* dlast, void* dq, void* dk, void* dv,
                  void* dg, void* dbeta, void* dstate0, void* workspace, size_t ws_bytes, void* stream) {
  DeltaSizes z;
  if (!delta_sizes(d, true, &z)) return RNN_EINVAL;
  if (d->T > 0 && (!q || !k || !v || !tape || !dq || !dk || !dv || !dg || !dbeta || !workspace)) return RNN_EINVAL;
  const void* ptrs[] = {q, k, v, tape, dO, dlast, dq, dk, dv, dg, dbeta, dstate0, workspace};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (!al4(lengths)) return RNN_EINVAL;
  cudaStream_t st = (cudaStream_t)stream;
  if (d->T == 0) {
    const size_t bytes = (size_t)d->B * d->N * d->Dk * d->Dv * sizeof(float);
    if (!dstate0) return RNN_OK;
    return cuda_status(dlast ? cudaMemcpyAsync(dstate0, dlast, bytes, cudaMemcpyDeviceToDevice, st)
                             : cudaMemsetAsync(dstate0, 0, bytes, st));
  }
  if (tape_bytes < 256 + z.tape || ws_bytes < 256 + z.bwd) return RNN_ENOSPC;
  char* w = (char*)workspace;
  auto fill = [&](auto& a) {
    a.q = q; a.k = k; a.v = v; a.lengths = lengths; a.scale = scale;
    a.dO = dO; a.dlast = (const float*)dlast;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = (float*)dg; a.dbeta = (float*)dbeta; a.ds0 = (float*)dstate0;
    if (z.part) {
      a.pq = (float*)(w + z.bwd - 2 * z.part);
      a.pk = (float*)(w + z.bwd - z.part);
    }
  };
  if (z.bf) {
    DeltaTcArgs a = delta_tc_args(d, z, tape, true);
    fill(a);
    a.dSh = (bf16*)w;
    a.dYl = (bf16*)(w += z.S);
    a.dots = (float*)(w += z.Z);
    a.edge = (float*)(w += z.dots);
    a.near = (float*)(w += z.edge);
    a.cross = (float*)(w += z.near);
    a.Ht = (float*)(w += z.cross);
    a.St = (float*)(w += z.H);
    return cuda_status(delta_tc_bwd_launch(z.BV, a, st));
  }
  DeltaArgs a = delta_args(d, z, tape);
  fill(a);
  a.dS = (bf16*)w;
  a.dY = (bf16*)(w + z.S);
  return cuda_status(delta_bwd_launch(a, st));
}

int rnn_delta_step(int rows, int slots, int Nk, int N, int Dk, int Dv, int dtype, const void* q, const void* k,
                   const void* v, const void* g, const void* beta, const int* slot, const void* pool, void* pool_out,
                   float scale, void* o, void* status, void* stream) {
  if (rows < 0 || slots < 1 || !delta_heads_ok(Nk, N, Dk, Dv, dtype) || (!slot && rows > slots)) return RNN_EINVAL;
  if (!pool || !pool_out || (rows > 0 && (!q || !k || !v || !g || !beta || !o))) return RNN_EINVAL;
  const void* ptrs[] = {q, k, v, g, beta, pool, pool_out, o};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (!al4(slot) || !al4(status)) return RNN_EINVAL;
  if (!pools_apart(pool, pool_out, (size_t)slots * N * Dk * Dv * sizeof(float))) return RNN_EINVAL;
  const int tiles = (Dv + 31) / 32;
  if ((long long)rows * N * tiles > INT_MAX) return RNN_EINVAL;
  if (rows == 0) return RNN_OK;
  StepArgs a{rows, slots, Nk, N, Dk, Dv, tiles, q, k, v, (const float*)g, (const float*)beta, slot, (const float*)pool,
             (float*)pool_out, scale, o, (unsigned*)status};
  const unsigned grid = (unsigned)((long long)rows * N * tiles);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == RNN_BF16) {
    if (Dv % 4 == 0) delta_step_kernel<bf16, 4><<<grid, 256, 0, st>>>(a);
    else delta_step_kernel<bf16, 1><<<grid, 256, 0, st>>>(a);
  } else {
    if (Dv % 4 == 0) delta_step_kernel<float, 4><<<grid, 256, 0, st>>>(a);
    else delta_step_kernel<float, 1><<<grid, 256, 0, st>>>(a);
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
