// Group norm with an activation, channels last (include/rnn.h): statistics over
// the W channels of one group of one row,
//   m = mean x (0 where not centred), r = (mean (x - m)^2 + eps)^-1/2,
//   n = (x - m) r, t = n w + b, y = act(t), or t act(z) with a gate z.
// Backward: dt = dy act'(t), or dy act(z) and dz = dy t act'(z); dn = dt w,
//   dx = r (dn - mean dn - n mean(dn n)) (without mean dn where not centred),
//   dw = sum over rows of dt n, db of dt.
// All in fp32. The backward takes the statistics from x again: x is read in any
// case, and nothing is kept from the forward.
#include <limits.h>
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "rnn.h"

namespace rnn {
namespace {

typedef __nv_bfloat16 bf16;

struct NormArgs {
  long long rows;
  int G, W, act, centered;
  float eps;
  const void *x, *w, *b, *gate, *dy;
  void *y, *dx, *dgate;
  float* part;  // [gridDim.x][2][C]: sums of dt n and dt over a CTA's rows, or null
  int lanes, gp, rp;  // threads of a group; groups and rows that a CTA takes at once
  // channels that warp k of a group's several has
  __device__ int share_of(int k, int vec, int nv) const {
    int n = 0;
    for (int v = 0; v < nv; ++v) n += max(0, min(32, (W + vec - 1) / vec - (k * 32 + v * lanes))) * vec;
    return n;
  }
};

// VEC values of T as they are loaded: 16 bytes, a pair, or one value
template <typename T, int VEC> struct Raw {
  uint4 v;
  __device__ void load(const T* p) { v = __ldcs((const uint4*)p); }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&x)[VEC]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};
template <typename T> struct Raw<T, 2> {
  alignas(2 * sizeof(T)) T v[2];
  __device__ void load(const T* p) {
    if constexpr (sizeof(T) == 4) *(float2*)v = *(const float2*)p;
    else *(uint32_t*)v = *(const uint32_t*)p;
  }
  __device__ void zero() { v[0] = v[1] = from_f<T>(0.0f); }
  __device__ void get(float (&x)[2]) const { x[0] = to_f(v[0]), x[1] = to_f(v[1]); }
};
template <typename T> struct Raw<T, 1> {
  T v;
  __device__ void load(const T* p) { v = *p; }
  __device__ void zero() { v = from_f<T>(0.0f); }
  __device__ void get(float (&x)[1]) const { x[0] = to_f(v); }
};
template <typename T, int VEC> __device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  Raw<T, VEC> r;
  r.load(p);
  r.get(v);
}
template <typename T, int VEC> __device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    p[0] = from_f<T>(v[0]);
  } else if constexpr (VEC == 2) {
    if constexpr (sizeof(T) == 4) *(float2*)p = make_float2(v[0], v[1]);
    else *(__nv_bfloat162*)p = __floats2bfloat162_rn(v[0], v[1]);
  } else if constexpr (sizeof(T) == 4) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *(const uint32_t*)&h;
    }
    *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The sigmoid: bf16 storage takes the approximate exponential and reciprocal
// (2^-21 together), fp32 the exact ones.
template <typename T> __device__ __forceinline__ float sigm(float x) {
  if constexpr (sizeof(T) == 2) return rcp_fast(1.0f + exp2_fast(-1.4426950408889634f * x));
  else return 1.0f / (1.0f + expf(-x));
}
// act(x) and, for the backward, its slope
template <typename T> __device__ __forceinline__ float act_of(int act, float x) {
  if (act == RNN_ACT_NONE) return x;
  const float s = sigm<T>(x);
  return act == RNN_ACT_SILU ? x * s : s;
}
template <typename T> __device__ __forceinline__ void act_both(int act, float x, float& a, float& slope) {
  if (act == RNN_ACT_NONE) {
    a = x;
    slope = 1.0f;
    return;
  }
  // s and s (1 - s) from e = exp(-|x|): 1 - s would be the rounding of s at an open gate
  float e, r;
  if constexpr (sizeof(T) == 2) {
    e = exp2_fast(-1.4426950408889634f * fabsf(x));
    r = rcp_fast(1.0f + e);
  } else {
    e = expf(-fabsf(x));
    r = 1.0f / (1.0f + e);
  }
  const float s = x < 0.0f ? e * r : r, c = e * r * r;
  a = act == RNN_ACT_SILU ? x * s : s;
  slope = act == RNN_ACT_SILU ? fmaf(x, c, s) : c;
}

// The sum over `lanes` (a power of two up to 32) lanes of a warp.
__device__ __forceinline__ float lane_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// What the warps of a group (MANY: of several whole warps) have, through red [8]:
// one barrier; red may be written again only behind the next one.
template <typename V> __device__ __forceinline__ void share(V* red, V v) {
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
}

// What both directions do with a value once the statistics are known.
template <typename T, bool GATE>
__device__ __forceinline__ float forward_value(int act, float n, float w, float b, float z) {
  const float t = fmaf(n, w, b);
  return GATE ? t * act_of<T>(act, z) : act_of<T>(act, t);
}
// dt (returned) and dz
template <typename T, bool GATE>
__device__ __forceinline__ float backward_value(int act, float n, float w, float b, float z, float dy, float& dz) {
  const float t = fmaf(n, w, b);
  float a, slope;
  act_both<T>(act, GATE ? z : t, a, slope);
  dz = dy * t * slope;
  return GATE ? dy * a : dy * slope;
}

// Groups of up to 256 * NV vectors (of VEC channels): `lanes` threads (a power of
// two; MANY: of several warps) hold a group's channels in registers. A CTA takes
// gp groups of rp rows at once, the same groups for all its rows, so that a
// thread's sums of dw and db are over one set of columns. One pass over the data,
// bound by DRAM: measured 75 us forward (floor 59) and 145 backward (floor 99) for
// 65536 rows x 8 groups of 128, bf16, gated; 23 and 41 us (floors 10 and 15) for
// 16384 rows of one group of 1024, where the two sums of a row that eight warps
// share are waited for. Four CTAs an SM forward, with few spills, against one with
// none: 34 us and 47 (30000 rows x 16 of 64, gated); backward they cost more (85 us
// against 66), and it keeps its registers.
template <typename T, int VEC, int NV, bool GATE, bool BWD, bool MANY>
__global__ void __launch_bounds__(256, BWD ? (VEC * NV > 8 ? 1 : 2) : (VEC * NV > 16 ? 2 : 4)) norm_kernel(NormArgs p) {
  extern __shared__ float sums[];  // [2][gp * W], BWD with p.part
  __shared__ float4 stats[2][8];  // in turn: forward, one barrier a row stands between a row's reads and the writes two rows on
  __shared__ float2 red[8];
  const int li = threadIdx.x % p.lanes, slot = threadIdx.x / p.lanes;
  const int gi = slot % p.gp, ri = slot / p.gp;
  const int g = blockIdx.y * p.gp + gi;
  const bool on = ri < p.rp && g < p.G;
  const long long C = (long long)p.G * p.W;
  const float inv = 1.0f / (float)p.W;
  const int many = MANY ? p.lanes >> 5 : 1, lanes = MANY ? 32 : p.lanes, w0 = (threadIdx.x >> 5) & ~(many - 1);
  float w[NV][VEC], b[NV][VEC];
  bool have[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (li + v * p.lanes) * VEC;
    have[v] = on && c < p.W;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[v][e] = 1.0f, b[v][e] = 0.0f;
    if (have[v] && p.w) load_vec<T, VEC>((const T*)p.w + (size_t)g * p.W + c, w[v]);
    if (have[v] && p.b) load_vec<T, VEC>((const T*)p.b + (size_t)g * p.W + c, b[v]);
  }
  float dw[BWD ? NV : 1][VEC], db[BWD ? NV : 1][VEC];
  if constexpr (BWD) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) dw[v][e] = db[v][e] = 0.0f;
  }
  __shared__ float part[8];  // channels of a group's warp
  if constexpr (MANY) {
    if (threadIdx.x < many) part[threadIdx.x] = (float)p.share_of(threadIdx.x, VEC, NV);
    __syncthreads();
  }
  const float mine = MANY ? 1.0f / fmaxf(part[(threadIdx.x >> 5) - w0], 1.0f) : inv;
  // A row's values are loaded while the one before is worked on. All threads of a
  // warp stay in the loop: the sums are over the warp's lanes.
  Raw<T, VEC> rx[NV], rz[GATE ? NV : 1], rd[BWD ? NV : 1];
  auto load = [&](long long r) {
    const bool live = on && r < p.rows;
    const size_t at = (size_t)(live ? r : 0) * C + (size_t)(on ? g : 0) * p.W;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (li + v * p.lanes) * VEC;
      if (live && have[v]) {
        rx[v].load((const T*)p.x + at + c);
        if constexpr (GATE) rz[v].load((const T*)p.gate + at + c);
        if constexpr (BWD) rd[v].load((const T*)p.dy + at + c);
      } else {
        rx[v].zero();
        if constexpr (GATE) rz[v].zero();
        if constexpr (BWD) rd[v].zero();
      }
    }
  };
  const long long step = (long long)gridDim.x * p.rp;
  int turn = 0;
  load((long long)blockIdx.x * p.rp + ri);
  for (long long r0 = (long long)blockIdx.x * p.rp; r0 < p.rows; r0 += step) {
    const long long r = r0 + ri;
    const bool live = on && r < p.rows;
    const size_t at = (size_t)(live ? r : 0) * C + (size_t)(on ? g : 0) * p.W;
    float x[NV][VEC], z[GATE ? NV : 1][VEC], dy[BWD ? NV : 1][VEC];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      rx[v].get(x[v]);
      if constexpr (GATE) rz[v].get(z[v]);
      if constexpr (BWD) rd[v].get(dy[v]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += x[v][e];
    }
    if (r0 + step < p.rows) load(r + step);
    // The mean, and around it the sums of d = x - mean and of its squares: the
    // first is the mean's own rounding, which a mean far above the spread makes
    // large beside d. Where a group has several warps each does so by itself, and
    // the distances of their means to the first one's join them.
    s = p.centered ? lane_sum(s, lanes) : 0.0f;
    float mean = s * mine;
    float q = 0.0f, e1 = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = have[v] ? x[v][e] - mean : 0.0f;
        if constexpr (!MANY) x[v][e] = d;
        e1 += d;
        q = fmaf(d, d, q);
      }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      q += __shfl_xor_sync(0xffffffffu, q, o);
      e1 += __shfl_xor_sync(0xffffffffu, e1, o);
    }
    if (!p.centered) e1 = 0.0f;
    if constexpr (MANY) {
      const float4* st = stats[turn] + w0;
      share(stats[turn], make_float4(mean, e1, q, 0.0f));
      turn ^= 1;
      mean = st[0].x;
      q = e1 = 0.0f;
      for (int k = 0; k < many; ++k) {
        const float4 r = st[k];
        const float n = part[k], d = r.x - mean;
        q += r.z + d * fmaf(n, d, 2.0f * r.y);
        e1 += fmaf(n, d, r.y);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[v][e] = x[v][e] - mean;
    }
    e1 *= inv;
    q = fmaf(-e1 * e1, (float)p.W, q);
    if (q < 0.0f) q = 0.0f;  // a NaN stays one
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[v][e] = have[v] ? x[v][e] - e1 : 0.0f;
    const float rstd = 1.0f / sqrtf(fmaf(q, inv, p.eps));
    if constexpr (!BWD) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!live || !have[v]) continue;
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          y[e] = forward_value<T, GATE>(p.act, x[v][e] * rstd, w[v][e], b[v][e], GATE ? z[GATE ? v : 0][e] : 0.0f);
        store_vec<T, VEC>((T*)p.y + at + (li + v * p.lanes) * VEC, y);
      }
    } else {
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float n = x[v][e] * rstd;
          float dz;
          const float dt = backward_value<T, GATE>(p.act, n, w[v][e], b[v][e], GATE ? z[GATE ? v : 0][e] : 0.0f, dy[v][e], dz);
          if constexpr (GATE) z[v][e] = dz;
          if (live && have[v]) {
            dw[v][e] = fmaf(dt, n, dw[v][e]);
            db[v][e] += dt;
          }
          x[v][e] = n;
          const float dn = live && have[v] ? dt * w[v][e] : 0.0f;
          dy[v][e] = dn;
          s1 += dn;
          s2 = fmaf(dn, n, s2);
        }
      for (int o = lanes >> 1; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
      if constexpr (MANY) {
        share(red, make_float2(s1, s2));
        s1 = s2 = 0.0f;
        for (int k = 0; k < many; ++k) {
          s1 += red[w0 + k].x;
          s2 += red[w0 + k].y;
        }
      } else {
        __syncwarp();
      }
      s1 = p.centered ? s1 * inv : 0.0f;
      s2 *= inv;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!live || !have[v]) continue;
        const size_t to = at + (li + v * p.lanes) * VEC;
        float dx[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) dx[e] = rstd * (dy[v][e] - s1 - x[v][e] * s2);
        store_vec<T, VEC>((T*)p.dx + to, dx);
        if constexpr (GATE) store_vec<T, VEC>((T*)p.dgate + to, z[v]);
      }
    }
  }
  if constexpr (BWD) {
    if (!p.part) return;
    // the CTA's rows, one after the other, then its sums to its own place
    const int n = p.gp * p.W;
    for (int q = 0; q < p.rp; ++q) {
      if (on && ri == q) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (!have[v]) continue;
          const int c = gi * p.W + (li + v * p.lanes) * VEC;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            sums[c + e] = (q ? sums[c + e] : 0.0f) + dw[v][e];
            sums[n + c + e] = (q ? sums[n + c + e] : 0.0f) + db[v][e];
          }
        }
      }
      __syncthreads();
    }
    const long long c0 = (long long)blockIdx.y * n;
    for (int c = threadIdx.x; c < n; c += 256)
      if (c0 + c < C) {
        p.part[(size_t)blockIdx.x * 2 * C + c0 + c] = sums[c];
        p.part[((size_t)blockIdx.x * 2 + 1) * C + c0 + c] = sums[n + c];
      }
  }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += red[i];
  return s;
}

// Wider groups, or rows that are not whole vectors: a CTA takes one group, the
// row in shared memory. dw and db are summed into this CTA's place of p.part.
template <typename T, bool GATE, bool BWD> __global__ void __launch_bounds__(512) norm_wide_kernel(NormArgs p) {
  extern __shared__ float sm[];
  float *xs = sm, *ds = sm + p.W, *dw = sm + 2 * p.W, *db = sm + 3 * p.W;  // ds, dw, db: BWD
  __shared__ float red[16];
  const int g = blockIdx.y, W = p.W;
  const long long C = (long long)p.G * W;
  const T* w = p.w ? (const T*)p.w + (size_t)g * W : nullptr;
  const T* b = p.b ? (const T*)p.b + (size_t)g * W : nullptr;
  const float inv = 1.0f / (float)W;
  if (BWD && p.part)
    for (int c = threadIdx.x; c < W; c += 512) dw[c] = db[c] = 0.0f;
  for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const size_t at = (size_t)r * C + (size_t)g * W;
    const T* x = (const T*)p.x + at;
    float s = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x; c < W; c += 512) {
      const float v = to_f(x[c]);
      xs[c] = v;
      s += v;
    }
    const float mean = p.centered ? block_sum(s, red) * inv : 0.0f;
    s = 0.0f;
    float e1 = 0.0f;  // the mean's own rounding
    for (int c = threadIdx.x; c < W; c += 512) {
      const float v = xs[c] - mean;
      xs[c] = v;
      e1 += v;
    }
    e1 = p.centered ? block_sum(e1, red) * inv : 0.0f;
    for (int c = threadIdx.x; c < W; c += 512) {
      const float v = xs[c] - e1;
      xs[c] = v;
      s = fmaf(v, v, s);
    }
    const float rstd = 1.0f / sqrtf(fmaf(block_sum(s, red), inv, p.eps));
    if constexpr (!BWD) {
#pragma unroll 4
      for (int c = threadIdx.x; c < W; c += 512)
        ((T*)p.y)[at + c] = from_f<T>(forward_value<T, GATE>(p.act, xs[c] * rstd, w ? to_f(w[c]) : 1.0f, b ? to_f(b[c]) : 0.0f,
                                                             GATE ? to_f(((const T*)p.gate)[at + c]) : 0.0f));
    } else {
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 2
      for (int c = threadIdx.x; c < W; c += 512) {
        const float n = xs[c] * rstd, wc = w ? to_f(w[c]) : 1.0f;
        float dz;
        const float dt = backward_value<T, GATE>(p.act, n, wc, b ? to_f(b[c]) : 0.0f, GATE ? to_f(((const T*)p.gate)[at + c]) : 0.0f,
                                                 to_f(((const T*)p.dy)[at + c]), dz);
        if constexpr (GATE) ((T*)p.dgate)[at + c] = from_f<T>(dz);
        if (p.part) {
          dw[c] = fmaf(dt, n, dw[c]);
          db[c] += dt;
        }
        const float dn = dt * wc;
        xs[c] = n;
        ds[c] = dn;
        s1 += dn;
        s2 = fmaf(dn, n, s2);
      }
      s1 = block_sum(s1, red) * inv;
      if (!p.centered) s1 = 0.0f;
      s2 = block_sum(s2, red) * inv;
      for (int c = threadIdx.x; c < W; c += 512) ((T*)p.dx)[at + c] = from_f<T>(rstd * (ds[c] - s1 - xs[c] * s2));
    }
  }
  if (BWD && p.part)
    for (int c = threadIdx.x; c < W; c += 512) {
      p.part[(size_t)blockIdx.x * 2 * C + (size_t)g * W + c] = dw[c];
      p.part[((size_t)blockIdx.x * 2 + 1) * C + (size_t)g * W + c] = db[c];
    }
}

// out[c] = sum of part[k][c], k in order; 32 columns a block
template <typename T>
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* part, int parts, long long C, T* dw, T* db) {
  __shared__ float red[32][33];
  const long long c = (long long)blockIdx.x * 32 + (threadIdx.x & 31);  // of 2 C
  const int k0 = threadIdx.x >> 5;
  float s = 0.0f;
  if (c < 2 * C)
#pragma unroll 4
    for (int k = k0; k < parts; k += 32) s += part[(size_t)k * 2 * C + c];
  red[k0][threadIdx.x & 31] = s;
  __syncthreads();
  if (k0 == 0 && c < 2 * C) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += red[k][threadIdx.x];
    if (c < C) {
      if (dw) dw[c] = from_f<T>(t);
    } else if (db) {
      db[c - C] = from_f<T>(t);
    }
  }
}

// ---- host ------------------------------------------------------------------------
int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RNN_OK;
  fprintf(stderr, "librnn_gb300: CUDA error: %s\n", cudaGetErrorString(e));
  return RNN_ECUDA;
}
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int NORM_MAX_W = RNN_NORM_MAX_WIDTH;

bool norm_ok(long long rows, int G, int W, int dtype) {
  return rows >= 0 && rows < (1LL << 40) && G >= 1 && W >= 1 && W <= NORM_MAX_W && (long long)G * W <= (1 << 28) &&
         G <= 65535 && (dtype == RNN_F32 || dtype == RNN_BF16);
}

// How a problem is laid over the GPU: vectors of vec values, nv of them a
// thread (0: the wide kernel), and the grid.
struct NormPlan {
  int vec, nv, lanes, gp, rp;
  unsigned gx, gy;
};
NormPlan norm_plan(long long rows, int G, int W, int dtype, bool bwd) {
  NormPlan p{};
  const int full = dtype == RNN_BF16 ? 8 : 4;
  p.vec = W % full == 0 ? full : W % 2 == 0 ? 2 : 1;
  const int n = (W + p.vec - 1) / p.vec;  // vectors of a group; below, of a thread: at most, and while threads are to be had
  // Threads before vectors: a group of several warps is slower by its barrier and
  // faster by its loads in flight. Backward, 2 KB rows (1024 bf16) at one vector a
  // thread take 44 us and at two 64; forward two are as fast, and 8 KB rows gain
  // (22 us against 27).
  const int most = p.vec == 1 ? 8 : p.vec == 2 ? 4 : 2, some = p.vec == 1 ? 4 : p.vec == 2 || !bwd ? 2 : 1;
  if (n > 256 * most) {
    p.gp = p.rp = 1;
    p.gy = (unsigned)G;
  } else {
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes < n) p.lanes *= 2;
    while (p.lanes < 256 && p.lanes * some < n) p.lanes *= 2;
    p.nv = 1;
    while (p.nv * p.lanes < n) p.nv *= 2;
    const int slots = 256 / p.lanes;
    p.gp = G < slots ? G : slots;
    p.rp = slots / p.gp;
    p.gy = (unsigned)((G + p.gp - 1) / p.gp);
  }
  const long long want = (rows + p.rp - 1) / p.rp;
  long long most_ctas = (long long)device_sms() * (p.nv && p.nv * p.vec <= (bwd ? 8 : 16) ? 4 : 2) / p.gy;  // about what an SM holds
  if (most_ctas < 1) most_ctas = 1;
  p.gx = (unsigned)(want < 1 ? 1 : want < most_ctas ? want : most_ctas);
  return p;
}

template <typename T, int VEC, int NV, bool MANY> auto norm_kernel_of(bool gate, bool bwd) {
  return bwd ? (gate ? norm_kernel<T, VEC, NV, true, true, MANY> : norm_kernel<T, VEC, NV, false, true, MANY>)
             : (gate ? norm_kernel<T, VEC, NV, true, false, MANY> : norm_kernel<T, VEC, NV, false, false, MANY>);
}
template <typename T, int VEC, int NV> cudaError_t narrow(const NormPlan& pl, const NormArgs& a, bool bwd, cudaStream_t st) {
  void (*k)(NormArgs) = pl.lanes > 32 ? norm_kernel_of<T, VEC, NV, true>(a.gate, bwd) : norm_kernel_of<T, VEC, NV, false>(a.gate, bwd);
  const size_t sm = bwd && a.part ? (size_t)2 * pl.gp * a.W * 4 : 0;
  cudaError_t e = set_smem_attr((const void*)k, sm);
  if (e != cudaSuccess) return e;
  k<<<dim3(pl.gx, pl.gy), 256, sm, st>>>(a);
  note_launch();
  return cudaGetLastError();
}
template <typename T, int VEC> cudaError_t launch_nv(const NormPlan& pl, const NormArgs& a, bool bwd, cudaStream_t st) {
  if (pl.nv == 1) return narrow<T, VEC, 1>(pl, a, bwd, st);
  if (pl.nv == 2) return narrow<T, VEC, 2>(pl, a, bwd, st);
  if constexpr (VEC <= 2) {
    if (pl.nv == 4) return narrow<T, VEC, 4>(pl, a, bwd, st);
  }
  if constexpr (VEC == 1) return narrow<T, 1, 8>(pl, a, bwd, st);
  return cudaErrorInvalidValue;
}
template <typename T> cudaError_t launch(const NormPlan& pl, const NormArgs& a, bool bwd, cudaStream_t st) {
  constexpr int FULL = 16 / sizeof(T);
  if (pl.nv) return pl.vec == 1 ? launch_nv<T, 1>(pl, a, bwd, st) : pl.vec == 2 ? launch_nv<T, 2>(pl, a, bwd, st) : launch_nv<T, FULL>(pl, a, bwd, st);
  void (*k)(NormArgs) = bwd ? (a.gate ? norm_wide_kernel<T, true, true> : norm_wide_kernel<T, false, true>)
                            : (a.gate ? norm_wide_kernel<T, true, false> : norm_wide_kernel<T, false, false>);
  const size_t sm = (size_t)(bwd ? (a.part ? 4 : 2) : 1) * a.W * 4;
  cudaError_t e = set_smem_attr((const void*)k, sm);
  if (e != cudaSuccess) return e;
  k<<<dim3(pl.gx, pl.gy), 512, sm, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

NormArgs norm_args(const NormPlan& pl, long long rows, int G, int W, int act, int centered, float eps) {
  NormArgs a{};
  a.rows = rows; a.G = G; a.W = W; a.act = act; a.centered = centered; a.eps = eps;
  a.lanes = pl.lanes; a.gp = pl.gp; a.rp = pl.rp;
  return a;
}

}  // namespace
}  // namespace rnn

using namespace rnn;

extern "C" {

size_t rnn_group_norm_workspace_size(long long rows, int groups, int width, int dtype) {
  if (!norm_ok(rows, groups, width, dtype)) return 0;
  return 256 + (size_t)norm_plan(rows, groups, width, dtype, true).gx * 2 * groups * width * sizeof(float);
}

int rnn_group_norm_fwd(long long rows, int groups, int width, int dtype, int act, int centered, float eps, const void* x,
                       const void* w, const void* b, const void* gate, void* y, void* stream) {
  if (!norm_ok(rows, groups, width, dtype) || act < RNN_ACT_NONE || act > RNN_ACT_SIGMOID || !(eps >= 0)) return RNN_EINVAL;
  if (rows > 0 && (!x || !y)) return RNN_EINVAL;
  const void* ptrs[] = {x, w, b, gate, y};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (rows == 0) return RNN_OK;
  const NormPlan pl = norm_plan(rows, groups, width, dtype, false);
  NormArgs a = norm_args(pl, rows, groups, width, act, centered, eps);
  a.x = x; a.w = w; a.b = b; a.gate = gate; a.y = y;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == RNN_BF16 ? launch<bf16>(pl, a, false, st) : launch<float>(pl, a, false, st));
}

int rnn_group_norm_bwd(long long rows, int groups, int width, int dtype, int act, int centered, float eps, const void* x,
                       const void* w, const void* b, const void* gate, const void* dy, void* dx, void* dgate, void* dw,
                       void* db, void* workspace, size_t ws_bytes, void* stream) {
  if (!norm_ok(rows, groups, width, dtype) || act < RNN_ACT_NONE || act > RNN_ACT_SIGMOID || !(eps >= 0)) return RNN_EINVAL;
  if (rows > 0 && (!x || !dy || !dx || !gate != !dgate)) return RNN_EINVAL;
  const void* ptrs[] = {x, w, b, gate, dy, dx, dgate, dw, db, workspace};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  cudaStream_t st = (cudaStream_t)stream;
  const size_t C = (size_t)groups * width, e = dtype == RNN_BF16 ? 2 : 4;
  if (rows == 0) {
    int rc = dw ? cuda_status(cudaMemsetAsync(dw, 0, C * e, st)) : RNN_OK;
    return rc || !db ? rc : cuda_status(cudaMemsetAsync(db, 0, C * e, st));
  }
  const NormPlan pl = norm_plan(rows, groups, width, dtype, true);
  NormArgs a = norm_args(pl, rows, groups, width, act, centered, eps);
  a.x = x; a.w = w; a.b = b; a.gate = gate; a.dy = dy; a.dx = dx; a.dgate = dgate;
  if (dw || db) {
    if (!workspace) return RNN_EINVAL;
    if (ws_bytes < rnn_group_norm_workspace_size(rows, groups, width, dtype)) return RNN_ENOSPC;
    a.part = (float*)workspace;
  }
  int rc = cuda_status(dtype == RNN_BF16 ? launch<bf16>(pl, a, true, st) : launch<float>(pl, a, true, st));
  if (rc || !a.part) return rc;
  const unsigned blocks = (unsigned)((2 * C + 31) / 32);
  if (dtype == RNN_BF16) norm_sums_kernel<bf16><<<blocks, 1024, 0, st>>>(a.part, (int)pl.gx, (long long)C, (bf16*)dw, (bf16*)db);
  else norm_sums_kernel<float><<<blocks, 1024, 0, st>>>(a.part, (int)pl.gx, (long long)C, (float*)dw, (float*)db);
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
