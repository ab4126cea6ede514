// Pointwise part of the gated linear scan: gates, recurrence coefficients and
// their derivatives, fp32 arithmetic.
//
// linear (gates i, f, g, o at the LSTM's positions; i, f, o sigmoids):
//   c_t = f c_{t-1} + i g,  h_t = o c_t
// linear_coupled (gates f, g):
//   h_t = c_t = f c_{t-1} + (1 - f) g
// With delta_t the gradient of c_t (from h_t and from every later step):
//   linear:  da_i = delta g i (1-i), da_f = delta c_{t-1} f (1-f),
//            da_g = delta i, da_o = dh c o (1-o)
//   coupled: da_f = delta (c_{t-1} - g) f (1-f), da_g = delta (1-f)
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cells.cuh"
#include "rnn.h"

namespace rnn {

// Bit of the device status word: an index (token, slot) out of range. The
// bounded waits' STATUS_TIMEOUT is the other bit.
constexpr unsigned STATUS_RANGE = 2;

enum { GATED_LINEAR = 0, GATED_COUPLED = 1 };
__host__ __device__ constexpr int gated_gates(int fn) { return fn == GATED_LINEAR ? 4 : 2; }

constexpr int GATED_CHUNK = RNN_GATED_CHUNK;  // steps between kept states
constexpr int ACT_BLOCK = RNN_ACT_BLOCK;      // rows (steps) that share an 8-bit scale

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16(v); }

// ---- N channels of a lane as one value ------------------------------------------
// N = 2 (bf16 storage): the packed fp32 pair instructions of sm_100 and later
// take one issue slot for both channels. N = 1 (fp32 storage): plain fp32.
template <int N> struct FV { float v[N]; };
template <int N> __device__ __forceinline__ FV<N> splat(float a) {
  FV<N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.v[i] = a;
  return r;
}
__device__ __forceinline__ uint64_t pair_bits(const FV<2>& a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.v[0]), "f"(a.v[1]));
  return r;
}
__device__ __forceinline__ FV<2> pair_of(uint64_t b) {
  FV<2> r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.v[0]), "=f"(r.v[1]) : "l"(b));
  return r;
}
__device__ __forceinline__ FV<2> fma(const FV<2>& a, const FV<2>& b, const FV<2>& c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return pair_of(d);
}
__device__ __forceinline__ FV<2> mul(const FV<2>& a, const FV<2>& b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_of(d);
}
__device__ __forceinline__ FV<2> add(const FV<2>& a, const FV<2>& b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_of(d);
}
__device__ __forceinline__ FV<1> fma(const FV<1>& a, const FV<1>& b, const FV<1>& c) { return {{fmaf(a.v[0], b.v[0], c.v[0])}}; }
__device__ __forceinline__ FV<1> mul(const FV<1>& a, const FV<1>& b) { return {{a.v[0] * b.v[0]}}; }
__device__ __forceinline__ FV<1> add(const FV<1>& a, const FV<1>& b) { return {{a.v[0] + b.v[0]}}; }
template <int N> __device__ __forceinline__ FV<N> one_minus(const FV<N>& a) { return fma(a, splat<N>(-1.0f), splat<N>(1.0f)); }

// A gate's biased pre-activation, as its function wants it: z itself, or, for
// the sigmoids of bf16 storage, -z log2 e (the factor sits in `mul_of` and in
// the prepared bias), so that exp(-z) is one base-2 exponential.
template <int FN> __host__ __device__ constexpr bool gate_is_linear(int g) { return FN == GATED_LINEAR ? g == 2 : g == 1; }
template <int FN, int N> __device__ __forceinline__ constexpr float mul_of(int g) {
  return N == 1 || gate_is_linear<FN>(g) ? 1.0f : -1.4426950408889634f;
}
// the smaller one; a NaN stays one (fminf would hide it)
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// e = exp(-z). For fp32 z log2 e in two parts, the product and what its
// rounding and the constant's left out, so that e keeps the exponential's own
// 2^-22; z held to -88 .. 88 (e finite, NaN stays), where the sigmoid has
// reached 0 and 1: 12 instructions to a sigmoid where expf and a division take
// about twice that.
__device__ __forceinline__ FV<2> exp_neg(const FV<2>& t) { return {{exp2_fast(t.v[0]), exp2_fast(t.v[1])}}; }
__device__ __forceinline__ FV<1> exp_neg(const FV<1>& z) {
  const float x = min_nan(max_nan(-z.v[0], -88.0f), 88.0f);
  const float t = x * 1.44269502f, l = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269502f, -t));  // log2 e = 1.44269502 + 1.926e-8
  const float e = exp2_fast(t);
  return {{fmaf(e, l * 0.693147181f, e)}};
}
__device__ __forceinline__ FV<2> rcp(const FV<2>& d) { return {{rcp_fast(d.v[0]), rcp_fast(d.v[1])}}; }
__device__ __forceinline__ FV<1> rcp(const FV<1>& d) {
  const float r = rcp_fast(d.v[0]);
  return {{fmaf(r, fmaf(-d.v[0], r, 1.0f), r)}};
}
// 1 / d to a rounding, d <= 1.7e38 for N = 2 (one Newton step on the
// approximate reciprocal): the factor f of a long memory enters every later
// state, and the approximation alone, off to one side by up to 2^-23, moved
// the fp32 state of a channel that remembers 2000 steps by 2e-4.
__device__ __forceinline__ FV<2> rcp_full(const FV<2>& d) {
  const FV<2> r = rcp(d);
  return fma(r, fma(mul(d, splat<2>(-1.0f)), r, splat<2>(1.0f)), r);
}
__device__ __forceinline__ FV<1> rcp_full(const FV<1>& d) { return rcp(d); }

template <int N> __device__ __forceinline__ FV<N> sigmoid(const FV<N>& z) { return rcp(add(exp_neg(z), splat<N>(1.0f))); }
// The forget gate of `linear`. The bound keeps the Newton step finite where
// the reciprocal is 0 already.
__device__ __forceinline__ FV<2> sigmoid_full(const FV<2>& z) {
  FV<2> d = add(exp_neg(z), splat<2>(1.0f));
  d.v[0] = min_nan(d.v[0], 1.7e38f);
  d.v[1] = min_nan(d.v[1], 1.7e38f);
  return rcp_full(d);
}
__device__ __forceinline__ FV<1> sigmoid_full(const FV<1>& z) { return sigmoid(z); }
// f = sigmoid(z) and n = 1 - f, both to full relative accuracy (the coupled
// cell uses n itself as the input gate). fp32: with e = exp(-|z|), which cannot
// overflow, 1 / (1 + e) and e / (1 + e), the larger one f where z > 0. bf16
// storage: f = 1 / (1 + e) and n = e f with e = exp(-z) bounded by 2^125, so that
// n becomes 1; the least f, 2^-125 (1 / (1 + e) rounds to no less, so f stays
// non-negative), is taken off again, so that a gate of -infinity is 0. (The
// other form takes 156 + 323 us, this one 150 + 311, at B=32 T=4096 C=1024.)
__device__ __forceinline__ void sigmoid_both(const FV<2>& t, FV<2>& f, FV<2>& n) {
  const FV<2> e = exp_neg(FV<2>{{min_nan(t.v[0], 125.0f), min_nan(t.v[1], 125.0f)}});
  const FV<2> r = rcp_full(add(e, splat<2>(1.0f)));
  n = mul(e, r);
  f = add(r, splat<2>(-2.350988702e-38f));
}
__device__ __forceinline__ void sigmoid_both(const FV<1>& z, FV<1>& f, FV<1>& n) {
  const FV<1> e = exp_neg(FV<1>{{fabsf(z.v[0])}}), hi = rcp(add(e, splat<1>(1.0f))), lo = mul(e, hi);
  const bool open = z.v[0] > 0.0f;
  f.v[0] = open ? hi.v[0] : lo.v[0];
  n.v[0] = open ? lo.v[0] : hi.v[0];
}

// f and u of c = f c' + u from the gates z[G]
template <int FN, int N> __device__ __forceinline__ void gated_coeff(const FV<N>* z, FV<N>& f, FV<N>& u) {
  if (FN == GATED_LINEAR) {
    f = sigmoid_full(z[1]);
    u = mul(sigmoid(z[0]), z[2]);
  } else {
    FV<N> n;
    sigmoid_both(z[0], f, n);
    u = mul(n, z[1]);
  }
}
// da[G] of one step from its gates, f, c' (0 after a reset), c, dh and the
// gradient x that reaches c from later steps; x becomes f delta, what the
// step passes on (0 after a reset goes by f = 0).
template <int FN, int N>
__device__ __forceinline__ void gated_grad(const FV<N>* z, const FV<N>& f, const FV<N>& cp, const FV<N>& c, const FV<N>& dh,
                                           FV<N>& x, FV<N>* da) {
  if (FN == GATED_LINEAR) {
    const FV<N> i = sigmoid(z[0]), o = sigmoid(z[3]);
    const FV<N> e = mul(dh, o), delta = add(x, e);
    x = mul(f, delta);
    da[2] = mul(delta, i);
    da[0] = mul(da[2], mul(z[2], one_minus(i)));
    da[1] = mul(x, mul(cp, one_minus(f)));
    da[3] = mul(e, mul(c, one_minus(o)));
  } else {
    FV<N> s, n;
    sigmoid_both(z[0], s, n);
    const FV<N> delta = add(x, dh);
    x = mul(f, delta);
    da[1] = mul(delta, n);
    da[0] = mul(mul(da[1], s), fma(z[1], splat<N>(-1.0f), cp));
  }
}

// ---- 8-bit checkpoints ------------------------------------------------------
// The scale of a block is 2^e with the smallest e >= -126 whose 127 steps
// hold the block's largest magnitude: of amax = m 2^k (1 <= m < 2) it is
// k - 6, one more when m > 127/64; at most 121, so that no q unpacks to an
// infinity (magnitudes past 127 2^121 = 3.38e38 saturate). Stored as the byte
// e + 127 (1 .. 248); 255 marks a block that held an infinity or a NaN.
constexpr unsigned ACT_NONFINITE = 255;
__device__ __forceinline__ unsigned act_scale_byte(float amax) {
  const unsigned bits = __float_as_uint(amax);
  if (bits >= 0x7f800000u) return ACT_NONFINITE;
  const int k = (int)(bits >> 23) - 127;
  const int e = k - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (unsigned)(min(max(e, -126), 121) + 127);
}
// 2^e and 2^-e of a scale byte (the byte of a non-finite block: NaN and 0)
__device__ __forceinline__ float act_scale(unsigned byte) {
  return byte == ACT_NONFINITE ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}
__device__ __forceinline__ float act_inv_scale(unsigned byte) {
  return byte == ACT_NONFINITE ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// The largest magnitudes of the channels in a 4-byte word of the storage type,
// in its bits (an infinity or NaN stays one), and the fp32 bits of channel v.
template <typename T> __device__ __forceinline__ uint32_t mag_max(uint32_t top, uint32_t x);
template <> __device__ __forceinline__ uint32_t mag_max<float>(uint32_t top, uint32_t x) { return max(top, x & 0x7fffffffu); }
template <> __device__ __forceinline__ uint32_t mag_max<__nv_bfloat16>(uint32_t top, uint32_t x) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(x & 0x7fff7fffu));
  return r;
}
template <typename T> __device__ __forceinline__ uint32_t mag_bits(uint32_t top, int v) {
  return sizeof(T) == 4 ? top : v ? top & 0xffff0000u : top << 16;
}
// q of N channels, each in the low byte of its word: a / 2^e + 1.5 2^23 rounds to
// nearest even (the product is exact, so one fused instruction) and leaves q
// there. `huge`: some block may saturate (act_scale_byte).
template <int N> __device__ __forceinline__ FV<N> quant(const FV<N>& a, const FV<N>& inv, bool huge) {
  if (huge) {
    FV<N> t = mul(a, inv);
#pragma unroll
    for (int v = 0; v < N; ++v) t.v[v] = fminf(fmaxf(t.v[v], -127.0f), 127.0f);
    return add(t, splat<N>(12582912.0f));
  }
  return fma(a, inv, splat<N>(12582912.0f));
}
// the low bytes of two words, in the low half
__device__ __forceinline__ uint32_t low_bytes(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
}

}  // namespace rnn
