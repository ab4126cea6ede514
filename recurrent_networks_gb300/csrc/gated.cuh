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

// 1 / d to a rounding (one Newton step on the approximate reciprocal): the
// factor f of a long memory enters every later state, and the approximation
// alone, off to one side by up to 2^-23, moved the fp32 state of a channel
// that remembers 2000 steps by 2e-4.
template <bool FAST> __device__ __forceinline__ float rcp_full(float d) {
  if (!FAST) return 1.0f / d;
  const float r = rcp_fast(d);
  return fmaf(r, fmaf(-d, r, 1.0f), r);
}
template <bool FAST> __device__ __forceinline__ float sig_full(float x) {
  if (!FAST) return 1.0f / (1.0f + expf(-x));
  // the bound keeps the Newton step finite; the reciprocal is 0 there already
  return rcp_full<FAST>(fminf(1.0f + exp2_fast(-1.4426950408889634f * x), 1.7e38f));
}
// s = sigmoid(x) and n = 1 - s without cancellation: e = exp(-x), s = 1 / (1 + e),
// n = e s. An e past the fp32 range leaves s = 0 and n = 0 (instead of inf * 0):
// n only ever enters the product s n, which is 0 there.
template <bool FAST> __device__ __forceinline__ void sig_pair(float x, float& s, float& n) {
  const float e = FAST ? exp2_fast(-1.4426950408889634f * x) : expf(-x);
  s = FAST ? rcp_fast(1.0f + e) : 1.0f / (1.0f + e);
  n = s * fminf(e, 3e38f);
}
// s = sigmoid(x) and n = sigmoid(-x), both to full relative accuracy (from
// exp(-|x|) <= 1): the coupled cell uses n itself as the input gate.
template <bool FAST> __device__ __forceinline__ void sig_both(float x, float& s, float& n) {
  const float e = FAST ? exp2_fast(-1.4426950408889634f * fabsf(x)) : expf(-fabsf(x));
  const float r = rcp_full<FAST>(1.0f + e);
  const float er = e * r;
  s = x >= 0.0f ? r : er;
  n = x >= 0.0f ? er : r;
}

// f and u of c = f c' + u from the biased pre-activations a[G]
template <int FN, bool FAST> __device__ __forceinline__ void gated_coeff(const float* a, float& f, float& u) {
  if (FN == GATED_LINEAR) {
    f = sig_full<FAST>(a[1]);
    u = f_sigmoid<FAST>(a[0]) * a[2];
  } else {
    float n;
    sig_both<FAST>(a[0], f, n);
    u = n * a[1];
  }
}
// h from c
template <int FN, bool FAST> __device__ __forceinline__ float gated_out(const float* a, float c) {
  return FN == GATED_LINEAR ? f_sigmoid<FAST>(a[3]) * c : c;
}
// the part of delta that comes from dh of the same step
template <int FN, bool FAST> __device__ __forceinline__ float gated_into(const float* a, float dh) {
  return FN == GATED_LINEAR ? f_sigmoid<FAST>(a[3]) * dh : dh;
}
// da[G] of one step from its biased pre-activations, c' (0 after a reset), c,
// dh and delta
template <int FN, bool FAST>
__device__ __forceinline__ void gated_grad(const float* a, float cp, float c, float dh, float delta, float* da) {
  if (FN == GATED_LINEAR) {
    float s, n;
    sig_pair<FAST>(a[0], s, n);
    da[0] = delta * a[2] * (s * n);
    da[2] = delta * s;
    sig_pair<FAST>(a[1], s, n);
    da[1] = delta * cp * (s * n);
    sig_pair<FAST>(a[3], s, n);
    da[3] = dh * c * (s * n);
  } else {
    float s, n;
    sig_both<FAST>(a[0], s, n);
    da[0] = delta * (cp - a[1]) * (s * n);
    da[1] = delta * n;
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
__device__ __forceinline__ int act_quant(float x, float inv) { return max(-127, min(127, __float2int_rn(x * inv))); }

}  // namespace rnn
