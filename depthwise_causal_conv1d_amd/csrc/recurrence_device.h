// recurrence_device.h -- the gate arithmetic of the gated linear recurrence,
// shared by its forward, backward and one-token kernels.
//
//   r = sigmoid(gate_a), i = sigmoid(gate_x)
//   log a = -k r,  k = decay_scale * softplus(decay)   (per channel)
//   m = sqrt(1 - a^2),  h_t = a_t h_{t-1} + m_t i_t x_t
//
// Everything is fp32.  The hardware exp2, reciprocal and square roots are
// good to about 1 ulp, and 1 - a^2 keeps its relative precision near a = 1
// through expm1 (below).  A sigmoid's relative error grows with a negative
// gate, whose product with log2 e is rounded before exp2: about 5 units of
// 2^-24 at -5, 9 at -10, 17 at -20, 32 at -40 (carrying the product in two parts
// would mend it for three more instructions each, of the prefill's 35 an
// element); below -88 it is zero.
#pragma once

#include "lane_tokens.h"

namespace sconv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMarkTokens = 32;  // tokens between two checkpoints of the state

// Per-channel constants of the decay.
struct Decay {
  float k;       // decay_scale * softplus(decay)
  float k2;      // twice that
  float k_log2;  // -k in powers of two
};

// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|) <= 1, to a few ulp.
// log1p(e) = 2 artanh(z), z = e / (2 + e) <= 1/3, by its power series.  The
// product |v| log2 e is carried in two parts, or exp would lose |v| / 2 ulp.
// |v| ends at 200, where e is zero already: the parts of an infinite product
// would be inf - inf.  k ends at 2^126, where a is zero at every gate above
// -80: times a closed gate's r = 0 it is zero, which an infinity is not.
// (Both comparisons leave a NaN as it is.)
constexpr float kMaxDecay = 8.50705917e37f;  // 2^126
__device__ __forceinline__ Decay make_decay(float decay, float scale) {
  const float least = -__builtin_fabsf(decay), v = least < -200.0f ? -200.0f : least;
  const float t = v * kLog2e;
  const float rest = __builtin_fmaf(v, kLog2e, -t) + v * 1.92596299e-8f;  // log2 e - kLog2e
  float e = __builtin_amdgcn_exp2f(t);
  e = __builtin_fmaf(e, rest * 0.693147181f, e);
  const float z = e * __builtin_amdgcn_rcpf(2.0f + e), w = z * z;
  float s = 1.0f / 13;
  s = __builtin_fmaf(s, w, 1.0f / 11);
  s = __builtin_fmaf(s, w, 1.0f / 9);
  s = __builtin_fmaf(s, w, 1.0f / 7);
  s = __builtin_fmaf(s, w, 1.0f / 5);
  s = __builtin_fmaf(s, w, 1.0f / 3);
  s = __builtin_fmaf(s, w, 1.0f);
  const float sp = __builtin_fmaf(2.0f * z, s, decay > 0.f ? decay : 0.f);
  Decay d;
  d.k = scale * sp > kMaxDecay ? kMaxDecay : scale * sp;
  d.k2 = 2.0f * d.k;
  d.k_log2 = d.k * -kLog2e;
  return d;
}

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
}

// 1 - a^2 from w = -2 log a >= 0 and a itself.  For w < 0.35 it is
// w (1 - e^-w)/w with the quotient's Chebyshev interpolant of degree 4
// (relative error 1.4e-8, coefficients computed for this file); above,
// 1 - a^2 >= 0.29 and the difference loses at most two bits.
__device__ __forceinline__ float one_minus_square(float w, float a) {
  float q = 7.211245596408844e-3f;
  q = __builtin_fmaf(q, w, -4.133187234401703e-2f);
  q = __builtin_fmaf(q, w, 1.6662530601024628e-1f);
  q = __builtin_fmaf(q, w, -4.9999821186065674e-1f);
  q = __builtin_fmaf(q, w, 1.0f);
  const float near = w * q, far = __builtin_fmaf(-a, a, 1.0f);
  return w < 0.35f ? near : far;
}

// One token's gates.
struct Gates {
  float r, i, a, m;
};

__device__ __forceinline__ Gates make_gates(float ga, float gx, const Decay& d) {
  Gates g;
  g.r = sigmoid(ga);
  g.i = sigmoid(gx);
  g.a = __builtin_amdgcn_exp2f(d.k_log2 * g.r);
  g.m = __builtin_amdgcn_sqrtf(one_minus_square(d.k2 * g.r, g.a));
  return g;
}

// The same with 1/m for the backward pass: zero where m is zero (the limit
// of every gradient that it enters, since it comes with a factor m^2).
struct GatesInv {
  float r, i, a, m, inv_m;
};

__device__ __forceinline__ GatesInv make_gates_inv(float ga, float gx, const Decay& d) {
  GatesInv g;
  g.r = sigmoid(ga);
  g.i = sigmoid(gx);
  g.a = __builtin_amdgcn_exp2f(d.k_log2 * g.r);
  const float m2 = one_minus_square(d.k2 * g.r, g.a);
  // Zero below the normal range, but a NaN stays one.
  const float inv = __builtin_amdgcn_rsqf(m2);
  g.inv_m = m2 < 1.17549435e-38f ? 0.0f : inv;
  g.m = m2 * g.inv_m;
  return g;
}

}  // namespace sconv
