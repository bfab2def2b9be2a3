// recurrence_device.h -- the gate arithmetic of the gated linear recurrence,
// shared by its forward, backward and one-token kernels.
//
//   r = sigmoid(gate_a), i = sigmoid(gate_x)
//   log a = -k r,  k = decay_scale * softplus(decay)   (per channel)
//   m = sqrt(1 - a^2),  h_t = a_t h_{t-1} + m_t i_t x_t
//
// Everything is fp32.  The hardware exp2, reciprocal and square roots are
// good to about 1 ulp, and every use of them here is relative: a gate near
// one keeps 1 - a^2 exact to a few ulp through expm1 (below), so a state
// that decays over thousands of tokens keeps the precision of its inputs.
#pragma once

#include "sconv_device.h"

namespace sconv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMarkTokens = 64;  // tokens between two checkpoints of the state

// Per-channel constants of the decay.
struct Decay {
  float k;       // decay_scale * softplus(decay)
  float k_log2;  // the same in powers of two
};

__device__ __forceinline__ Decay make_decay(float decay, float scale) {
  // softplus; past 20 it equals its argument in fp32
  const float sp = decay > 20.f ? decay : log1pf(expf(decay));
  Decay d;
  d.k = scale * sp;
  d.k_log2 = d.k * kLog2e;
  return d;
}

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
}

// 1 - a^2 from y = 2 log a <= 0 and a itself.  For y > -0.7 it is
// -y (e^y - 1)/y with the quotient's Chebyshev interpolant of degree 5 on
// [-0.7, 0] (relative error 1.1e-8, coefficients computed for this file);
// below, 1 - a^2 >= 0.5 and the difference loses at most one bit.  A result
// below the smallest normal number counts as zero.
__device__ __forceinline__ float one_minus_square(float y, float a) {
  float q = 1.0332433739677072e-3f;
  q = __builtin_fmaf(q, y, 8.06795246899128e-3f);
  q = __builtin_fmaf(q, y, 4.157276451587677e-2f);
  q = __builtin_fmaf(q, y, 1.6665145754814148e-1f);
  q = __builtin_fmaf(q, y, 4.9999910593032837e-1f);
  q = __builtin_fmaf(q, y, 1.0f);
  const float near = -y * q, far = __builtin_fmaf(-a, a, 1.0f);
  return y > -0.7f ? near : far;
}

// One token's gates.
struct Gates {
  float r, i, a, m;
};

__device__ __forceinline__ Gates make_gates(float ga, float gx, const Decay& d) {
  Gates g;
  g.r = sigmoid(ga);
  g.i = sigmoid(gx);
  g.a = __builtin_amdgcn_exp2f(-d.k_log2 * g.r);
  g.m = __builtin_amdgcn_sqrtf(one_minus_square(-2.0f * d.k * g.r, g.a));
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
  g.a = __builtin_amdgcn_exp2f(-d.k_log2 * g.r);
  const float m2 = one_minus_square(-2.0f * d.k * g.r, g.a);
  // Zero below the normal range, but a NaN stays one.
  const float inv = __builtin_amdgcn_rsqf(m2);
  g.inv_m = m2 < 1.17549435e-38f ? 0.0f : inv;
  g.m = m2 * g.inv_m;
  return g;
}

// ---------------------------------------------------------------- eight tokens of a lane

constexpr int kLaneTokens = 8;                     // consecutive tokens of one lane
constexpr int kChunkTokens = 64 * kLaneTokens;     // tokens of one wave

// Raw bits of a lane's eight tokens of one channel.
template <typename D>
struct Raw8 {
  using S = typename D::storage;
  static constexpr int kPacks = kLaneTokens / D::kVec16;
  using P = Pack<D, D::kVec16>;
  struct Elems { S e[kLaneTokens]; };
  P p[kPacks];

  // Tokens [t, t + 8) of a row of `total` tokens.  VEC: tokens contiguous,
  // rows 16-byte aligned, t a multiple of 8.  Tokens past the row's end read
  // as zero bits; tokens of other sequences are read and not used.
  template <bool VEC>
  __device__ __forceinline__ void load(const S* row, int64_t stride, int64_t t, int64_t total) {
    if (VEC && t + kLaneTokens <= total) {
#pragma unroll
      for (int q = 0; q < kPacks; ++q) p[q].load_nt(row + t + q * D::kVec16);
    } else {
      Elems v;
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e)
        v.e[e] = t + e < total ? row[(t + e) * stride] : (S)0;
      __builtin_memcpy(p, &v, sizeof v);
    }
  }

  __device__ __forceinline__ void to_float(float (&f)[kLaneTokens]) const {
#pragma unroll
    for (int q = 0; q < kPacks; ++q) {
      float g[D::kVec16];
      p[q].to_float(g);
#pragma unroll
      for (int e = 0; e < D::kVec16; ++e) f[q * D::kVec16 + e] = g[e];
    }
  }

  __device__ __forceinline__ void from_float(const float (&f)[kLaneTokens]) {
#pragma unroll
    for (int q = 0; q < kPacks; ++q) {
      float g[D::kVec16];
#pragma unroll
      for (int e = 0; e < D::kVec16; ++e) g[e] = f[q * D::kVec16 + e];
      p[q].from_float(g);
    }
  }

  // Store the tokens of [t, t + 8) that lie in [start, end).
  template <bool VEC>
  __device__ __forceinline__ void store(S* row, int64_t stride, int64_t t, int64_t start,
                                        int64_t end) const {
    if (VEC && t >= start && t + kLaneTokens <= end) {
#pragma unroll
      for (int q = 0; q < kPacks; ++q) p[q].store_nt(row + t + q * D::kVec16);
    } else {
      Elems v;
      __builtin_memcpy(&v, p, sizeof v);
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e)
        if (t + e >= start && t + e < end) row[(t + e) * stride] = v.e[e];
    }
  }
};

// ---------------------------------------------------------------- scans of h -> P h + H

// v of another lane by a DPP move; lanes that the move has no source for,
// and rows outside ROWS, get `other`.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float lane_move(float other, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(v), CTRL,
                                                    ROWS, 0xF, false));
}

// One step of an inclusive scan: this lane's map after the moved lane's.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ void compose(float& P, float& H) {
  const float p = lane_move<CTRL, ROWS>(1.0f, P), h = lane_move<CTRL, ROWS>(0.0f, H);
  H = __builtin_fmaf(P, h, H);
  P *= p;
}

// Maps of lanes 0..l composed, in ascending lane order (row_shr 1, 2, 4, 8
// inside rows of 16 lanes, then the last lane of a row to the next row, then
// lane 31 to the upper half).
__device__ __forceinline__ void scan_wave_up(float& P, float& H) {
  compose<0x111>(P, H);
  compose<0x112>(P, H);
  compose<0x114>(P, H);
  compose<0x118>(P, H);
  compose<0x142, 0xA>(P, H);
  compose<0x143, 0xC>(P, H);
}

// The same inside each row of 16 lanes, in descending lane order (row_shl).
__device__ __forceinline__ void scan_row_down(float& P, float& H) {
  compose<0x101>(P, H);
  compose<0x102>(P, H);
  compose<0x104>(P, H);
  compose<0x108>(P, H);
}

__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

template <typename D>
__device__ __forceinline__ typename D::storage round_to(float v) {
  if constexpr (sizeof(typename D::storage) == 2)
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    return v;
}

}  // namespace sconv
