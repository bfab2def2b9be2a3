// lane_tokens.h -- eight consecutive tokens of one channel in a lane, and the
// cross-lane moves between them: shared by the gated linear recurrence and
// the conv's gradients.
#pragma once

#include "sconv_device.h"

namespace sconv {

template <typename D>
__device__ __forceinline__ typename D::storage round_to(float v) {
  if constexpr (sizeof(typename D::storage) == 2)
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    return v;
}

// Workgroups of ragged work: N consecutive logical ones on each XCD in turn,
// so that one long sequence spreads over every XCD (a contiguous run of
// workgroups on each left seven of them waiting for the longest: 671 us
// against 321 us for 16 ragged sequences of 4096 channels), while the N that
// share lines meet in one L2.  A bijection on [0, G).
template <uint32_t N>
__device__ __forceinline__ uint32_t xcd_groups(uint32_t g, uint32_t G) {
  if (g >= G / (8 * N) * (8 * N)) return g;
  const uint32_t xcd = g % 8, idx = g / 8;
  return (idx / N * 8 + xcd) * N + idx % N;
}

// Keeps the instructions before it and behind it apart, where the compiler
// would start them all at once and hold more registers than it gains.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

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
  // A 16-byte access at any element: sequences that start anywhere and rows of
  // an odd length keep vector lanes (a wave's lanes still cover whole lines
  // between them).  Ordinary loads: lanes share lines when a token starts off
  // a 16-byte boundary and in fp32 (two loads a lane), and streaming loads
  // read such lines twice (16 ragged fp32 sequences of 4096 channels, forward
  // and gradients: 987 us streaming, 810 us so; aligned bf16 loses 2.5%).
  // Streaming stores: 398 against 419 us for 8 x 4096 x 8192 bf16.
  typedef typename P::raw_t any_raw __attribute__((aligned(sizeof(S))));
  P p[kPacks];

  // Tokens [t, t + 8) of a row of `total` tokens.  VEC: tokens contiguous.
  // Tokens past the row's end read as zero bits; tokens of other sequences
  // are read and not used.
  template <bool VEC>
  __device__ __forceinline__ void load(const S* row, int64_t stride, int64_t t, int64_t total) {
    if (VEC && t + kLaneTokens <= total) {
#pragma unroll
      for (int q = 0; q < kPacks; ++q)
        p[q].raw = *reinterpret_cast<const any_raw*>(row + t + q * D::kVec16);
    } else {
      Elems v;
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e) {
        v.e[e] = t + e < total ? row[(t + e) * (VEC ? 1 : stride)] : (S)0;
        if (VEC) in_order();  // a row's end only: not worth eight addresses at once
      }
      __builtin_memcpy(p, &v, sizeof v);
    }
  }

  // Token e (a constant) as a float.
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(S) == 2) {
      const uint32_t w = p[0].raw[e / 2];
      return __uint_as_float(e % 2 ? w & 0xFFFF0000u : w << 16);
    } else {
      return __uint_as_float(p[e / 4].raw[e % 4]);
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

  // Store the tokens of [t, t + 8) that lie before `end`.
  template <bool VEC>
  __device__ __forceinline__ void store(S* row, int64_t stride, int64_t t, int64_t end) const {
    if (VEC && t + kLaneTokens <= end) {
#pragma unroll
      for (int q = 0; q < kPacks; ++q)
        __builtin_nontemporal_store(p[q].raw,
                                    reinterpret_cast<any_raw*>(row + t + q * D::kVec16));
    } else {
      Elems v;
      __builtin_memcpy(&v, p, sizeof v);
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e) {
        if (t + e < end) row[(t + e) * (VEC ? 1 : stride)] = v.e[e];
        in_order();
      }
    }
  }
};

// The sequence of the unit-th largest length (ties: the lower index first), so
// that the longest start first and the shortest fill the end.  Up to 64
// sequences, one a lane; more are taken as they come.
__device__ __forceinline__ int by_length(const int32_t* qsl, int32_t batch, int unit) {
  if (batch > 64 || batch == 1) return unit;
  const int lane = threadIdx.x & 63;
  const int n = lane < batch ? qsl[lane + 1] - qsl[lane] : -1;
  int rank = 0;
  for (int j = 0; j < batch; ++j) {
    const int m = __builtin_amdgcn_readlane(n, j);
    rank += m > n || (m == n && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < batch && rank == unit));
}

// The first of `batch` sequences that does not end before row lo (batch: none).
__device__ __forceinline__ int first_sequence(const int32_t* qsl, int32_t batch, int64_t lo) {
  int n = 0;
  for (int i0 = 0; i0 < batch; i0 += 64) {
    const int i = i0 + (threadIdx.x & 63);
    const bool done = i < batch && qsl[i + 1] < lo;
    const int k = __popcll(__ballot(done));
    n += k;
    if (k < 64) break;
  }
  return n;
}

// ---------------------------------------------------------------- scans of h -> P h + H

// v of another lane by a DPP move; lanes that the move has no source for,
// and rows outside ROWS, get `other`.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float lane_move(float other, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(v), CTRL,
                                                    ROWS, 0xF, false));
}

// One step of an inclusive scan: this lane's map after that of the lane which
// the DPP move names (lanes without one keep their own).  Two instructions
// that take the move as an operand (the compiler made six: the identities,
// the moves, the products); the wait is the one a DPP operand needs behind a
// write.  P and H are written last by vector instructions, all lanes active.
#define SCONV_COMPOSE(NAME, MOVE)                                      \
  __device__ __forceinline__ void NAME(float& P, float& H) {           \
    asm("s_nop 1\n\t"                                                  \
        "v_fmac_f32_dpp %1, %1, %0 " MOVE " bank_mask:0xf\n\t"         \
        "v_mul_f32_dpp %0, %0, %0 " MOVE " bank_mask:0xf"              \
        : "+v"(P), "+v"(H));                                           \
  }
SCONV_COMPOSE(compose_shr1, "row_shr:1 row_mask:0xf")
SCONV_COMPOSE(compose_shr2, "row_shr:2 row_mask:0xf")
SCONV_COMPOSE(compose_shr4, "row_shr:4 row_mask:0xf")
SCONV_COMPOSE(compose_shr8, "row_shr:8 row_mask:0xf")
SCONV_COMPOSE(compose_bcast15, "row_bcast:15 row_mask:0xa")
SCONV_COMPOSE(compose_bcast31, "row_bcast:31 row_mask:0xc")
SCONV_COMPOSE(compose_shl1, "row_shl:1 row_mask:0xf")
SCONV_COMPOSE(compose_shl2, "row_shl:2 row_mask:0xf")
SCONV_COMPOSE(compose_shl4, "row_shl:4 row_mask:0xf")
SCONV_COMPOSE(compose_shl8, "row_shl:8 row_mask:0xf")
#undef SCONV_COMPOSE

// Maps of lanes 0..l composed, in ascending lane order (row_shr 1, 2, 4, 8
// inside rows of 16 lanes, then the last lane of a row to the next row, then
// lane 31 to the upper half).
__device__ __forceinline__ void scan_wave_up(float& P, float& H) {
  compose_shr1(P, H);
  compose_shr2(P, H);
  compose_shr4(P, H);
  compose_shr8(P, H);
  compose_bcast15(P, H);
  compose_bcast31(P, H);
}

// The same inside each row of 16 lanes, in descending lane order (row_shl).
__device__ __forceinline__ void scan_row_down(float& P, float& H) {
  compose_shl1(P, H);
  compose_shl2(P, H);
  compose_shl4(P, H);
  compose_shl8(P, H);
}

__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace sconv
