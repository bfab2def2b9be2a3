// delta_walk.h -- how the kernels that walk a sequence's chunks bring a chunk
// into LDS: K, Q, two sets of frags, three vectors and the workgroup's columns
// of one more tensor.  A chunk's loads are issued before the chunk ahead of it
// is worked on and wait in registers meanwhile.
#pragma once

#include "delta_rule.h"

namespace sconv {

template <typename D, int KP, int NW> struct WalkLds {
  using S = typename D::storage;
  static constexpr int C = kDeltaChunk<D>;
  using Rows = LdsRows<D, KP>;
  using Cols = LdsRows<D, 16 * NW>;
  __attribute__((aligned(16))) S k[C * Rows::LD];
  __attribute__((aligned(16))) S q[C * Rows::LD];
  __attribute__((aligned(16))) S x[C * Cols::LD];
  __attribute__((aligned(16))) char f[2 * kDeltaFrags<C> * kFragBytes];
  __attribute__((aligned(16))) float v[3 * C];
};

template <typename D, int KP, int NW> struct WalkStage {
  using L = WalkLds<D, KP, NW>;
  using S = typename D::storage;
  using E = typename Tile<D>::Exact;
  static constexpr int C = L::C, THREADS = 64 * NW;
  static constexpr int KN = C * KP / 8, XN = C * 2 * NW, FN = 2 * kDeltaFrags<C> * kFragBytes / 16;
  static constexpr int KO = (KN + THREADS - 1) / THREADS, XO = XN / THREADS, FO = FN / THREADS;
  static_assert(XN % THREADS == 0 && FN % THREADS == 0 && 3 * C <= THREADS);
  E k[KO], q[KO], x[XO];
  u32x4 f[FO];
  float v;

  // tk, tq, tx: the heads' first rows; the chunk's rows are t0 .. end - 1.
  // vec: K's, Q's and x's rows are of 16-byte vectors.
  template <bool VEC>
  __device__ __forceinline__ void fetch_rows(const DeltaParams& p, const S* tk, const S* tq,
                                             const S* tx, int64_t x_t, int32_t col0, int32_t t0,
                                             int32_t end) {
#pragma unroll
    for (int o = 0; o < KO; ++o) {
      const int i = threadIdx.x + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
      k[o] = load8<D, VEC>(tk + t0 * p.k_t, p.k_t, t, end - t0, c0, p.K);
      q[o] = load8<D, VEC>(tq + t0 * p.q_t, p.q_t, t, end - t0, c0, p.K);
    }
#pragma unroll
    for (int o = 0; o < XO; ++o) {
      const int i = threadIdx.x + o * THREADS, t = i / (2 * NW), c0 = i % (2 * NW) * 8;
      x[o] = load8<D, VEC>(tx + t0 * x_t, x_t, t, end - t0, col0 + c0, p.V);
    }
  }
  __device__ __forceinline__ void fetch(const DeltaParams& p, const S* tk, const S* tq, const S* tx,
                                        int64_t x_t, bool vec, int32_t col0, int32_t t0,
                                        int32_t end, const char* frags, const float* vectors) {
    if (vec) fetch_rows<true>(p, tk, tq, tx, x_t, col0, t0, end);
    else fetch_rows<false>(p, tk, tq, tx, x_t, col0, t0, end);
    const u32x4* from = reinterpret_cast<const u32x4*>(frags);
#pragma unroll
    for (int o = 0; o < FO; ++o) f[o] = from[threadIdx.x + o * THREADS];
    v = vectors[threadIdx.x < 3 * C ? threadIdx.x : 0];
  }
  // len: tokens of the chunk
  __device__ __forceinline__ void stage(L& l, const DeltaParams& p, int32_t col0, int32_t len) const {
#pragma unroll
    for (int o = 0; o < KO; ++o) {
      const int i = threadIdx.x + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
      const int n = t < len ? p.K - c0 : 0;
      if (KN % THREADS == 0 || i < KN) {
        L::Rows::put8(l.k, t, c0, mask8<D>(k[o], n));
        L::Rows::put8(l.q, t, c0, mask8<D>(q[o], n));
      }
    }
#pragma unroll
    for (int o = 0; o < XO; ++o) {
      const int i = threadIdx.x + o * THREADS, t = i / (2 * NW), c0 = i % (2 * NW) * 8;
      L::Cols::put8(l.x, t, c0, mask8<D>(x[o], t < len ? p.V - col0 - c0 : 0));
    }
#pragma unroll
    for (int o = 0; o < FO; ++o) reinterpret_cast<u32x4*>(l.f)[threadIdx.x + o * THREADS] = f[o];
    if (threadIdx.x < 3 * C) l.v[threadIdx.x] = v;
  }
};

// A wave's 16 columns of a K x V matrix in accumulator tiles: f(index, value)
// for every entry it has, and the values that f returns in their place.
template <int KT, typename F>
__device__ __forceinline__ void each_entry(f32x4 (&s)[KT], int K, int V, int col, int col_end, F&& f) {
  const int g = (threadIdx.x & 63) >> 4;
  if (K == 16 * KT && col_end <= V) {  // of the whole wave
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = f((int64_t)(16 * t + 4 * g + e) * V + col, s[t][e]);
    return;
  }
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = 16 * t + 4 * g + e;
      if (k < K && col < V) s[t][e] = f((int64_t)k * V + col, s[t][e]);
    }
}

}  // namespace sconv
