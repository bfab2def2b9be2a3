// delta_walk.h -- how the kernels that walk a sequence's chunks bring a chunk
// into LDS: K, Q, two sets of frags, three vectors and the workgroup's columns
// of one more tensor.  A chunk's loads are issued before the chunk ahead of it
// is worked on and wait in registers meanwhile.
#pragma once

#include "delta_rule.h"
#include "row_lanes.h"

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
  static constexpr int XW = 2 * NW;  // octets of a row of x
  static constexpr int KN = C * KP / 8, XN = C * XW, FN = 2 * kDeltaFrags<C> * kFragBytes / 16;
  static constexpr int KO = (KN + THREADS - 1) / THREADS, XO = XN / THREADS, FO = FN / THREADS;
  static_assert(XN % THREADS == 0 && FN % THREADS == 0 && 3 * C <= THREADS);
  E k[KO], q[KO], x[XO];
  u32x4 f[FO];
  float v;

  // Whole chunks of whole rows: a row is a uniform address and a lane's 32-bit
  // offset, and nothing is masked (a third of the walk's vector instructions
  // were addresses and masks).
  uint32_t k_off, q_off, x_off;
  static constexpr int KR = THREADS / (KP / 8), XR = THREADS / XW;  // rows of one piece a thread

  const S *tk, *tq, *tx;  // the heads' first rows
  int64_t x_t;
  int32_t col0;
  bool vec, whole;  // rows of 16-byte vectors; no row ends inside the tiles

  __device__ __forceinline__ void init(const DeltaParams& p, const S* k_, const S* q_, const S* x_,
                                       int64_t x_t_, bool vec_, int32_t col0_) {
    tk = k_, tq = q_, tx = x_, x_t = x_t_, vec = vec_, col0 = col0_;
    whole = vec && p.K == KP && col0 + 16 * NW <= p.V && KN % THREADS == 0;
    const int t = threadIdx.x / (KP / 8), c0 = threadIdx.x % (KP / 8) * 8, es = sizeof(S);
    k_off = (uint32_t)(t * p.k_t + c0) * es;
    q_off = (uint32_t)(t * p.q_t + c0) * es;
    x_off = (uint32_t)(threadIdx.x / XW * x_t + threadIdx.x % XW * 8 + col0) * es;
  }
  // The other chunks.  Where the thread's number comes from is hidden, or all
  // these addresses would be made ahead of the loop and held there.
  template <bool VEC>
  __device__ __forceinline__ void fetch_rows(const DeltaParams& p, int32_t t0, int32_t end) {
    const int tid = (int)lane_offset(threadIdx.x);
#pragma unroll
    for (int o = 0; o < KO; ++o) {
      const int i = tid + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
      k[o] = load8<D, VEC>(tk + t0 * p.k_t, p.k_t, t, end - t0, c0, p.K);
      q[o] = load8<D, VEC>(tq + t0 * p.q_t, p.q_t, t, end - t0, c0, p.K);
    }
#pragma unroll
    for (int o = 0; o < XO; ++o) {
      const int i = tid + o * THREADS, t = i / XW, c0 = i % XW * 8;
      x[o] = load8<D, VEC>(tx + t0 * x_t, x_t, t, end - t0, col0 + c0, p.V);
    }
  }
  static __device__ __forceinline__ E at(const S* row, uint32_t off) {
    const S* m = in_row(row, off);
    if constexpr (sizeof(S) == 2) return {__builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(m))};
    else return {*reinterpret_cast<const f32x4*>(m), *reinterpret_cast<const f32x4*>(m + 4)};
  }
  // The chunk's rows are t0 .. end - 1.
  __device__ __forceinline__ void fetch(const DeltaParams& p, int32_t t0, int32_t end,
                                        const char* frags, const float* vectors) {
    if (whole && t0 + C <= end) {
#pragma unroll
      for (int o = 0; o < KO; ++o) {
        k[o] = at(tk + (t0 + o * KR) * p.k_t, k_off);
        q[o] = at(tq + (t0 + o * KR) * p.q_t, q_off);
      }
#pragma unroll
      for (int o = 0; o < XO; ++o) x[o] = at(tx + (t0 + o * XR) * x_t, x_off);
    } else if (vec) {
      fetch_rows<true>(p, t0, end);
    } else {
      fetch_rows<false>(p, t0, end);
    }
#pragma unroll
    for (int o = 0; o < FO; ++o)
      f[o] = *reinterpret_cast<const u32x4*>(in_row(frags + o * THREADS * 16, threadIdx.x * 16u));
    v = *in_row(vectors, (threadIdx.x < 3 * C ? threadIdx.x : 0) * 4u);
  }
  // len: tokens of the chunk
  template <bool MASK> __device__ __forceinline__ void stage_rows(L& l, const DeltaParams& p, int32_t len) const {
    const int tid = MASK ? (int)lane_offset(threadIdx.x) : threadIdx.x;
#pragma unroll
    for (int o = 0; o < KO; ++o) {
      const int i = tid + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
      const int n = t < len ? p.K - c0 : 0;
      if (KN % THREADS == 0 || i < KN) {
        L::Rows::put8(l.k, t, c0, MASK ? mask8<D>(k[o], n) : k[o]);
        L::Rows::put8(l.q, t, c0, MASK ? mask8<D>(q[o], n) : q[o]);
      }
    }
#pragma unroll
    for (int o = 0; o < XO; ++o) {
      const int i = tid + o * THREADS, t = i / XW, c0 = i % XW * 8;
      L::Cols::put8(l.x, t, c0, MASK ? mask8<D>(x[o], t < len ? p.V - col0 - c0 : 0) : x[o]);
    }
  }
  __device__ __forceinline__ void stage(L& l, const DeltaParams& p, int32_t len) const {
    if (whole && len >= C) stage_rows<false>(l, p, len);
    else stage_rows<true>(l, p, len);
#pragma unroll
    for (int o = 0; o < FO; ++o) reinterpret_cast<u32x4*>(l.f)[threadIdx.x + o * THREADS] = f[o];
    if (threadIdx.x < 3 * C) l.v[threadIdx.x] = v;
  }
};

// A wave's 16 columns of a K x V matrix in memory and in accumulator tiles.  A
// row is a uniform address and a lane's 32-bit offset: 64-bit addresses for
// every lane and row, made once ahead of the loop, would take 64 registers.
template <bool STORE, int KT>
__device__ __forceinline__ void state_columns(f32x4 (&s)[KT], std::conditional_t<STORE, float, const float>* m,
                                              int K, int V, int col, int col_end) {
  const int g = (threadIdx.x & 63) >> 4;
  const uint32_t off = lane_offset((uint32_t)(4 * g * V + col) * 4u);
  auto all = [&](auto in) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!in(16 * t + 4 * g + e)) continue;
        auto* at = in_row(m + (int64_t)(16 * t + e) * V, off);
        if constexpr (STORE) *at = s[t][e];
        else s[t][e] = *at;
      }
  };
  if (K == 16 * KT && col_end <= V) all([](int) { return true; });  // of the whole wave
  else all([&](int k) { return k < K && col < V; });
}

// The products of a chunk's K (and Q) with 16 columns of a state: x = K S, y =
// Q S.  K's and Q's operands alternate, each loaded while the other's products
// run; `last` loads what comes next, behind the last of Q's.
template <typename D, typename Rows, int KS, int NT, bool BOTH, typename F>
__device__ __forceinline__ void rows_times_state(const typename D::storage* lk, const typename D::storage* lq,
                                                 const f32x4 (&s)[2 * KS], f32x4 (&x)[NT], f32x4 (&y)[NT],
                                                 int lane, F&& last) {
  using T = Tile<D>;
  typename T::Exact kf[2][NT], qf[NT];
  typename T::Split sp[2];
  auto load = [&](const typename D::storage* m, int c, typename T::Exact (&to)[NT]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) to[t] = Rows::rows(m, 16 * t, 32 * c, lane);
  };
  load(lk, 0, kf[0]);
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = y[t] = zero4();
  sp[0] = T::split(s[0], s[1]);
#pragma unroll
  for (int c = 0; c < KS; ++c) {
    constexpr int B = BOTH ? 0 : 1;  // K alone: its own operands alternate
    if constexpr (BOTH) {
      load(lq, c, qf);
    } else {
      if (c + 1 < KS) load(lk, c + 1, kf[(c + 1) & B]);
      else last();
    }
    keep_order();
    if (!BOTH && c + 1 < KS) sp[(c + 1) & 1] = T::split(s[2 * c + 2], s[2 * c + 3]);
    each_part<T::kExactSplit>([&](auto P) {
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t] = T::template part<P>(kf[c & B][t], sp[c & 1], x[t]);
    });
    keep_order();
    if constexpr (BOTH) {
      if (c + 1 < KS) load(lk, c + 1, kf[0]);
      else last();
      keep_order();
      if (c + 1 < KS) sp[(c + 1) & 1] = T::split(s[2 * c + 2], s[2 * c + 3]);
      each_part<T::kExactSplit>([&](auto P) {
#pragma unroll
        for (int t = 0; t < NT; ++t) y[t] = T::template part<P>(qf[t], sp[c & 1], y[t]);
      });
      keep_order();
    }
  }
}

// x += (the triangle's frags) y: lower rows meet columns of steps c <= t / 2,
// upper ones c >= t / 2.
template <typename D, bool LOWER, int NF, typename Y, int NT>
__device__ __forceinline__ void triangle_times(const typename Tile<D>::Split (&tri)[NF],
                                               const Y (&y)[NT / 2], f32x4 (&x)[NT]) {
  using T = Tile<D>;
  constexpr int C = 16 * NT, CS = NT / 2;
  constexpr int N = std::is_same<Y, typename T::Split>::value ? T::kSplitSplit : T::kSplitExact;
  each_part<CS * N>([&](auto P) {
    constexpr int c = P / N;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (LOWER ? c <= t / 2 : c >= t / 2)
        x[t] = T::template part<P % N>(tri[LOWER ? lower_frag<C>(t, c) : upper_frag<C>(t, c)], y[c], x[t]);
  });
}

template <typename D, int NF>
__device__ __forceinline__ void load_triangle(typename Tile<D>::Split (&tri)[NF], const char* f, int lane) {
#pragma unroll
  for (int x = 0; x < NF; ++x) tri[x] = Tile<D>::get(f + x * kFragBytes, lane);
}

// s += M^T u for M's rows in LDS, 16 columns of u; half of M's operands are
// loaded while the other half's products run.
template <typename D, typename Rows, int KT, int CS>
__device__ __forceinline__ void cols_times(const typename D::storage* m,
                                           const typename Tile<D>::Fine (&u)[CS], f32x4 (&s)[KT], int lane) {
  using T = Tile<D>;
  constexpr int H = KT / 2;
  typename T::Exact f[2][H];
  auto load = [&](int i) {
#pragma unroll
    for (int t = 0; t < H; ++t) f[i & 1][t] = Rows::cols(m, 32 * (i / 2), 16 * (H * (i & 1) + t), lane);
  };
  load(0);
#pragma unroll
  for (int i = 0; i < 2 * CS; ++i) {
    if (i + 1 < 2 * CS) load(i + 1);
    keep_order();
    each_part<T::kExactFine>([&](auto P) {
#pragma unroll
      for (int t = 0; t < H; ++t) {
        f32x4& to = s[H * (i & 1) + t];
        to = T::template part<P>(f[i & 1][t], u[i / 2], to);
      }
    });
    keep_order();
  }
}

}  // namespace sconv
