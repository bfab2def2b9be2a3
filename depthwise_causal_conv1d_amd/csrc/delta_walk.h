// delta_walk.h -- how the kernels that walk a sequence's chunks bring a chunk
// into LDS: K, Q, two sets of frags, their vectors and the workgroup's columns
// of one more tensor.
//
// Where the walks fill the chip (eight waves a workgroup), a chunk's loads go
// out between the products of the chunk ahead of it and wait in registers.
// Where they do not, a chain of chunks is what takes the time: four waves
// compute and four more load, stage into a second buffer and store outputs
// meanwhile (2 x 8192 tokens of 16 heads bf16, forward and backward walk, with states
// stored as rows: 524 and 556 us, without them 597 and 640; as they are now 443 and 471).
#pragma once

#include "delta_rule.h"
#include "row_lanes.h"

namespace sconv {

// A workgroup's sequence, value head and block of columns; see delta_walk_grid.
struct WalkPlace {
  int32_t b, h, kh, block;
  __device__ __forceinline__ WalkPlace(const DeltaParams& p, int32_t cols) {
    const uint32_t L = blockIdx.x, m = L / (uint32_t)p.spread, n = (uint32_t)(p.group * cols);
    const uint32_t pair = m / n * (uint32_t)p.spread + L % (uint32_t)p.spread, i = m % n;
    const uint32_t key_heads = p.heads / p.group;
    b = (int32_t)(pair / key_heads), kh = (int32_t)(pair % key_heads);
    h = kh * p.group + (int32_t)i / cols, block = (int32_t)i % cols;
  }
};

template <typename D, int KP, int NW> struct WalkLds {
  using S = typename D::storage;
  static constexpr int C = kDeltaChunk<D>;
  using Rows = LdsRows<D, KP>;
  using Cols = LdsRows<D, 16 * NW>;
  __attribute__((aligned(16))) S k[C * Rows::LD];
  __attribute__((aligned(16))) S q[C * Rows::LD];
  __attribute__((aligned(16))) S x[C * Cols::LD];
  __attribute__((aligned(16))) char f[2 * kDeltaFrags<C> * kFragBytes];
  __attribute__((aligned(16))) float v[kWalkVectors<D, C>];
};

template <typename D, int KP, int NW, bool VEC> struct WalkStage {
  using L = WalkLds<D, KP, NW>;
  using S = typename D::storage;
  using E = typename Tile<D>::Exact;
  static constexpr int C = L::C, THREADS = 64 * NW;
  static constexpr int XW = 2 * NW;  // octets of a row of x
  static constexpr int KN = C * KP / 8, XN = C * XW, FN = 2 * kDeltaFrags<C> * kFragBytes / 16;
  static constexpr int KO = (KN + THREADS - 1) / THREADS, XO = XN / THREADS, FO = FN / THREADS;
  static constexpr int VN = kWalkVectors<D, C>, VO = (VN + THREADS - 1) / THREADS;
  static_assert(XN % THREADS == 0 && FN % THREADS == 0);
  E k[KO], q[KO], x[XO];
  u32x4 f[FO];
  float v[VO];

  // A thread's column of each tensor in bytes (fp32: of its second half too),
  // made once; a chunk's rows end at `end`, and lanes behind it load its last.
  uint32_t k_c[2], x_c[2];
  const S *tk, *tq, *tx;  // the heads' first rows
  int64_t x_t;
  int32_t col0;
  int id;      // of THREADS
  bool whole;  // no row ends inside the tiles

  static __device__ __forceinline__ void columns(uint32_t (&c)[2], int c0, int W) {
    c[0] = (uint32_t)(c0 < W ? c0 : 0) * (uint32_t)sizeof(S);
    c[1] = (uint32_t)(c0 + 4 < W ? c0 + 4 : 0) * (uint32_t)sizeof(S);
  }
  __device__ __forceinline__ void init(const DeltaParams& p, const S* k_, const S* q_, const S* x_,
                                       int64_t x_t_, int32_t col0_, int id_) {
    id = id_;
    tk = k_, tq = q_, tx = x_, x_t = x_t_, col0 = col0_;
    whole = p.K == KP && col0 + 16 * NW <= p.V;
    columns(k_c, id % (KP / 8) * 8, p.K);
    columns(x_c, col0 + id % XW * 8, p.V);
  }
  static __device__ __forceinline__ E at(const S* rows, uint32_t row, const uint32_t (&c)[2]) {
    if constexpr (sizeof(S) == 2)
      return {__builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(in_row(rows, row + c[0])))};
    else
      return {*reinterpret_cast<const f32x4*>(in_row(rows, row + c[0])),
              *reinterpret_cast<const f32x4*>(in_row(rows, row + c[1]))};
  }
  // The chunk's rows are t0 .. end - 1.  One path of loads: where paths with
  // loads meet, the compiler waits for those of either, and on this machine a
  // wait for loads is one for stores as well (4000 of a chunk's 13000 cycles).
  // Piece P of N of it: a wave stands still while the memory pipes are full, so
  // a chunk's loads go out between the products of the one ahead of it.
  template <int P, int N>
  __device__ __forceinline__ void fetch(const DeltaParams& p, int32_t t0, int32_t end,
                                        const char* frags, const float* vectors) {
    const S *rk = tk + t0 * p.k_t, *rq = tq + t0 * p.q_t, *rx = tx + t0 * x_t;
    const int32_t last = end - t0 - 1;
    constexpr int ALL = 2 * KO + XO + FO + VO, LO = ALL * P / N, HI = ALL * (P + 1) / N;
    // hidden, or all these addresses would be made ahead of the loop and held
    const int tid = VEC ? id : (int)lane_offset(id);
    auto rows = [&](const S* m, int64_t ld, int i, int wide, const uint32_t (&c)[2], int c0, int W) {
      const int t = i / wide;
      if constexpr (VEC) return at(m, (uint32_t)min(t, last) * (uint32_t)ld * (uint32_t)sizeof(S), c);
      else return load8<D, false>(m, ld, t, last + 1, c0 + i % wide * 8, W);
    };
#pragma unroll
    for (int n = LO; n < HI; ++n) {
      if (n < KO) {
        k[n] = rows(rk, p.k_t, tid + n * THREADS, KP / 8, k_c, 0, p.K);
      } else if (n < 2 * KO) {
        q[n - KO] = rows(rq, p.q_t, tid + (n - KO) * THREADS, KP / 8, k_c, 0, p.K);
      } else if (n < 2 * KO + XO) {
        x[n - 2 * KO] = rows(rx, x_t, tid + (n - 2 * KO) * THREADS, XW, x_c, col0, p.V);
      } else if (n < 2 * KO + XO + FO) {
        const int o = n - 2 * KO - XO;
        f[o] = *reinterpret_cast<const u32x4*>(in_row(frags + o * THREADS * 16, id * 16u));
      } else {
        const int o = n - 2 * KO - XO - FO, at = id + o * THREADS;
        v[o] = *in_row(vectors, (at < VN ? at : 0) * 4u);
      }
    }
  }
  // len: tokens of the chunk
  template <bool MASK> __device__ __forceinline__ void stage_rows(L& l, const DeltaParams& p, int32_t len) const {
    const int tid = MASK ? (int)lane_offset(id) : id;
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
    for (int o = 0; o < FO; ++o) reinterpret_cast<u32x4*>(l.f)[id + o * THREADS] = f[o];
#pragma unroll
    for (int o = 0; o < VO; ++o)
      if ((o + 1) * THREADS <= VN || id + o * THREADS < VN) l.v[id + o * THREADS] = v[o];
  }
};

// Rows t0 .. end - 1 of an output that waits in x, to memory.
template <typename Stage, typename D, bool VEC>
__device__ __forceinline__ void put_rows(const typename Stage::L& l, typename D::storage* out, int64_t ld, int32_t V,
                                         int32_t cols0, int32_t t0, int32_t end, int id) {
  using S = typename D::storage;
#pragma unroll
  for (int o = 0; o < Stage::XO; ++o) {
    const int x = id + o * Stage::THREADS, t = x / Stage::XW, c0 = x % Stage::XW * 8;
    if (t < end - t0) {
      const auto y = Stage::L::Cols::get8(l.x, t, c0);
      if constexpr (VEC)
        put_row8<D>(in_row(out + t0 * ld, (uint32_t)t * (uint32_t)ld * (uint32_t)sizeof(S)), cols0 + c0, V, true, y);
      else
        put_row8<D>(out + (int64_t)(t0 + t) * ld, cols0 + c0, V, false, y);
    }
  }
}

// Ends what is in flight: loads ahead of a loop would make their registers'
// first use inside it a wait for the loop's own.
__device__ __forceinline__ void wait_for_all() { __builtin_amdgcn_s_waitcnt(0); }

// A wave's 16 columns of a K x V state in its slot and in accumulator tiles.  A
// row is a uniform address and a lane's 32-bit offset.
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

// Piece P of N of the same columns to a chunk's tiles: one store of 1 KB a
// tile.  (As rows of V floats a walk's chunk took 3000 of 9500 cycles for its
// 32 stores of 64-byte pieces.)
template <int P, int N, int KT>
__device__ __forceinline__ void put_tiles(const f32x4 (&s)[KT], float* m, int K, int lane) {
#pragma unroll
  for (int t = KT * P / N; t < KT * (P + 1) / N; ++t)
    if (16 * t < K) *reinterpret_cast<f32x4*>(in_row(m + t * 256, lane * 16u)) = s[t];
}

// The products of a chunk's K (and Q) with 16 columns of a state: x = K S, y
// = Q S.  K's and Q's operands alternate, each loaded while the other's products
// run; `last` loads what comes next, behind the last of them.  piece(j) issues
// what else there is for memory, j of kGroups.
template <int KS, bool BOTH> constexpr int kGroups = BOTH ? 2 * KS : KS;
template <typename D, typename Rows, int KS, int NT, bool BOTH, typename F, typename G>
__device__ __forceinline__ void rows_times_state(const typename D::storage* lk, const typename D::storage* lq,
                                                 const f32x4 (&s)[2 * KS], f32x4 (&x)[NT],
                                                 f32x4 (&y)[NT], int lane, F&& last, G&& piece) {
  using T = Tile<D>;
  typename T::Exact kf[2][NT], qf[NT];
  typename T::Fine sp[2];
  auto load = [&](const typename D::storage* m, int c, typename T::Exact (&to)[NT]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) to[t] = Rows::rows(m, 16 * t, 32 * c, lane);
  };
  auto split = [&](int c) { sp[c & 1] = T::fine(s[2 * c], s[2 * c + 1]); };
  load(lk, 0, kf[0]);
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = y[t] = zero4();
  split(0);
  each_part<KS>([&](auto c) {
    constexpr int B = BOTH ? 0 : 1;  // K alone: its own operands alternate
    if constexpr (BOTH) {
      load(lq, c, qf);
    } else {
      if constexpr (c + 1 < KS) load(lk, c + 1, kf[(c + 1) & B]);
      else last();
    }
    piece(std::integral_constant<int, BOTH ? 2 * c : c>());
    keep_order();
    if constexpr (!BOTH && c + 1 < KS) split(c + 1);
    each_part<T::kExactFine>([&](auto P) {
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t] = T::template part<P>(kf[c & B][t], sp[c & 1], x[t]);
    });
    keep_order();
    if constexpr (BOTH) {
      if constexpr (c + 1 < KS) load(lk, c + 1, kf[0]);
      else last();
      piece(std::integral_constant<int, 2 * c + 1>());
      keep_order();
      if constexpr (c + 1 < KS) split(c + 1);
      each_part<T::kExactFine>([&](auto P) {
#pragma unroll
        for (int t = 0; t < NT; ++t) y[t] = T::template part<P>(qf[t], sp[c & 1], y[t]);
      });
      keep_order();
    }
  });
}

// x += (the triangle's frags) y: lower rows meet columns of steps c <= t / 2,
// upper ones c >= t / 2.  y is an operand made with the factor whose inverse is
// `down`; rows: the inverses of the factors of the triangle's rows of tiles.
template <typename D, bool LOWER, int NF, typename Y, int NT>
__device__ __forceinline__ void triangle_times(const typename Tile<D>::Pair (&tri)[NF], const Y (&y)[NT / 2],
                                               f32x4 (&x)[NT], float down, const f32x4& rows) {
  using T = Tile<D>;
  constexpr int C = 16 * NT, CS = NT / 2;
  constexpr int N = std::is_same<Y, typename T::Pair>::value ? T::kPairPair : T::kPairHalf;
  f32x4 own[NT];
  if constexpr (T::kScaled) {
#pragma unroll
    for (int t = 0; t < NT; ++t) own[t] = zero4();
  }
  f32x4(&to)[NT] = T::kScaled ? own : x;
  each_part<CS * N>([&](auto P) {
    constexpr int c = P / N;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (LOWER ? c <= t / 2 : c >= t / 2)
        to[t] = T::template part<P % N>(tri[LOWER ? lower_frag<C>(t, c) : upper_frag<C>(t, c)], y[c], to[t]);
  });
  if constexpr (T::kScaled) {
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] += own[t] * (rows[t] * down);
  }
}

template <typename D, int NF>
__device__ __forceinline__ void load_triangle(typename Tile<D>::Pair (&tri)[NF], const char* f, int lane) {
#pragma unroll
  for (int x = 0; x < NF; ++x) tri[x] = Tile<D>::get(f + x * kFragBytes, lane);
}

// A column's tiles as operands beside a triangle; returns the inverse of their factor.
template <typename D, int NT>
__device__ __forceinline__ float pair_tiles(const f32x4 (&u)[NT], typename Tile<D>::Pair (&o)[NT / 2]) {
  float most = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) most = max4(u[t], most);
  const Pow2 by(Tile<D>::kScaled ? groups_max(most) : 1.f);
#pragma unroll
  for (int c = 0; c < NT / 2; ++c) o[c] = Tile<D>::pair(u[2 * c], u[2 * c + 1], by.up);
  return by.down;
}

template <typename D, int NT>
__device__ __forceinline__ void fine_tiles(const f32x4 (&u)[NT], typename Tile<D>::Fine (&o)[NT / 2]) {
#pragma unroll
  for (int c = 0; c < NT / 2; ++c) o[c] = Tile<D>::fine(u[2 * c], u[2 * c + 1]);
}

// s += M^T u for M's rows in LDS, 16 columns of u; half of M's operands are
// loaded while the other half's products run.
template <typename D, typename Rows, int KT, int CS>
__device__ __forceinline__ void cols_times(const typename D::storage* m,
                                           const typename Tile<D>::Fine (&u)[CS], f32x4 (&s)[KT],
                                           int lane) {
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
