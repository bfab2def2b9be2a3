// gated_delta_grad.hip -- gradients of the gated delta rule, for gfx950.
//
// With the names of delta_rule.h, in a chunk whose state after it has the
// gradient dS1:
//   dU = P^T dO + e^(G_C - G) (K dS1),  dR = T^T dU = dU + N^T dU
//   dS0 = e^(G_C) dS1 + scale Q^T (e^G dO) - K^T (e^G beta dR)
// One kernel walks the chunks from the end with dS in registers, as the
// forward walks them, and leaves dS1 and dR of every chunk; then every chunk's
// gradients are independent.  With E_P = scale e (dO U^T) (i >= j), E_A =
// e (dR U^T) (i > j):
//   dV = beta dR,  dQ = scale e^G (dO S0^T) + E_P K
//   Z = e^G (dR S0^T) + E_A K             (dk as read: -beta Z)
//   M = e^(G_C - G) (U dS1^T)             (dk as written into S1)
//   W = E_P^T Q - (beta E_A)^T K          (dk as written for later tokens)
//   dK = M + W - beta Z,  dbeta = rowsum(dR V) - k.Z
// A gate g_t closes between the tokens j < t and i >= t, and only what passes
// it enters its gradient.  With z_ij = E_P k_j.q_i - beta_i E_A k_i.k_j (i > j) and
// s_i = e^G (scale q.(dO S0^T) - beta k.(dR S0^T))_i, what token i reads of S0:
//   dg_t = sum_(i >= t) s_i + sum_(j < t) (k.M)_j + sum_(i >= t > j) z_ij
//          + e^(G_C) <dS1, S0>
// Every term has the factor e^(g_t), and none is a difference of larger ones: the
// gradient of a gate that is nearly closed keeps its digits.
#include "delta_host.h"
#include "delta_prep.h"
#include "delta_walk.h"
#include "norm_rows.h"

namespace sconv {

struct DeltaBwd {
  DeltaParams p;
  const void* dout;
  int64_t do_t, do_h;
  const float *marks, *dfinal;
  float *dinitial, *dstates, *drows;  // drows: dR's accumulator tiles
  int64_t df_slot, di_slot;
  void *dq, *dk, *dv, *dg, *db;
  int64_t dq_t, dq_h, dk_t, dk_h, dv_t, dv_h, dg_t, dg_h, db_t, db_h;
  int32_t do_vec, grads_vec;
};

// Where a lane's part of dR's tiles of 16 columns lies: 1 KB a tile of 16 tokens.
template <int C>
__device__ __forceinline__ f32x4* delta_row_tiles(float* drows, int64_t at, int32_t V, int32_t tile, int lane) {
  return reinterpret_cast<f32x4*>(drows + (at * tiles16(V) + tile) * 16 * C) + lane;
}

// One workgroup walks a sequence's chunks from the last, for one value head
// and 16 columns a wave of NW; LOAD: as many waves more load.  Bound as the
// forward's walk: 2 x 8192 tokens, 16 heads of 128 x 128 bf16 in 471 us (640
// with rows of states stored as they lie and no loaders).
template <typename D, int KP, int NW, bool LOAD, bool VEC>
__global__ __launch_bounds__(LOAD ? 128 * NW : 64 * NW, 2) void delta_back_kernel(DeltaBwd a) {
  using T = Tile<D>;
  using S = typename D::storage;
  constexpr int C = kDeltaChunk<D>, NT = C / 16, KS = KP / 32, KT = KP / 16, CS = C / 32;
  constexpr int NF = kDeltaFrags<C>, PIECES = kGroups<KS, false>;
  using Stage = WalkStage<D, KP, NW, VEC>;
  using Rows = typename Stage::L::Rows;
  using Cols = typename Stage::L::Cols;
  __shared__ typename Stage::L lds[2];

  const DeltaParams& p = a.p;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const WalkPlace place(p, (p.V + 16 * NW - 1) / (16 * NW));
  const int32_t b = place.b, h = place.h, kh = place.kh;
  if (b >= p.batch) return;
  const int32_t slot = p.slots ? p.slots[b] : b;
  if (p.slots && slot == p.pad) return;
  const int32_t start = p.qsl[b], end = p.qsl[b + 1];
  const int32_t cols0 = place.block * 16 * NW;
  const int32_t chunks = (end - start + C - 1) / C, row0 = start / C + b;
  const int64_t KV = (int64_t)p.K * p.V;
  const S* q = static_cast<const S*>(p.q) + kh * p.q_h;
  const S* k = static_cast<const S*>(p.k) + kh * p.k_h;
  const S* dout = static_cast<const S*>(a.dout) + h * a.do_h;
  Stage next;
  next.init(p, k, q, dout, a.do_t, cols0, threadIdx.x % Stage::THREADS);
  auto fetch = [&](int32_t i, auto P, auto N) {
    const int64_t at = (int64_t)(row0 + i) * p.heads + h;
    next.template fetch<decltype(P)::value, decltype(N)::value>(
        p, start + i * C, end, p.frags + (at * (3 * NF) + NF) * kFragBytes, p.vectors + at * kDeltaVectors<C>);
  };
  auto stage = [&](int32_t i, typename Stage::L& l) { next.stage(l, p, end - (start + i * C)); };
  constexpr std::integral_constant<int, 0> kFirst;
  constexpr std::integral_constant<int, 1> kWhole;

  if (LOAD && wave >= NW) {  // as the forward's
    if (chunks > 0) {
      fetch(chunks - 1, kFirst, kWhole);
      stage(chunks - 1, lds[(chunks - 1) & 1]);
      if constexpr (VEC) fetch(max(chunks - 2, 0), kFirst, kWhole);
    }
    __syncthreads();
    for (int32_t i = chunks - 1; i >= 0; --i) {
      if constexpr (!VEC) fetch(max(i - 1, 0), kFirst, kWhole);
      if (i > 0) stage(i - 1, lds[(i - 1) & 1]);
      if constexpr (VEC) keep_order(), fetch(max(i - 2, 0), kFirst, kWhole);
      __syncthreads();
    }
    return;
  }

  const int32_t c16 = 16 * wave, col = cols0 + c16 + r, ends = cols0 + c16 + 16;
  f32x4 s[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) s[t] = zero4();
  if (a.dfinal) state_columns<false>(s, a.dfinal + slot * a.df_slot + h * KV, p.K, p.V, col, ends);
  wait_for_all();
  if (!LOAD && chunks > 0) {
    fetch(chunks - 1, kFirst, kWhole);
    stage(chunks - 1, lds[(chunks - 1) & 1]);
  }
  __syncthreads();
  for (int32_t i = chunks - 1; i >= 0; --i) {
    const typename Stage::L& l = lds[i & 1];
    const int64_t at = (int64_t)(row0 + i) * p.heads + h;
    float* mark = a.dstates + at * delta_state_floats(p.K, p.V) + (ends / 16 - 1) * tiles16(p.K) * 256;
    f32x4 u[NT], none[NT];    // K dS, then dU, then dR
    typename T::Exact go[CS]; // dO
    typename T::Pair tri[NF], us[CS];
    rows_times_state<D, Rows, KS, NT, false>(
        l.k, l.q, s, u, none, lane,
        [&] {
#pragma unroll
          for (int c = 0; c < CS; ++c) go[c] = Cols::cols(l.x, 32 * c, c16, lane);
          load_triangle<D>(tri, l.f + NF * kFragBytes, lane);
        },
        [&](auto P) {
          if constexpr (!LOAD) fetch(max(i - 1, 0), P, std::integral_constant<int, PIECES>());
          if (ends - 16 < p.V) put_tiles<decltype(P)::value, PIECES>(s, mark, p.K, lane);
        });
#pragma unroll
    for (int t = 0; t < NT; ++t) u[t] *= lds4(l.v + C + 16 * t + 4 * g);
    {  // P^T dO; the factors of P^T's columns go by dO's rows
      const f32x4 steps = lds4(l.v + kDeltaFactors<C> + 4);
      f32x4 y[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = T::value(go[t / 2], 4 * (t & 1) + e);
          y[t][e] = T::kScaled ? x * steps[t / 2] : x;
        }
      float most = 0.f;
      if constexpr (T::kScaled) {
#pragma unroll
        for (int t = 0; t < NT; ++t) most = max4(y[t], most);
        most = groups_max(most);
      }
      const Pow2 by(most);
      typename T::Half half[CS];
#pragma unroll
      for (int c = 0; c < CS; ++c) half[c] = T::half(y[2 * c], y[2 * c + 1], by.up);
      triangle_times<D, false>(tri, half, u, by.down, (f32x4){1.f, 1.f, 1.f, 1.f});
    }
    keep_order();
    load_triangle<D>(tri, l.f, lane);
    keep_order();
    const float down = pair_tiles<D>(u, us);
    const float whole = l.v[C - 1];
    typename T::Fine fine[CS];
#pragma unroll
    for (int t = 0; t < KT; ++t) s[t] *= whole;
#pragma unroll
    for (int c = 0; c < CS; ++c) {
      f32x4 y[2];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const f32x4 gam = lds4(l.v + 32 * c + 16 * o + 4 * g) * p.scale;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[o][e] = gam[e] * T::value(go[c], 4 * o + e);
      }
      fine[c] = T::fine(y[0], y[1]);
    }
    triangle_times<D, false>(tri, us, u, down, lds4(l.v + kDeltaFactors<C>));
    keep_order();
    cols_times<D, Rows>(l.q, fine, s, lane);
    if (ends - 16 < p.V) {
      f32x4* to = delta_row_tiles<C>(a.drows, at, p.V, ends / 16 - 1, lane);
#pragma unroll
      for (int t = 0; t < NT; ++t) to[64 * t] = u[t];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
      u[t] *= -(lds4(l.v + 16 * t + 4 * g) * lds4(l.v + 2 * C + 16 * t + 4 * g));
    fine_tiles<D>(u, fine);
    cols_times<D, Rows>(l.k, fine, s, lane);
    if (!LOAD && i > 0) stage(i - 1, lds[(i - 1) & 1]);
    __syncthreads();
  }
  if (a.dinitial) {
    if (!(p.has && p.has[b])) {
#pragma unroll
      for (int t = 0; t < KT; ++t) s[t] = zero4();
    }
    state_columns<true>(s, a.dinitial + slot * a.di_slot + h * KV, p.K, p.V, col, ends);
  }
}

template <int CTRL> __device__ __forceinline__ float lanes_moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Four lanes' four values transposed: entry j of lane q of a quad is entry q of
// its lane j.
__device__ __forceinline__ f32x4 quad_transposed(const f32x4& a, int r) {
  const bool odd = r & 1, high = r & 2;
  f32x4 m;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float keep = odd ? a[i + 1] : a[i], other = lanes_moved<0xB1>(odd ? a[i] : a[i + 1]);
    m[i] = odd ? other : keep, m[i + 1] = odd ? keep : other;
  }
  f32x4 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = high ? m[2 + i] : m[i], other = lanes_moved<0x4E>(high ? m[i] : m[2 + i]);
    o[i] = high ? other : keep, o[2 + i] = high ? keep : other;
  }
  return o;
}

// N values (16 or 8) of every lane summed over the 16 lanes of its group; lane
// r gets the sum of value r % N.  A step halves the values: a lane keeps one half
// and gives its partner the other (15 additions where 16 sums over 16 lanes
// take 64, and one store).
template <int N> __device__ __forceinline__ float sums16(float (&v)[N], int r) {
  static_assert(N == 16 || N == 8);
  auto step = [&](auto ctrl, auto half, bool upper) {
    constexpr int H = decltype(half)::value;
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const float keep = upper ? v[H + j] : v[j], give = upper ? v[j] : v[H + j];
      v[j] = keep + lanes_moved<decltype(ctrl)::value>(give);
    }
  };
  using std::integral_constant;
  if constexpr (N == 16) {
    step(integral_constant<int, 0x140>(), integral_constant<int, 8>(), (r & 8) != 0);  // mirrored
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += lanes_moved<0x140>(v[j]);
  }
  step(integral_constant<int, 0x141>(), integral_constant<int, 4>(), (r & 4) != 0);  // halves mirrored
  step(integral_constant<int, 0x1B>(), integral_constant<int, 2>(), (r & 2) != 0);   // lanes 3 2 1 0
  step(integral_constant<int, 0xB1>(), integral_constant<int, 1>(), (r & 1) != 0);   // lanes 1 0 3 2
  return v[0];
}

// Sums of the values of the 16 lanes of a group that come before a lane (without
// its own), and of those from it on.
__device__ __forceinline__ float sum_before(float v) {
  v = lanes_moved<0x111>(v);  // shifted up by one, zero at the start
  v += lanes_moved<0x111>(v);
  v += lanes_moved<0x112>(v);
  v += lanes_moved<0x114>(v);
  return v + lanes_moved<0x118>(v);
}
__device__ __forceinline__ float sum_from(float v) {
  v += lanes_moved<0x101>(v);
  v += lanes_moved<0x102>(v);
  v += lanes_moved<0x104>(v);
  return v + lanes_moved<0x108>(v);
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Row of tile n of a lower triangle of 4 x 4 tiles, counted row by row.
__device__ __forceinline__ int tile_row(int n) { return n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0; }

// LDS of a workgroup below: K, Q, dO (bf16: as fp16), the parts of U and dR (later of
// three triangles), vectors, sums of the waves.
template <typename D, int KP> struct GradLds {
  using S = typename D::storage;
  static constexpr int C = kDeltaChunk<D>, NW = KP / 16, PARTS = sizeof(S) == 2 ? 2 : 1;
  static constexpr int BIG = C * LdsRows<D, KP>::LD, SMALL = C * LdsRows<D, C>::LD;
  __attribute__((aligned(16))) S k[BIG];
  __attribute__((aligned(16))) S q[BIG];
  __attribute__((aligned(16))) S dout[BIG];
  union {
    struct { S u[PARTS * BIG], r[PARTS * BIG]; };
    S e[3 * PARTS * SMALL];  // E_P, E_A, beta E_A
    __attribute__((aligned(16))) char align_;
  };
  __attribute__((aligned(16))) char f[kDeltaFrags<C> * kFragBytes];  // N
  __attribute__((aligned(16))) float v[kDeltaVectors<C>];
  float part[NW][4][C], dots[NW];
  // the waves' largest |dO|, |dR| and |U| of a block of columns
  float most[NW][3];
  // row sums of E_A k.k
  __attribute__((aligned(16))) float za[C / 16 * (C / 16 + 1) / 2][16];
  // of a tile of z: its rows' and columns' sums (of one on the diagonal, in place
  // of the latter, what passes each of its gates)
  __attribute__((aligned(16))) float z[2][C / 16 * (C / 16 + 1) / 2][16];
};

// One workgroup: all gradients of a chunk's tokens for one key head, its value
// heads one after another (dq and dk add up in registers, in that order).
// Columns come in blocks of KP, 16 a wave; then a wave owns 16 of K.
// 2 x 8192 tokens of 16 heads of 128 x 128 bf16: 469 us for 1.3 GB, 2.8 TB/s.  One
// workgroup a CU (its tiles take 150 KB of LDS), whose loads and products therefore
// do not overlap: LDS, then registers, bound how many run.  ONE: the value channels are
// one block, so what adds up over blocks lives behind its first products alone and
// nothing is spilled (182 of 256 registers, 251 with shared key heads; with blocks 32
// to 79 are: 8 x 4096 tokens, 16 key and 32 value heads, all of backward 2590 us so,
// 2280 with ONE).  Registers are bounded for two workgroups a CU at KP = 64 too, where
// bf16 tiles leave room for one: fp32 ones do for two (4 x 2048 tokens, heads of 64 x
// 100: 396 us, with twice the registers 421).  bf16: dO, dR, U and the states enter as fp16 parts with one factor a
// block (states: a channel and step) of 22 bits; the triangles E beside K and Q as two
// bf16 parts, 16 bits, which only dq and dk, rounded to bf16, take.  So fp32 dg and
// dbeta are 3.5e-7 and 2.9e-7 of their norm off (with 16 bits throughout 4e-6).
template <typename D, int KP, bool GROUPED, bool ONE, bool VEC>
__global__ __launch_bounds__(4 * KP, 2) void delta_grad_kernel(DeltaBwd a) {
  using T = Tile<D>;
  using S = typename D::storage;
  using L = GradLds<D, KP>;
  using Rows = LdsRows<D, KP>;
  constexpr bool kB = sizeof(S) == 2;
  constexpr int C = L::C, NT = C / 16, KS = KP / 32, KT = KP / 16, CS = C / 32, NW = L::NW;
  constexpr int NF = kDeltaFrags<C>, THREADS = 64 * NW, PARTS = L::PARTS, BIG = L::BIG, SMALL = L::SMALL;
  constexpr int TILES = NT * (NT + 1) / 2, MINE = (TILES + NW - 1) / NW;
  using Tri = LdsRows<D, C>;
  __shared__ L l;

  const DeltaParams& p = a.p;
  // Hidden anew in every loop below: all that is computed from them would
  // otherwise be computed once ahead of the loops and spilled there.
  int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = uniform(tid >> 6);
  auto hide = [&] {
    tid = (int)lane_offset((uint32_t)tid);
    lane = tid & 63, r = lane & 15, g = lane >> 4;
  };
  const int32_t row = blockIdx.x, kh = blockIdx.y;
  const DeltaChunk ch = delta_find<C>(p, row);
  if (ch.len == 0) return;
  const int kt16 = tiles16(p.K);

  auto put_split = [&](S* m, int planes, int at, float v) {
    if constexpr (kB) {
      const uint16_t hi = __builtin_bit_cast(uint16_t, (__bf16)v);
      m[at] = hi;
      m[at + planes] = __builtin_bit_cast(uint16_t, (__bf16)(v - bf16_bits_to_float(hi)));
    } else {
      m[at] = v;
    }
  };
  auto rows2 = [&](const S* m, int t0, int c0) {
    if constexpr (kB) return T::as_pair(Rows::rows(m, t0, c0, lane), Rows::rows(m + BIG, t0, c0, lane));
    else return Rows::rows(m, t0, c0, lane);
  };
  // The factor of a block of columns' U, dR or dO: from every wave's largest.
  auto factor = [&](int which) {
    float most = 0.f;
#pragma unroll
    for (int n = 0; n < NW; ++n) most = fmaxf(most, l.most[n][which]);
    return Pow2(most);
  };
  auto tri_rows = [&](const S* m, int t0, int c0) {
    if constexpr (kB)
      return typename T::Split{Tri::rows(m, t0, c0, lane).v, Tri::rows(m + SMALL, t0, c0, lane).v};
    else
      return Tri::rows(m, t0, c0, lane);
  };
  auto tri_cols = [&](const S* m, int t0, int c0) {
    if constexpr (kB)
      return typename T::Split{Tri::cols(m, t0, c0, lane).v, Tri::cols(m + SMALL, t0, c0, lane).v};
    else
      return Tri::cols(m, t0, c0, lane);
  };
  // columns w0 .. of the chunk's rows of two tensors, to registers and on to LDS
  constexpr int N8 = C * KP / 8 / THREADS;
  static_assert(C * KP / 8 % THREADS == 0);
  typedef typename T::Exact Octets[N8];
  auto load2 = [&](Octets& x1, Octets& x2, const S* m1, int64_t ld1, const S* m2, int64_t ld2, int w0,
                   int W) {
#pragma unroll
    for (int o = 0; o < N8; ++o) {
      const int i = tid + o * THREADS, t = i / (KP / 8), c0 = w0 + i % (KP / 8) * 8;
      x1[o] = load8<D, VEC>(m1, ld1, t, ch.len, c0, W);
      x2[o] = load8<D, VEC>(m2, ld2, t, ch.len, c0, W);
    }
  };
  auto masked = [&](const typename T::Exact& x, int o, int w0, int W) {
    const int i = tid + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
    return mask8<D>(x, t < ch.len ? W - w0 - c0 : 0);
  };
  auto stage2 = [&](S* l1, S* l2, const Octets& x1, const Octets& x2, int w0, int W, auto&& first) {
#pragma unroll
    for (int o = 0; o < N8; ++o) {
      const int i = tid + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
      Rows::put8(l1, t, c0, first(masked(x1[o], o, w0, W)));
      Rows::put8(l2, t, c0, masked(x2[o], o, w0, W));
    }
  };
  auto as_is = [](const typename T::Exact& x) { return x; };
  // a tile back to memory, 16 bytes a lane where rows are of such vectors
  auto put_tile = [&](S* m, int64_t ld, int w0, int W, auto&& octet) {
#pragma unroll
    for (int o = 0; o < N8; ++o) {
      const int i = tid + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
      if (t < ch.len) put_row8<D>(m + t * ld, w0 + c0, W, VEC, octet(t, c0));
    }
  };

  Octets x1, x2;
  load2(x1, x2, static_cast<const S*>(p.k) + ch.t0 * p.k_t + kh * p.k_h, p.k_t,
        static_cast<const S*>(p.q) + ch.t0 * p.q_t + kh * p.q_h, p.q_t, 0, p.K);
  f32x4 dq[NT], dk[NT];
  if constexpr (GROUPED) {
#pragma unroll
    for (int t = 0; t < NT; ++t) dq[t] = dk[t] = zero4();
  }

  for (int32_t gh = 0; gh < (GROUPED ? p.group : 1); ++gh) {
    hide();
    const int32_t h = kh * p.group + gh;
    const int64_t at = (int64_t)row * p.heads + h;
    const int64_t state = at * delta_state_floats(p.K, p.V);
    const float *s0 = a.marks + state, *ds = a.dstates + state;
    const S* v = static_cast<const S*>(p.v) + ch.t0 * p.v_t + h * p.v_h;
    const S* dout = static_cast<const S*>(a.dout) + ch.t0 * a.do_t + h * a.do_h;

    f32x4 mq[NT], mz[NT], mw[NT];  // dO S0^T, dR S0^T, U dS1^T
    f32x4 ep[MINE], ea[MINE];      // tiles of dO U^T and dR U^T
    float dot = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) mq[t] = mz[t] = mw[t] = zero4();
#pragma unroll
    for (int m = 0; m < MINE; ++m) ep[m] = ea[m] = zero4();

    for (int32_t v0 = 0; ONE ? v0 == 0 : v0 < p.V; v0 += KP) {
      hide();
      const int c16 = 16 * wave;
      // everything that the block needs from memory, before anything waits
      Octets xo, xv;
      load2(xo, xv, dout, a.do_t, v, p.v_t, v0, p.V);
      const bool first = v0 == 0;
      float vec = 0.f;
      if (first) vec = p.vectors[at * kDeltaVectors<C> + min(tid, kDeltaVectors<C> - 1)];
      static_assert(kDeltaVectors<C> <= THREADS || KP == 64, "a vector entry a thread");
      f32x4 st[KT], y[NT];  // S0's columns, dR
#pragma unroll
      for (int t = 0; t < KT; ++t) st[t] = zero4();
#pragma unroll
      for (int t = 0; t < NT; ++t) y[t] = zero4();
      const int tile0 = (v0 + c16) / 16 * kt16;
      if (v0 + c16 < p.V) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
          if (t < kt16) st[t] = lds4(in_row(s0 + (tile0 + t) * 256, lane * 16u));
      }
      if (v0 + c16 < p.V) {
        const f32x4* from = delta_row_tiles<C>(a.drows, at, p.V, (v0 + c16) / 16, lane);
#pragma unroll
        for (int t = 0; t < NT; ++t) y[t] = from[64 * t];
      }
      constexpr int F16 = NF * kFragBytes / 16, FO = (F16 + THREADS - 1) / THREADS;
      u32x4 nf[FO];
      if (first) {
        const u32x4* from = reinterpret_cast<const u32x4*>(p.frags + at * (3 * NF) * kFragBytes);
#pragma unroll
        for (int o = 0; o < FO; ++o) nf[o] = from[min(tid + o * THREADS, F16 - 1)];
      }
      if constexpr (kB) {  // behind the columns' end dR is zero
        typename T::u16x2 o_most = 0;
        float r_most = 0.f;
#pragma unroll
        for (int o = 0; o < N8; ++o) o_most = T::larger(masked(xo[o], o, v0, p.V), o_most);
#pragma unroll
        for (int t = 0; t < NT; ++t) r_most = max4(y[t], r_most);
        const float x = __uint_as_float((uint32_t)(o_most[0] > o_most[1] ? o_most[0] : o_most[1]) << 16);
        const float dm = groups_max(lanes_reduce<16>(x, Larger())), rm = groups_max(lanes_reduce<16>(r_most, Larger()));
        if (lane == 0) l.most[wave][0] = dm, l.most[wave][1] = rm;
      }
      __syncthreads();  // the last reads of dO, U, dR and the triangles
      if (gh == 0 && first) stage2(l.k, l.q, x1, x2, 0, p.K, as_is);
      // V lies in U's place until U replaces it
      float o_down = 1.f, r_up = 1.f, r_down = 1.f, u_down = 1.f;
      if constexpr (kB) {
        const Pow2 by_o = factor(0), by_r = factor(1);
        o_down = by_o.down, r_up = by_r.up, r_down = by_r.down;
        stage2(l.dout, l.u, xo, xv, v0, p.V, [&](const typename T::Exact& x) { return T::scaled(x, by_o.up); });
      } else {
        stage2(l.dout, l.u, xo, xv, v0, p.V, as_is);
      }
      if (first) {
#pragma unroll
        for (int o = 0; o < FO; ++o)
          if (F16 % THREADS == 0 || tid + o * THREADS < F16)
            reinterpret_cast<u32x4*>(l.f)[tid + o * THREADS] = nf[o];
        for (int x = tid; x < kDeltaVectors<C>; x += THREADS)
          l.v[x] = x == tid ? vec : p.vectors[at * kDeltaVectors<C> + x];
      }
      __syncthreads();
      f32x4 u[NT], none[NT];
      float rv[4 * NT];
      typename T::Exact vv[CS];
      typename T::Pair tri[NF];
      rows_times_state<D, Rows, KS, NT, false>(l.k, l.q, st, u, none, lane, [&] {
#pragma unroll
        for (int c = 0; c < CS; ++c) vv[c] = Rows::cols(l.u, 32 * c, c16, lane);
        load_triangle<D>(tri, l.f, lane);
      }, [](auto) {});
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const f32x4 gam = lds4(l.v + 16 * t + 4 * g), bt = lds4(l.v + 2 * C + 16 * t + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = T::value(vv[t / 2], 4 * (t & 1) + e);
          u[t][e] = bt[e] * (x - gam[e] * u[t][e]);
          rv[4 * t + e] = y[t][e] * x;
        }
      }
      {  // rowsum(dR V), this wave's columns
        const float sv = sums16(rv, r);
        float* to = &l.part[wave][3][16 * (r >> 2) + 4 * g + (r & 3)];
        if (r < 4 * NT) *to = first ? sv : *to + sv;
      }
      {
        typename T::Pair us[CS];
        const float down = pair_tiles<D>(u, us);
        triangle_times<D, true>(tri, us, u, down, lds4(l.v + kDeltaFactors<C> + kFactorsN));
      }
      // the first step's rows of S0 and dS1 are on their way over the barrier
      const int steps = (min(KP, p.V - v0) + 31) / 32;
      f32x4 w[2][2], z[2][2];
      // A tile's lane has four rows of K and one column; this lane's channel of
      // K is one row and four columns of it: quads of lanes trade them.
      auto load_states = [&](int c) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int tile = min(v0 / 16 + 2 * c + o, tiles16(p.V) - 1) * kt16 + min(wave, kt16 - 1);
          const uint32_t from = (uint32_t)(16 * (r >> 2) + 4 * g + (r & 3)) * 16u;
          w[c & 1][o] = lds4(in_row(s0 + tile * 256, from));
          z[c & 1][o] = lds4(in_row(ds + tile * 256, from));
        }
      };
      load_states(0);
      float u_up = 1.f;
      if constexpr (kB) {
        float most = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) most = max4(u[t], most);
        most = groups_max(lanes_reduce<16>(most, Larger()));
        if (lane == 0) l.most[wave][2] = most;
        __syncthreads();
        const Pow2 by_u = factor(2);
        u_up = by_u.up, u_down = by_u.down;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (16 * t + 4 * g + e) * Rows::LD + Rows::pos(c16 + r);
          if constexpr (kB) {
            T::put_pair(l.u[i], l.u[i + BIG], u[t][e] * u_up);
            T::put_pair(l.r[i], l.r[i + BIG], y[t][e] * r_up);
          } else {
            l.u[i] = u[t][e], l.r[i] = y[t][e];
          }
        }
      __syncthreads();
      put_tile(static_cast<S*>(a.dv) + ch.t0 * a.dv_t + h * a.dv_h, a.dv_t, v0, p.V,
               [&](int t, int c0) {
                 const float bt = l.v[2 * C + t];
                 S o[8];
                 const auto hi = Rows::get8(l.r, t, c0);
                 if constexpr (kB) {
                   const auto dr = T::as_pair(hi, Rows::get8(l.r + BIG, t, c0));
                   const float by = bt * r_down;
#pragma unroll
                   for (int e = 0; e < 8; ++e) o[e] = delta_round<D>(by * T::value(dr, e));
                 } else {
#pragma unroll
                   for (int e = 0; e < 8; ++e) o[e] = bt * T::value(hi, e);
                 }
                 return T::join(o);
               });
      // products over this block's columns
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        if (c >= steps) break;
        if (c + 1 < steps) load_states(c + 1);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const bool in = wave < kt16 && v0 / 16 + 2 * c + o < tiles16(p.V);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[c & 1][o][e] = in ? w[c & 1][o][e] : 0.f, z[c & 1][o][e] = in ? z[c & 1][o][e] : 0.f;
            dot = fmaf(w[c & 1][o][e], z[c & 1][o][e], dot);
          }
          w[c & 1][o] = quad_transposed(w[c & 1][o], r);
          z[c & 1][o] = quad_transposed(z[c & 1][o], r);
        }
        // a lane's channel of the states, its largest of these columns near 2^14
        float w_most = 0.f, z_most = 0.f;
        if constexpr (kB) {
          w_most = groups_max(max4(w[c & 1][1], max4(w[c & 1][0], 0.f)));
          z_most = groups_max(max4(z[c & 1][1], max4(z[c & 1][0], 0.f)));
        }
        const Pow2 by_w(w_most), by_z(z_most);
        const auto sw = T::pair(w[c & 1][0], w[c & 1][1], by_w.up), sz = T::pair(z[c & 1][0], z[c & 1][1], by_z.up);
        const float q_real = o_down * by_w.down, z_real = r_down * by_w.down, w_real = u_down * by_z.down;
        typename T::Half fo[2];
        typename T::Pair fr[2], fu[2];
        auto load_rows = [&](int t) {
          fo[t & 1] = T::as_half(Rows::rows(l.dout, 16 * t, 32 * c, lane));
          fr[t & 1] = rows2(l.r, 16 * t, 32 * c);
          fu[t & 1] = rows2(l.u, 16 * t, 32 * c);
        };
        load_rows(0);
        f32x4 sums[2][3];
        auto add_sums = [&](int t) {
          if constexpr (kB) {
            mq[t] += sums[t & 1][0] * q_real;
            mz[t] += sums[t & 1][1] * z_real;
            mw[t] += sums[t & 1][2] * w_real;
          }
        };
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t + 1 < NT) load_rows(t + 1);
          keep_order();
          if constexpr (kB) sums[t & 1][0] = sums[t & 1][1] = sums[t & 1][2] = zero4();
          f32x4 &sq = kB ? sums[t & 1][0] : mq[t], &sr = kB ? sums[t & 1][1] : mz[t], &su = kB ? sums[t & 1][2] : mw[t];
          each_part<T::kPairPair>([&](auto P) {
            if constexpr (P < T::kHalfPair) sq = T::template part<P>(fo[t & 1], sw, sq);
            sr = T::template part<P>(fr[t & 1], sw, sr);
            su = T::template part<P>(fu[t & 1], sz, su);
          });
          if (t > 0) add_sums(t - 1);
          keep_order();
        }
        add_sums(NT - 1);
      }
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        const int want = wave + m * NW;
        if (want >= TILES) break;
        const int I = tile_row(want), J = want - I * (I + 1) / 2;
        f32x4 sp = kB ? zero4() : ep[m], sa = kB ? zero4() : ea[m];
        for (int c = 0; c < steps; ++c) {
          const auto uf = rows2(l.u, 16 * J, 32 * c), rf = rows2(l.r, 16 * I, 32 * c);
          const auto of = T::as_half(Rows::rows(l.dout, 16 * I, 32 * c, lane));
          each_part<T::kPairPair>([&](auto P) {
            if constexpr (P < T::kHalfPair) sp = T::template part<P>(of, uf, sp);
            sa = T::template part<P>(rf, uf, sa);
          });
        }
        if constexpr (kB) ep[m] += sp * (o_down * u_down), ea[m] += sa * (r_down * u_down);
        else ep[m] = sp, ea[m] = sa;
      }
    }
    __syncthreads();
    hide();
    // the triangles, with zeros above the diagonal of every 32 columns
    {
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        const int want = wave + m * NW;
        if (want >= TILES) break;
        const int I = tile_row(want), J = want - I * (I + 1) / 2;
        const int j = 16 * J + r;
        f32x4 qk = zero4(), kk = zero4(), z, ak;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const auto kj = Rows::rows(l.k, 16 * J, 32 * s, lane);
          qk = T::mul(Rows::rows(l.q, 16 * I, 32 * s, lane), kj, qk);
          kk = T::mul(Rows::rows(l.k, 16 * I, 32 * s, lane), kj, kk);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * I + 4 * g + e, x = i * Tri::LD + Tri::pos(j);
          constexpr float kLog2e = 1.44269504088896340736f;
          const float* G = l.v + kDeltaSums<C>;
          const float d = (G[i] - G[j]) + (G[C + i] - G[C + j]);
          const float dec = __builtin_amdgcn_exp2f(i >= j ? d * kLog2e : 0.f);
          const float pv = i >= j ? p.scale * dec * ep[m][e] : 0.f;
          const float av = i > j ? dec * ea[m][e] : 0.f;
          put_split(l.e, SMALL, x, pv);
          put_split(l.e + PARTS * SMALL, SMALL, x, av);
          put_split(l.e + 2 * PARTS * SMALL, SMALL, x, l.v[2 * C + i] * av);
          ak[e] = av * kk[e];
          z[e] = i > j ? pv * qk[e] - l.v[2 * C + i] * ak[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) ak[e] = lanes_reduce<16>(ak[e], Add());
        if (r == 0) *reinterpret_cast<f32x4*>(&l.za[want][4 * g]) = ak;
        if (I == J) {  // the tile's rows i >= t and columns j < t, lane r's t
          float passes = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float before = sum_before(z[e]);
            passes += 4 * g + e >= r ? before : 0.f;
          }
          passes = sum_groups(passes);
          if (g == 0) l.z[1][want][r] = passes;
        } else {
          const float cols = sum_groups((z[0] + z[1]) + (z[2] + z[3]));
          if (g == 0) l.z[1][want][r] = cols;
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = lanes_reduce<16>(z[e], Add());
          if (r == 0) *reinterpret_cast<f32x4*>(&l.z[0][want][4 * g]) = z;
        }
        if (I == J && I % 2 == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = (16 * I + 4 * g + e) * Tri::LD + Tri::pos(j + 16);
#pragma unroll
            for (int o = 0; o < 3; ++o) put_split(l.e + o * PARTS * SMALL, SMALL, x, 0.f);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 gam = lds4(l.v + 16 * t + 4 * g);
      mq[t] *= p.scale * gam;
      mz[t] *= gam;
      mw[t] *= lds4(l.v + C + 16 * t + 4 * g);
    }
    // rows' sums over this wave's channels, one quantity after the other
    const bool last = gh + 1 == p.group;
    const int kidx = 16 * wave + r, mine = 16 * (r >> 2) + 4 * g + (r & 3);
    auto row_sums = [&](float* to, auto&& f) {
      float v[4 * NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * t + e] = f(t, e, (16 * t + 4 * g + e) * Rows::LD + Rows::pos(kidx));
      const float sum = sums16(v, r);
      if (r < 4 * NT) to[mine] = sum;
    };
    row_sums(l.part[wave][0], [&](int t, int e, int i) {
      const float bt = l.v[2 * C + 16 * t + 4 * g + e];
      return to_float<D>(l.q[i]) * mq[t][e] - bt * (to_float<D>(l.k[i]) * mz[t][e]);
    });
    row_sums(l.part[wave][1], [&](int t, int e, int i) { return to_float<D>(l.k[i]) * mw[t][e]; });
    row_sums(l.part[wave][2], [&](int t, int e, int i) { return to_float<D>(l.k[i]) * mz[t][e]; });
    __syncthreads();
    f32x4 w[NT], neg[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) w[t] = neg[t] = zero4();
#pragma unroll
    for (int c = 0; c < CS; ++c) {
      const auto kf = Rows::cols(l.k, 32 * c, 16 * wave, lane), qf = Rows::cols(l.q, 32 * c, 16 * wave, lane);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (c <= t / 2) {
          const auto x = tri_rows(l.e, 16 * t, 32 * c), y = tri_rows(l.e + PARTS * SMALL, 16 * t, 32 * c);
          each_part<T::kSplitExact>([&](auto P) {
            mq[t] = T::template part<P>(x, kf, mq[t]);
            mz[t] = T::template part<P>(y, kf, mz[t]);
          });
        }
        if (c >= t / 2) {
          const auto x = tri_cols(l.e, 32 * c, 16 * t), y = tri_cols(l.e + 2 * PARTS * SMALL, 32 * c, 16 * t);
          each_part<T::kSplitExact>([&](auto P) {
            w[t] = T::template part<P>(x, qf, w[t]);
            neg[t] = T::template part<P>(y, kf, neg[t]);
          });
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) w[t] -= neg[t];
    // dq and dk, over the value heads; this wave's channels of Q and K have
    // been read for the last time
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 gk = mw[t] + w[t] - lds4(l.v + 2 * C + 16 * t + 4 * g) * mz[t], gq = mq[t];
      if constexpr (GROUPED) gq = dq[t] += gq, gk = dk[t] += gk;
      if (!GROUPED || last) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (16 * t + 4 * g + e) * Rows::LD + Rows::pos(kidx);
          l.q[i] = delta_round<D>(gq[e]);
          l.k[i] = delta_round<D>(gk[e]);
        }
      }
    }
    dot = lanes_reduce<64>(dot, Add());
    if (lane == 0) l.dots[wave] = dot;
    __syncthreads();
    if (wave == 0) {
      const int t = lane;
      float own = 0.f, km = 0.f, sz = 0.f, sv = 0.f, all = 0.f;
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const int x = t < C ? t : 0;
        own += l.part[n][0][x], km += l.part[n][1][x], sz += l.part[n][2][x], sv += l.part[n][3][x];
        all += l.dots[n];
      }
      if (t >= C) own = km = 0.f;
      // what passes gate t, of z's tiles: those below and left of its own whole,
      // those below it up to its column, those left of it from its row on
      const int I = t < C ? t / 16 : 0, at16 = t % 16;
      float whole = 0.f, below = 0.f, left = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < i; ++j) {
          const int n = i * (i + 1) / 2 + j;
          const float rs = l.z[0][n][at16], cs = l.z[1][n][at16];
          whole += i > I && j < I ? rs : 0.f;
          below += j == I ? cs : 0.f;
          left += i == I ? rs : 0.f;
        }
      const float pairs = lanes_reduce<16>(whole, Add()) + sum_before(below) + sum_from(left) +
                          l.z[1][I * (I + 3) / 2][at16];
      // k.Z of token t: what it reads of S0, and of the tokens ahead of it
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) sz += i == I ? l.za[i * (i + 1) / 2 + j][at16] : 0.f;
      float before = __shfl_up(km, 1, 64), after = own;
      before = lane > 0 ? before : 0.f;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const float x = __shfl_up(before, d, 64), y = __shfl_down(after, d, 64);
        if (lane >= d) before += x;
        if (lane + d < 64) after += y;
      }
      if (t < ch.len) {
        const float dg = (after + before) + (pairs + l.v[C - 1] * all);
        const float db = sv - sz;
        const int64_t tok = ch.t0 + t;
        if (p.gates_f32) {
          static_cast<float*>(a.dg)[tok * a.dg_t + h * a.dg_h] = dg;
          static_cast<float*>(a.db)[tok * a.db_t + h * a.db_h] = db;
        } else {
          static_cast<S*>(a.dg)[tok * a.dg_t + h * a.dg_h] = delta_round<D>(dg);
          static_cast<S*>(a.db)[tok * a.db_t + h * a.db_h] = delta_round<D>(db);
        }
      }
    }
  }
  // the barrier above also ends the writes of the tiles below
  put_tile(static_cast<S*>(a.dq) + ch.t0 * a.dq_t + kh * a.dq_h, a.dq_t, 0, p.K,
           [&](int t, int c0) { return Rows::get8(l.q, t, c0); });
  put_tile(static_cast<S*>(a.dk) + ch.t0 * a.dk_t + kh * a.dk_h, a.dk_t, 0, p.K,
           [&](int t, int c0) { return Rows::get8(l.k, t, c0); });
}

template <typename D, int KP>
static int delta_backward(DeltaBwd a, int64_t rows, hipStream_t stream) {
  const char* what = "gated_delta_rule_varlen_bwd";
  const DeltaParams& p = a.p;
  if (int rc = delta_prepare<D, KP, true>(what, p, rows, stream)) return rc;
  const bool vec = p.qk_vec && a.do_vec;
  const dim3 walk(512);
  bool wide = false;
  if constexpr (sizeof(typename D::storage) == 2) {
    wide = delta_wide(p);
    if (wide) {
      const dim3 grid = delta_walk_grid(a.p, (p.V + 127) / 128);
      if (vec) hipLaunchKernelGGL((delta_back_kernel<D, KP, 8, false, true>), grid, walk, 0, stream, a);
      else hipLaunchKernelGGL((delta_back_kernel<D, KP, 8, false, false>), grid, walk, 0, stream, a);
    }
  }
  if (!wide) {
    const dim3 grid = delta_walk_grid(a.p, (p.V + 63) / 64);
    if (vec) hipLaunchKernelGGL((delta_back_kernel<D, KP, 4, true, true>), grid, walk, 0, stream, a);
    else hipLaunchKernelGGL((delta_back_kernel<D, KP, 4, true, false>), grid, walk, 0, stream, a);
  }
  if (int rc = check_launch(what)) return rc;
  auto gradients = [&](auto one) {
    constexpr bool ONE = decltype(one)::value;
    const dim3 chunks((uint32_t)rows, p.heads / p.group), threads(4 * KP);
    if (!(vec && p.v_vec && a.grads_vec))
      hipLaunchKernelGGL((delta_grad_kernel<D, KP, true, ONE, false>), chunks, threads, 0, stream, a);
    else if (p.group > 1)
      hipLaunchKernelGGL((delta_grad_kernel<D, KP, true, ONE, true>), chunks, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((delta_grad_kernel<D, KP, false, ONE, true>), chunks, threads, 0, stream, a);
  };
  if (p.V <= KP) gradients(std::true_type());
  else gradients(std::false_type());
  return check_launch(what);
}

}  // namespace sconv

extern "C" int gated_delta_rule_varlen_bwd(
    const void* dout, int64_t do_stride_t, int64_t do_stride_h, const void* q, int64_t q_stride_t,
    int64_t q_stride_h, const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v,
    int64_t v_stride_t, int64_t v_stride_h, const void* g, int64_t g_stride_t, int64_t g_stride_h,
    const void* beta, int64_t b_stride_t, int64_t b_stride_h, float scale,
    const float* checkpoints, int64_t checkpoint_rows, const int32_t* query_start_loc,
    int32_t batch, const int32_t* cache_indices, const uint8_t* has_initial_state,
    int64_t num_slots, const float* dfinal_states, int64_t df_stride_slot, float* dinitial_states,
    int64_t di_stride_slot, void* dq, int64_t dq_stride_t, int64_t dq_stride_h, void* dk,
    int64_t dk_stride_t, int64_t dk_stride_h, void* dv, int64_t dv_stride_t, int64_t dv_stride_h,
    void* dg, int64_t dg_stride_t, int64_t dg_stride_h, void* dbeta, int64_t db_stride_t,
    int64_t db_stride_h, float* workspace, int64_t workspace_floats, int64_t total_T,
    int32_t key_heads, int32_t value_heads, int32_t K, int32_t V, int32_t dtype,
    int32_t gate_dtype, int32_t pad_slot_id, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* what = "gated_delta_rule_varlen_bwd";
  DeltaBwd a = {};
  DeltaCall c = {what, total_T, batch, key_heads, value_heads, K, V, dtype, gate_dtype};
  if (int rc = delta_sizes(c)) return rc;
  if (batch == 0 || value_heads == 0 || V == 0) return SCONV_OK;
  if (int rc = delta_grids(c)) return rc;
  if (!query_start_loc) return fail(SCONV_ERR_INVALID, "%s: NULL query_start_loc", what);
  if (int rc = delta_inputs(c, a.p, q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v,
                            v_stride_t, v_stride_h, g, g_stride_t, g_stride_h, beta, b_stride_t,
                            b_stride_h, scale))
    return rc;
  if ((total_T > 0 && !dout) || !checkpoints) return fail(SCONV_ERR_INVALID, "%s: NULL input", what);
  if (do_stride_t < 0 || do_stride_h < 0) return fail(SCONV_ERR_INVALID, "%s: negative stride", what);
  delta_packing(a.p, query_start_loc, cache_indices, has_initial_state, pad_slot_id);
  const int64_t rows = delta_rows(total_T, batch, delta_chunk(dtype));
  if (checkpoint_rows < rows || !aligned16(checkpoints))
    return fail(SCONV_ERR_INVALID, "%s: %lld checkpoint rows, needs %lld at 16 bytes", what,
                (long long)checkpoint_rows, (long long)rows);
  const bool indexed = cache_indices != nullptr;
  DeltaBuffer df, di, oq, ok, ov, og, ob;
  if (int rc = delta_pool(c, dfinal_states, num_slots, df_stride_slot, indexed, "dfinal_states", &df))
    return rc;
  if (int rc = delta_pool(c, dinitial_states, num_slots, di_stride_slot, indexed, "dinitial_states", &di))
    return rc;
  const int64_t gs = elem_size(gate_dtype);
  if (int rc = delta_output(c, dq, dq_stride_t, dq_stride_h, key_heads, K, "dq", &oq)) return rc;
  if (int rc = delta_output(c, dk, dk_stride_t, dk_stride_h, key_heads, K, "dk", &ok)) return rc;
  if (int rc = delta_output(c, dv, dv_stride_t, dv_stride_h, value_heads, V, "dv", &ov)) return rc;
  if (int rc = delta_output(c, dg, dg_stride_t, dg_stride_h, value_heads, 1, "dg", &og, gs)) return rc;
  if (int rc = delta_output(c, dbeta, db_stride_t, db_stride_h, value_heads, 1, "dbeta", &ob, gs))
    return rc;
  const DeltaSpace s = delta_space(total_T, batch, value_heads, K, V, dtype);
  if (!workspace || workspace_floats < s.bwd || !aligned16(workspace))
    return fail(SCONV_ERR_INVALID, "%s: workspace needs %lld floats at 16 bytes", what,
                (long long)s.bwd);
  // dinitial_states may be dfinal_states itself; otherwise they share nothing
  const bool same = dfinal_states && dinitial_states == dfinal_states && di_stride_slot == df_stride_slot;
  if (!same && delta_overlap(df, di))
    return fail(SCONV_ERR_INVALID, "%s: dfinal_states and dinitial_states overlap", what);
  const DeltaBuffer marks = delta_block(checkpoints, rows * value_heads * delta_state_floats(K, V) * 4);
  const DeltaBuffer work = delta_block(workspace, s.bwd * 4);
  const DeltaBuffer od = delta_tensor(dout, do_stride_t, do_stride_h, total_T, value_heads, V,
                                      elem_size(dtype));
  for (const DeltaBuffer& o : {oq, ok, ov, og, ob, di, work})
    if (delta_overlap(o, marks) || delta_overlap(o, od) || (!same && delta_overlap(o, df) && o.p != di.p))
      return fail(SCONV_ERR_INVALID, "%s: an output overlaps an input", what);
  if (int rc = delta_disjoint(c, a.p, {oq, ok, ov, og, ob, di, work})) return rc;
  a.p.vectors = workspace;
  a.p.frags = reinterpret_cast<char*>(workspace + s.vectors);
  a.drows = workspace + s.bwd_rows;
  a.dstates = workspace + s.bwd_states;
  a.dout = dout, a.do_t = do_stride_t, a.do_h = do_stride_h;
  a.marks = checkpoints, a.dfinal = dfinal_states, a.df_slot = df_stride_slot;
  a.dinitial = dinitial_states, a.di_slot = di_stride_slot;
  a.dq = dq, a.dq_t = dq_stride_t, a.dq_h = dq_stride_h;
  a.dk = dk, a.dk_t = dk_stride_t, a.dk_h = dk_stride_h;
  a.dv = dv, a.dv_t = dv_stride_t, a.dv_h = dv_stride_h;
  a.dg = dg, a.dg_t = dg_stride_t, a.dg_h = dg_stride_h;
  a.db = dbeta, a.db_t = db_stride_t, a.db_h = db_stride_h;
  const int64_t n = 16 / elem_size(dtype);
  a.do_vec = delta_vec(dout, do_stride_t, do_stride_h, V, n);
  a.grads_vec = delta_vec(dv, dv_stride_t, dv_stride_h, V, n) && delta_vec(dq, dq_stride_t, dq_stride_h, K, n) &&
                delta_vec(dk, dk_stride_t, dk_stride_h, K, n);
  if (dtype == SCONV_BF16)
    return K <= 64 ? delta_backward<Bf16, 64>(a, rows, stream) : delta_backward<Bf16, 128>(a, rows, stream);
  return K <= 64 ? delta_backward<F32, 64>(a, rows, stream) : delta_backward<F32, 128>(a, rows, stream);
}
