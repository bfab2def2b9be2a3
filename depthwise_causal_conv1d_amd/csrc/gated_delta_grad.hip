// gated_delta_grad.hip -- gradients of the gated delta rule, for gfx950.
//
// With the names of delta_rule.h, in a chunk whose state after it has the
// gradient dS1:
//   dU = P^T dO + e^(G_C - G) (K dS1),  dR = T^T dU = dU + N^T dU
//   dS0 = e^(G_C) dS1 + scale Q^T (e^G dO) - K^T (e^G beta dR)
// One kernel walks the chunks from the end with dS in registers, as the
// forward walks them, and leaves dS1 of every chunk; then every chunk's
// gradients are independent.  With E_P = scale e (dO U^T) (i >= j), E_A =
// e (dR U^T) (i > j):
//   dV = beta dR,  dQ = scale e^G (dO S0^T) + E_P K
//   Z = e^G (dR S0^T) + E_A K             (dk as read: -beta Z)
//   M = e^(G_C - G) (U dS1^T)             (dk as written into S1)
//   W = E_P^T Q - (beta E_A)^T K          (dk as written for later tokens)
//   dK = M + W - beta Z,  dbeta = rowsum(dR V) - k.Z
// The gradient of a running sum G_i is q.dq - beta k.Z - k.W - k.M, that of
// G_C adds <dS1, S1> = e^(G_C) <dS1, S0> + sum k.M; so
//   dg_t = sum_(i >= t) (q.dq - beta k.Z - k.W)_i + sum_(j < t) (k.M)_j
//          + e^(G_C) <dS1, S0>
// in which the parts that would cancel are left out.
#include "delta_host.h"
#include "delta_prep.h"
#include "delta_walk.h"

namespace sconv {

struct DeltaBwd {
  DeltaParams p;
  const void* dout;
  int64_t do_t, do_h;
  const float *marks, *dfinal;
  float *dinitial, *dstates;
  int64_t df_slot, di_slot;
  void *dq, *dk, *dv, *dg, *db;
  int64_t dq_t, dq_h, dk_t, dk_h, dv_t, dv_h, dg_t, dg_h, db_t, db_h;
  int32_t do_vec;
};

// One workgroup walks a sequence's chunks from the last, for one value head
// and 16 columns a wave.
template <typename D, int KP, int NW>
__global__ __launch_bounds__(64 * NW, NW / 4) void delta_back_kernel(DeltaBwd a) {
  using T = Tile<D>;
  using S = typename D::storage;
  constexpr int C = kDeltaChunk<D>, NT = C / 16, KS = KP / 32, KT = KP / 16, CS = C / 32;
  constexpr int NF = kDeltaFrags<C>;
  using Stage = WalkStage<D, KP, NW>;
  using Rows = typename Stage::L::Rows;
  using Cols = typename Stage::L::Cols;
  __shared__ typename Stage::L l;

  const DeltaParams& p = a.p;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int32_t h = blockIdx.y, b = blockIdx.z, kh = h / p.group;
  const int32_t slot = p.slots ? p.slots[b] : b;
  if (p.slots && slot == p.pad) return;
  const int32_t start = p.qsl[b], end = p.qsl[b + 1];
  const int32_t cols0 = blockIdx.x * 16 * NW, c16 = 16 * wave, col = cols0 + c16 + r;
  const int64_t KV = (int64_t)p.K * p.V;

  f32x4 s[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) s[t] = zero4();
  const int32_t ends = cols0 + c16 + 16;
  if (a.dfinal) state_columns<false>(s, a.dfinal + slot * a.df_slot + h * KV, p.K, p.V, col, ends);
  const S* q = static_cast<const S*>(p.q) + kh * p.q_h;
  const S* k = static_cast<const S*>(p.k) + kh * p.k_h;
  const S* dout = static_cast<const S*>(a.dout) + h * a.do_h;
  const int32_t row0 = start / C + b;
  Stage next;
  auto fetch = [&](int32_t i) {
    const int64_t at = (int64_t)(row0 + i) * p.heads + h;
    next.fetch(p, k, q, dout, a.do_t, p.qk_vec && a.do_vec, cols0, start + i * C, end,
               p.frags + (at * (3 * NF) + NF) * kFragBytes, p.vectors + at * kDeltaVectors<C>);
  };
  const int32_t chunks = (end - start + C - 1) / C;
  if (chunks > 0) fetch(chunks - 1);
  for (int32_t i = chunks - 1; i >= 0; --i) {
    __syncthreads();
    next.stage(l, p, cols0, end - (start + i * C));
    __syncthreads();
    if (i > 0) fetch(i - 1);
    state_columns<true>(s, a.dstates + ((int64_t)(row0 + i) * p.heads + h) * KV, p.K, p.V, col, ends);
    f32x4 u[NT], none[NT];     // K dS, then dU, then dR
    typename T::Exact go[CS];  // dO
    typename T::Split tri[NF], us[CS];
    rows_times_state<D, Rows, KS, NT, false>(l.k, l.q, s, u, none, lane, [&] {
#pragma unroll
      for (int c = 0; c < CS; ++c) go[c] = Cols::cols(l.x, 32 * c, c16, lane);
      load_triangle<D>(tri, l.f + NF * kFragBytes, lane);
    });
#pragma unroll
    for (int t = 0; t < NT; ++t) u[t] *= lds4(l.v + C + 16 * t + 4 * g);
    triangle_times<D, false>(tri, go, u);
    keep_order();
    load_triangle<D>(tri, l.f, lane);
    keep_order();
#pragma unroll
    for (int c = 0; c < CS; ++c) us[c] = T::split(u[2 * c], u[2 * c + 1]);
    const float whole = l.v[C - 1];
#pragma unroll
    for (int t = 0; t < KT; ++t) s[t] *= whole;
    typename T::Fine fine[CS];
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
    triangle_times<D, false>(tri, us, u);
    keep_order();
    cols_times<D, Rows>(l.q, fine, s, lane);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      u[t] *= -(lds4(l.v + 16 * t + 4 * g) * lds4(l.v + 2 * C + 16 * t + 4 * g));
#pragma unroll
    for (int c = 0; c < CS; ++c) fine[c] = T::fine(u[2 * c], u[2 * c + 1]);
    cols_times<D, Rows>(l.k, fine, s, lane);
  }
  if (a.dinitial) {
    if (!(p.has && p.has[b])) {
#pragma unroll
      for (int t = 0; t < KT; ++t) s[t] = zero4();
    }
    state_columns<true>(s, a.dinitial + slot * a.di_slot + h * KV, p.K, p.V, col, ends);
  }
}

// v summed over the 16 lanes of a group; all of them get it.
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) v += __shfl_xor(v, d, 64);
  return v;
}

// LDS of a workgroup below: K, Q, dO, the parts of U and dR (later of three
// triangles), vectors, sums of the waves.
template <typename D, int KP>
constexpr int kGradParts = sizeof(typename D::storage) == 2 ? 2 : 1;
template <typename D, int KP> constexpr int kGradBig = kDeltaChunk<D> * LdsRows<D, KP>::LD;
template <typename D, int KP>
constexpr int kGradSmall = kDeltaChunk<D> * LdsRows<D, kDeltaChunk<D>>::LD;
template <typename D, int KP>
constexpr int kGradShared = kGradParts<D, KP> * (3 * kGradSmall<D, KP> > 2 * kGradBig<D, KP>
                                                     ? 3 * kGradSmall<D, KP> : 2 * kGradBig<D, KP>);
template <typename D, int KP>
constexpr int kGradLds = (3 * kGradBig<D, KP> + kGradShared<D, KP>) * (int)sizeof(typename D::storage) +
                         4 * (kDeltaVectors<kDeltaChunk<D>> + KP / 16 * (4 * kDeltaChunk<D> + 1));

// One workgroup: all gradients of a chunk's tokens for one key head, its value
// heads one after another (dq and dk add up in registers, in that order).
// Columns come in blocks of KP, 16 a wave; then a wave owns 16 of K.
template <typename D, int KP>
__global__ __launch_bounds__(4 * KP, KP == 128 ? 2 : 1) void delta_grad_kernel(DeltaBwd a) {
  using T = Tile<D>;
  using S = typename D::storage;
  constexpr bool kB = sizeof(S) == 2;
  constexpr int C = kDeltaChunk<D>, NT = C / 16, KS = KP / 32, CS = C / 32, NW = KP / 16;
  constexpr int NF = kDeltaFrags<C>, THREADS = 64 * NW, PARTS = kGradParts<D, KP>;
  constexpr int TILES = NT * (NT + 1) / 2, MINE = (TILES + NW - 1) / NW;
  using Rows = LdsRows<D, KP>;
  using Tri = LdsRows<D, C>;
  constexpr int BIG = kGradBig<D, KP>, SMALL = kGradSmall<D, KP>;
  __shared__ __attribute__((aligned(16))) char lds[kGradLds<D, KP>];
  S* lk = reinterpret_cast<S*>(lds);
  S* lq = lk + BIG;
  S* ldo = lq + BIG;
  S* lu = ldo + BIG;           // PARTS planes each
  S* lr = lu + PARTS * BIG;
  S* le = lu;                  // E_P, E_A, beta E_A over U and dR once those are read
  float* lv = reinterpret_cast<float*>(lu + kGradShared<D, KP>);  // the chunk's vectors
  float* part = lv + kDeltaVectors<C>;                     // [NW][4][C]
  float* dots = part + NW * 4 * C;                         // [NW]

  const DeltaParams& p = a.p;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int32_t row = blockIdx.x, kh = blockIdx.y;
  const DeltaChunk ch = delta_find<C>(p, row);
  if (ch.len == 0) return;
  const int64_t KV = (int64_t)p.K * p.V;

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
    if constexpr (kB)
      return typename T::Split{Rows::rows(m, t0, c0, lane).v, Rows::rows(m + BIG, t0, c0, lane).v};
    else
      return Rows::rows(m, t0, c0, lane);
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

  // columns w0 .. of the chunk's rows of two tensors
  auto stage2 = [&](S* l1, S* l2, const S* m1, int64_t ld1, const S* m2, int64_t ld2, int w0, int W,
                    bool vec) {
    constexpr int N = C * KP / 8 / THREADS;
    static_assert(C * KP / 8 % THREADS == 0);
    typename T::Exact x1[N], x2[N];
    auto load = [&](auto v) {
#pragma unroll
      for (int o = 0; o < N; ++o) {
        const int i = threadIdx.x + o * THREADS, t = i / (KP / 8), c0 = w0 + i % (KP / 8) * 8;
        x1[o] = load8<D, decltype(v)::value>(m1, ld1, t, ch.len, c0, W);
        x2[o] = load8<D, decltype(v)::value>(m2, ld2, t, ch.len, c0, W);
      }
    };
    if (vec) load(std::true_type()); else load(std::false_type());
#pragma unroll
    for (int o = 0; o < N; ++o) {
      const int i = threadIdx.x + o * THREADS, t = i / (KP / 8), c0 = i % (KP / 8) * 8;
      const int n = t < ch.len ? W - w0 - c0 : 0;
      Rows::put8(l1, t, c0, mask8<D>(x1[o], n));
      Rows::put8(l2, t, c0, mask8<D>(x2[o], n));
    }
  };
  // K and Q of the chunk
  {
    const S* q = static_cast<const S*>(p.q) + (int64_t)ch.t0 * p.q_t + kh * p.q_h;
    const S* k = static_cast<const S*>(p.k) + (int64_t)ch.t0 * p.k_t + kh * p.k_h;
    stage2(lk, lq, k, p.k_t, q, p.q_t, 0, p.K, p.qk_vec);
  }

  f32x4 dq[NT], dk[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) dq[t] = zero4(), dk[t] = zero4();
  const int kidx = 16 * wave + r;  // this lane's channel of K

  for (int32_t gh = 0; gh < p.group; ++gh) {
    const int32_t h = kh * p.group + gh;
    const int64_t at = (int64_t)row * p.heads + h;
    const char* frags = p.frags + at * (3 * NF) * kFragBytes;
    const float *s0 = a.marks + at * KV, *ds = a.dstates + at * KV;
    const S* v = static_cast<const S*>(p.v) + (int64_t)ch.t0 * p.v_t + h * p.v_h;
    const S* dout = static_cast<const S*>(a.dout) + (int64_t)ch.t0 * a.do_t + h * a.do_h;
    S* dv = static_cast<S*>(a.dv) + (int64_t)ch.t0 * a.dv_t + h * a.dv_h;

    f32x4 mq[NT], mz[NT], mw[NT];  // dO S0^T, dR S0^T, U dS1^T
    f32x4 ep[MINE], ea[MINE];      // tiles of dO U^T and dR U^T
    f32x4 rv[NT];                  // rowsum(dR V), this lane's columns
    float dot = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) mq[t] = mz[t] = mw[t] = rv[t] = zero4();
#pragma unroll
    for (int m = 0; m < MINE; ++m) ep[m] = ea[m] = zero4();

    for (int32_t v0 = 0; v0 < p.V; v0 += KP) {
      __syncthreads();  // the last reads of dO, U, dR and the triangles
      // V lies in U's place until U replaces it
      stage2(ldo, lu, dout, a.do_t, v, p.v_t, v0, p.V, a.do_vec && p.v_vec);
      if (v0 == 0)
        for (int x = threadIdx.x; x < kDeltaVectors<C>; x += THREADS)
          lv[x] = p.vectors[at * kDeltaVectors<C> + x];
      __syncthreads();
      const int c16 = 16 * wave, col = v0 + c16 + r;
      f32x4 u[NT], y[NT];
      {
        f32x4 x[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] = y[t] = zero4();
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          f32x4 w[2], z[2];
#pragma unroll
          for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = 32 * c + 16 * o + 4 * g + e;
              const bool in = k < p.K && col < p.V;
              w[o][e] = in ? s0[(int64_t)k * p.V + col] : 0.f;
              z[o][e] = in ? ds[(int64_t)k * p.V + col] : 0.f;
            }
          const auto sw = T::split(w[0], w[1]), sz = T::split(z[0], z[1]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const auto kf = Rows::rows(lk, 16 * t, 32 * c, lane);
            x[t] = T::mul(kf, sw, x[t]);
            y[t] = T::mul(kf, sz, y[t]);
          }
        }
        f32x4 vv[NT];
#pragma unroll
        for (int c = 0; c < CS; ++c) {
          const auto w = Rows::cols(lu, 32 * c, c16, lane);
#pragma unroll
          for (int e = 0; e < 8; ++e) vv[2 * c + e / 4][e % 4] = T::value(w, e);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
          u[t] = lds4(lv + 2 * C + 16 * t + 4 * g) * (vv[t] - lds4(lv + 16 * t + 4 * g) * x[t]);
        typename T::Split us[CS];
#pragma unroll
        for (int c = 0; c < CS; ++c) us[c] = T::split(u[2 * c], u[2 * c + 1]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c <= t / 2; ++c)
            u[t] = T::mul(T::get(frags + lower_frag<C>(t, c) * kFragBytes, lane), us[c], u[t]);
        // dU
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          y[t] *= lds4(lv + C + 16 * t + 4 * g);
#pragma unroll
          for (int c = t / 2; c < CS; ++c)
            y[t] = T::mul(T::get(frags + (2 * NF + upper_frag<C>(t, c)) * kFragBytes, lane),
                          Rows::cols(ldo, 32 * c, c16, lane), y[t]);
        }
#pragma unroll
        for (int c = 0; c < CS; ++c) us[c] = T::split(y[2 * c], y[2 * c + 1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int c = t / 2; c < CS; ++c)
            y[t] = T::mul(T::get(frags + (NF + upper_frag<C>(t, c)) * kFragBytes, lane), us[c], y[t]);
          rv[t] += y[t] * vv[t];
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const f32x4 bt = lds4(lv + 2 * C + 16 * t + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 16 * t + 4 * g + e;
          put_split(lu, BIG, x * Rows::LD + Rows::pos(c16 + r), u[t][e]);
          put_split(lr, BIG, x * Rows::LD + Rows::pos(c16 + r), y[t][e]);
          if (x < ch.len && col < p.V) dv[(int64_t)x * a.dv_t + col] = delta_round<D>(bt[e] * y[t][e]);
        }
      }
      __syncthreads();
      // products over this block's columns
      const int steps = (min(KP, p.V - v0) + 31) / 32;
      for (int c = 0; c < steps; ++c) {
        f32x4 w[2], z[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int vc = v0 + 32 * c + 16 * o + 4 * g;
          w[o] = z[o] = zero4();
          if (kidx < p.K) {
            const int64_t i = (int64_t)kidx * p.V + vc;
            if (p.V % 4 == 0) {
              if (vc < p.V) w[o] = lds4(s0 + i), z[o] = lds4(ds + i);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (vc + e < p.V) w[o][e] = s0[i + e], z[o][e] = ds[i + e];
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = fmaf(w[o][e], z[o][e], dot);
        }
        const auto sw = T::split(w[0], w[1]), sz = T::split(z[0], z[1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mq[t] = T::mul(Rows::rows(ldo, 16 * t, 32 * c, lane), sw, mq[t]);
          mz[t] = T::mul(rows2(lr, 16 * t, 32 * c), sw, mz[t]);
          mw[t] = T::mul(rows2(lu, 16 * t, 32 * c), sz, mw[t]);
        }
      }
      int I = 0, J = 0, n = 0;
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        const int want = wave + m * NW;
        if (want >= TILES) break;
        for (; n < want; ++n) J == I ? (++I, J = 0) : ++J;
        for (int c = 0; c < steps; ++c) {
          const auto uf = rows2(lu, 16 * J, 32 * c);
          ep[m] = T::mul(Rows::rows(ldo, 16 * I, 32 * c, lane), uf, ep[m]);
          ea[m] = T::mul(rows2(lr, 16 * I, 32 * c), uf, ea[m]);
        }
      }
    }
    __syncthreads();
    // the triangles, with zeros above the diagonal of every 32 columns
    {
      int I = 0, J = 0, n = 0;
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        const int want = wave + m * NW;
        if (want >= TILES) break;
        for (; n < want; ++n) J == I ? (++I, J = 0) : ++J;
        const int j = 16 * J + r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * I + 4 * g + e, x = i * Tri::LD + Tri::pos(j);
          float dec = 0.f;
          if (i >= j) dec = expf((lv[3 * C + i] - lv[3 * C + j]) + (lv[4 * C + i] - lv[4 * C + j]));
          const float pv = i >= j ? p.scale * dec * ep[m][e] : 0.f;
          const float av = i > j ? dec * ea[m][e] : 0.f;
          put_split(le, SMALL, x, pv);
          put_split(le + PARTS * SMALL, SMALL, x, av);
          put_split(le + 2 * PARTS * SMALL, SMALL, x, lv[2 * C + i] * av);
        }
        if (I == J && I % 2 == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = (16 * I + 4 * g + e) * Tri::LD + Tri::pos(j + 16);
#pragma unroll
            for (int o = 0; o < 3; ++o) put_split(le + o * PARTS * SMALL, SMALL, x, 0.f);
          }
        }
      }
    }
    __syncthreads();
    f32x4 w[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 gam = lds4(lv + 16 * t + 4 * g);
      mq[t] *= p.scale * gam;
      mz[t] *= gam;
      mw[t] *= lds4(lv + C + 16 * t + 4 * g);
      w[t] = zero4();
    }
#pragma unroll
    for (int c = 0; c < CS; ++c) {
      const auto kf = Rows::cols(lk, 32 * c, 16 * wave, lane), qf = Rows::cols(lq, 32 * c, 16 * wave, lane);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (c <= t / 2) {
          mq[t] = T::mul(tri_rows(le, 16 * t, 32 * c), kf, mq[t]);
          mz[t] = T::mul(tri_rows(le + PARTS * SMALL, 16 * t, 32 * c), kf, mz[t]);
        }
        if (c >= t / 2) {
          f32x4 neg = T::mul(tri_cols(le + 2 * PARTS * SMALL, 32 * c, 16 * t), kf, zero4());
          w[t] = T::mul(tri_cols(le, 32 * c, 16 * t), qf, w[t] - neg);
        }
      }
    }
    // rows' sums over this wave's channels, and the sums over value heads
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 bt = lds4(lv + 2 * C + 16 * t + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = 16 * t + 4 * g + e, i = x * Rows::LD + Rows::pos(kidx);
        const float kv = to_float<D>(lk[i]), qv = to_float<D>(lq[i]);
        const float kz = kv * mz[t][e];
        const float own = sum16(qv * mq[t][e] - bt[e] * kz - kv * w[t][e]);
        const float km = sum16(kv * mw[t][e]), sz = sum16(kz), sv = sum16(rv[t][e]);
        if (r == 0) {
          float* to = part + wave * 4 * C + x;
          to[0] = own, to[C] = km, to[2 * C] = sz, to[3 * C] = sv;
        }
        dq[t][e] += mq[t][e];
        dk[t][e] += mw[t][e] + w[t][e] - bt[e] * mz[t][e];
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d, 64);
    if (lane == 0) dots[wave] = dot;
    __syncthreads();
    if (wave == 0) {
      const int t = lane;
      float own = 0.f, km = 0.f, sz = 0.f, sv = 0.f, all = 0.f;
      for (int n = 0; n < NW; ++n) {
        const float* from = part + n * 4 * C + (t < C ? t : 0);
        own += from[0], km += from[C], sz += from[2 * C], sv += from[3 * C];
        all += dots[n];
      }
      if (t >= C) own = km = 0.f;
      double before = km, after = own;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const double x = __shfl_up(before, d, 64), y2 = __shfl_down(after, d, 64);
        if (lane >= d) before += x;
        if (lane + d < 64) after += y2;
      }
      if (t < ch.len) {
        float dg = (float)(after + (before - km) + (double)lv[C - 1] * all);
        const float db = sv - sz;
        // behind a closed gate the parts cancel but for their roundings
        const float gt = lv[3 * C + t] + lv[4 * C + t] - (t ? lv[3 * C + t - 1] + lv[4 * C + t - 1] : 0.f);
        if (gt < -104.f) dg = 0.f;  // e^g is zero in fp32
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
  S* oq = static_cast<S*>(a.dq) + (int64_t)ch.t0 * a.dq_t + kh * a.dq_h + kidx;
  S* ok = static_cast<S*>(a.dk) + (int64_t)ch.t0 * a.dk_t + kh * a.dk_h + kidx;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = 16 * t + 4 * g + e;
      if (x < ch.len && kidx < p.K) {
        oq[(int64_t)x * a.dq_t] = delta_round<D>(dq[t][e]);
        ok[(int64_t)x * a.dk_t] = delta_round<D>(dk[t][e]);
      }
    }
}

template <typename D, int KP>
static int delta_backward(const DeltaBwd& a, int64_t rows, hipStream_t stream) {
  const char* what = "gated_delta_rule_varlen_bwd";
  const DeltaParams& p = a.p;
  hipLaunchKernelGGL((delta_prep_kernel<D, KP, true>), dim3((uint32_t)rows, p.heads), dim3(64), 0,
                     stream, p);
  if (int rc = check_launch(what)) return rc;
  if (delta_wide(p))
    hipLaunchKernelGGL((delta_back_kernel<D, KP, 8>), dim3((p.V + 127) / 128, p.heads, p.batch),
                       dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((delta_back_kernel<D, KP, 4>), dim3((p.V + 63) / 64, p.heads, p.batch),
                       dim3(256), 0, stream, a);
  if (int rc = check_launch(what)) return rc;
  hipLaunchKernelGGL((delta_grad_kernel<D, KP>), dim3((uint32_t)rows, p.heads / p.group),
                     dim3(4 * KP), 0, stream, a);
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
  if (!query_start_loc) return fail(SCONV_ERR_INVALID, "%s: NULL query_start_loc", what);
  if (int rc = delta_inputs(c, a.p, q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v,
                            v_stride_t, v_stride_h, g, g_stride_t, g_stride_h, beta, b_stride_t,
                            b_stride_h, scale))
    return rc;
  if ((total_T > 0 && !dout) || !checkpoints) return fail(SCONV_ERR_INVALID, "%s: NULL input", what);
  if (do_stride_t < 0 || do_stride_h < 0) return fail(SCONV_ERR_INVALID, "%s: negative stride", what);
  delta_packing(c, a.p, query_start_loc, cache_indices, has_initial_state, pad_slot_id);
  const int64_t rows = delta_rows(total_T, batch, delta_chunk(dtype));
  const int64_t KV = (int64_t)K * V;
  if (checkpoint_rows < rows)
    return fail(SCONV_ERR_INVALID, "%s: %lld checkpoint rows, needs %lld", what,
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
  const DeltaBuffer marks = delta_block(checkpoints, rows * value_heads * KV * 4);
  const DeltaBuffer work = delta_block(workspace, s.bwd * 4);
  const DeltaBuffer od = delta_tensor(dout, do_stride_t, do_stride_h, total_T, value_heads, V,
                                      elem_size(dtype));
  for (const DeltaBuffer& o : {oq, ok, ov, og, ob, di, work})
    if (delta_overlap(o, marks) || delta_overlap(o, od) || (!same && delta_overlap(o, df) && o.p != di.p))
      return fail(SCONV_ERR_INVALID, "%s: an output overlaps an input", what);
  if (int rc = delta_disjoint(c, a.p, {oq, ok, ov, og, ob, di, work})) return rc;
  a.p.vectors = workspace;
  a.p.frags = reinterpret_cast<char*>(workspace + s.vectors);
  a.dstates = workspace + s.bwd_states;
  a.dout = dout, a.do_t = do_stride_t, a.do_h = do_stride_h;
  a.marks = checkpoints, a.dfinal = dfinal_states, a.df_slot = df_stride_slot;
  a.dinitial = dinitial_states, a.di_slot = di_stride_slot;
  a.dq = dq, a.dq_t = dq_stride_t, a.dq_h = dq_stride_h;
  a.dk = dk, a.dk_t = dk_stride_t, a.dk_h = dk_stride_h;
  a.dv = dv, a.dv_t = dv_stride_t, a.dv_h = dv_stride_h;
  a.dg = dg, a.dg_t = dg_stride_t, a.dg_h = dg_stride_h;
  a.db = dbeta, a.db_t = db_stride_t, a.db_h = db_stride_h;
  a.do_vec = delta_vec(dout, do_stride_t, do_stride_h, V, 16 / elem_size(dtype));
  if (dtype == SCONV_BF16)
    return K <= 64 ? delta_backward<Bf16, 64>(a, rows, stream) : delta_backward<Bf16, 128>(a, rows, stream);
  return K <= 64 ? delta_backward<F32, 64>(a, rows, stream) : delta_backward<F32, 128>(a, rows, stream);
}
