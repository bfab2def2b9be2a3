// delta_prep.h -- the kernel that prepares the chunks of a gated delta rule
// call: what a chunk needs that does not depend on the state, for all chunks
// at once, laid out as the operands that the walking kernels read.
//
// One wave a chunk and value head.  k.k and k.q run on the matrix cores from
// registers.  T = (I + A)^-1 is built in LDS: lanes solve the 16 x 16
// diagonal blocks column by column, then pairs of blocks meet by
//   [T0, 0; T1 (-A10) T0, T1]
// in fp32 matrix products.  Log decays are summed in 64 bits and kept as two
// floats: e_ij is the exponential of a difference of sums.
#pragma once

#include <type_traits>

#include "delta_rule.h"
#include "norm_rows.h"

namespace sconv {

// 16 x 16 x 16 fp32 product of X (rows in LDS) and an operand in registers
// whose entry e of lane group g is row 4 g + e.
__device__ __forceinline__ f32x4 mul16(const f32x4& x, const f32x4& y, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
  return c;
}

struct Larger {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// A lower triangle of 16 x 16 tiles in LDS, tile after tile; a row of 20 floats
// lets 16 rows be read 16 bytes each without bank conflicts.
constexpr int kTileLd = 20, kTileFloats = 16 * kTileLd;
__host__ __device__ constexpr int tile_at(int I, int J) { return (I * (I + 1) / 2 + J) * kTileFloats; }

// T = (I + A)^-1 in place: m holds A strictly below the diagonal (anything above).
template <int C>
__device__ __forceinline__ void unit_lower_inverse(float* m, int lane) {
  const int r = lane & 15, g = lane >> 4;
  if (lane < C) {
    float* d = m + (g * (g + 3) / 2) * kTileFloats;  // tile (g, g)
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == r ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const f32x4 a = lds4(d + i * kTileLd + j);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < i) s = fmaf(-a[e], x[j + e], s);
      }
      x[i] = s;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i * kTileLd + r] = x[i];
  }
  __syncthreads();
  auto rows = [&](int I, int J) { return lds4(m + tile_at(I, J) + r * kTileLd + 4 * g); };
  auto cols = [&](int I, int J) {
    const float* at = m + tile_at(I, J) + 4 * g * kTileLd + r;
    return (f32x4){at[0], at[kTileLd], at[2 * kTileLd], at[3 * kTileLd]};
  };
  auto store = [&](int I, int J, const f32x4& t) {
    float* at = m + tile_at(I, J) + 4 * g * kTileLd + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e * kTileLd] = -t[e];
  };
  f32x4 pair[C / 32];
#pragma unroll
  for (int P = 0; P < C / 32; ++P) pair[P] = mul16(rows(2 * P + 1, 2 * P), cols(2 * P, 2 * P), zero4());
#pragma unroll
  for (int P = 0; P < C / 32; ++P) pair[P] = mul16(rows(2 * P + 1, 2 * P + 1), pair[P], zero4());
  __syncthreads();
#pragma unroll
  for (int P = 0; P < C / 32; ++P) store(2 * P + 1, 2 * P, pair[P]);
  __syncthreads();
  if constexpr (C == 64) {
    f32x4 w[2][2], t[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      w[a][1] = mul16(rows(2 + a, 1), cols(1, 1), zero4());
      w[a][0] = mul16(rows(2 + a, 0), cols(0, 0), zero4());
      w[a][0] = mul16(rows(2 + a, 1), cols(1, 0), w[a][0]);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      t[0][b] = mul16(rows(2, 2), w[0][b], zero4());
      t[1][b] = mul16(rows(3, 2), w[0][b], zero4());
      t[1][b] = mul16(rows(3, 3), w[1][b], t[1][b]);
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) store(2 + a, b, t[a][b]);
    __syncthreads();
  }
}

// FWD: frags N (lower), P (lower).  Gradients: N (lower), N^T (upper), P^T (upper).
template <int C, bool GRAD> constexpr int kPrepFrags = (GRAD ? 3 : 2) * kDeltaFrags<C>;

// One wave a chunk and value head.  Bound by latency: three waves a SIMD are
// what the LDS of a triangle leaves room for (8 x 4096 tokens, 32 heads of 128
// channels bf16: 172 us, 0.8 GB; with whole squares in LDS, which leave room
// for two, 198 against 162 at the time).  The value heads of a key head
// read the same rows, so they come 8 workgroups apart: on one XCD, soon after.
// Rows that are not aligned come entry by entry and take registers for two waves; of
// more than 64 channels they spill 17, with gradients 58 (4 x 2048 tokens, 8 heads of
// 100: 48 and 57 us).
template <typename D, int KP, bool GRAD, bool VEC>
__global__ __launch_bounds__(64, VEC ? 3 : 2) void delta_prep_kernel(DeltaParams p) {
  using T = Tile<D>;
  using S = typename D::storage;
  constexpr int C = kDeltaChunk<D>, NT = C / 16, KS = KP / 32, NF = kDeltaFrags<C>;
  __shared__ __attribute__((aligned(16))) float m[NT * (NT + 1) / 2 * kTileFloats];
  __shared__ __attribute__((aligned(16))) float gh[C], gl[C], bt[C];
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const int32_t x = blockIdx.x >> 3, row = x / p.group * 8 + (blockIdx.x & 7);
  const int32_t h = blockIdx.y * p.group + x % p.group;
  const DeltaChunk c = delta_find<C>(p, row);
  if (c.len == 0) return;

  const int32_t kh = h / p.group;
  const S* q = static_cast<const S*>(p.q) + (int64_t)c.t0 * p.q_t + kh * p.q_h;
  const S* k = static_cast<const S*>(p.k) + (int64_t)c.t0 * p.k_t + kh * p.k_h;
  typename T::Exact kf[NT][KS], qf[2][KS];
  auto load = [&](const S* m, int64_t ld, int I, typename T::Exact (&to)[KS]) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
      to[s] = load8<D, VEC>(m, ld, 16 * I + r, c.len, 32 * s + 8 * g, p.K);
  };
  auto mask = [&](int I, typename T::Exact (&x)[KS]) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
      x[s] = mask8<D>(x[s], 16 * I + r < c.len ? p.K - (32 * s + 8 * g) : 0);
  };
#pragma unroll
  for (int I = 0; I < NT; ++I) load(k, p.k_t, I, kf[I]);
  load(q, p.q_t, 0, qf[0]);

  const int64_t at = (int64_t)row * p.heads + h;
  char* frags = p.frags + at * kPrepFrags<C, GRAD> * kFragBytes;
  float* vec = p.vectors + at * kDeltaVectors<C>;
  {
    const int64_t t = c.t0 + min(lane, c.len - 1);
    const bool live = lane < c.len;
    const float gv = delta_bound(delta_gate(p, p.g, t * p.g_t + h * p.g_h));
    const float bv = delta_gate(p, p.beta, t * p.b_t + h * p.b_h);
    double sum = live ? (double)gv : 0.0;
    const float b = live ? bv : 0.f;
#pragma unroll
    for (int d = 1; d < C; d *= 2) {
      const double o = __shfl_up(sum, d, 64);
      if (lane >= d) sum += o;
    }
    const double whole = __shfl(sum, C - 1, 64);
    if (lane < C) {
      gh[lane] = (float)sum;
      gl[lane] = (float)(sum - (double)(float)sum);
      bt[lane] = b;
      vec[lane] = expf((float)sum);
      vec[C + lane] = expf((float)(whole - sum));
      vec[2 * C + lane] = b;
      if constexpr (GRAD) {
        vec[kDeltaSums<C> + lane] = gh[lane];
        vec[kDeltaSums<C> + C + lane] = gl[lane];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int I = 0; I < NT; ++I) mask(I, kf[I]);
  // A factor for entries of which a lane has none above `most`; its inverse goes to
  // the vectors.
  auto factor = [&](float most, int at) {
    if constexpr (!T::kScaled) return 1.f;
    const Pow2 by(groups_max(lanes_reduce<16>(most, Larger())));
    if (lane == 0) vec[kDeltaFactors<C> + at] = by.down;
    return by.up;
  };
  // Tiles of A and P, e_ij once for both.  An accumulator is then a piece of a
  // frag as it lies: rows j and columns i for P's, rows i and columns j for P^T's.
  constexpr float kLog2e = 1.44269504088896340736f;
  f32x4 pt[NT][NT];
#pragma unroll
  for (int I = 0; I < NT; ++I) {
    if (I + 1 < NT) load(q, p.q_t, I + 1, qf[(I + 1) & 1]);
    mask(I, qf[I & 1]);
#pragma unroll
    for (int J = 0; J <= I; ++J) {
      f32x4 a = zero4(), w = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        a = GRAD ? T::mul(kf[I][s], kf[J][s], a) : T::mul(kf[J][s], kf[I][s], a);
        w = GRAD ? T::mul(qf[I & 1][s], kf[J][s], w) : T::mul(kf[J][s], qf[I & 1][s], w);
      }
      const int lane_t = 16 * (GRAD ? J : I) + r, four = 16 * (GRAD ? I : J) + 4 * g;
      const float h1 = gh[lane_t], l1 = gl[lane_t], b1 = bt[lane_t];
      const f32x4 h4 = lds4(gh + four), l4 = lds4(gl + four), b4 = lds4(bt + four);
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = GRAD ? four + e : lane_t, j = GRAD ? lane_t : four + e;
        const float d = GRAD ? (h4[e] - h1) + (l4[e] - l1) : (h1 - h4[e]) + (l1 - l4[e]);
        const float dec = __builtin_amdgcn_exp2f(i >= j ? d * kLog2e : 0.f);
        x[e] = (GRAD ? b4[e] : b1) * dec * a[e];
        pt[I][J][e] = i >= j ? p.scale * dec * w[e] : 0.f;
      }
      if constexpr (GRAD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) m[tile_at(I, J) + (4 * g + e) * kTileLd + r] = x[e];
      } else {
        *reinterpret_cast<f32x4*>(m + tile_at(I, J) + r * kTileLd + 4 * g) = x;
      }
    }
    if constexpr (!GRAD) {
      float most = 0.f;
#pragma unroll
      for (int J = 0; J <= I; ++J) most = max4(pt[I][J], most);
      const float up = factor(most, 4 + I);
#pragma unroll
      for (int s = 0; s <= I / 2; ++s)
        T::put(frags + (NF + lower_frag<C>(I, s)) * kFragBytes, lane,
               T::pair(pt[I][2 * s], 2 * s + 1 <= I ? pt[I][2 * s + 1] : zero4(), up));
    } else if (I % 2 == 1) {  // P^T's columns of this step are complete, its rows are not
      float most = 0.f;
#pragma unroll
      for (int J = 0; J <= I; ++J) {
        most = max4(pt[I][J], most);
        if (J < I) most = max4(pt[I - 1][J], most);
      }
      const float up = factor(most, 4 + I / 2);
#pragma unroll
      for (int J = 0; J <= I; ++J)
        T::put(frags + (2 * NF + upper_frag<C>(J, I / 2)) * kFragBytes, lane,
               T::pair(J <= I - 1 ? pt[I - 1][J] : zero4(), pt[I][J], up));
    }
  }
  __syncthreads();
  unit_lower_inverse<C>(m, lane);
  // N = T - I; what lies above the diagonal of a frag's 32 columns is zero
#pragma unroll
  for (int R = 0; R < NT; ++R) {
    f32x4 x[C / 32][2];
    float most = 0.f;
#pragma unroll
    for (int s = 0; s <= R / 2; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int J = 2 * s + u;
        x[s][u] = J <= R ? lds4(m + tile_at(R, J <= R ? J : 0) + r * kTileLd + 4 * g) : zero4();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (J == R) x[s][u][e] = 4 * g + e < r ? x[s][u][e] : 0.f;
        most = max4(x[s][u], most);
      }
    const float up = factor(most, (GRAD ? kFactorsN : 0) + R);
#pragma unroll
    for (int s = 0; s <= R / 2; ++s)
      T::put(frags + lower_frag<C>(R, s) * kFragBytes, lane, T::pair(x[s][0], x[s][1], up));
  }
  if constexpr (GRAD) {
#pragma unroll
    for (int R = 0; R < NT; ++R) {
      f32x4 x[C / 32][2];
      float most = 0.f;
#pragma unroll
      for (int s = R / 2; s < C / 32; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int I = 2 * s + u;
          const float* at = m + tile_at(I >= R ? I : R, R) + 4 * g * kTileLd + r;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[s][u][e] = I >= R ? at[e * kTileLd] : 0.f;
            if (I == R) x[s][u][e] = r < 4 * g + e ? x[s][u][e] : 0.f;
          }
          most = max4(x[s][u], most);
        }
      const float up = factor(most, R);
#pragma unroll
      for (int s = R / 2; s < C / 32; ++s)
        T::put(frags + (NF + upper_frag<C>(R, s)) * kFragBytes, lane, T::pair(x[s][0], x[s][1], up));
    }
  }
}

template <typename D, int KP, bool GRAD>
static int delta_prepare(const char* what, const DeltaParams& p, int64_t rows, hipStream_t stream) {
  const dim3 grid((uint32_t)(cdiv(rows, 8) * 8 * p.group), p.heads / p.group), wave(64);
  if (p.qk_vec) hipLaunchKernelGGL((delta_prep_kernel<D, KP, GRAD, true>), grid, wave, 0, stream, p);
  else hipLaunchKernelGGL((delta_prep_kernel<D, KP, GRAD, false>), grid, wave, 0, stream, p);
  return check_launch(what);
}

}  // namespace sconv
