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

namespace sconv {

// 16 x 16 x 16 fp32 product of X (rows in LDS) and an operand in registers
// whose entry e of lane group g is row 4 g + e.
__device__ __forceinline__ f32x4 mul16(const f32x4& x, const f32x4& y, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
  return c;
}

// T = (I + A)^-1 in place: m [C][LD] holds A strictly below the diagonal.
template <int C, int LD>
__device__ __forceinline__ void unit_lower_inverse(float* m, int lane) {
  const int r = lane & 15, g = lane >> 4;
  if (lane < C) {
    float* d = m + (16 * g) * LD + 16 * g;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == r ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const f32x4 a = lds4(d + i * LD + j);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < i) s = fmaf(-a[e], x[j + e], s);
      }
      x[i] = s;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i * LD + r] = x[i];
  }
  __syncthreads();
  auto rows = [&](int I, int J) { return lds4(m + (16 * I + r) * LD + 16 * J + 4 * g); };
  auto cols = [&](int I, int J) {
    const float* at = m + (16 * I + 4 * g) * LD + 16 * J + r;
    return (f32x4){at[0], at[LD], at[2 * LD], at[3 * LD]};
  };
  auto store = [&](int I, int J, const f32x4& t) {
    float* at = m + (16 * I + 4 * g) * LD + 16 * J + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e * LD] = -t[e];
  };
  f32x4 pair[C / 32];
#pragma unroll
  for (int P = 0; P < C / 32; ++P) {
    const f32x4 w = mul16(rows(2 * P + 1, 2 * P), cols(2 * P, 2 * P), zero4());
    pair[P] = mul16(rows(2 * P + 1, 2 * P + 1), w, zero4());
  }
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

template <typename D, int KP, bool GRAD>
__global__ __launch_bounds__(64) void delta_prep_kernel(DeltaParams p) {
  using T = Tile<D>;
  using S = typename D::storage;
  constexpr int C = kDeltaChunk<D>, NT = C / 16, KS = KP / 32, LD = C + 4, NF = kDeltaFrags<C>;
  __shared__ float m[C * LD];
  __shared__ float gh[C], gl[C], bt[C];
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const int32_t row = blockIdx.x, h = blockIdx.y;
  const DeltaChunk c = delta_find<C>(p, row);
  if (c.len == 0) return;

  const int64_t at = (int64_t)row * p.heads + h;
  char* frags = p.frags + at * kPrepFrags<C, GRAD> * kFragBytes;
  float* vec = p.vectors + at * kDeltaVectors<C>;
  {
    const int64_t t = c.t0 + lane;
    const bool live = lane < c.len;
    double sum = live ? (double)delta_bound(delta_gate(p, p.g, t * p.g_t + h * p.g_h)) : 0.0;
    const float b = live ? delta_gate(p, p.beta, t * p.b_t + h * p.b_h) : 0.f;
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
      vec[3 * C + lane] = gh[lane];
      vec[4 * C + lane] = gl[lane];
    }
  }
  __syncthreads();
  auto decay = [&](int i, int j) { return expf((gh[i] - gh[j]) + (gl[i] - gl[j])); };

  const int32_t kh = h / p.group;
  const S* q = static_cast<const S*>(p.q) + (int64_t)c.t0 * p.q_t + kh * p.q_h;
  const S* k = static_cast<const S*>(p.k) + (int64_t)c.t0 * p.k_t + kh * p.k_h;
  typename T::Exact kf[NT][KS], qf[NT][KS];
  auto load = [&](auto v) {
#pragma unroll
    for (int I = 0; I < NT; ++I)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        kf[I][s] = load8<D, decltype(v)::value>(k, p.k_t, 16 * I + r, c.len, 32 * s + 8 * g, p.K);
        qf[I][s] = load8<D, decltype(v)::value>(q, p.q_t, 16 * I + r, c.len, 32 * s + 8 * g, p.K);
      }
  };
  if (p.qk_vec) load(std::true_type()); else load(std::false_type());
#pragma unroll
  for (int I = 0; I < NT; ++I)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int n = 16 * I + r < c.len ? p.K - (32 * s + 8 * g) : 0;
      kf[I][s] = mask8<D>(kf[I][s], n);
      qf[I][s] = mask8<D>(qf[I][s], n);
    }
  // A into LDS
#pragma unroll
  for (int I = 0; I < NT; ++I)
#pragma unroll
    for (int J = 0; J < NT; ++J) {
      f32x4 a = zero4();
      if (J <= I) {
#pragma unroll
        for (int s = 0; s < KS; ++s) a = T::mul(kf[I][s], kf[J][s], a);
      }
      const int j = 16 * J + r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * I + 4 * g + e;
        m[i * LD + j] = i > j ? bt[i] * decay(i, j) * a[e] : 0.f;
      }
    }
  // P or P^T from registers
  f32x4 pt[NT][NT];
#pragma unroll
  for (int I = 0; I < NT; ++I)
#pragma unroll
    for (int J = 0; J < NT; ++J) {
      pt[I][J] = zero4();
      if (J > I) continue;
      f32x4 a = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s)
        a = GRAD ? T::mul(qf[I][s], kf[J][s], a) : T::mul(kf[J][s], qf[I][s], a);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * I + (GRAD ? 4 * g + e : r), j = 16 * J + (GRAD ? r : 4 * g + e);
        pt[I][J][e] = i >= j ? p.scale * decay(i, j) * a[e] : 0.f;
      }
    }
#pragma unroll
  for (int R = 0; R < NT; ++R)
#pragma unroll
    for (int s = 0; s < C / 32; ++s) {
      if constexpr (GRAD) {
        if (s >= R / 2)
          T::put(frags + (2 * NF + upper_frag<C>(R, s)) * kFragBytes, lane,
                 T::split(pt[2 * s][R], pt[2 * s + 1][R]));
      } else {
        if (s <= R / 2)
          T::put(frags + (NF + lower_frag<C>(R, s)) * kFragBytes, lane,
                 T::split(pt[R][2 * s], pt[R][2 * s + 1]));
      }
    }
  __syncthreads();
  unit_lower_inverse<C, LD>(m, lane);
  // N = T - I; what lies above the diagonal of a frag's 32 columns is zero
#pragma unroll
  for (int R = 0; R < NT; ++R)
#pragma unroll
    for (int s = 0; s <= R / 2; ++s) {
      f32x4 x[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * R + r, j = 32 * s + 16 * u + 4 * g + e;
          x[u][e] = j < i ? m[i * LD + j] : 0.f;
        }
      T::put(frags + lower_frag<C>(R, s) * kFragBytes, lane, T::split(x[0], x[1]));
    }
  if constexpr (GRAD) {
#pragma unroll
    for (int R = 0; R < NT; ++R)
#pragma unroll
      for (int s = R / 2; s < C / 32; ++s) {
        f32x4 x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 16 * R + r, i = 32 * s + 16 * u + 4 * g + e;
            x[u][e] = j < i ? m[i * LD + j] : 0.f;
          }
        T::put(frags + (NF + upper_frag<C>(R, s)) * kFragBytes, lane, T::split(x[0], x[1]));
      }
  }
}

}  // namespace sconv
