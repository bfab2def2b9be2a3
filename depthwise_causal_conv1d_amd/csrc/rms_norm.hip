// rms_norm.hip -- root-mean-square norm of rows with the residual's
// addition, with an output in the rows' type or in 8 bits with scales, and
// its gradients, for gfx950.
//
//   s = x + residual, out = s * rsqrt(mean(s^2) + eps) * weight
//   8 bits: scale = max |out| over a group / 448, code = e4m3(out / scale)
#include "column_sum.h"
#include "lane_tokens.h"
#include "plane_host.h"

#include <initializer_list>
#include <type_traits>

namespace sconv {

constexpr int kNormThreads = 256;
constexpr float kFp8Max = 448.f;               // largest e4m3 value
constexpr float kFp8MinScale = 1.17549435e-38f;  // keeps a row of zeros finite

struct NormParams {
  const void *x, *res, *w;
  void *sum, *out;
  float* scales;
  int64_t x_rs, r_rs, s_rs, o_rs, sc_rs, rows;
  int32_t dim, group;  // group: channels that share a scale
  float eps;
};

// v combined over groups of N consecutive lanes (a power of two); every lane
// gets the result.  Up to 16 lanes by DPP moves inside a row.
template <int N, typename T, typename F>
__device__ __forceinline__ T lanes_reduce(T v, F&& f) {
  auto step = [&](auto ctrl) {
    constexpr int C = decltype(ctrl)::value;
    const int m = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), C, 0xF, 0xF, true);
    v = f(v, __builtin_bit_cast(T, m));
  };
  if constexpr (N >= 2) step(std::integral_constant<int, 0xB1>());   // lanes 1 0 3 2
  if constexpr (N >= 4) step(std::integral_constant<int, 0x4E>());   // lanes 2 3 0 1
  if constexpr (N >= 8) step(std::integral_constant<int, 0x141>());  // half rows mirrored
  if constexpr (N >= 16) step(std::integral_constant<int, 0x140>()); // rows mirrored
  if constexpr (N >= 32) v = f(v, __shfl_xor(v, 16, 64));
  if constexpr (N >= 64) v = f(v, __shfl_xor(v, 32, 64));
  return v;
}

struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// Sum over the workgroup; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = lanes_reduce<64>(v, Add());
  const int wave = threadIdx.x >> 6, n = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) lds[wave] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < n; ++i) t += lds[i];
  __syncthreads();
  return t;
}

// |v| as bits: the order of the bits is that of the values, and a NaN is
// above every number, so that a NaN reaches the scale.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) * (1.0f / kFp8Max);
  return s < kFp8MinScale ? kFp8MinScale : s;
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xFF);
}

// V codes of v / scale, one store.  The quotient is the nearest fp32 one: the
// product with 1 / scale alone falls on the other side of a border between
// two codes now and then.  The product's remainder mends it (exact, since
// it is a multiple of the last place of v) where no place is lost below fp32's
// range; there, and at an infinite or NaN scale, the division itself
// (everywhere: 103 against 101 us for 17408 x 4096 bf16, 11.6 against 11.0 for
// 4096 x 1001 fp32).
constexpr float kFp8NearScale = 8.0779357e-28f;  // 2^-90
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&v)[V], float scale) {
  float y[V];
  if (scale >= kFp8NearScale && scale < INFINITY) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float near = v[e] * inv;
      y[e] = __builtin_fmaf(__builtin_fmaf(-scale, near, v[e]), inv, near);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = v[e] / scale;
  }
  if constexpr (V == 1) {
    *q = to_e4m3(y[0]);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[e], y[e + 1], 0, false);
      w[e / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[e + 2], y[e + 3], lo, true);
    }
    __builtin_memcpy(__builtin_assume_aligned(q, V), w, V);
  }
}

// One workgroup per row, which it reads three times: rows too long for the
// registers (8192 x 8196 fp32 332 us, 8192 x 8192 in registers 202), and groups of
// channels at unaligned rows, a few threads and four barriers a group (8192 x
// 4096 bf16 in groups of 128 and 32: 701 and 2634 us, aligned 44).
template <typename D, bool Q>
__global__ __launch_bounds__(kNormThreads) void norm_fwd_simple(const NormParams p) {
  using S = typename D::storage;
  __shared__ float lds[kNormThreads / 64];
  __shared__ uint32_t amax;
  const int64_t row = blockIdx.x;
  const S* x = static_cast<const S*>(p.x) + row * p.x_rs;
  const S* res = p.res ? static_cast<const S*>(p.res) + row * p.r_rs : nullptr;
  const S* w = static_cast<const S*>(p.w);
  S* sum = p.sum ? static_cast<S*>(p.sum) + row * p.s_rs : nullptr;
  auto at = [&](int c) { return load_as_float<D>(x + c) + (res ? load_as_float<D>(res + c) : 0.f); };
  float sq = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
    const float v = at(c);
    sq = __builtin_fmaf(v, v, sq);
  }
  const float mean = block_sum(sq, lds) / (float)p.dim;
  const float rstd = 1.0f / sqrtf(mean + p.eps);
  for (int g = 0; g < p.dim; g += p.group) {
    float scale = 1.f;
    if constexpr (Q) {
      if (threadIdx.x == 0) amax = 0;
      __syncthreads();
      uint32_t m = 0;
      for (int c = g + threadIdx.x; c < g + p.group; c += kNormThreads)
        m = max(m, abs_bits(at(c) * rstd * load_as_float<D>(w + c)));
      atomicMax(&amax, m);
      __syncthreads();
      scale = scale_of(amax);
      if (threadIdx.x == 0) p.scales[row * p.sc_rs + g / p.group] = scale;
      __syncthreads();
    }
    for (int c = g + threadIdx.x; c < g + p.group; c += kNormThreads) {
      const float v = at(c);
      const float y = v * rstd * load_as_float<D>(w + c);
      if (sum) sum[c] = round_to<D>(v);
      if constexpr (Q) static_cast<uint8_t*>(p.out)[row * p.o_rs + c] = to_e4m3(y / scale);
      else static_cast<S*>(p.out)[row * p.o_rs + c] = round_to<D>(y);
    }
  }
}

// A row in registers, read once: T threads (one wave, or the workgroup's
// four) hold NV vectors of V channels each.  Bound by the bytes of the rows;
// weight comes from the caches.  G: lanes that share a scale (0: the row).
// 17408 x 4096 bf16 to 8 bits with the residual, groups of 128: 90 us
// (5.5 TB/s).  Ordinary stores: the kernel alone gains 3% by streaming ones, but
// loses more in what reads the output and the sum next (with a copy of both,
// ordinary and streaming: 2048 x 4096 bf16 29 and 32 us, 32768 x 4096 411 and 422).
template <typename D, int V, int NV, int T, bool Q, int G>
__global__ __launch_bounds__(kNormThreads) void norm_fwd_kernel(const NormParams p) {
  using S = typename D::storage;
  using P = Pack<D, V>;
  constexpr int kRows = kNormThreads / T, kWaves = T / 64;
  __shared__ float lsum[kWaves];
  __shared__ uint32_t lmax[kWaves];
  const int t = threadIdx.x % T, wave = t >> 6;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / T;
  if (row >= p.rows) return;  // with a barrier below, a workgroup has one row
  const S* x = static_cast<const S*>(p.x) + row * p.x_rs;
  const S* res = static_cast<const S*>(p.res) + row * p.r_rs;
  const S* w = static_cast<const S*>(p.w);
  S* sum = static_cast<S*>(p.sum) + row * p.s_rs;
  P xv[NV], rv[NV], wv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * T + t) * V;
    xv[j].zero();
    rv[j].zero();
    wv[j].zero();
    if (c < p.dim) {
      xv[j].load(x + c);
      if (p.res) rv[j].load(res + c);
      wv[j].load(w + c);
    }
  }
  float s[NV][V], sq = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[V];
    xv[j].to_float(s[j]);
    if (p.res) {
      rv[j].to_float(f);
#pragma unroll
      for (int e = 0; e < V; ++e) s[j][e] += f[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sq = __builtin_fmaf(s[j][e], s[j][e], sq);
  }
  sq = lanes_reduce<64>(sq, Add());
  if constexpr (kWaves > 1) {
    if ((t & 63) == 0) lsum[wave] = sq;
    __syncthreads();
    sq = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) sq += lsum[i];
  }
  const float rstd = 1.0f / sqrtf(sq / (float)p.dim + p.eps);
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * T + t) * V;
    if (p.sum && c < p.dim) {
      P o;
      o.from_float(s[j]);
      o.store(sum + c);
    }
    float f[V];
    wv[j].to_float(f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s[j][e] = s[j][e] * rstd * f[e];
      if constexpr (Q && G == 0) amax = Max()(amax, c < p.dim ? abs_bits(s[j][e]) : 0u);
    }
  }
  float scale = 1.f;
  if constexpr (Q && G == 0) {
    amax = lanes_reduce<64>(amax, Max());
    if constexpr (kWaves > 1) {
      if ((t & 63) == 0) lmax[wave] = amax;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWaves; ++i) amax = Max()(amax, lmax[i]);
    }
    scale = scale_of(amax);
    if (t == 0) p.scales[row * p.sc_rs] = scale;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * T + t) * V;
    if constexpr (Q) {
      if constexpr (G > 0) {
        amax = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) amax = Max()(amax, abs_bits(s[j][e]));
        scale = scale_of(lanes_reduce<(G > 0 ? G : 1)>(amax, Max()));
        if (t % (G > 0 ? G : 1) == 0 && c < p.dim) p.scales[row * p.sc_rs + c / p.group] = scale;
      }
      if (c < p.dim) store_codes(static_cast<uint8_t*>(p.out) + row * p.o_rs + c, s[j], scale);
    } else if (c < p.dim) {
      P o;
      o.from_float(s[j]);
      o.store(static_cast<S*>(p.out) + row * p.o_rs + c);
    }
  }
}

struct NormBwdParams {
  const void *dout, *x, *w, *dres;
  void* dx;
  float* partial;  // [workgroups, dim]
  int64_t do_rs, x_rs, dr_rs, dx_rs, rows;
  int32_t dim;
  float eps;
};

// dx = rstd (w dout - x^ mean(w dout x^)) + dresidual, x^ = x rstd;
// dweight's share of this workgroup's rows.  Rows too long for the registers.
template <typename D>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_simple(const NormBwdParams p) {
  using S = typename D::storage;
  __shared__ float lds[kNormThreads / 64];
  const S* w = static_cast<const S*>(p.w);
  float* part = p.partial + (int64_t)blockIdx.x * p.dim;
  for (int c = threadIdx.x; c < p.dim; c += kNormThreads) part[c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const S* x = static_cast<const S*>(p.x) + row * p.x_rs;
    const S* g = static_cast<const S*>(p.dout) + row * p.do_rs;
    const S* dr = p.dres ? static_cast<const S*>(p.dres) + row * p.dr_rs : nullptr;
    S* dx = static_cast<S*>(p.dx) + row * p.dx_rs;
    float sq = 0.f, dot = 0.f;
    for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
      const float v = load_as_float<D>(x + c);
      sq = __builtin_fmaf(v, v, sq);
      dot = __builtin_fmaf(load_as_float<D>(g + c) * load_as_float<D>(w + c), v, dot);
    }
    const float mean = block_sum(sq, lds) / (float)p.dim;
    const float rstd = 1.0f / sqrtf(mean + p.eps);
    const float proj = block_sum(dot, lds) * rstd / (float)p.dim;
    for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
      const float hat = load_as_float<D>(x + c) * rstd, gv = load_as_float<D>(g + c);
      float v = rstd * (gv * load_as_float<D>(w + c) - hat * proj);
      if (dr) v += load_as_float<D>(dr + c);
      part[c] = __builtin_fmaf(gv, hat, part[c]);
      dx[c] = round_to<D>(v);
    }
  }
}

// Rows in registers: T threads hold NV vectors of V channels of a row, walk
// every kRows * gridDim-th row, and keep dweight's sums of their channels.
// The next row's loads are issued before this row's sums are exchanged.
// 32768 x 4096 bf16: 199 us (5.4 TB/s); 1023 x 1001 fp32: 11 us, latency.
template <typename D, int V, int NV, int T>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_kernel(const NormBwdParams p) {
  using S = typename D::storage;
  using P = Pack<D, V>;
  constexpr int kRows = kNormThreads / T, kWaves = T / 64;
  __shared__ float2 lsum[2][kWaves];
  const int t = threadIdx.x % T, wave = t >> 6, mine = threadIdx.x / T;
  const S* w = static_cast<const S*>(p.w);
  P wv[NV], xv[NV], gv[NV], dv[NV];
  float dw[NV][V];
  auto fetch = [&](int64_t row) {
    const S* x = static_cast<const S*>(p.x) + row * p.x_rs;
    const S* g = static_cast<const S*>(p.dout) + row * p.do_rs;
    const S* dr = static_cast<const S*>(p.dres) + row * p.dr_rs;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      if (c < p.dim) {
        xv[j].load(x + c);
        gv[j].load(g + c);
        if (p.dres) dv[j].load(dr + c);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * T + t) * V;
    wv[j].zero();
    xv[j].zero();
    gv[j].zero();
    dv[j].zero();
    if (c < p.dim) wv[j].load(w + c);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + mine;
  if (row < p.rows) fetch(row);
  for (int turn = 0; row < p.rows; row += step, turn ^= 1) {
    float x[NV][V], g[NV][V], d[NV][V], sq = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
      xv[j].to_float(x[j]);
      gv[j].to_float(g[j]);
      dv[j].to_float(d[j]);
      wv[j].to_float(f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sq = __builtin_fmaf(x[j][e], x[j][e], sq);
        dot = __builtin_fmaf(g[j][e] * f[e], x[j][e], dot);
      }
    }
    if (row + step < p.rows) fetch(row + step);
    sq = lanes_reduce<64>(sq, Add());
    dot = lanes_reduce<64>(dot, Add());
    if constexpr (kWaves > 1) {
      if ((t & 63) == 0) lsum[turn][wave] = make_float2(sq, dot);
      __syncthreads();
      sq = dot = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        sq += lsum[turn][i].x;
        dot += lsum[turn][i].y;
      }
    }
    const float n = (float)p.dim;
    const float rstd = 1.0f / sqrtf(sq / n + p.eps);
    const float proj = dot * rstd / n;
    S* dx = static_cast<S*>(p.dx) + row * p.dx_rs;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      float f[V], y[V];
      wv[j].to_float(f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hat = x[j][e] * rstd;
        dw[j][e] = __builtin_fmaf(g[j][e], hat, dw[j][e]);
        y[e] = rstd * (g[j][e] * f[e] - hat * proj) + d[j][e];
      }
      if (c < p.dim) {
        P o;
        o.from_float(y);
        o.store(dx + c);
      }
    }
  }
  // the waves' sums of one channel, in the order of the waves
  float* part = p.partial + (int64_t)blockIdx.x * p.dim;
  if constexpr (kRows > 1) {
    constexpr int kWide = NV * T * V;
    __shared__ float lds[kRows][kWide];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) lds[mine][(j * T + t) * V + e] = dw[j][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
      float a = 0.f;
#pragma unroll
      for (int q = 0; q < kRows; ++q) a += lds[q][c];
      part[c] = a;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      if (c < p.dim) {
#pragma unroll
        for (int e = 0; e < V; ++e) part[c + e] = dw[j][e];
      }
    }
  }
}

__global__ __launch_bounds__(kSumCols * kSumGroups) void norm_dweight_kernel(const float* partial,
                                                                             float* dweight,
                                                                             int32_t dim,
                                                                             int32_t n) {
  column_sum(partial, n, dim, [&](int64_t c, float v) { dweight[c] = v; });
}

// How many vectors of a row T threads hold: the smallest instance that
// covers dim, 0 if none does.
static int norm_vectors(int32_t dim, int V, int T) {
  const int64_t need = cdiv(dim, (int64_t)V * T);
  if (V > 1) return need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : 0;
  return need <= 4 ? 4 : need <= 16 ? 16 : need <= 32 ? 32 : 0;
}

// Threads of a row: a wave where it holds the row in two vectors a lane (16
// single elements), which spares the barriers; else four waves, however many
// the rows: with a wave for rows of four and eight vectors, 17408 x 4096 bf16 to
// 8 bits takes 102 us (four waves 90), 4096 x 4096 30 (24), 17408 x 2048 fp32 97 (83).
static int norm_threads(int32_t dim, int V) {
  return cdiv(dim, (int64_t)V * 64) <= (V > 1 ? 2 : 16) ? 64 : 256;
}

// group: channels that share a scale, 0 for the row.
template <typename D, int V, int NV, int T>
static void launch_norm_fwd(bool quant, int group, const NormParams& p, hipStream_t s) {
  const dim3 g((uint32_t)cdiv(p.rows, kNormThreads / T)), th(kNormThreads);
  if (!quant) hipLaunchKernelGGL((norm_fwd_kernel<D, V, NV, T, false, 0>), g, th, 0, s, p);
  else if (group == 0) hipLaunchKernelGGL((norm_fwd_kernel<D, V, NV, T, true, 0>), g, th, 0, s, p);
  else if constexpr (V > 1) {
    switch (group) {
      case 32: hipLaunchKernelGGL((norm_fwd_kernel<D, V, NV, T, true, 32 / V>), g, th, 0, s, p); break;
      case 64: hipLaunchKernelGGL((norm_fwd_kernel<D, V, NV, T, true, 64 / V>), g, th, 0, s, p); break;
      case 128: hipLaunchKernelGGL((norm_fwd_kernel<D, V, NV, T, true, 128 / V>), g, th, 0, s, p); break;
      default: hipLaunchKernelGGL((norm_fwd_kernel<D, V, NV, T, true, 256 / V>), g, th, 0, s, p); break;
    }
  }
}

template <typename D, int V>
static void launch_norm_fwd_n(int nv, int T, bool quant, int group, const NormParams& p,
                              hipStream_t s) {
  if constexpr (V > 1) {
    if (T == 64) {
      if (nv == 1) launch_norm_fwd<D, V, 1, 64>(quant, group, p, s);
      else launch_norm_fwd<D, V, 2, 64>(quant, group, p, s);
    } else {
      if (nv == 1) launch_norm_fwd<D, V, 1, 256>(quant, group, p, s);
      else if (nv == 2) launch_norm_fwd<D, V, 2, 256>(quant, group, p, s);
      else if (nv == 4) launch_norm_fwd<D, V, 4, 256>(quant, group, p, s);
      else launch_norm_fwd<D, V, 8, 256>(quant, group, p, s);
    }
  } else {
    if (T == 64) {
      if (nv == 4) launch_norm_fwd<D, 1, 4, 64>(quant, 0, p, s);
      else launch_norm_fwd<D, 1, 16, 64>(quant, 0, p, s);
    } else {
      if (nv <= 16) launch_norm_fwd<D, 1, 16, 256>(quant, 0, p, s);
      else launch_norm_fwd<D, 1, 32, 256>(quant, 0, p, s);
    }
  }
}

template <typename D, int V>
static void launch_norm_bwd_n(int nv, int T, const NormBwdParams& p, uint32_t grid, hipStream_t s) {
  const dim3 g(grid), th(kNormThreads);
  if constexpr (V > 1) {
    if (T == 64) {
      if (nv == 1) hipLaunchKernelGGL((norm_bwd_kernel<D, V, 1, 64>), g, th, 0, s, p);
      else hipLaunchKernelGGL((norm_bwd_kernel<D, V, 2, 64>), g, th, 0, s, p);
    } else {
      if (nv == 1) hipLaunchKernelGGL((norm_bwd_kernel<D, V, 1, 256>), g, th, 0, s, p);
      else if (nv == 2) hipLaunchKernelGGL((norm_bwd_kernel<D, V, 2, 256>), g, th, 0, s, p);
      else if (nv == 4) hipLaunchKernelGGL((norm_bwd_kernel<D, V, 4, 256>), g, th, 0, s, p);
      else hipLaunchKernelGGL((norm_bwd_kernel<D, V, 8, 256>), g, th, 0, s, p);
    }
  } else {
    if (T == 64) {
      if (nv == 4) hipLaunchKernelGGL((norm_bwd_kernel<D, 1, 4, 64>), g, th, 0, s, p);
      else hipLaunchKernelGGL((norm_bwd_kernel<D, 1, 16, 64>), g, th, 0, s, p);
    } else {
      if (nv <= 16) hipLaunchKernelGGL((norm_bwd_kernel<D, 1, 16, 256>), g, th, 0, s, p);
      else hipLaunchKernelGGL((norm_bwd_kernel<D, 1, 32, 256>), g, th, 0, s, p);
    }
  }
}

// Every row starts on a multiple of V elements, and holds whole vectors.
static bool norm_vec(std::initializer_list<Plane> planes, int64_t V) {
  for (const Plane& a : planes)
    if (!a.empty() && (a.nc % V != 0 || (a.nt > 1 && a.st % V != 0) || !aligned_to(a.p, V * a.es)))
      return false;
  return true;
}

// Workgroups of the backward pass, and rows of its workspace: four rows each at
// least (a row a wave where a wave holds one; single rows were no faster, 1023 x
// 8192 fp32 forward and gradients 52 us both).  At most one a CU where registers
// hold the rows, since each walks them with the next one's loads in flight and
// leaves a row of partial sums (forward and gradients with 1024 and with 256:
// 32768 x 4096 bf16 401 and 373 us, 8192 x 4096 106 and 96, 8192 x 1001 fp32 68 and
// 60); four a CU for wider rows, which are read twice (4096 x 20000 bf16: 977 and
// 1995).  The width tells them apart whatever the type and alignment, which a
// workspace's size does not know.
static int64_t norm_parts(int64_t rows, int32_t dim) {
  const int64_t most = dim <= 8192 ? 256 : 1024;
  return rows < 4 * most ? cdiv(rows, 4) : most;
}

}  // namespace sconv

extern "C" int rms_norm_fwd(const void* x, int64_t x_stride_r, const void* residual,
                            int64_t residual_stride_r, const void* weight, float eps,
                            void* residual_out, int64_t residual_out_stride_r, void* out,
                            int64_t out_stride_r, float* scales, int64_t scales_stride_r,
                            int32_t group_size, int64_t rows, int32_t dim, int32_t dtype,
                            int32_t out_dtype, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "rms_norm_fwd";
  const bool quant = out_dtype == SCONV_E4M3;
  if (rows < 0 || dim < 0) return fail(SCONV_ERR_INVALID, "%s: rows and dim must be >= 0", fn);
  if (!valid_dtype(dtype)) return fail(SCONV_ERR_INVALID, "%s: unknown dtype %d", fn, dtype);
  if (out_dtype != dtype && !quant)
    return fail(SCONV_ERR_INVALID, "%s: out_dtype %d is neither the input's nor e4m3", fn, out_dtype);
  if (!(eps >= 0.f) || !(eps <= 3.0e38f))
    return fail(SCONV_ERR_INVALID, "%s: eps must be finite and >= 0", fn);
  if (group_size < 0 || (group_size > 0 && !quant))
    return fail(SCONV_ERR_INVALID, "%s: group_size=%d without an 8-bit output", fn, group_size);
  if (group_size > 0 && group_size != 32 && group_size != 64 && group_size != 128 && group_size != 256)
    return fail(SCONV_ERR_UNSUPPORTED, "%s: group_size=%d is none of 32, 64, 128, 256", fn, group_size);
  if (group_size > 0 && dim % group_size != 0)
    return fail(SCONV_ERR_INVALID, "%s: group_size=%d does not divide dim=%d", fn, group_size, dim);
  if (rows == 0 || dim == 0) return SCONV_OK;
  if (!x || !weight || !out || (quant && !scales))
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  if (residual_out && !residual)
    return fail(SCONV_ERR_INVALID, "%s: residual_out without residual", fn);
  const int64_t es = elem_size(dtype), oes = quant ? 1 : es;
  const int64_t groups = quant ? (group_size ? dim / group_size : 1) : 0;
  const Plane px = plane(x, 1, x_stride_r, dim, rows, es);
  const Plane pr = plane(residual, 1, residual_stride_r, residual ? dim : 0, rows, es);
  const Plane ps = plane(residual_out, 1, residual_out_stride_r, residual_out ? dim : 0, rows, es);
  const Plane po = plane(out, 1, out_stride_r, dim, rows, oes);
  const Plane pc = plane(scales, 1, scales_stride_r, groups, rows, 4);
  if (!px.readable() || !pr.readable())
    return fail(SCONV_ERR_INVALID, "%s: strides must be >= 0", fn);
  if (!ps.writable() || !po.writable() || !pc.writable())
    return fail(SCONV_ERR_INVALID, "%s: an output's rows overlap each other", fn);
  const Plane in[2] = {px, pr}, ou[3] = {po, ps, pc};
  for (int i = 0; i < 3; ++i) {
    for (const Plane& a : in)  // a row is read before it is written: in place is fine
      if (!(i < 2 && same_plane(ou[i], a)) && planes_overlap(ou[i], a))
        return fail(SCONV_ERR_INVALID, "%s: an output partially overlaps x or residual", fn);
    if (overlap(ou[i].p, ou[i].bytes(), weight, dim * es))
      return fail(SCONV_ERR_INVALID, "%s: an output overlaps weight", fn);
    for (int j = 0; j < i; ++j)
      if (planes_overlap(ou[i], ou[j])) return fail(SCONV_ERR_INVALID, "%s: two outputs overlap", fn);
  }
  NormParams p = {};
  p.x = x; p.res = residual; p.w = weight; p.sum = residual_out; p.out = out; p.scales = scales;
  p.x_rs = px.st; p.r_rs = pr.st; p.s_rs = ps.st; p.o_rs = po.st; p.sc_rs = pc.st; p.rows = rows;
  p.dim = dim; p.group = group_size ? group_size : dim; p.eps = eps;
  if (!valid_grid(rows, kNormThreads)) return fail(SCONV_ERR_UNSUPPORTED, "%s: too many rows", fn);
  const int vec16 = (int)(16 / es);
  const bool vec = norm_vec({px, pr, ps, po}, vec16) && aligned16(weight);
  const int V = vec ? vec16 : 1, T = norm_threads(dim, V), nv = norm_vectors(dim, V, T);
  if (nv > 0 && (vec || group_size == 0)) {
    if (dtype == SCONV_BF16) {
      if (vec) launch_norm_fwd_n<Bf16, 8>(nv, T, quant, group_size, p, stream);
      else launch_norm_fwd_n<Bf16, 1>(nv, T, quant, 0, p, stream);
    } else {
      if (vec) launch_norm_fwd_n<F32, 4>(nv, T, quant, group_size, p, stream);
      else launch_norm_fwd_n<F32, 1>(nv, T, quant, 0, p, stream);
    }
    return check_launch(fn);
  }
  const dim3 grid((uint32_t)rows), th(kNormThreads);
  if (dtype == SCONV_BF16) {
    if (quant) hipLaunchKernelGGL((norm_fwd_simple<Bf16, true>), grid, th, 0, stream, p);
    else hipLaunchKernelGGL((norm_fwd_simple<Bf16, false>), grid, th, 0, stream, p);
  } else {
    if (quant) hipLaunchKernelGGL((norm_fwd_simple<F32, true>), grid, th, 0, stream, p);
    else hipLaunchKernelGGL((norm_fwd_simple<F32, false>), grid, th, 0, stream, p);
  }
  return check_launch(fn);
}

extern "C" int rms_norm_bwd_workspace(int64_t rows, int32_t dim, int64_t* floats) {
  using namespace sconv;
  clear_error();
  if (rows < 0 || dim < 0 || !floats)
    return fail(SCONV_ERR_INVALID, "rms_norm_bwd_workspace: rows and dim must be >= 0, floats not NULL");
  *floats = norm_parts(rows, dim) * dim;
  return SCONV_OK;
}

extern "C" int rms_norm_bwd(const void* dout, int64_t dout_stride_r, const void* x,
                            int64_t x_stride_r, const void* weight, float eps,
                            const void* dresidual, int64_t dresidual_stride_r, void* dx,
                            int64_t dx_stride_r, float* dweight, float* workspace,
                            int64_t workspace_floats, int64_t rows, int32_t dim, int32_t dtype,
                            hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "rms_norm_bwd";
  if (rows < 0 || dim < 0) return fail(SCONV_ERR_INVALID, "%s: rows and dim must be >= 0", fn);
  if (!valid_dtype(dtype)) return fail(SCONV_ERR_INVALID, "%s: unknown dtype %d", fn, dtype);
  if (!(eps >= 0.f) || !(eps <= 3.0e38f))
    return fail(SCONV_ERR_INVALID, "%s: eps must be finite and >= 0", fn);
  if (dim == 0) return SCONV_OK;
  if (!dweight || (rows > 0 && (!dout || !x || !weight || !dx || !workspace)))
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  const int64_t parts = norm_parts(rows, dim), need = parts * dim;
  if (workspace_floats < need)
    return fail(SCONV_ERR_INVALID, "%s: workspace holds %lld floats, %lld needed", fn,
                (long long)workspace_floats, (long long)need);
  const int64_t es = elem_size(dtype);
  const Plane in[3] = {plane(dout, 1, dout_stride_r, dim, rows, es),
                       plane(x, 1, x_stride_r, dim, rows, es),
                       plane(dresidual, 1, dresidual_stride_r, dresidual ? dim : 0, rows, es)};
  const Plane po = plane(dx, 1, dx_stride_r, dim, rows, es);
  for (const Plane& a : in) {
    if (!a.readable()) return fail(SCONV_ERR_INVALID, "%s: strides must be >= 0", fn);
    // a row is read before it is written: in place is fine
    if (!same_plane(po, a) && planes_overlap(po, a))
      return fail(SCONV_ERR_INVALID, "%s: dx partially overlaps an input", fn);
  }
  if (!po.writable()) return fail(SCONV_ERR_INVALID, "%s: dx's rows overlap each other", fn);
  const struct { const void* p; int64_t n; } wr[3] = {
      {dx, po.bytes()}, {dweight, (int64_t)dim * 4}, {workspace, need * 4}};
  for (int i = 0; i < 3; ++i) {
    bool bad = rows > 0 && overlap(wr[i].p, wr[i].n, weight, dim * es);
    for (const Plane& a : in) bad = bad || (i > 0 && overlap(wr[i].p, wr[i].n, a.p, a.bytes()));
    for (int j = 0; j < i; ++j) bad = bad || overlap(wr[i].p, wr[i].n, wr[j].p, wr[j].n);
    if (bad) return fail(SCONV_ERR_INVALID, "%s: an output or the workspace overlaps another buffer", fn);
  }
  NormBwdParams p = {};
  p.dout = dout; p.x = x; p.w = weight; p.dres = dresidual; p.dx = dx; p.partial = workspace;
  p.do_rs = in[0].st; p.x_rs = in[1].st; p.dr_rs = in[2].st; p.dx_rs = po.st; p.rows = rows;
  p.dim = dim; p.eps = eps;
  if (rows > 0) {
    const int vec16 = (int)(16 / es);
    const bool vec = norm_vec({in[0], in[1], in[2], po}, vec16) && aligned16(weight);
    const int V = vec ? vec16 : 1, T = norm_threads(dim, V), nv = norm_vectors(dim, V, T);
    const uint32_t grid = (uint32_t)parts;
    if (nv > 0) {
      if (dtype == SCONV_BF16) {
        if (vec) launch_norm_bwd_n<Bf16, 8>(nv, T, p, grid, stream);
        else launch_norm_bwd_n<Bf16, 1>(nv, T, p, grid, stream);
      } else {
        if (vec) launch_norm_bwd_n<F32, 4>(nv, T, p, grid, stream);
        else launch_norm_bwd_n<F32, 1>(nv, T, p, grid, stream);
      }
    } else if (dtype == SCONV_BF16) {
      hipLaunchKernelGGL(norm_bwd_simple<Bf16>, dim3(grid), dim3(kNormThreads), 0, stream, p);
    } else {
      hipLaunchKernelGGL(norm_bwd_simple<F32>, dim3(grid), dim3(kNormThreads), 0, stream, p);
    }
    if (const int rc = check_launch(fn)) return rc;
  }
  hipLaunchKernelGGL(norm_dweight_kernel, dim3((uint32_t)cdiv(dim, kSumCols)),
                     dim3(kSumCols * kSumGroups), 0, stream, workspace, dweight, dim,
                     (int32_t)parts);
  return check_launch(fn);
}
