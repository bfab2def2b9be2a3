// layer_norm.hip -- layer norm of rows with the residual's addition, and its
// gradients, for gfx950.
//
//   s = x + residual, n = (s - mean(s)) * rsqrt(mean((s - mean)^2) + eps),
//   out = n * weight + bias
// The variance is a sum over differences from the mean, and the mean's own
// rounding is taken out of it: the same exchange sums the differences, whose mean
// r is what the first mean was off by, so that n = (d - r) * rsqrt(mean(d^2) - r^2
// + eps).  A row far from zero keeps its digits (4096 channels of 4321.1: outputs of
// 1e-8 where a mean that is left as it is gives 0.15); it costs a second exchange
// between the waves of a row.
#include "column_sum.h"
#include "lane_tokens.h"
#include "norm_rows.h"

namespace sconv {

struct LayerParams {
  const void *x, *res, *w, *b;
  void *sum, *out;
  int64_t x_rs, r_rs, s_rs, o_rs, rows;
  int32_t dim;
  float eps;
};

template <int CTRL> __device__ __forceinline__ float moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The sums of the waves of a row, N = 1, 2 or 4 of them; one LDS row an exchange,
// so one barrier.  A lane keeps one half of several sums and gives its neighbour the
// other, so that lane i % N ends with sum i: 7 moves for four sums (24 one by one;
// 32768 x 4096 bf16 gradients with dresidual, four sums a row: 189 us, one by one 201).
template <int N, int kWaves>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*lds)[N], int t) {
  static_assert(N == 1 || N == 2 || N == 4);
  float x;
  if constexpr (N == 1) {
    x = lanes_reduce<64>(v[0], Add());
  } else {
    const bool odd = t & 1, high = t & 2;
    x = (odd ? v[1] : v[0]) + moved<0xB1>(odd ? v[0] : v[1]);  // lanes 1 0 3 2
    if constexpr (N == 4) {
      const float y = (odd ? v[3] : v[2]) + moved<0xB1>(odd ? v[2] : v[3]);
      x = (high ? y : x) + moved<0x4E>(high ? x : y);  // lanes 2 3 0 1
    } else {
      x += moved<0x4E>(x);
    }
    x += moved<0x124>(x);  // four lanes on, of sixteen
    x += moved<0x128>(x);  // eight
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
  }
  if constexpr (kWaves > 1) {
    if ((t & 63) < N) lds[t >> 6][t & 63] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v[i] += lds[w][i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i));
  }
}

// Of a row, from the sums of the differences d from its rounded mean: their own
// mean, and 1 / the standard deviation around it.
struct RowScale {
  float rest, rstd;
  __device__ __forceinline__ RowScale(float sum, float squares, float n, float eps) {
    rest = sum / n;
    // fused: rest's square is not rounded, so infinite squares stay so (rstd 0)
    const float var = __builtin_fmaf(-rest, rest, squares / n);
    rstd = 1.0f / sqrtf((var < 0.f ? 0.f : var) + eps);  // a NaN stays one
  }
  __device__ __forceinline__ float operator()(float d) const { return __builtin_fmaf(d, rstd, -(rest * rstd)); }
};

// One workgroup a row, which it reads three times: rows too long for the registers.
template <typename D>
__global__ __launch_bounds__(kNormThreads) void layer_fwd_simple(const LayerParams p) {
  using S = typename D::storage;
  __shared__ float lds[kNormThreads / 64];
  const int64_t row = blockIdx.x;
  const S* x = static_cast<const S*>(p.x) + row * p.x_rs;
  const S* res = p.res ? static_cast<const S*>(p.res) + row * p.r_rs : nullptr;
  const S *w = static_cast<const S*>(p.w), *b = static_cast<const S*>(p.b);
  S* sum = p.sum ? static_cast<S*>(p.sum) + row * p.s_rs : nullptr;
  auto at = [&](int c) { return load_as_float<D>(x + c) + (res ? load_as_float<D>(res + c) : 0.f); };
  float m = 0.f, sum1 = 0.f, sq = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += kNormThreads) m += at(c);
  const float mean = block_sum(m, lds) / (float)p.dim;
  for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
    const float d = at(c) - mean;
    sum1 += d;
    sq = __builtin_fmaf(d, d, sq);
  }
  const float all = block_sum(sum1, lds);
  const RowScale norm(all, block_sum(sq, lds), (float)p.dim, p.eps);
  for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
    const float v = at(c);
    if (sum) sum[c] = round_to<D>(v);
    static_cast<S*>(p.out)[row * p.o_rs + c] = round_to<D>(
        norm(v - mean) * load_as_float<D>(w + c) + (b ? load_as_float<D>(b + c) : 0.f));
  }
}

// A row in registers, read once: T threads (one wave, or the workgroup's
// four) hold NV vectors of V channels each.  Bytes bound it: 32768 x 4096 bf16
// with the residual 174 us, 6.2 TB/s; 256 x 1024 3.7 us, a load's latency and two
// exchanges.
template <typename D, int V, int NV, int T>
__global__ __launch_bounds__(kNormThreads) void layer_fwd_kernel(const LayerParams p) {
  using S = typename D::storage;
  using P = Pack<D, V>;
  constexpr int kRows = kNormThreads / T, kWaves = T / 64;
  __shared__ float lmean[kWaves][1], lsum[kWaves][2];
  const int t = threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / T;
  if (row >= p.rows) return;  // with a barrier below, a workgroup has one row
  const S* x = static_cast<const S*>(p.x) + row * p.x_rs;
  const S* res = static_cast<const S*>(p.res) + row * p.r_rs;
  const S *w = static_cast<const S*>(p.w), *b = static_cast<const S*>(p.b);
  P xv[NV], rv[NV], wv[NV], bv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * T + t) * V;
    xv[j].zero();
    rv[j].zero();
    wv[j].zero();
    bv[j].zero();
    if (c < p.dim) {
      xv[j].load(x + c);
      if (p.res) rv[j].load(res + c);
      wv[j].load(w + c);
      if (p.b) bv[j].load(b + c);
    }
  }
  float s[NV][V], m[1] = {0.f}, sums[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[V];
    xv[j].to_float(s[j]);
    rv[j].to_float(f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (p.res) s[j][e] += f[e];
      m[0] += s[j][e];
    }
  }
  row_sums<1, kWaves>(m, lmean, t);
  const float mean = m[0] / (float)p.dim;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * T + t) * V;
    if (p.sum && c < p.dim) {
      P o;
      o.from_float(s[j]);
      o.store(static_cast<S*>(p.sum) + row * p.s_rs + c);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s[j][e] = c < p.dim ? s[j][e] - mean : 0.f;
      sums[0] += s[j][e];
      sums[1] = __builtin_fmaf(s[j][e], s[j][e], sums[1]);
    }
  }
  row_sums<2, kWaves>(sums, lsum, t);
  const RowScale norm(sums[0], sums[1], (float)p.dim, p.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * T + t) * V;
    float f[V], h[V];
    wv[j].to_float(f);
    bv[j].to_float(h);
#pragma unroll
    for (int e = 0; e < V; ++e) s[j][e] = __builtin_fmaf(norm(s[j][e]), f[e], h[e]);
    if (c < p.dim) {
      P o;
      o.from_float(s[j]);
      o.store(static_cast<S*>(p.out) + row * p.o_rs + c);
    }
  }
}

struct LayerBwdParams {
  const void *dout, *x, *w, *dres;
  void* dx;
  float* partial;  // [workgroups, 2, dim]: dweight's and dbias's shares
  int64_t do_rs, x_rs, dr_rs, dx_rs, rows;
  int32_t dim;
  float eps;
};

// dx = rstd (w dout - mean(w dout) - n mean(w dout n)) + dresidual; the
// shares of this workgroup's rows in dweight and dbias.  Rows too long for
// the registers.  The shares are added up in memory, which with the second read of
// a row is what it costs (4096 x 32768 bf16: 1580 us, 0.5 TB/s of its own bytes).
template <typename D>
__global__ __launch_bounds__(kNormThreads) void layer_bwd_simple(const LayerBwdParams p) {
  using S = typename D::storage;
  __shared__ float lds[kNormThreads / 64];
  const S* w = static_cast<const S*>(p.w);
  float* dw = p.partial + (int64_t)blockIdx.x * 2 * p.dim;
  float* db = dw + p.dim;
  for (int c = threadIdx.x; c < p.dim; c += kNormThreads) dw[c] = db[c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const S* x = static_cast<const S*>(p.x) + row * p.x_rs;
    const S* g = static_cast<const S*>(p.dout) + row * p.do_rs;
    const S* dr = p.dres ? static_cast<const S*>(p.dres) + row * p.dr_rs : nullptr;
    S* dx = static_cast<S*>(p.dx) + row * p.dx_rs;
    const float n = (float)p.dim;
    float m = 0.f, sum1 = 0.f, sq = 0.f, one = 0.f, dot = 0.f;
    for (int c = threadIdx.x; c < p.dim; c += kNormThreads) m += load_as_float<D>(x + c);
    const float mean = block_sum(m, lds) / n;
    for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
      const float d = load_as_float<D>(x + c) - mean;
      const float wg = load_as_float<D>(g + c) * load_as_float<D>(w + c);
      sum1 += d;
      sq = __builtin_fmaf(d, d, sq);
      one += wg;
      dot = __builtin_fmaf(wg, d, dot);
    }
    const float all = block_sum(sum1, lds);
    const RowScale norm(all, block_sum(sq, lds), n, p.eps);
    const float ones = block_sum(one, lds), rstd = norm.rstd;
    const float flat = ones / n, proj = (block_sum(dot, lds) - norm.rest * ones) * rstd / n;
    for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
      const float hat = norm(load_as_float<D>(x + c) - mean), gv = load_as_float<D>(g + c);
      float v = rstd * (gv * load_as_float<D>(w + c) - flat - hat * proj);
      if (dr) v += load_as_float<D>(dr + c);
      dw[c] = __builtin_fmaf(gv, hat, dw[c]);
      db[c] += gv;
      dx[c] = round_to<D>(v);
    }
  }
}

// Rows in registers: T threads hold NV vectors of V channels of a row, walk
// every kRows * gridDim-th row, and keep the weights' sums of their channels.
// The next row's loads are issued before this row's sums are exchanged, so a
// workgroup always has a row under way: bytes bound it (32768 x 4096 bf16 162 us,
// 5.0 TB/s; with dresidual 189, 5.7 TB/s), and for few rows two launches' latency
// (1023 x 1001 fp32: 13 + 4 us).  16384 bf16 channels spill 45 registers of 512,
// and are still faster than the two-pass kernel (4096 x 16384: 250 us; 4096 x
// 12001, which that one takes, 462).
template <typename D, int V, int NV, int T>
__global__ __launch_bounds__(kNormThreads) void layer_bwd_kernel(const LayerBwdParams p) {
  using S = typename D::storage;
  using P = Pack<D, V>;
  constexpr int kRows = kNormThreads / T, kWaves = T / 64;
  // each is written behind the other's barrier
  __shared__ float lmean[kWaves][1], lsum[kWaves][4];
  const int t = threadIdx.x % T, mine = threadIdx.x / T;
  const S* w = static_cast<const S*>(p.w);
  P wv[NV], xv[NV], gv[NV], dv[NV];
  float dw[NV][V], db[NV][V];
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
    for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + mine;
  if (row < p.rows) fetch(row);
  const float n = (float)p.dim;
  for (; row < p.rows; row += step) {
    float x[NV][V], g[NV][V], d[NV][V], m[1] = {0.f}, sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xv[j].to_float(x[j]);
      gv[j].to_float(g[j]);
      dv[j].to_float(d[j]);
#pragma unroll
      for (int e = 0; e < V; ++e) m[0] += x[j][e];
    }
    if (row + step < p.rows) fetch(row + step);
    row_sums<1, kWaves>(m, lmean, t);
    const float mean = m[0] / n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      float f[V];
      wv[j].to_float(f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] = c < p.dim ? x[j][e] - mean : 0.f;
        const float wg = g[j][e] * f[e];
        sums[0] = __builtin_fmaf(x[j][e], x[j][e], sums[0]);
        sums[1] += wg;
        sums[2] = __builtin_fmaf(wg, x[j][e], sums[2]);
        sums[3] += x[j][e];
      }
    }
    row_sums<4, kWaves>(sums, lsum, t);
    const RowScale norm(sums[3], sums[0], n, p.eps);
    const float rstd = norm.rstd;
    const float flat = sums[1] / n, proj = (sums[2] - norm.rest * sums[1]) * rstd / n;
    S* dx = static_cast<S*>(p.dx) + row * p.dx_rs;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      float f[V], y[V];
      wv[j].to_float(f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hat = norm(x[j][e]);
        dw[j][e] = __builtin_fmaf(g[j][e], hat, dw[j][e]);
        db[j][e] += g[j][e];
        y[e] = rstd * (g[j][e] * f[e] - flat - hat * proj) + d[j][e];
      }
      if (c < p.dim) {
        P o;
        o.from_float(y);
        o.store(dx + c);
      }
    }
  }
  // the waves' sums of one channel, in the order of the waves
  float* part = p.partial + (int64_t)blockIdx.x * 2 * p.dim;
  if constexpr (kRows > 1) {
    constexpr int kWide = NV * T * V;
    __shared__ float lds[2][kRows][kWide];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        lds[0][mine][(j * T + t) * V + e] = dw[j][e];
        lds[1][mine][(j * T + t) * V + e] = db[j][e];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.dim; c += kNormThreads) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a = 0.f;
#pragma unroll
        for (int q = 0; q < kRows; ++q) a += lds[k][q][c];
        part[k * p.dim + c] = a;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      if (c < p.dim) {
#pragma unroll
        for (int e = 0; e < V; ++e) part[c + e] = dw[j][e], part[p.dim + c + e] = db[j][e];
      }
    }
  }
}

__global__ __launch_bounds__(kSumCols * kSumGroups) void layer_dweight_kernel(const float* partial,
                                                                              float* dweight,
                                                                              float* dbias,
                                                                              int32_t dim,
                                                                              int32_t n) {
  column_sum(partial, n, 2 * (int64_t)dim, [&](int64_t c, float v) {
    if (c < dim) dweight[c] = v;
    else if (dbias) dbias[c - dim] = v;
  });
}

template <typename D, int V, int NV, int T>
static void launch_layer(const LayerParams& p, hipStream_t s) {
  hipLaunchKernelGGL((layer_fwd_kernel<D, V, NV, T>), dim3((uint32_t)cdiv(p.rows, kNormThreads / T)),
                     dim3(kNormThreads), 0, s, p);
}
template <typename D, int V, int NV, int T>
static void launch_layer(const LayerBwdParams& p, uint32_t grid, hipStream_t s) {
  hipLaunchKernelGGL((layer_bwd_kernel<D, V, NV, T>), dim3(grid), dim3(kNormThreads), 0, s, p);
}

// The instance whose T threads hold a row in nv vectors.
template <typename D, int V, typename... A> static void launch_layer_n(int nv, int T, const A&... a) {
  if constexpr (V > 1) {
    if (T == 64) {
      if (nv == 1) launch_layer<D, V, 1, 64>(a...);
      else launch_layer<D, V, 2, 64>(a...);
    } else {
      if (nv == 1) launch_layer<D, V, 1, 256>(a...);
      else if (nv == 2) launch_layer<D, V, 2, 256>(a...);
      else if (nv == 4) launch_layer<D, V, 4, 256>(a...);
      else launch_layer<D, V, 8, 256>(a...);
    }
  } else {
    if (T == 64) {
      if (nv == 4) launch_layer<D, 1, 4, 64>(a...);
      else launch_layer<D, 1, 16, 64>(a...);
    } else {
      if (nv <= 16) launch_layer<D, 1, 16, 256>(a...);
      else launch_layer<D, 1, 32, 256>(a...);
    }
  }
}

// Workgroups of the backward pass; each writes its share of 2 dim sums, which
// costs more than a workgroup gains below four rows (1000 x 4096 bf16: 20.0 us,
// 25.9 with two rows each).  Where registers hold the rows one workgroup a CU
// keeps memory busy (8192 x 8192 bf16: 90 us, two 100), but for short rows from
// eight a workgroup on (2048 x 4096: 23 us, two 27): those of 8 KB (32768 x 4096
// bf16: 161 us, one 184, four 188; 16384 x 4096 fp32: 150, two 156), or with a
// fourth stream, dresidual, in vectors of 4 KB (8192 x 2048 bf16: 37, one 44;
// 32768 x 4096: 189, two 207).  Rows read twice are latency: four a CU (4096 x
// 12001: 463 us, one 1195) from two rows on (1024 x 12001: 192 us, from four 290).
static int64_t layer_parts(int64_t rows, bool is_short, bool held) {
  if (!held) return rows < 2048 ? cdiv(rows, 2) : 1024;
  if (rows < 4096) return rows < 1024 ? cdiv(rows, 4) : 256;
  return is_short ? 512 : 256;
}
// A workgroup's share of the weights' gradients is fp32 chains of its rows, then 64
// bits add the shares.  So that no chain is longer than kChain rows, a call whose
// workgroups would have more (in_hand rows at a time each) is several launches of
// as many (2^20 equal terms: 4e-6 off, in chains of 2048 3e-5).
constexpr int64_t kChain = 256;
static int64_t layer_launches(int64_t rows, int64_t parts, int in_hand) {
  return rows > 0 ? cdiv(rows, parts * in_hand * kChain) : 1;
}
// No fewer shares for either type, at any alignment: 8192 channels are always held.
static int64_t layer_parts_most(int64_t rows, int32_t dim) {
  return layer_parts(rows, dim <= 4096, dim <= 8192) + (rows > 256 * kChain ? rows / kChain : 0);
}

}  // namespace sconv

extern "C" int layer_norm_fwd(const void* x, int64_t x_stride_r, const void* residual,
                              int64_t residual_stride_r, const void* weight, const void* bias,
                              float eps, void* residual_out, int64_t residual_out_stride_r,
                              void* out, int64_t out_stride_r, int64_t rows, int32_t dim,
                              int32_t dtype, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "layer_norm_fwd";
  if (rows < 0 || dim < 0) return fail(SCONV_ERR_INVALID, "%s: rows and dim must be >= 0", fn);
  if (!valid_dtype(dtype)) return fail(SCONV_ERR_INVALID, "%s: unknown dtype %d", fn, dtype);
  if (!(eps >= 0.f) || !(eps <= 3.0e38f))
    return fail(SCONV_ERR_INVALID, "%s: eps must be finite and >= 0", fn);
  if (rows == 0 || dim == 0) return SCONV_OK;
  if (!x || !weight || !out) return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  if (residual_out && !residual)
    return fail(SCONV_ERR_INVALID, "%s: residual_out without residual", fn);
  const int64_t es = elem_size(dtype);
  const Plane px = plane(x, 1, x_stride_r, dim, rows, es);
  const Plane pr = plane(residual, 1, residual_stride_r, residual ? dim : 0, rows, es);
  const Plane ps = plane(residual_out, 1, residual_out_stride_r, residual_out ? dim : 0, rows, es);
  const Plane po = plane(out, 1, out_stride_r, dim, rows, es);
  if (!px.readable() || !pr.readable())
    return fail(SCONV_ERR_INVALID, "%s: strides must be >= 0", fn);
  if (!ps.writable() || !po.writable())
    return fail(SCONV_ERR_INVALID, "%s: an output's rows overlap each other", fn);
  for (const Plane& o : {po, ps}) {
    for (const Plane& a : {px, pr})  // a row is read before it is written: in place is fine
      if (!same_plane(o, a) && planes_overlap(o, a))
        return fail(SCONV_ERR_INVALID, "%s: an output partially overlaps x or residual", fn);
    if (overlap(o.p, o.bytes(), weight, dim * es) || (bias && overlap(o.p, o.bytes(), bias, dim * es)))
      return fail(SCONV_ERR_INVALID, "%s: an output overlaps weight or bias", fn);
  }
  if (planes_overlap(po, ps)) return fail(SCONV_ERR_INVALID, "%s: two outputs overlap", fn);
  LayerParams p = {};
  p.x = x; p.res = residual; p.w = weight; p.b = bias; p.sum = residual_out; p.out = out;
  p.x_rs = px.st; p.r_rs = pr.st; p.s_rs = ps.st; p.o_rs = po.st; p.rows = rows;
  p.dim = dim; p.eps = eps;
  if (!valid_grid(rows, kNormThreads)) return fail(SCONV_ERR_UNSUPPORTED, "%s: too many rows", fn);
  const int vec16 = (int)(16 / es);
  const bool vec = norm_vec({px, pr, ps, po}, vec16) && aligned16(weight) && aligned16(bias);
  const int V = vec ? vec16 : 1, T = norm_threads(dim, V), nv = norm_vectors(dim, V, T);
  if (nv > 0) {
    if (dtype == SCONV_BF16) {
      if (vec) launch_layer_n<Bf16, 8>(nv, T, p, stream);
      else launch_layer_n<Bf16, 1>(nv, T, p, stream);
    } else {
      if (vec) launch_layer_n<F32, 4>(nv, T, p, stream);
      else launch_layer_n<F32, 1>(nv, T, p, stream);
    }
  } else {
    const dim3 grid((uint32_t)rows), th(kNormThreads);
    if (dtype == SCONV_BF16) hipLaunchKernelGGL(layer_fwd_simple<Bf16>, grid, th, 0, stream, p);
    else hipLaunchKernelGGL(layer_fwd_simple<F32>, grid, th, 0, stream, p);
  }
  return check_launch(fn);
}

extern "C" int layer_norm_bwd_workspace(int64_t rows, int32_t dim, int64_t* floats) {
  using namespace sconv;
  clear_error();
  if (rows < 0 || dim < 0 || !floats)
    return fail(SCONV_ERR_INVALID, "layer_norm_bwd_workspace: rows and dim must be >= 0, floats not NULL");
  *floats = layer_parts_most(rows, dim) * 2 * dim;
  return SCONV_OK;
}

extern "C" int layer_norm_bwd(const void* dout, int64_t dout_stride_r, const void* x,
                              int64_t x_stride_r, const void* weight, float eps,
                              const void* dresidual, int64_t dresidual_stride_r, void* dx,
                              int64_t dx_stride_r, float* dweight, float* dbias, float* workspace,
                              int64_t workspace_floats, int64_t rows, int32_t dim, int32_t dtype,
                              hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "layer_norm_bwd";
  if (rows < 0 || dim < 0) return fail(SCONV_ERR_INVALID, "%s: rows and dim must be >= 0", fn);
  if (!valid_dtype(dtype)) return fail(SCONV_ERR_INVALID, "%s: unknown dtype %d", fn, dtype);
  if (!(eps >= 0.f) || !(eps <= 3.0e38f))
    return fail(SCONV_ERR_INVALID, "%s: eps must be finite and >= 0", fn);
  if (dim > (1 << 28)) return fail(SCONV_ERR_UNSUPPORTED, "%s: dim above 2^28", fn);
  if (dim == 0) return SCONV_OK;
  if (!dweight || (rows > 0 && (!dout || !x || !weight || !dx || !workspace)))
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  const int64_t need = layer_parts_most(rows, dim) * 2 * dim;
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
  const struct { const void* p; int64_t n; } wr[4] = {
      {dx, po.bytes()}, {dweight, (int64_t)dim * 4}, {dbias, dbias ? (int64_t)dim * 4 : 0},
      {workspace, need * 4}};
  for (int i = 0; i < 4; ++i) {
    bool bad = rows > 0 && overlap(wr[i].p, wr[i].n, weight, dim * es);
    for (const Plane& a : in) bad = bad || (i > 0 && overlap(wr[i].p, wr[i].n, a.p, a.bytes()));
    for (int j = 0; j < i; ++j) bad = bad || overlap(wr[i].p, wr[i].n, wr[j].p, wr[j].n);
    if (bad) return fail(SCONV_ERR_INVALID, "%s: an output or the workspace overlaps another buffer", fn);
  }
  LayerBwdParams p = {};
  p.dout = dout; p.x = x; p.w = weight; p.dres = dresidual; p.dx = dx; p.partial = workspace;
  p.do_rs = in[0].st; p.x_rs = in[1].st; p.dr_rs = in[2].st; p.dx_rs = po.st; p.rows = rows;
  p.dim = dim; p.eps = eps;
  const int vec16 = (int)(16 / es);
  const bool vec = norm_vec({in[0], in[1], in[2], po}, vec16) && aligned16(weight);
  const int V = vec ? vec16 : 1, T = norm_threads(dim, V), nv = norm_vectors(dim, V, T);
  const uint32_t grid = (uint32_t)layer_parts(rows, dim * es <= (dresidual && vec ? 4096 : 8192), nv > 0);
  // even parts of the rows, each with shares of its own
  const int64_t launches = layer_launches(rows, grid, nv > 0 ? kNormThreads / T : 1);
  const int64_t each = rows > 0 ? cdiv(rows, launches) : 1;
  for (int64_t at = 0; at < rows; at += each) {
    p.rows = rows - at < each ? rows - at : each;
    if (nv > 0) {
      if (dtype == SCONV_BF16) {
        if (vec) launch_layer_n<Bf16, 8>(nv, T, p, grid, stream);
        else launch_layer_n<Bf16, 1>(nv, T, p, grid, stream);
      } else {
        if (vec) launch_layer_n<F32, 4>(nv, T, p, grid, stream);
        else launch_layer_n<F32, 1>(nv, T, p, grid, stream);
      }
    } else if (dtype == SCONV_BF16) {
      hipLaunchKernelGGL(layer_bwd_simple<Bf16>, dim3(grid), dim3(kNormThreads), 0, stream, p);
    } else {
      hipLaunchKernelGGL(layer_bwd_simple<F32>, dim3(grid), dim3(kNormThreads), 0, stream, p);
    }
    if (const int rc = check_launch(fn)) return rc;
    p.dout = static_cast<const char*>(p.dout) + each * p.do_rs * es;
    p.x = static_cast<const char*>(p.x) + each * p.x_rs * es;
    if (p.dres) p.dres = static_cast<const char*>(p.dres) + each * p.dr_rs * es;
    p.dx = static_cast<char*>(p.dx) + each * p.dx_rs * es;
    p.partial += (int64_t)grid * 2 * dim;
  }
  hipLaunchKernelGGL(layer_dweight_kernel, dim3((uint32_t)cdiv(2 * (int64_t)dim, kSumCols)),
                     dim3(kSumCols * kSumGroups), 0, stream, workspace, dweight, dbias, dim,
                     (int32_t)(rows > 0 ? cdiv(rows, each) * grid : 0));
  return check_launch(fn);
}
