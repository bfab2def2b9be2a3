// conv_grad.hip -- gradients of the causal depthwise conv over packed
// variable-length sequences (causal_conv1d_varlen_fwd), for gfx950.
//
// With u a sequence's initial state followed by its inputs (logical index
// i >= -(W-1)), z_t = bias + sum_k w_k u_{t-(W-1)+k} and out = act(z):
//   dz_t = dout_t act'(z_t)
//   du_i = sum_l w_{W-1-l} dz_{i+l}  (+ the final state's gradient)
//   dw_k = sum_t dz_t u_{t-(W-1)+k},  dbias = sum_t dz_t
// z is recomputed from the inputs, so the forward saves nothing.
#include "column_sum.h"
#include "lane_tokens.h"
#include "row_lanes.h"
#include "plane_host.h"

namespace sconv {

struct ConvGradParams {
  const void *dout, *x, *w, *bias, *initial;
  const int32_t* qsl;
  const int32_t* cache_indices;
  const uint8_t* has_init;
  const void* dfinal;
  void *dinitial, *dx;
  float* partial;  // [parts, dim, W + 1]: dw, dbias of one sequence or segment
  int64_t do_sc, do_st, x_sc, x_st, w_sc, w_sk, dx_sc, dx_st;
  int64_t is_slot, is_c, is_k, df_slot, df_c, df_k, di_slot, di_c, di_k;
  int64_t total_T, num_pairs;
  int32_t strip, batch, dim, silu, pad_slot_id;
};

// dout * d silu(z) / dz
__device__ __forceinline__ float silu_grad(float z, float g) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  return g * s * __builtin_fmaf(z, 1.0f - s, 1.0f);
}

// The W - 1 dz after a run of tokens, or before the first: dz of tokens
// [t, t + W-1) of the sequence [start, end), from scalar loads.
template <typename D, int W>
struct Head {
  using S = typename D::storage;
  const S *x, *g;
  int64_t x_st, g_st, start, end;
  float s0[W];  // initial state, oldest first (W-1 used)
  float w[W], bias;
  bool silu;

  __device__ __forceinline__ float input(int64_t t) const {
    if (t >= start) return load_as_float<D>(x + t * x_st);
    return t >= start - (W - 1) ? pick(s0, (int)(t - start + W - 1)) : 0.f;
  }
  __device__ __forceinline__ void after(int64_t t, float (&dz)[W]) const {
    float u[2 * W];
#pragma unroll
    for (int k = 0; k < 2 * W - 2; ++k) u[k] = t + k - (W - 1) < end ? input(t + k - (W - 1)) : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      dz[j] = 0.f;
      if (j < W - 1 && t + j < end) {
        float z = bias;
#pragma unroll
        for (int k = 0; k < W; ++k) z = __builtin_fmaf(w[k], u[j + k], z);
        const float gv = load_as_float<D>(g + (t + j) * g_st);
        dz[j] = silu ? silu_grad(z, gv) : gv;
      }
    }
  }
};

// Tokens in lanes: a wave takes chunks of 512 tokens of one channel from the
// last to the first, lane l the tokens [8 l, 8 l + 8).  The inputs before a
// lane's tokens come from the lane below, the dz after them from the lane
// above, and across chunks from a load and from the chunk done before.
// Every byte of x and dout is read once; bound by that.  NW waves share a
// sequence, each with a run of its chunks (one dz past a run is recomputed).
// 8 x 4096 x 8192 bf16: 300 us with the sums' launch, 5.4 TB/s of 6 bytes an element.
template <typename D, bool VEC, int W, int NW>
__global__ __launch_bounds__(256, 4) void conv_grad_kernel(const ConvGradParams p) {
  using S = typename D::storage;
  constexpr int SL = W - 1, N = kLaneTokens, kPairs = 4 / NW;
  static_assert(NW == 1 || NW == 4, "a barrier is met by one pair only");
  __shared__ float sums[NW][W + 1];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int sub = wave % NW;
  const int64_t pair = (int64_t)xcd_groups<8>(blockIdx.x, gridDim.x) * kPairs + wave / NW;
  if (pair >= p.num_pairs) return;
  const int b = (int)(pair / p.dim), c = (int)(pair - (int64_t)b * p.dim);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  float* part = p.partial + pair * (W + 1);
  if (slot == p.pad_slot_id) {
    if (sub == 0 && lane <= W) part[lane] = 0.f;
    return;
  }
  const int64_t start = p.qsl[b], end = p.qsl[b + 1];
  const bool init = p.initial && p.has_init && p.has_init[b] != 0;
  Head<D, W> q;
  q.x = static_cast<const S*>(p.x) + c * p.x_sc;
  q.g = static_cast<const S*>(p.dout) + c * p.do_sc;
  q.x_st = p.x_st;
  q.g_st = p.do_st;
  q.start = start;
  q.end = end;
  q.silu = p.silu;
  q.bias = p.bias ? load_as_float<D>(static_cast<const S*>(p.bias) + c) : 0.f;
  float dfv[W], acc[W + 1];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    q.w[k] = load_as_float<D>(static_cast<const S*>(p.w) + c * p.w_sc + k * p.w_sk);
    q.s0[k] = k < SL && init ? load_as_float<D>(static_cast<const S*>(p.initial) + slot * p.is_slot +
                                                c * p.is_c + k * p.is_k) : 0.f;
    dfv[k] = k < SL && p.dfinal ? load_as_float<D>(static_cast<const S*>(p.dfinal) + slot * p.df_slot +
                                                   c * p.df_c + k * p.df_k) : 0.f;
    acc[k] = 0.f;
  }
  acc[W] = 0.f;
  S* dx = static_cast<S*>(p.dx) + c * p.dx_sc;

  // this wave's run of chunks [c_lo, c_hi), counted from the start
  const int64_t chunks = (end - start + kChunkTokens - 1) / kChunkTokens;
  const int64_t per = (chunks + NW - 1) / NW;
  const int64_t c_lo = sub * per, c_hi = c_lo + per < chunks ? c_lo + per : chunks;
  Raw8<D> rx, rg;
  S before[W];  // the inputs before the chunk (uniform)
  auto fetch = [&](int64_t base) {
    const int64_t t = base + lane * N;
    rx.template load<VEC>(q.x, p.x_st, t, p.total_T);
    rg.template load<VEC>(q.g, p.do_st, t, p.total_T);
#pragma unroll
    for (int m = 0; m < SL; ++m)
      before[m] = base - SL + m >= start ? q.x[(base - SL + m) * p.x_st] : (S)0;
  };
  float next[W];  // dz of the tokens after the chunk
  if (c_hi > c_lo) {
    fetch(start + (c_hi - 1) * kChunkTokens);
    q.after(start + c_hi * kChunkTokens, next);
  }
  for (int64_t ch = c_hi - 1; ch >= c_lo; --ch) {
    const int64_t base = start + ch * kChunkTokens, t = base + lane * N;
    float u[SL + N], dz[N + SL];
    {
      float f[N];
      rx.to_float(f);
#pragma unroll
      for (int e = 0; e < N; ++e) u[SL + e] = f[e];
      rg.to_float(f);
#pragma unroll
      for (int e = 0; e < N; ++e) dz[e] = f[e];
    }
    float head[W];
#pragma unroll
    for (int m = 0; m < SL; ++m) {
      head[m] = to_float<D>(before[m]);
      if (base - SL + m < start) head[m] = q.input(base - SL + m);
    }
    if (ch > c_lo) fetch(base - kChunkTokens);
    if (base + kChunkTokens > end) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        dz[e] = t + e < end ? dz[e] : 0.f;
        u[SL + e] = t + e < end ? u[SL + e] : 0.f;
      }
    }
#pragma unroll
    for (int m = 0; m < SL; ++m) u[m] = lane_move<0x138>(head[m], u[N + m]);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float z = q.bias;
#pragma unroll
      for (int k = 0; k < W; ++k) z = __builtin_fmaf(q.w[k], u[e + k], z);
      if (p.silu) dz[e] = silu_grad(z, dz[e]);
#pragma unroll
      for (int k = 0; k < W; ++k) acc[k] = __builtin_fmaf(dz[e], u[e + k], acc[k]);
      acc[W] += dz[e];
    }
#pragma unroll
    for (int m = 0; m < SL; ++m) {
      dz[N + m] = lane_move<0x130>(next[m], dz[m]);  // from the lane above
      next[m] = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(dz[m])));
    }
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      y[e] = 0.f;
#pragma unroll
      for (int l = 0; l < W; ++l) y[e] = __builtin_fmaf(q.w[W - 1 - l], dz[e + l], y[e]);
    }
    if (base + kChunkTokens > end - SL) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int64_t m = t + e - (end - SL);
        if (m >= 0 && m < SL) y[e] += pick(dfv, (int)m);
      }
    }
    Raw8<D> o;
    o.from_float(y);
    o.template store<VEC>(dx, p.dx_st, t, end);
  }
#pragma unroll
  for (int k = 0; k <= W; ++k) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) acc[k] += __shfl_xor(acc[k], d, 64);
  }
  if constexpr (NW > 1) {
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k <= W; ++k) sums[sub][k] = acc[k];
    }
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
      acc[k] = 0.f;
#pragma unroll
      for (int s = 0; s < NW; ++s) acc[k] += sums[s][k];
    }
  }
  if (sub != 0 || lane != 0) return;
#pragma unroll
  for (int k = 0; k <= W; ++k) part[k] = acc[k];
  if (SL > 0 && p.dinitial) {
    float dz[W];
    q.after(start, dz);
    S* di = static_cast<S*>(p.dinitial) + slot * p.di_slot + c * p.di_c;
    const int64_t L = end - start;
#pragma unroll
    for (int j = 0; j < SL; ++j) {  // logical index j - SL
      float du = 0.f;
#pragma unroll
      for (int l = SL - j; l < W; ++l) du = __builtin_fmaf(q.w[W - 1 - l], dz[j - SL + l], du);
      if (j >= L) du += pick(dfv, (int)(j - L));
      di[j * p.di_k] = init ? round_to<D>(du) : (S)0;
    }
  }
}

// Channels in lanes (rows of tokens): a wave walks a strip of rows forward
// with the last W inputs and dz of its V channels in registers; du_i is
// complete once dz_{i+W-1} is known, so a strip reads W-1 rows before it and
// W-1 after it again.  Strips lie on the flat token axis, whatever the
// sequences' lengths: a wave takes every sequence that its strip meets.
// 17409 x 4096 bf16: 115 us (83 at a copy's rate); 5003 x 1021 fp32: 19 us,
// the latency of a strip's chain of loads.  Ordinary stores: what reads dx next
// finds a small plane in the caches (with a copy of dx after it, ordinary and
// streaming: 5003 x 1021 fp32 27.6 and 29.2 us, 2048 x 4096 bf16 37.9 and 39.1; past
// the caches streaming wins, 17408 x 4096 175.7 and 171.8).
constexpr int kStripWaves = 4, kStripGroup = 8;

template <typename D, int V, int W>
__global__ __launch_bounds__(kStripWaves * 64) void conv_grad_rows_kernel(const ConvGradParams p) {
  using S = typename D::storage;
  using P = Pack<D, V>;
  constexpr int SL = W - 1, G = kStripGroup;
  __shared__ float sums[kStripWaves][W + 1][64 * V];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t slabs = (uint32_t)((p.dim + 64 * V - 1) / (64 * V));
  const uint32_t wg = xcd_contiguous(blockIdx.x, gridDim.x);
  const int seg = (int)(wg / slabs), total = (int)p.total_T;
  const int ch = ((int)(wg % slabs) * 64 + lane) * V;
  const bool live = ch < p.dim;
  const int c = live ? ch : p.dim - V;
  const int strip = seg * kStripWaves + wave;
  // The strip of the last row (of none: the first strip) also takes the
  // sequences that start at the end of the rows; strips past it are idle.
  const bool used = strip == 0 || (int64_t)strip * p.strip < total;
  const int lo = used ? strip * p.strip : total;
  const bool last = used && total - lo <= p.strip;
  const int hi = last ? total : used ? lo + p.strip : lo;
  const uint32_t off = (uint32_t)c * (uint32_t)sizeof(S);
  float w[W][V], bias[V], acc[W + 1][V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = p.bias ? load_as_float<D>(static_cast<const S*>(p.bias) + c + v) : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k)
      w[k][v] = load_as_float<D>(static_cast<const S*>(p.w) + (c + v) * p.w_sc + k * p.w_sk);
#pragma unroll
    for (int k = 0; k <= W; ++k) acc[k][v] = 0.f;
  }
  const S* x = static_cast<const S*>(p.x);
  const S* g = static_cast<const S*>(p.dout);
  S* dx = static_cast<S*>(p.dx);
  for (int b = used ? first_sequence(p.qsl, p.batch, lo) : p.batch; b < p.batch; ++b) {
    const int start = p.qsl[b], end = p.qsl[b + 1];
    if (start >= hi && !(last && p.dinitial)) break;  // an empty one has no other gradient
    const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
    const bool mine_first = start >= lo && (start < hi || last);
    const int from = start > lo ? start : lo, to = end < hi ? end : hi;
    if (slot == p.pad_slot_id || (from >= to && !(start == end && mine_first))) continue;
    const bool init = p.initial && p.has_init && p.has_init[b] != 0;
    auto state = [&](int i, int v) {  // initial state, logical index i in [-SL, 0)
      return init && i >= -SL ? load_as_float<D>(static_cast<const S*>(p.initial) + slot * p.is_slot +
                                                 (c + v) * p.is_c + (i + SL) * p.is_k) : 0.f;
    };
    float u[W][V], dz[W][V];
#pragma unroll
    for (int m = 0; m < W; ++m) {
#pragma unroll
      for (int v = 0; v < V; ++v) u[m][v] = dz[m][v] = 0.f;
      if (m >= 1) {  // u[1..SL]: the inputs before `from`
        const int t = from - W + m;
        if (t >= start) {
          P r;
          r.load(in_row(x + (int64_t)t * p.x_st, off));
          r.to_float(u[m]);
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) u[m][v] = state(t - start, v);
        }
      }
    }
    P rx[G], rg[G];
    auto fetch = [&](int t0) {
      load_rows(rx, x, p.x_st, t0, end, off);
      load_rows(rg, g, p.do_st, t0, end, off);
    };
    if (end > start) {
      fetch(from);
    } else {
#pragma unroll
      for (int r = 0; r < G; ++r) {
        rx[r].zero();
        rg[r].zero();
      }
    }
    for (int t0 = from; t0 < to + SL; t0 += G) {
      P cx[G], cg[G];
#pragma unroll
      for (int r = 0; r < G; ++r) {
        cx[r] = rx[r];
        cg[r] = rg[r];
      }
      if (t0 + G < to + SL && end > start) fetch(t0 + G);
#pragma unroll
      for (int r = 0; r < G; ++r) {
        const int t = t0 + r, i = t - SL;
        if (t >= to + SL) break;
        const bool in = t < end;
        float gf[V], xf[V], du[V];
        cx[r].to_float(xf);
        cg[r].to_float(gf);
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int k = 0; k + 1 < W; ++k) {
            u[k][v] = u[k + 1][v];
            dz[k][v] = dz[k + 1][v];
          }
          u[SL][v] = in ? xf[v] : 0.f;
          float z = bias[v];
#pragma unroll
          for (int k = 0; k < W; ++k) z = __builtin_fmaf(w[k][v], u[k][v], z);
          const float d = p.silu ? silu_grad(z, gf[v]) : gf[v];
          dz[SL][v] = in ? d : 0.f;
          const float own = t < to ? dz[SL][v] : 0.f;  // the rows after the strip are another's
#pragma unroll
          for (int k = 0; k < W; ++k) acc[k][v] = __builtin_fmaf(own, u[k][v], acc[k][v]);
          acc[W][v] += own;
          du[v] = 0.f;
#pragma unroll
          for (int l = 0; l < W; ++l) du[v] = __builtin_fmaf(w[W - 1 - l][v], dz[l][v], du[v]);
        }
        if (p.dfinal && i >= end - SL) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            du[v] += load_as_float<D>(static_cast<const S*>(p.dfinal) + slot * p.df_slot +
                                      (c + v) * p.df_c + (i - (end - SL)) * p.df_k);
        }
        if (i >= from) {
          P o;
          o.from_float(du);
          if (live) o.store(in_row(dx + (int64_t)i * p.dx_st, off));
        } else if (i < start && mine_first && p.dinitial && live) {
          S* di = static_cast<S*>(p.dinitial) + slot * p.di_slot + (i - start + SL) * p.di_k;
#pragma unroll
          for (int v = 0; v < V; ++v) di[(c + v) * p.di_c] = init ? round_to<D>(du[v]) : (S)0;
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k <= W; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) sums[wave][k][lane * V + v] = acc[k][v];
  }
  __syncthreads();
  if (wave != 0 || !live) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k <= W; ++k) {
      float a = 0.f;
#pragma unroll
      for (int s = 0; s < kStripWaves; ++s) a += sums[s][k][lane * V + v];
      p.partial[((int64_t)seg * p.dim + c + v) * (W + 1) + k] = a;
    }
  }
}

__global__ __launch_bounds__(kSumCols * kSumGroups) void conv_grad_sum_kernel(
    const float* partial, float* dweight, float* dbias, int32_t batch, int32_t dim, int32_t W) {
  column_sum(partial, batch, (int64_t)dim * (W + 1), [&](int64_t id, float v) {
    const int64_t c = id / (W + 1);
    const int k = (int)(id - c * (W + 1));
    if (k < W) dweight[c * W + k] = v;
    else if (dbias) dbias[c] = v;
  });
}

template <typename D, bool VEC, int NW>
static void launch_grad(int W, const ConvGradParams& p, uint32_t grid, hipStream_t s) {
  const dim3 g(grid), th(256);
  switch (W) {
    case 1: hipLaunchKernelGGL((conv_grad_kernel<D, VEC, 1, NW>), g, th, 0, s, p); break;
    case 2: hipLaunchKernelGGL((conv_grad_kernel<D, VEC, 2, NW>), g, th, 0, s, p); break;
    case 3: hipLaunchKernelGGL((conv_grad_kernel<D, VEC, 3, NW>), g, th, 0, s, p); break;
    default: hipLaunchKernelGGL((conv_grad_kernel<D, VEC, 4, NW>), g, th, 0, s, p); break;
  }
}

template <typename D, int V>
static void launch_grad_rows(int W, const ConvGradParams& p, uint32_t grid, hipStream_t s) {
  const dim3 g(grid), th(kStripWaves * 64);
  switch (W) {
    case 1: hipLaunchKernelGGL((conv_grad_rows_kernel<D, V, 1>), g, th, 0, s, p); break;
    case 2: hipLaunchKernelGGL((conv_grad_rows_kernel<D, V, 2>), g, th, 0, s, p); break;
    case 3: hipLaunchKernelGGL((conv_grad_rows_kernel<D, V, 3>), g, th, 0, s, p); break;
    default: hipLaunchKernelGGL((conv_grad_rows_kernel<D, V, 4>), g, th, 0, s, p); break;
  }
}

// Rows of a strip: long strips read fewer rows twice, short ones keep a
// small batch's chain short (5003 x 1021 fp32: 16 rows 21 us, 32 22, 64 26,
// 128 38; 17409 x 4096 bf16: 143, 117, 115, 127).
static int64_t strip_rows(int64_t total_T, int32_t dim) {
  return total_T * dim >= (int64_t)1 << 23 ? 64 : 16;
}

static int64_t grad_segments(int64_t total_T, int32_t dim) {
  const int64_t n = cdiv(total_T, strip_rows(total_T, dim) * kStripWaves);
  return n > 0 ? n : 1;  // sequences without tokens still have state gradients
}

// Parts of the workspace: the larger of the two kernels' counts, so that its
// size does not depend on strides.
static int64_t grad_floats(int64_t total_T, int32_t batch, int32_t dim, int32_t W) {
  const int64_t s = grad_segments(total_T, dim), parts = batch == 0 ? 0 : s > batch ? s : batch;
  return parts * dim * (W + 1);
}

}  // namespace sconv

extern "C" int causal_conv1d_varlen_bwd_workspace(int64_t total_T, int32_t batch, int32_t dim,
                                                  int32_t W, int64_t* floats) {
  using namespace sconv;
  clear_error();
  if (total_T < 0 || batch < 0 || dim < 0 || W < 1 || W > 4 || !floats)
    return fail(SCONV_ERR_INVALID, "causal_conv1d_varlen_bwd_workspace: sizes must be >= 0, W in "
                                   "[1, 4], floats not NULL");
  *floats = grad_floats(total_T, batch, dim, W);
  return SCONV_OK;
}

extern "C" int causal_conv1d_varlen_bwd(
    const void* dout, int64_t do_stride_c, int64_t do_stride_t, const void* x,
    int64_t x_stride_c, int64_t x_stride_t, const void* weight, int64_t w_stride_c,
    int64_t w_stride_k, const void* bias, const void* initial_states, int64_t is_stride_slot,
    int64_t is_stride_c, int64_t is_stride_k, int64_t num_slots, const int32_t* query_start_loc,
    int32_t batch, const int32_t* cache_indices, const uint8_t* has_initial_state,
    const void* dfinal_states, int64_t df_stride_slot, int64_t df_stride_c, int64_t df_stride_k,
    void* dinitial_states, int64_t di_stride_slot, int64_t di_stride_c, int64_t di_stride_k,
    void* dx, int64_t dx_stride_c, int64_t dx_stride_t, float* dweight, float* dbias,
    float* workspace, int64_t workspace_floats, int32_t dim, int64_t total_T, int32_t W,
    int32_t dtype, int32_t activation, int32_t pad_slot_id, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "causal_conv1d_varlen_bwd";
  if (batch < 0 || dim < 0 || total_T < 0)
    return fail(SCONV_ERR_INVALID, "%s: batch, dim and total_T must be >= 0", fn);
  if (total_T > INT32_MAX - 4096)  // token numbers are int32, as the offsets
    return fail(SCONV_ERR_UNSUPPORTED, "%s: total_T too large", fn);
  if (dim > 1 << 28)  // a lane's byte offset in a row is 32 bits
    return fail(SCONV_ERR_UNSUPPORTED, "%s: dim too large", fn);
  if (W < 1 || W > 4) return fail(SCONV_ERR_INVALID, "%s: W=%d outside [1, 4]", fn, W);
  if (!valid_dtype(dtype)) return fail(SCONV_ERR_INVALID, "%s: unknown dtype %d", fn, dtype);
  if (!valid_act(activation))
    return fail(SCONV_ERR_INVALID, "%s: unknown activation %d", fn, activation);
  if (dim == 0) return SCONV_OK;
  if (!weight || !dweight || (batch > 0 && (!query_start_loc || !workspace)) ||
      (batch > 0 && total_T > 0 && (!dout || !x || !dx)))
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  if (has_initial_state && !initial_states && W > 1)
    return fail(SCONV_ERR_INVALID, "%s: has_initial_state without initial_states", fn);
  if (W == 1) initial_states = dfinal_states = dinitial_states = nullptr;  // no state
  const bool any = initial_states || dfinal_states || dinitial_states;
  if (any && (num_slots < 1 || (!cache_indices && num_slots < batch)))
    return fail(SCONV_ERR_INVALID, "%s: state pool has fewer slots than needed", fn);
  if (w_stride_c < 0 || w_stride_k < 0 ||
      (initial_states && (is_stride_slot < 0 || is_stride_c < 0 || is_stride_k < 0)) ||
      (dfinal_states && (df_stride_slot < 0 || df_stride_c < 0 || df_stride_k < 0)) ||
      (dinitial_states && (di_stride_slot < 1 || di_stride_c < 1 || di_stride_k < 1)))
    return fail(SCONV_ERR_INVALID, "%s: strides too small", fn);
  const int64_t need = grad_floats(total_T, batch, dim, W);
  if (workspace_floats < need)
    return fail(SCONV_ERR_INVALID, "%s: workspace holds %lld floats, %lld needed", fn,
                (long long)workspace_floats, (long long)need);
  const int64_t es = elem_size(dtype);
  const Plane pg = plane(dout, do_stride_c, do_stride_t, dim, total_T, es);
  const Plane px = plane(x, x_stride_c, x_stride_t, dim, total_T, es);
  const Plane po = plane(dx, dx_stride_c, dx_stride_t, dim, total_T, es);
  if (!pg.readable() || !px.readable())
    return fail(SCONV_ERR_INVALID, "%s: strides must be >= 0", fn);
  if (!po.writable()) return fail(SCONV_ERR_INVALID, "%s: dx's elements overlap each other", fn);
  if (planes_overlap(po, pg) || planes_overlap(po, px))
    return fail(SCONV_ERR_INVALID, "%s: dx overlaps dout or x", fn);
  auto pool = [&](const void* q, int64_t ss, int64_t sc, int64_t sk) {
    return q ? ((num_slots - 1) * ss + (dim - 1) * sc + (W - 2) * sk + 1) * es : (int64_t)0;
  };
  struct Span { const void* p; int64_t n; };
  const Span rd[7] = {{dout, pg.bytes()}, {x, px.bytes()},
                      {weight, ((dim - 1) * w_stride_c + (W - 1) * w_stride_k + 1) * es},
                      {bias, bias ? dim * es : 0},
                      {initial_states, pool(initial_states, is_stride_slot, is_stride_c, is_stride_k)},
                      {dfinal_states, pool(dfinal_states, df_stride_slot, df_stride_c, df_stride_k)},
                      {nullptr, 0}};
  const Span wr[5] = {{dx, po.bytes()},
                      {dinitial_states, pool(dinitial_states, di_stride_slot, di_stride_c, di_stride_k)},
                      {dweight, (int64_t)dim * W * 4}, {dbias, dbias ? (int64_t)dim * 4 : 0},
                      {workspace, need * 4}};
  for (int i = 0; i < 5; ++i) {
    bool bad = false;
    for (int j = i == 0 ? 2 : 0; j < 6; ++j)  // dx against dout and x: done above
      bad = bad || overlap(wr[i].p, wr[i].n, rd[j].p, rd[j].n);
    for (int j = 0; j < i; ++j) bad = bad || overlap(wr[i].p, wr[i].n, wr[j].p, wr[j].n);
    if (bad) return fail(SCONV_ERR_INVALID, "%s: an output or the workspace overlaps another buffer", fn);
  }
  ConvGradParams p = {};
  p.dout = dout; p.x = x; p.w = weight; p.bias = bias; p.initial = initial_states;
  p.qsl = query_start_loc; p.cache_indices = cache_indices; p.has_init = has_initial_state;
  p.dfinal = dfinal_states; p.dinitial = dinitial_states; p.dx = dx; p.partial = workspace;
  p.do_sc = pg.sc; p.do_st = pg.st; p.x_sc = px.sc; p.x_st = px.st; p.w_sc = w_stride_c;
  p.w_sk = w_stride_k; p.dx_sc = po.sc; p.dx_st = po.st; p.is_slot = is_stride_slot;
  p.is_c = is_stride_c; p.is_k = is_stride_k; p.df_slot = df_stride_slot; p.df_c = df_stride_c;
  p.df_k = df_stride_k; p.di_slot = di_stride_slot; p.di_c = di_stride_c; p.di_k = di_stride_k;
  p.total_T = total_T; p.num_pairs = (int64_t)batch * dim; p.batch = batch; p.dim = dim;
  p.silu = activation == SCONV_ACT_SILU; p.pad_slot_id = pad_slot_id;
  const bool rows = dim > 1 && pg.sc == 1 && px.sc == 1 && po.sc == 1;
  int64_t parts = batch, grid = 0;
  int NW = 1, V = 1;
  bool vec = false;
  if (rows) {
    auto lanes = [&](const Plane& a) { return a.st % 2 == 0 && aligned_to(a.p, 2 * es); };
    V = dim % 2 == 0 && lanes(pg) && lanes(px) && lanes(po) ? 2 : 1;
    p.strip = (int32_t)strip_rows(total_T, dim);
    parts = grad_segments(total_T, dim);
    grid = parts * cdiv(dim, 64 * V);
  } else {
    vec = pg.st == 1 && px.st == 1 && po.st == 1;
    // Few (sequence, channel) pairs of several chunks: four waves for each.  With
    // four and with one, us: 1 x 65536 x 512 bf16 49 and 119, 1 x 8192 x 1024 18.5 and
    // 22.0, 2 x 4096 x 1024 21 and 18 (fp32 24 and 25), 2 x 8192 x 1024 27.5 and 28.2,
    // 3 x 4096 x 1024 25 and 21 (38 and 35), 6 x 1024 x 1024 27 and 18 (26 and 19),
    // 6 x 4096 x 1024 53 and 34 (69 both).
    NW = p.num_pairs < 2048 && total_T / (batch ? batch : 1) >= 2 * kChunkTokens ? 4 : 1;
    grid = cdiv(p.num_pairs, 4 / NW);
  }
  const int64_t sums = cdiv((int64_t)dim * (W + 1), kSumCols);
  if ((batch > 0 && !valid_grid(grid, 256)) || !valid_grid(sums, kSumCols * kSumGroups))
    return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
  if (batch > 0) {
    const uint32_t g = (uint32_t)grid;
    if (rows) {
      if (dtype == SCONV_BF16) {
        if (V == 2) launch_grad_rows<Bf16, 2>(W, p, g, stream);
        else launch_grad_rows<Bf16, 1>(W, p, g, stream);
      } else {
        if (V == 2) launch_grad_rows<F32, 2>(W, p, g, stream);
        else launch_grad_rows<F32, 1>(W, p, g, stream);
      }
    } else if (dtype == SCONV_BF16) {
      if (vec && NW == 1) launch_grad<Bf16, true, 1>(W, p, g, stream);
      else if (vec) launch_grad<Bf16, true, 4>(W, p, g, stream);
      else if (NW == 1) launch_grad<Bf16, false, 1>(W, p, g, stream);
      else launch_grad<Bf16, false, 4>(W, p, g, stream);
    } else {
      if (vec && NW == 1) launch_grad<F32, true, 1>(W, p, g, stream);
      else if (vec) launch_grad<F32, true, 4>(W, p, g, stream);
      else if (NW == 1) launch_grad<F32, false, 1>(W, p, g, stream);
      else launch_grad<F32, false, 4>(W, p, g, stream);
    }
    if (const int rc = check_launch(fn)) return rc;
  }
  hipLaunchKernelGGL(conv_grad_sum_kernel, dim3((uint32_t)sums), dim3(kSumCols * kSumGroups), 0,
                     stream, workspace,
                     dweight, dbias, (int32_t)(batch > 0 ? parts : 0), dim, W);
  return check_launch(fn);
}
