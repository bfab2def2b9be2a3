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
#include "sconv_host.h"

namespace sconv {

struct ConvGradParams {
  const void *dout, *x, *w, *bias, *initial;
  const int32_t* qsl;
  const int32_t* cache_indices;
  const uint8_t* has_init;
  const void* dfinal;
  void *dinitial, *dx;
  float* partial;  // [batch, dim, W + 1]: dw, dbias of one sequence
  int64_t do_sc, do_st, x_sc, x_st, w_sc, w_sk, dx_sc, dx_st;
  int64_t is_slot, is_c, is_k, df_slot, df_c, df_k, di_slot, di_c, di_k;
  int64_t total_T, num_pairs;
  int32_t batch, dim, silu, pad_slot_id;
};

template <typename D>
__device__ __forceinline__ typename D::storage rounded(float v) {
  if constexpr (sizeof(typename D::storage) == 2)
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    return v;
}

// dout * d silu(z) / dz
__device__ __forceinline__ float silu_grad(float z, float g) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  return g * s * __builtin_fmaf(z, 1.0f - s, 1.0f);
}

// One thread per (sequence, channel), token by token: du_i is complete once
// dz_{i+W-1} is known.
template <typename D, int W>
__global__ __launch_bounds__(64) void conv_grad_simple(const ConvGradParams p) {
  using S = typename D::storage;
  constexpr int SL = W - 1;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (id >= p.num_pairs) return;
  const int b = (int)(id / p.dim), c = (int)(id - (int64_t)b * p.dim);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  float* part = p.partial + id * (W + 1);
  if (slot == p.pad_slot_id) {
#pragma unroll
    for (int k = 0; k <= W; ++k) part[k] = 0.f;
    return;
  }
  const int64_t start = p.qsl[b], L = p.qsl[b + 1] - start;
  const bool init = p.initial && p.has_init && p.has_init[b] != 0;
  const S* x = static_cast<const S*>(p.x) + c * p.x_sc + start * p.x_st;
  const S* g = static_cast<const S*>(p.dout) + c * p.do_sc + start * p.do_st;
  S* dx = static_cast<S*>(p.dx) + c * p.dx_sc + start * p.dx_st;
  const S* df = p.dfinal ? static_cast<const S*>(p.dfinal) + slot * p.df_slot + c * p.df_c : nullptr;
  S* di = p.dinitial ? static_cast<S*>(p.dinitial) + slot * p.di_slot + c * p.di_c : nullptr;
  float w[W], u[W], dz[W], dw[W], db = 0.f;
  const float bias = p.bias ? load_as_float<D>(static_cast<const S*>(p.bias) + c) : 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    w[k] = load_as_float<D>(static_cast<const S*>(p.w) + c * p.w_sc + k * p.w_sk);
    dw[k] = dz[k] = u[k] = 0.f;
  }
#pragma unroll
  for (int m = 0; m < SL; ++m)  // u[W-1] is the current token's input
    if (init) u[m + 1] = load_as_float<D>(static_cast<const S*>(p.initial) + slot * p.is_slot + c * p.is_c + m * p.is_k);
  float dfv[W];
#pragma unroll
  for (int m = 0; m < SL; ++m) dfv[m] = df ? load_as_float<D>(df + m * p.df_k) : 0.f;
  for (int64_t t = 0; t < L + SL; ++t) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      u[k] = u[k + 1];
      dz[k] = dz[k + 1];
    }
    u[W - 1] = 0.f;
    dz[W - 1] = 0.f;
    if (t < L) {
      u[W - 1] = load_as_float<D>(x + t * p.x_st);
      float z = bias;
#pragma unroll
      for (int k = 0; k < W; ++k) z = __builtin_fmaf(w[k], u[k], z);
      const float gv = load_as_float<D>(g + t * p.do_st);
      dz[W - 1] = p.silu ? silu_grad(z, gv) : gv;
#pragma unroll
      for (int k = 0; k < W; ++k) dw[k] = __builtin_fmaf(dz[W - 1], u[k], dw[k]);
      db += dz[W - 1];
    }
    const int64_t i = t - SL;  // dz[l] = dz_{i+l}
    float du = 0.f;
#pragma unroll
    for (int l = 0; l < W; ++l) du = __builtin_fmaf(w[W - 1 - l], dz[l], du);
#pragma unroll
    for (int m = 0; m < SL; ++m)
      if (i == L - SL + m) du += dfv[m];
    if (i >= 0) dx[i * p.dx_st] = rounded<D>(du);
    else if (di) di[(i + SL) * p.di_k] = init ? rounded<D>(du) : rounded<D>(0.f);
  }
#pragma unroll
  for (int k = 0; k < W; ++k) part[k] = dw[k];
  part[W] = db;
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

template <typename D>
static void launch_conv_grad(int W, const ConvGradParams& p, uint32_t grid, hipStream_t s) {
  switch (W) {
    case 1: hipLaunchKernelGGL((conv_grad_simple<D, 1>), dim3(grid), dim3(64), 0, s, p); break;
    case 2: hipLaunchKernelGGL((conv_grad_simple<D, 2>), dim3(grid), dim3(64), 0, s, p); break;
    case 3: hipLaunchKernelGGL((conv_grad_simple<D, 3>), dim3(grid), dim3(64), 0, s, p); break;
    default: hipLaunchKernelGGL((conv_grad_simple<D, 4>), dim3(grid), dim3(64), 0, s, p); break;
  }
}

}  // namespace sconv

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
  const int64_t need = (int64_t)batch * dim * (W + 1);
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
  const int64_t grid = cdiv(p.num_pairs, 64), sums = cdiv((int64_t)dim * (W + 1), kSumCols);
  if ((batch > 0 && !valid_grid(grid, 64)) || !valid_grid(sums, kSumCols * kSumGroups))
    return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
  if (batch > 0) {
    if (dtype == SCONV_BF16) launch_conv_grad<Bf16>(W, p, (uint32_t)grid, stream);
    else launch_conv_grad<F32>(W, p, (uint32_t)grid, stream);
    if (const int rc = check_launch(fn)) return rc;
  }
  hipLaunchKernelGGL(conv_grad_sum_kernel, dim3((uint32_t)sums), dim3(kSumCols * kSumGroups), 0,
                     stream, workspace,
                     dweight, dbias, batch, dim, W);
  return check_launch(fn);
}
