// gated_recurrence.hip -- gated linear recurrence over packed
// variable-length sequences with a slot-indexed state pool (prefill), its
// gradients, and its one-token decode step, for gfx950.
//
// The recurrence is the layer step behind the short conv: it takes the
// conv's packing (query_start_loc), state slots and layouts.
#include "recurrence_device.h"
#include "sconv_host.h"

namespace sconv {

struct RecFwdParams {
  const void *x, *ga, *gx;
  const float* decay;
  float* states;
  const int32_t* qsl;
  const int32_t* cache_indices;
  const uint8_t* has_init;
  void* out;
  float* marks;
  int64_t x_sc, x_st, ga_sc, ga_st, gx_sc, gx_st, o_sc, o_st, ss_slot, total_T, num_pairs;
  float scale;
  int32_t batch, dim, pad_slot_id;
};

// One thread per (sequence, channel), token by token.
template <typename D>
__global__ __launch_bounds__(64) void rec_fwd_simple(const RecFwdParams p) {
  using S = typename D::storage;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (id >= p.num_pairs) return;
  const int b = (int)(id / p.dim), c = (int)(id - (int64_t)b * p.dim);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (slot == p.pad_slot_id) return;
  const Decay d = make_decay(p.decay[c], p.scale);
  const bool init = p.states && p.has_init && p.has_init[b] != 0;
  float h = init ? p.states[slot * p.ss_slot + c] : 0.f;
  const int64_t start = p.qsl[b], end = p.qsl[b + 1];
  const S* x = static_cast<const S*>(p.x) + c * p.x_sc;
  const S* ga = static_cast<const S*>(p.ga) + c * p.ga_sc;
  const S* gx = static_cast<const S*>(p.gx) + c * p.gx_sc;
  S* out = static_cast<S*>(p.out) + c * p.o_sc;
  for (int64_t t = start; t < end; ++t) {
    if (p.marks && (t == start || t % kMarkTokens == 0))
      p.marks[(t / kMarkTokens + b) * p.dim + c] = h;
    const Gates g = make_gates(load_as_float<D>(ga + t * p.ga_st), load_as_float<D>(gx + t * p.gx_st), d);
    h = __builtin_fmaf(g.a, h, g.m * (g.i * load_as_float<D>(x + t * p.x_st)));
    out[t * p.o_st] = round_to<D>(h);
  }
  if (p.states) p.states[slot * p.ss_slot + c] = h;
}

struct RecBwdParams {
  const void *dout, *x, *ga, *gx;
  const float *decay, *marks;
  const int32_t* qsl;
  const int32_t* cache_indices;
  const uint8_t* has_init;
  const float* dfinal;
  float* dinitial;
  void *dx, *dga, *dgx;
  float* partial;  // [batch, dim] sums over tokens of r * dlog a
  int64_t do_sc, do_st, x_sc, x_st, ga_sc, ga_st, gx_sc, gx_st;
  int64_t dx_sc, dx_st, dga_sc, dga_st, dgx_sc, dgx_st;
  int64_t df_slot, di_slot, total_T, num_pairs;
  float scale;
  int32_t batch, dim, pad_slot_id;
};

// One thread per (sequence, channel): block by block of 128 tokens from the
// end, the states of a block from its checkpoint, then its gradients.
template <typename D>
__global__ __launch_bounds__(64) void rec_bwd_simple(const RecBwdParams p) {
  using S = typename D::storage;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (id >= p.num_pairs) return;
  const int b = (int)(id / p.dim), c = (int)(id - (int64_t)b * p.dim);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (slot == p.pad_slot_id) {
    p.partial[id] = 0.f;
    return;
  }
  const Decay d = make_decay(p.decay[c], p.scale);
  const int64_t start = p.qsl[b], end = p.qsl[b + 1];
  const S* dout = static_cast<const S*>(p.dout) + c * p.do_sc;
  const S* x = static_cast<const S*>(p.x) + c * p.x_sc;
  const S* ga = static_cast<const S*>(p.ga) + c * p.ga_sc;
  const S* gx = static_cast<const S*>(p.gx) + c * p.gx_sc;
  S* dx = static_cast<S*>(p.dx) + c * p.dx_sc;
  S* dga = static_cast<S*>(p.dga) + c * p.dga_sc;
  S* dgx = static_cast<S*>(p.dgx) + c * p.dgx_sc;
  float s = p.dfinal ? p.dfinal[slot * p.df_slot + c] : 0.f;  // a_{t+1} dh_{t+1}
  float acc = 0.f;
  float before[kMarkTokens];
  for (int64_t blk = (end - 1) / kMarkTokens; end > start && blk >= start / kMarkTokens; --blk) {
    const int64_t lo = blk * kMarkTokens > start ? blk * kMarkTokens : start;
    const int64_t hi = (blk + 1) * kMarkTokens < end ? (blk + 1) * kMarkTokens : end;
    float h = p.marks[(blk + b) * p.dim + c];
    for (int64_t t = lo; t < hi; ++t) {
      before[t - lo] = h;
      const Gates g = make_gates(load_as_float<D>(ga + t * p.ga_st), load_as_float<D>(gx + t * p.gx_st), d);
      h = __builtin_fmaf(g.a, h, g.m * (g.i * load_as_float<D>(x + t * p.x_st)));
    }
    for (int64_t t = hi - 1; t >= lo; --t) {
      const GatesInv g = make_gates_inv(load_as_float<D>(ga + t * p.ga_st), load_as_float<D>(gx + t * p.gx_st), d);
      const float xv = load_as_float<D>(x + t * p.x_st);
      const float dh = s + load_as_float<D>(dout + t * p.do_st);
      s = g.a * dh;
      const float vx = dh * (g.m * g.i);
      const float dlog = s * (before[t - lo] - g.a * g.inv_m * (g.i * xv));
      acc = __builtin_fmaf(dlog, g.r, acc);
      dx[t * p.dx_st] = round_to<D>(vx);
      dgx[t * p.dgx_st] = round_to<D>(vx * xv * (1.f - g.i));
      dga[t * p.dga_st] = round_to<D>(-d.k * dlog * (g.r * (1.f - g.r)));
    }
  }
  p.partial[id] = acc;
  const bool init = p.has_init && p.has_init[b] != 0;
  if (p.dinitial) p.dinitial[slot * p.di_slot + c] = init ? s : 0.f;
}

// ddecay[c] = -scale sigmoid(decay[c]) * the sequences' sums, in their order.
__global__ __launch_bounds__(64) void rec_ddecay_kernel(const float* partial, const float* decay,
                                                        float* ddecay, int32_t batch, int32_t dim,
                                                        float scale) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= dim) return;
  float acc = 0.f;
  for (int b = 0; b < batch; ++b) acc += partial[(int64_t)b * dim + c];
  ddecay[c] = -scale * sigmoid(decay[c]) * acc;
}

struct RecUpdParams {
  const void *x, *ga, *gx;
  const float* decay;
  float* states;
  const int32_t* idx;
  void* out;
  int64_t x_rs, ga_rs, gx_rs, o_rs, ss_slot;
  float scale;
  int32_t batch, dim, pad_slot_id;
};

template <typename D>
__global__ __launch_bounds__(64) void rec_update_kernel(const RecUpdParams p) {
  using S = typename D::storage;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (id >= (int64_t)p.batch * p.dim) return;
  const int b = (int)(id / p.dim), c = (int)(id - (int64_t)b * p.dim);
  const int64_t slot = p.idx ? (int64_t)p.idx[b] : (int64_t)b;
  if (slot == p.pad_slot_id) return;
  const Decay d = make_decay(p.decay[c], p.scale);
  const Gates g = make_gates(load_as_float<D>(static_cast<const S*>(p.ga) + b * p.ga_rs + c),
                             load_as_float<D>(static_cast<const S*>(p.gx) + b * p.gx_rs + c), d);
  float* st = p.states + slot * p.ss_slot + c;
  const float xv = load_as_float<D>(static_cast<const S*>(p.x) + b * p.x_rs + c);
  const float h = __builtin_fmaf(g.a, *st, g.m * (g.i * xv));
  *st = h;
  static_cast<S*>(p.out)[b * p.o_rs + c] = round_to<D>(h);
}

// ---------------------------------------------------------------- host

// Checks shared by the two packed entry points; `fn` names the caller.
static int rec_check(const char* fn, int32_t batch, int32_t dim, int64_t total_T, int32_t dtype,
                     float scale) {
  if (batch < 0 || dim < 0 || total_T < 0)
    return fail(SCONV_ERR_INVALID, "%s: batch, dim and total_T must be >= 0", fn);
  if (!valid_dtype(dtype)) return fail(SCONV_ERR_INVALID, "%s: unknown dtype %d", fn, dtype);
  if (!(scale > 0.f) || !(scale <= 3.0e38f))
    return fail(SCONV_ERR_INVALID, "%s: decay_scale must be positive and finite", fn);
  return SCONV_OK;
}

static int64_t mark_rows(int64_t total_T, int32_t batch) {
  return cdiv(total_T, kMarkTokens) + batch;
}

}  // namespace sconv

extern "C" int gated_linear_recurrence_checkpoint_rows(int64_t total_T, int32_t batch,
                                                       int64_t* rows) {
  using namespace sconv;
  clear_error();
  const char* fn = "gated_linear_recurrence_checkpoint_rows";
  if (total_T < 0 || batch < 0 || !rows)
    return fail(SCONV_ERR_INVALID, "%s: total_T and batch must be >= 0, rows not NULL", fn);
  *rows = mark_rows(total_T, batch);
  return SCONV_OK;
}

extern "C" int gated_linear_recurrence_varlen_fwd(
    const void* x, int64_t x_stride_c, int64_t x_stride_t, const void* gate_a,
    int64_t ga_stride_c, int64_t ga_stride_t, const void* gate_x, int64_t gx_stride_c,
    int64_t gx_stride_t, const float* decay, float decay_scale, float* states, int64_t num_slots,
    int64_t st_stride_slot, const int32_t* query_start_loc, int32_t batch,
    const int32_t* cache_indices, const uint8_t* has_initial_state, void* out,
    int64_t out_stride_c, int64_t out_stride_t, float* checkpoints, int64_t checkpoint_rows,
    int32_t dim, int64_t total_T, int32_t dtype, int32_t pad_slot_id, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "gated_linear_recurrence_varlen_fwd";
  if (const int rc = rec_check(fn, batch, dim, total_T, dtype, decay_scale)) return rc;
  if (batch == 0 || dim == 0) return SCONV_OK;
  if (!query_start_loc || !decay || (total_T > 0 && (!x || !gate_a || !gate_x || !out)))
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  if (!states && has_initial_state)
    return fail(SCONV_ERR_INVALID, "%s: has_initial_state without states", fn);
  if (states && (num_slots < 1 || (!cache_indices && num_slots < batch)))
    return fail(SCONV_ERR_INVALID, "%s: state pool has fewer slots than needed", fn);
  if (states && st_stride_slot < dim && num_slots > 1)
    return fail(SCONV_ERR_INVALID, "%s: state slot stride smaller than dim", fn);
  if (checkpoints && checkpoint_rows < mark_rows(total_T, batch))
    return fail(SCONV_ERR_INVALID, "%s: checkpoints hold %lld rows, %lld needed", fn,
                (long long)checkpoint_rows, (long long)mark_rows(total_T, batch));
  const int64_t es = elem_size(dtype);
  const Plane px = plane(x, x_stride_c, x_stride_t, dim, total_T, es);
  const Plane pa = plane(gate_a, ga_stride_c, ga_stride_t, dim, total_T, es);
  const Plane pg = plane(gate_x, gx_stride_c, gx_stride_t, dim, total_T, es);
  const Plane po = plane(out, out_stride_c, out_stride_t, dim, total_T, es);
  if (!px.readable() || !pa.readable() || !pg.readable())
    return fail(SCONV_ERR_INVALID, "%s: strides must be >= 0", fn);
  if (!po.writable()) return fail(SCONV_ERR_INVALID, "%s: out's elements overlap each other", fn);
  if (!same_plane(po, px) && planes_overlap(po, px))
    return fail(SCONV_ERR_INVALID, "%s: out partially overlaps x", fn);
  if (planes_overlap(po, pa) || planes_overlap(po, pg))
    return fail(SCONV_ERR_INVALID, "%s: out overlaps a gate", fn);
  const int64_t sb = states ? ((num_slots - 1) * st_stride_slot + dim) * 4 : 0;
  const int64_t mb = checkpoints ? mark_rows(total_T, batch) * dim * 4 : 0;
  if (overlap(states, sb, x, px.bytes()) || overlap(states, sb, gate_a, pa.bytes()) ||
      overlap(states, sb, gate_x, pg.bytes()) || overlap(states, sb, out, po.bytes()) ||
      overlap(checkpoints, mb, x, px.bytes()) || overlap(checkpoints, mb, gate_a, pa.bytes()) ||
      overlap(checkpoints, mb, gate_x, pg.bytes()) || overlap(checkpoints, mb, out, po.bytes()) ||
      overlap(checkpoints, mb, states, sb))
    return fail(SCONV_ERR_INVALID, "%s: states or checkpoints overlap another buffer", fn);
  RecFwdParams p = {};
  p.x = x; p.ga = gate_a; p.gx = gate_x; p.decay = decay; p.states = states;
  p.qsl = query_start_loc; p.cache_indices = cache_indices; p.has_init = has_initial_state;
  p.out = out; p.marks = checkpoints;
  p.x_sc = px.sc; p.x_st = px.st; p.ga_sc = pa.sc; p.ga_st = pa.st; p.gx_sc = pg.sc;
  p.gx_st = pg.st; p.o_sc = po.sc; p.o_st = po.st; p.ss_slot = st_stride_slot;
  p.total_T = total_T; p.num_pairs = (int64_t)batch * dim; p.scale = decay_scale;
  p.batch = batch; p.dim = dim; p.pad_slot_id = pad_slot_id;
  const int64_t grid = cdiv(p.num_pairs, 64);
  if (!valid_grid(grid, 64)) return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
  if (dtype == SCONV_BF16)
    hipLaunchKernelGGL(rec_fwd_simple<Bf16>, dim3((uint32_t)grid), dim3(64), 0, stream, p);
  else
    hipLaunchKernelGGL(rec_fwd_simple<F32>, dim3((uint32_t)grid), dim3(64), 0, stream, p);
  return check_launch(fn);
}

extern "C" int gated_linear_recurrence_varlen_bwd(
    const void* dout, int64_t do_stride_c, int64_t do_stride_t, const void* x,
    int64_t x_stride_c, int64_t x_stride_t, const void* gate_a, int64_t ga_stride_c,
    int64_t ga_stride_t, const void* gate_x, int64_t gx_stride_c, int64_t gx_stride_t,
    const float* decay, float decay_scale, const float* checkpoints, int64_t checkpoint_rows,
    const int32_t* query_start_loc, int32_t batch, const int32_t* cache_indices,
    const uint8_t* has_initial_state, int64_t num_slots, const float* dfinal_states,
    int64_t df_stride_slot, float* dinitial_states, int64_t di_stride_slot, void* dx,
    int64_t dx_stride_c, int64_t dx_stride_t, void* dgate_a, int64_t dga_stride_c,
    int64_t dga_stride_t, void* dgate_x, int64_t dgx_stride_c, int64_t dgx_stride_t,
    float* ddecay, float* workspace, int64_t workspace_floats, int32_t dim, int64_t total_T,
    int32_t dtype, int32_t pad_slot_id, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "gated_linear_recurrence_varlen_bwd";
  if (const int rc = rec_check(fn, batch, dim, total_T, dtype, decay_scale)) return rc;
  if (dim == 0) return SCONV_OK;
  if (!decay || !ddecay ||
      (batch > 0 && (!query_start_loc || !workspace || !checkpoints)) ||
      (batch > 0 && total_T > 0 &&
       (!dout || !x || !gate_a || !gate_x || !dx || !dgate_a || !dgate_x)))
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  if ((dfinal_states || dinitial_states) &&
      (num_slots < 1 || (!cache_indices && num_slots < batch)))
    return fail(SCONV_ERR_INVALID, "%s: state gradients have fewer slots than needed", fn);
  if (num_slots > 1 && ((dfinal_states && df_stride_slot < dim) ||
                        (dinitial_states && di_stride_slot < dim)))
    return fail(SCONV_ERR_INVALID, "%s: state slot stride smaller than dim", fn);
  if (batch > 0 && checkpoint_rows < mark_rows(total_T, batch))
    return fail(SCONV_ERR_INVALID, "%s: checkpoints hold %lld rows, %lld needed", fn,
                (long long)checkpoint_rows, (long long)mark_rows(total_T, batch));
  if (batch > 0 && workspace_floats < (int64_t)batch * dim)
    return fail(SCONV_ERR_INVALID, "%s: workspace holds %lld floats, %lld needed", fn,
                (long long)workspace_floats, (long long)batch * dim);
  const int64_t es = elem_size(dtype);
  const Plane in[4] = {plane(dout, do_stride_c, do_stride_t, dim, total_T, es),
                       plane(x, x_stride_c, x_stride_t, dim, total_T, es),
                       plane(gate_a, ga_stride_c, ga_stride_t, dim, total_T, es),
                       plane(gate_x, gx_stride_c, gx_stride_t, dim, total_T, es)};
  const Plane ou[3] = {plane(dx, dx_stride_c, dx_stride_t, dim, total_T, es),
                       plane(dgate_a, dga_stride_c, dga_stride_t, dim, total_T, es),
                       plane(dgate_x, dgx_stride_c, dgx_stride_t, dim, total_T, es)};
  // Small float buffers that are written: state gradients, ddecay, workspace.
  const int64_t dib = dinitial_states ? ((num_slots - 1) * di_stride_slot + dim) * 4 : 0;
  const int64_t dfb = dfinal_states ? ((num_slots - 1) * df_stride_slot + dim) * 4 : 0;
  const int64_t mb = batch > 0 ? mark_rows(total_T, batch) * dim * 4 : 0;
  const struct { const void* p; int64_t n; } wr[3] = {
      {dinitial_states, dib}, {ddecay, (int64_t)dim * 4}, {workspace, (int64_t)batch * dim * 4}};
  for (const Plane& a : in)
    if (!a.readable()) return fail(SCONV_ERR_INVALID, "%s: strides must be >= 0", fn);
  for (int i = 0; i < 3; ++i) {
    if (!ou[i].writable())
      return fail(SCONV_ERR_INVALID, "%s: a gradient's elements overlap each other", fn);
    for (const Plane& a : in)
      if (planes_overlap(ou[i], a))
        return fail(SCONV_ERR_INVALID, "%s: a gradient overlaps an input", fn);
    for (int j = 0; j < i; ++j)
      if (planes_overlap(ou[i], ou[j]))
        return fail(SCONV_ERR_INVALID, "%s: two gradients overlap", fn);
    if (overlap(ou[i].p, ou[i].bytes(), checkpoints, mb) ||
        overlap(ou[i].p, ou[i].bytes(), dfinal_states, dfb))
      return fail(SCONV_ERR_INVALID, "%s: a gradient overlaps an input", fn);
  }
  for (int i = 0; i < 3; ++i) {
    bool bad = overlap(wr[i].p, wr[i].n, checkpoints, mb) ||
               overlap(wr[i].p, wr[i].n, decay, (int64_t)dim * 4);
    for (const Plane& a : in) bad = bad || overlap(wr[i].p, wr[i].n, a.p, a.bytes());
    for (const Plane& a : ou) bad = bad || overlap(wr[i].p, wr[i].n, a.p, a.bytes());
    for (int j = 0; j < i; ++j) bad = bad || overlap(wr[i].p, wr[i].n, wr[j].p, wr[j].n);
    // dinitial may be dfinal itself: each element is read before it is written
    const bool self = i == 0 && dinitial_states == dfinal_states && di_stride_slot == df_stride_slot;
    bad = bad || (!self && overlap(wr[i].p, wr[i].n, dfinal_states, dfb));
    if (bad)
      return fail(SCONV_ERR_INVALID,
                  "%s: state gradients, ddecay or workspace overlap another buffer", fn);
  }
  RecBwdParams p = {};
  p.dout = dout; p.x = x; p.ga = gate_a; p.gx = gate_x; p.decay = decay; p.marks = checkpoints;
  p.qsl = query_start_loc; p.cache_indices = cache_indices; p.has_init = has_initial_state;
  p.dfinal = dfinal_states; p.dinitial = dinitial_states; p.dx = dx; p.dga = dgate_a;
  p.dgx = dgate_x; p.partial = workspace;
  p.do_sc = in[0].sc; p.do_st = in[0].st; p.x_sc = in[1].sc; p.x_st = in[1].st;
  p.ga_sc = in[2].sc; p.ga_st = in[2].st; p.gx_sc = in[3].sc; p.gx_st = in[3].st;
  p.dx_sc = ou[0].sc; p.dx_st = ou[0].st; p.dga_sc = ou[1].sc; p.dga_st = ou[1].st;
  p.dgx_sc = ou[2].sc; p.dgx_st = ou[2].st; p.df_slot = df_stride_slot;
  p.di_slot = di_stride_slot; p.total_T = total_T; p.num_pairs = (int64_t)batch * dim;
  p.scale = decay_scale; p.batch = batch; p.dim = dim; p.pad_slot_id = pad_slot_id;
  const int64_t grid = cdiv(p.num_pairs, 64);
  if (batch > 0 && !valid_grid(grid, 64))
    return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
  if (batch > 0) {
    if (dtype == SCONV_BF16)
      hipLaunchKernelGGL(rec_bwd_simple<Bf16>, dim3((uint32_t)grid), dim3(64), 0, stream, p);
    else
      hipLaunchKernelGGL(rec_bwd_simple<F32>, dim3((uint32_t)grid), dim3(64), 0, stream, p);
    if (const int rc = check_launch(fn)) return rc;
  }
  hipLaunchKernelGGL(rec_ddecay_kernel, dim3((uint32_t)cdiv(dim, 64)), dim3(64), 0, stream,
                     workspace, decay, ddecay, batch, dim, decay_scale);
  return check_launch(fn);
}

extern "C" int gated_linear_recurrence_update(
    const void* x, int64_t x_stride_b, const void* gate_a, int64_t ga_stride_b,
    const void* gate_x, int64_t gx_stride_b, const float* decay, float decay_scale,
    float* states, int64_t num_slots, int64_t st_stride_slot, const int32_t* state_indices,
    void* out, int64_t out_stride_b, int32_t batch, int32_t dim, int32_t dtype,
    int32_t pad_slot_id, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "gated_linear_recurrence_update";
  if (const int rc = rec_check(fn, batch, dim, 0, dtype, decay_scale)) return rc;
  if (batch == 0 || dim == 0) return SCONV_OK;
  if (!x || !gate_a || !gate_x || !decay || !states || !out)
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  if (num_slots < 1 || (!state_indices && num_slots < batch))
    return fail(SCONV_ERR_INVALID, "%s: state pool has fewer slots than rows", fn);
  if (num_slots > 1 && st_stride_slot < dim)
    return fail(SCONV_ERR_INVALID, "%s: state slot stride smaller than dim", fn);
  const int64_t es = elem_size(dtype);
  const Plane px = plane(x, 1, x_stride_b, dim, batch, es);
  const Plane pa = plane(gate_a, 1, ga_stride_b, dim, batch, es);
  const Plane pg = plane(gate_x, 1, gx_stride_b, dim, batch, es);
  const Plane po = plane(out, 1, out_stride_b, dim, batch, es);
  if (!px.readable() || !pa.readable() || !pg.readable())
    return fail(SCONV_ERR_INVALID, "%s: strides must be >= 0", fn);
  if (!po.writable()) return fail(SCONV_ERR_INVALID, "%s: out's rows overlap each other", fn);
  if (!same_plane(po, px) && planes_overlap(po, px))
    return fail(SCONV_ERR_INVALID, "%s: out partially overlaps x", fn);
  if (planes_overlap(po, pa) || planes_overlap(po, pg))
    return fail(SCONV_ERR_INVALID, "%s: out overlaps a gate", fn);
  const int64_t sb = ((num_slots - 1) * st_stride_slot + dim) * 4;
  if (overlap(states, sb, x, px.bytes()) || overlap(states, sb, gate_a, pa.bytes()) ||
      overlap(states, sb, gate_x, pg.bytes()) || overlap(states, sb, out, po.bytes()))
    return fail(SCONV_ERR_INVALID, "%s: states overlap another buffer", fn);
  RecUpdParams p = {};
  p.x = x; p.ga = gate_a; p.gx = gate_x; p.decay = decay; p.states = states;
  p.idx = state_indices; p.out = out; p.x_rs = px.st; p.ga_rs = pa.st; p.gx_rs = pg.st;
  p.o_rs = po.st; p.ss_slot = st_stride_slot; p.scale = decay_scale; p.batch = batch;
  p.dim = dim; p.pad_slot_id = pad_slot_id;
  const int64_t grid = cdiv((int64_t)batch * dim, 64);
  if (!valid_grid(grid, 64)) return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
  if (dtype == SCONV_BF16)
    hipLaunchKernelGGL(rec_update_kernel<Bf16>, dim3((uint32_t)grid), dim3(64), 0, stream, p);
  else
    hipLaunchKernelGGL(rec_update_kernel<F32>, dim3((uint32_t)grid), dim3(64), 0, stream, p);
  return check_launch(fn);
}
