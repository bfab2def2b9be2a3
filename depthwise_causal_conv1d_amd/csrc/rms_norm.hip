// rms_norm.hip -- root-mean-square norm of rows with the residual's
// addition, with an output in the rows' type or in 8 bits with scales, and
// its gradients, for gfx950.
//
//   s = x + residual, out = s * rsqrt(mean(s^2) + eps) * weight
//   8 bits: scale = max |out| over a group / 448, code = e4m3(out / scale)
#include "sconv_device.h"
#include "sconv_host.h"

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

template <typename D>
__device__ __forceinline__ typename D::storage norm_round(float v) {
  if constexpr (sizeof(typename D::storage) == 2)
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sum over the workgroup; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = wave_sum(v);
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

// One workgroup per row, which it reads three times.
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
      if (sum) sum[c] = norm_round<D>(v);
      if constexpr (Q) static_cast<uint8_t*>(p.out)[row * p.o_rs + c] = to_e4m3(y / scale);
      else static_cast<S*>(p.out)[row * p.o_rs + c] = norm_round<D>(y);
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
// dweight's share of this workgroup's rows.
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
      dx[c] = norm_round<D>(v);
    }
  }
}

// dweight: the workgroups' sums, added in their order.
__global__ __launch_bounds__(64) void norm_dweight_kernel(const float* partial, float* dweight,
                                                          int32_t dim, int32_t n) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= dim) return;
  float acc = 0.f;
  for (int i = 0; i < n; ++i) acc += partial[(int64_t)i * dim + c];
  dweight[c] = acc;
}

// Workgroups of the backward pass, and rows of its workspace.
static int64_t norm_parts(int64_t rows) { return rows < 512 ? rows : 512; }

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
  *floats = norm_parts(rows) * dim;
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
  const int64_t parts = norm_parts(rows), need = parts * dim;
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
    const dim3 grid((uint32_t)parts), th(kNormThreads);
    if (dtype == SCONV_BF16) hipLaunchKernelGGL(norm_bwd_simple<Bf16>, grid, th, 0, stream, p);
    else hipLaunchKernelGGL(norm_bwd_simple<F32>, grid, th, 0, stream, p);
    if (const int rc = check_launch(fn)) return rc;
  }
  hipLaunchKernelGGL(norm_dweight_kernel, dim3((uint32_t)cdiv(dim, 64)), dim3(64), 0, stream,
                     workspace, dweight, dim, (int32_t)parts);
  return check_launch(fn);
}
