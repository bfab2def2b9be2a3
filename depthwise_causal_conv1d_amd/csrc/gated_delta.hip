// gated_delta.hip -- the gated delta rule over packed sequences and its
// one-token update, for gfx950.  The mathematics is in delta_rule.h.
#include "delta_prep.h"
#include "delta_host.h"
#include "delta_walk.h"

namespace sconv {

struct DeltaFwd {
  DeltaParams p;
  float* states;
  int64_t st_slot;
  void* out;
  int64_t o_t, o_h;
  float* marks;
  int32_t o_vec;
};

// One workgroup walks a sequence's chunks for one value head, 16 columns a
// wave of NW; LOAD: as many waves more load and store.  An output chunk waits in
// LDS, in V's place, for the next one's staging.
// Bound by the chain of chunks: a wave of the matrix cores' small tiles feeds
// them from LDS, where every wave reads all of K and Q.  8 x 4096 tokens, 32 heads
// of 128 x 128 bf16, eight waves: 434 us (546 when the clock falls in a long run),
// 1.25 GB, 6.8 us a chunk; 364 us with states of two parts, which lose digits.
// 2 x 8192 tokens of 16 heads with checkpoints, four waves and loaders: 443 us, 3.5 us
// a chunk.  fp32 is bound by the rate of 16 x 16 x 4 products, an eighth of the bf16
// ones': 224 of 32 cycles a wave are 3.0 of the 3.4 us of a chunk of 32 x 128 x 77.
template <typename D, int KP, int NW, bool LOAD, bool VEC>
__global__ __launch_bounds__(LOAD ? 128 * NW : 64 * NW, 2) void delta_walk_kernel(DeltaFwd a) {
  using T = Tile<D>;
  using S = typename D::storage;
  constexpr int C = kDeltaChunk<D>, NT = C / 16, KS = KP / 32, KT = KP / 16, CS = C / 32;
  constexpr int NF = kDeltaFrags<C>, PIECES = kGroups<KS, true>;
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
  const S* v = static_cast<const S*>(p.v) + h * p.v_h;
  S* out = static_cast<S*>(a.out) + h * a.o_h;
  Stage next;
  const int id = threadIdx.x % Stage::THREADS;
  next.init(p, k, q, v, p.v_t, cols0, id);
  auto fetch = [&](int32_t i, auto P, auto N) {
    const int64_t at = (int64_t)(row0 + i) * p.heads + h;
    next.template fetch<decltype(P)::value, decltype(N)::value>(
        p, start + i * C, end, p.frags + at * (2 * NF) * kFragBytes, p.vectors + at * kDeltaVectors<C>);
  };
  constexpr std::integral_constant<int, 0> kFirst;
  constexpr std::integral_constant<int, 1> kWhole;
  auto put_out = [&](int32_t i, const typename Stage::L& l) {
    put_rows<Stage, D, VEC>(l, out, a.o_t, p.V, cols0, start + i * C, end, id);
  };

  if (LOAD && wave >= NW) {
    // Aligned rows' loads are under way over the barrier before the one in which they are
    // staged (1 x 8192 x 16 heads: 430 -> 414 us; entries of others take registers that
    // are not there: 16 ragged fp32 prompts 253 -> 275).  Behind the last chunk it is
    // fetched again: a branch would make loads wait.
    if (chunks > 0) {
      fetch(0, kFirst, kWhole);
      next.stage(lds[0], p, end - start);
      if constexpr (VEC) fetch(min(1, chunks - 1), kFirst, kWhole);
    }
    __syncthreads();
    for (int32_t i = 0; i < chunks; ++i) {
      if constexpr (!VEC) fetch(min(i + 1, chunks - 1), kFirst, kWhole), keep_order();
      if (i > 0) put_out(i - 1, lds[(i + 1) & 1]);
      if (i + 1 < chunks) next.stage(lds[(i + 1) & 1], p, end - (start + (i + 1) * C));
      if constexpr (VEC) keep_order(), fetch(min(i + 2, chunks - 1), kFirst, kWhole);
      __syncthreads();
    }
    if (chunks > 0) put_out(chunks - 1, lds[(chunks - 1) & 1]);
    return;
  }

  const int32_t c16 = 16 * wave, col = cols0 + c16 + r, ends = cols0 + c16 + 16;
  f32x4 s[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) s[t] = zero4();
  float* state = a.states ? a.states + slot * a.st_slot + h * KV : nullptr;
  if (p.has && p.has[b]) state_columns<false>(s, state, p.K, p.V, col, ends);
  wait_for_all();
  if (!LOAD && chunks > 0) {
    fetch(0, kFirst, kWhole);
    next.stage(lds[0], p, end - start);
  }
  __syncthreads();
  for (int32_t i = 0; i < chunks; ++i) {
    typename Stage::L& l = lds[i & 1];
    if (!LOAD && i > 0) put_out(i - 1, lds[(i + 1) & 1]);
    float* mark = nullptr;
    if (a.marks && ends - 16 < p.V)
      mark = a.marks + ((int64_t)(row0 + i) * p.heads + h) * delta_state_floats(p.K, p.V) +
             (ends / 16 - 1) * tiles16(p.K) * 256;
    f32x4 u[NT], y[NT];  // K S, then R, then U; Q S, then O
    typename T::Exact vv[CS];
    typename T::Pair tri[NF], us[CS];
    rows_times_state<D, Rows, KS, NT, true>(
        l.k, l.q, s, u, y, lane,
        [&] {
#pragma unroll
          for (int c = 0; c < CS; ++c) vv[c] = Cols::cols(l.x, 32 * c, c16, lane);
          load_triangle<D>(tri, l.f, lane);
        },
        [&](auto P) {
          if constexpr (!LOAD) fetch(min(i + 1, chunks - 1), P, std::integral_constant<int, PIECES>());
          if (mark) put_tiles<decltype(P)::value, PIECES>(s, mark, p.K, lane);
        });
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 gam = lds4(l.v + 16 * t + 4 * g), bt = lds4(l.v + 2 * C + 16 * t + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[t][e] = bt[e] * (T::value(vv[t / 2], 4 * (t & 1) + e) - gam[e] * u[t][e]);
        y[t][e] *= p.scale * gam[e];
      }
    }
    float down = pair_tiles<D>(u, us);
    triangle_times<D, true>(tri, us, u, down, lds4(l.v + kDeltaFactors<C>));
    keep_order();
    load_triangle<D>(tri, l.f + NF * kFragBytes, lane);
    keep_order();
    down = pair_tiles<D>(u, us);
    const float whole = l.v[C - 1];
    typename T::Fine fine[CS];
#pragma unroll
    for (int t = 0; t < NT; ++t) u[t] *= lds4(l.v + C + 16 * t + 4 * g);
    fine_tiles<D>(u, fine);
#pragma unroll
    for (int t = 0; t < KT; ++t) s[t] *= whole;
    triangle_times<D, true>(tri, us, y, down, lds4(l.v + kDeltaFactors<C> + 4));
    keep_order();
    cols_times<D, Rows>(l.k, fine, s, lane);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        l.x[(16 * t + 4 * g + e) * Cols::LD + Cols::pos(c16 + r)] = delta_round<D>(y[t][e]);
    if (!LOAD && i + 1 < chunks) next.stage(lds[(i + 1) & 1], p, end - (start + (i + 1) * C));
    __syncthreads();
  }
  if (!LOAD && chunks > 0) put_out(chunks - 1, lds[(chunks - 1) & 1]);
  if (state) state_columns<true>(s, state, p.K, p.V, col, ends);
}

// ---------------------------------------------------------------- one token

struct DeltaUpdate {
  DeltaParams p;  // rows instead of tokens
  float* states;
  int64_t st_slot;
  void* out;
  int64_t o_t, o_h;
};

// One workgroup a row, value head and CL * VEC columns of the state, which it
// reads and writes once.  Both products with the old state are summed in one
// pass, since S^T q = S'^T q + (k.q) u: one meeting of the row groups.  The state
// stays in registers between its read and its write, so bytes bound it: 247
// rows x 32 heads of 128 x 128 take 208 us, 5.0 TB/s (a large copy reaches 5.1);
// 4 x 16 of 64 x 64 5.4 us, the latency of a load, a barrier and a store.
template <typename D, int CL, int VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void delta_update_kernel(DeltaUpdate a) {
  using S = typename D::storage;
  typedef float vf __attribute__((ext_vector_type(VEC)));
  constexpr int RG = THREADS / CL, RPG = kDeltaMaxK / RG;
  __shared__ float lk[kDeltaMaxK], lq[kDeltaMaxK];
  __shared__ float part[2][RG][CL * VEC];
  const DeltaParams& p = a.p;
  const int32_t b = blockIdx.z, h = blockIdx.y, kh = h / p.group;
  const int32_t slot = p.slots ? p.slots[b] : b;
  if (p.slots && slot == p.pad) return;
  const int cl = threadIdx.x % CL, rg = threadIdx.x / CL;
  const int32_t col = (blockIdx.x * CL + cl) * VEC;
  const bool on = col < p.V;
  float* state = a.states + slot * a.st_slot + (int64_t)h * p.K * p.V + col;
  vf s[RPG];
#pragma unroll
  for (int j = 0; j < RPG; ++j) {
    const int k = rg + RG * j;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[j][e] = 0.f;
    if (on && k < p.K) s[j] = *reinterpret_cast<const vf*>(state + (int64_t)k * p.V);
  }
  for (int k = threadIdx.x; k < kDeltaMaxK; k += THREADS) {
    lk[k] = k < p.K ? load_as_float<D>(static_cast<const S*>(p.k) + b * p.k_t + kh * p.k_h + k) : 0.f;
    lq[k] = k < p.K ? load_as_float<D>(static_cast<const S*>(p.q) + b * p.q_t + kh * p.q_h + k) : 0.f;
  }
  const float decay = expf(delta_bound(delta_gate(p, p.g, b * p.g_t + h * p.g_h)));
  const float beta = delta_gate(p, p.beta, b * p.b_t + h * p.b_h);
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    v[e] = on ? load_as_float<D>(static_cast<const S*>(p.v) + b * p.v_t + h * p.v_h + col + e) : 0.f;
  __syncthreads();
  vf x, y;
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = 0.f, y[e] = 0.f;
#pragma unroll
  for (int j = 0; j < RPG; ++j) {
    s[j] *= decay;
    x += s[j] * lk[rg + RG * j];
    y += s[j] * lq[rg + RG * j];
  }
  *reinterpret_cast<vf*>(&part[0][rg][cl * VEC]) = x;
  *reinterpret_cast<vf*>(&part[1][rg][cl * VEC]) = y;
  float kq = 0.f;
  {
    const int l = threadIdx.x & 63;
    kq = lk[l] * lq[l] + lk[l + 64] * lq[l + 64];
#pragma unroll
    for (int d = 32; d > 0; d /= 2) kq += __shfl_xor(kq, d, 64);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = 0.f, y[e] = 0.f;
#pragma unroll
  for (int w = 0; w < RG; ++w) {
    x += *reinterpret_cast<const vf*>(&part[0][w][cl * VEC]);
    y += *reinterpret_cast<const vf*>(&part[1][w][cl * VEC]);
  }
  vf u;
#pragma unroll
  for (int e = 0; e < VEC; ++e) u[e] = beta * (v[e] - x[e]);
  if (!on) return;
#pragma unroll
  for (int j = 0; j < RPG; ++j) {
    const int k = rg + RG * j;
    if (k < p.K) *reinterpret_cast<vf*>(state + (int64_t)k * p.V) = s[j] + u * lk[k];
  }
  if (rg == 0) {
    S* out = static_cast<S*>(a.out) + b * a.o_t + h * a.o_h + col;
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = delta_round<D>(p.scale * (y[e] + kq * u[e]));
  }
}

template <typename D, int KP>
static int delta_forward(DeltaFwd a, int64_t rows, hipStream_t stream) {
  const DeltaParams& p = a.p;
  if (int rc = delta_prepare<D, KP, false>("gated_delta_rule_varlen_fwd", p, rows, stream)) return rc;
  const bool vec = p.qk_vec && p.v_vec && a.o_vec;
  const dim3 threads(512);
  bool wide = false;
  if constexpr (sizeof(typename D::storage) == 2) {
    wide = delta_wide(p);
    if (wide) {
      const dim3 grid = delta_walk_grid(a.p, (p.V + 127) / 128);
      if (vec) hipLaunchKernelGGL((delta_walk_kernel<D, KP, 8, false, true>), grid, threads, 0, stream, a);
      else hipLaunchKernelGGL((delta_walk_kernel<D, KP, 8, false, false>), grid, threads, 0, stream, a);
    }
  }
  if (!wide) {
    const dim3 grid = delta_walk_grid(a.p, (p.V + 63) / 64);
    if (vec) hipLaunchKernelGGL((delta_walk_kernel<D, KP, 4, true, true>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((delta_walk_kernel<D, KP, 4, true, false>), grid, threads, 0, stream, a);
  }
  return check_launch("gated_delta_rule_varlen_fwd");
}

template <typename D, int CL, int VEC, int THREADS>
static void delta_update_launch(const DeltaUpdate& a, hipStream_t stream) {
  const int cols = CL * VEC;
  hipLaunchKernelGGL((delta_update_kernel<D, CL, VEC, THREADS>),
                     dim3((a.p.V + cols - 1) / cols, a.p.heads, a.p.batch), dim3(THREADS), 0,
                     stream, a);
}

// Eight groups of rows, so that a thread has up to 16 loads under way (256
// rows x 32 heads of 64 x 64: 57 us with eight groups, 62 with four, 103 with
// sixteen; 128 x 128: 218, 350 with two, 308 with sixteen); half the columns a
// workgroup where the head has no more.  States whose rows do not start on 16 bytes go by
// single elements (64 x 63: 60 us; 66 with four groups, 118 of 128 columns).
template <typename D> static void delta_update_pick(const DeltaUpdate& a, hipStream_t stream) {
  const DeltaParams& p = a.p;
  const bool vec = p.V % 4 == 0 && aligned16(a.states) && a.st_slot % 4 == 0;
  if (!vec) delta_update_launch<D, 64, 1, 512>(a, stream);
  else if (p.V <= 64) delta_update_launch<D, 16, 4, 128>(a, stream);
  else delta_update_launch<D, 32, 4, 256>(a, stream);
}

}  // namespace sconv

extern "C" int gated_delta_rule_checkpoint_rows(int64_t total_T, int32_t batch, int32_t dtype,
                                                int64_t* rows) {
  using namespace sconv;
  clear_error();
  if (total_T < 0 || batch < 0 || !valid_dtype(dtype) || !rows)
    return fail(SCONV_ERR_INVALID, "gated_delta_rule_checkpoint_rows: bad argument");
  *rows = delta_rows(total_T, batch, delta_chunk(dtype));
  return SCONV_OK;
}

extern "C" int gated_delta_rule_workspace(int64_t total_T, int32_t batch, int32_t heads, int32_t K,
                                          int32_t V, int32_t dtype, int64_t* fwd_floats,
                                          int64_t* bwd_floats) {
  using namespace sconv;
  clear_error();
  if (total_T < 0 || batch < 0 || heads < 0 || K < 0 || V < 0 || !valid_dtype(dtype) ||
      !fwd_floats || !bwd_floats)
    return fail(SCONV_ERR_INVALID, "gated_delta_rule_workspace: bad argument");
  const DeltaSpace s = delta_space(total_T, batch, heads, K, V, dtype);
  *fwd_floats = s.fwd;
  *bwd_floats = s.bwd;
  return SCONV_OK;
}

extern "C" int gated_delta_rule_varlen_fwd(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k, int64_t k_stride_t,
    int64_t k_stride_h, const void* v, int64_t v_stride_t, int64_t v_stride_h, const void* g,
    int64_t g_stride_t, int64_t g_stride_h, const void* beta, int64_t b_stride_t,
    int64_t b_stride_h, float scale, float* states, int64_t num_slots, int64_t st_stride_slot,
    const int32_t* query_start_loc, int32_t batch, const int32_t* cache_indices,
    const uint8_t* has_initial_state, void* out, int64_t out_stride_t, int64_t out_stride_h,
    float* checkpoints, int64_t checkpoint_rows, float* workspace, int64_t workspace_floats,
    int64_t total_T, int32_t key_heads, int32_t value_heads, int32_t K, int32_t V, int32_t dtype,
    int32_t gate_dtype, int32_t pad_slot_id, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* what = "gated_delta_rule_varlen_fwd";
  DeltaFwd a = {};
  DeltaCall c = {what, total_T, batch, key_heads, value_heads, K, V, dtype, gate_dtype};
  if (int rc = delta_sizes(c)) return rc;
  if (batch == 0 || value_heads == 0 || V == 0) return SCONV_OK;
  if (int rc = delta_grids(c)) return rc;
  if (!query_start_loc) return fail(SCONV_ERR_INVALID, "%s: NULL query_start_loc", what);
  if (int rc = delta_inputs(c, a.p, q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v,
                            v_stride_t, v_stride_h, g, g_stride_t, g_stride_h, beta, b_stride_t,
                            b_stride_h, scale))
    return rc;
  delta_packing(a.p, query_start_loc, cache_indices, has_initial_state, pad_slot_id);
  if (has_initial_state && !states)
    return fail(SCONV_ERR_INVALID, "%s: has_initial_state without states", what);
  DeltaBuffer pool, o;
  if (int rc = delta_pool(c, states, num_slots, st_stride_slot, cache_indices != nullptr, "states",
                          &pool))
    return rc;
  if (int rc = delta_output(c, out, out_stride_t, out_stride_h, value_heads, V, "out", &o)) return rc;
  const int64_t rows = delta_rows(total_T, batch, delta_chunk(dtype));
  if (checkpoints && (checkpoint_rows < rows || !aligned16(checkpoints)))
    return fail(SCONV_ERR_INVALID, "%s: %lld checkpoint rows, needs %lld at 16 bytes", what,
                (long long)checkpoint_rows, (long long)rows);
  const DeltaSpace s = delta_space(total_T, batch, value_heads, K, V, dtype);
  if (!workspace || workspace_floats < s.fwd || !aligned16(workspace))
    return fail(SCONV_ERR_INVALID, "%s: workspace needs %lld floats at 16 bytes", what,
                (long long)s.fwd);
  const DeltaBuffer marks = delta_block(checkpoints, checkpoints ? rows * value_heads * delta_state_floats(K, V) * 4 : 0);
  const DeltaBuffer work = delta_block(workspace, s.fwd * 4);
  if (int rc = delta_disjoint(c, a.p, {o, pool, marks, work}, /*out may be v=*/out == v &&
                              out_stride_t == v_stride_t && out_stride_h == v_stride_h))
    return rc;
  a.p.vectors = workspace;
  a.p.frags = reinterpret_cast<char*>(workspace + s.vectors);
  a.states = states, a.st_slot = st_stride_slot;
  a.out = out, a.o_t = out_stride_t, a.o_h = out_stride_h;
  a.o_vec = delta_vec(out, out_stride_t, out_stride_h, V, 16 / elem_size(dtype));
  a.marks = checkpoints;
  if (dtype == SCONV_BF16)
    return K <= 64 ? delta_forward<Bf16, 64>(a, rows, stream) : delta_forward<Bf16, 128>(a, rows, stream);
  return K <= 64 ? delta_forward<F32, 64>(a, rows, stream) : delta_forward<F32, 128>(a, rows, stream);
}

extern "C" int gated_delta_rule_update(
    const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* k, int64_t k_stride_b,
    int64_t k_stride_h, const void* v, int64_t v_stride_b, int64_t v_stride_h, const void* g,
    int64_t g_stride_b, int64_t g_stride_h, const void* beta, int64_t b_stride_b,
    int64_t b_stride_h, float scale, float* states, int64_t num_slots, int64_t st_stride_slot,
    const int32_t* state_indices, void* out, int64_t out_stride_b, int64_t out_stride_h,
    int32_t batch, int32_t key_heads, int32_t value_heads, int32_t K, int32_t V, int32_t dtype,
    int32_t gate_dtype, int32_t pad_slot_id, hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* what = "gated_delta_rule_update";
  DeltaUpdate a = {};
  DeltaCall c = {what, batch, batch, key_heads, value_heads, K, V, dtype, gate_dtype};
  if (int rc = delta_sizes(c)) return rc;
  if (batch == 0 || value_heads == 0 || V == 0) return SCONV_OK;
  if (int rc = delta_inputs(c, a.p, q, q_stride_b, q_stride_h, k, k_stride_b, k_stride_h, v,
                            v_stride_b, v_stride_h, g, g_stride_b, g_stride_h, beta, b_stride_b,
                            b_stride_h, scale))
    return rc;
  delta_packing(a.p, nullptr, state_indices, nullptr, pad_slot_id);
  if (!states) return fail(SCONV_ERR_INVALID, "%s: NULL states", what);
  DeltaBuffer pool, o;
  if (int rc = delta_pool(c, states, num_slots, st_stride_slot, state_indices != nullptr, "states",
                          &pool))
    return rc;
  if (int rc = delta_output(c, out, out_stride_b, out_stride_h, value_heads, V, "out", &o)) return rc;
  if (int rc = delta_disjoint(c, a.p, {o, pool}, out == v && out_stride_b == v_stride_b &&
                              out_stride_h == v_stride_h))
    return rc;
  a.states = states, a.st_slot = st_stride_slot;
  a.out = out, a.o_t = out_stride_b, a.o_h = out_stride_h;
  if (dtype == SCONV_BF16) delta_update_pick<Bf16>(a, stream);
  else delta_update_pick<F32>(a, stream);
  return check_launch(what);
}
