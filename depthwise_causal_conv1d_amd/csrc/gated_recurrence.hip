// gated_recurrence.hip -- gated linear recurrence over packed
// variable-length sequences with a slot-indexed state pool (prefill), its
// gradients, and its one-token decode step, for gfx950.
//
// The recurrence is the layer step behind the short conv: it takes the
// conv's packing (query_start_loc), state slots and layouts.
#include <initializer_list>

#include "column_sum.h"
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

// The checkpoint row of sequence b's token start + rel (rel a multiple of
// 64): rows of later sequences lie behind it, since a sequence of L tokens has
// ceil(L / 64) of them and ends less than 64 ceil(L / 64) after its start.
__device__ __forceinline__ int64_t mark_row(int64_t start, int b, int64_t rel) {
  return start / kMarkTokens + b + rel / kMarkTokens;
}

// ---------------------------------------------------------------- tokens in lanes

// A wave takes a chunk of 512 tokens of one channel, counted from the
// sequence's start, lane l the tokens [8 l, 8 l + 8) of it.  The
// recurrence is a composition of maps h -> a h + u: a lane composes its
// eight, the wave its lanes (six DPP steps), and NW waves that walk one
// sequence together exchange their chunks' maps through LDS, so that no
// state ever waits for another workgroup and every input is read once.
// Tokens outside the sequence are the identity (a = 1, u = 0).
template <typename D, bool VEC, int NW>
__global__ __launch_bounds__(NW > 4 ? NW * 64 : 256) void rec_fwd_kernel(const RecFwdParams p) {
  using S = typename D::storage;
  constexpr int kWaves = NW > 4 ? NW : 4;
  constexpr int kPairs = kWaves / NW;  // (sequence, channel) pairs of a workgroup
  static_assert(kPairs == 1 || NW == 1, "a barrier is met by one pair only");
  __shared__ float2 maps[2][kPairs][NW];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int sub = wave % NW, mine = wave / NW;
  const int64_t pair = (int64_t)xcd_groups<8>(blockIdx.x, gridDim.x) * kPairs + mine;
  if (pair >= p.num_pairs) return;  // NW waves of one pair leave together
  const int b = (int)(pair / p.dim), c = (int)(pair - (int64_t)b * p.dim);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (slot == p.pad_slot_id) return;
  const int64_t start = p.qsl[b], end = p.qsl[b + 1];
  const Decay d = make_decay(p.decay[c], p.scale);
  float carry = p.has_init && p.has_init[b] != 0 ? p.states[slot * p.ss_slot + c] : 0.f;
  const S* x = static_cast<const S*>(p.x) + c * p.x_sc;  // may be out
  const S* ga = static_cast<const S*>(p.ga) + c * p.ga_sc;
  const S* gx = static_cast<const S*>(p.gx) + c * p.gx_sc;
  S* out = static_cast<S*>(p.out) + c * p.o_sc;

  Raw8<D> rx, ra, rg;
  auto fetch = [&](int64_t base) {
    const int64_t t = base + lane * kLaneTokens;
    if (base < end) {
      rx.template load<VEC>(x, p.x_st, t, p.total_T);
      ra.template load<VEC>(ga, p.ga_st, t, p.total_T);
      rg.template load<VEC>(gx, p.gx_st, t, p.total_T);
    }
  };
  const int64_t first = start + sub * kChunkTokens;
  if (end > start) fetch(first);
  int turn = 0;
  for (int64_t base = first; base - sub * kChunkTokens < end; base += NW * kChunkTokens, turn ^= 1) {
    const int64_t t = base + lane * kLaneTokens;
    float a[kLaneTokens], u[kLaneTokens];
    float P = 1.f, H = 0.f;
    const bool any = base < end;
    if (any) {
      float xf[kLaneTokens], gf[kLaneTokens];
      rx.to_float(xf);
      ra.to_float(a);
      rg.to_float(gf);
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e) {
        const Gates g = make_gates(a[e], gf[e], d);
        a[e] = g.a;
        u[e] = g.m * (g.i * xf[e]);
      }
      if (base + kChunkTokens > end) {
#pragma unroll
        for (int e = 0; e < kLaneTokens; ++e) {
          const bool in = t + e < end;
          a[e] = in ? a[e] : 1.f;
          u[e] = in ? u[e] : 0.f;
        }
      }
      fetch(base + NW * kChunkTokens);
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e) {
        H = __builtin_fmaf(a[e], H, u[e]);
        P *= a[e];
      }
      scan_wave_up(P, H);
    }
    float h = carry;
    if constexpr (NW == 1) {
      carry = __builtin_fmaf(last_lane(P), carry, last_lane(H));
    } else {
      if (lane == 63) maps[turn][mine][sub] = make_float2(P, H);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        const float2 f = maps[turn][mine][q];
        if (q == sub) h = carry;
        carry = __builtin_fmaf(f.x, carry, f.y);
      }
    }
    if (!any) continue;
    h = __builtin_fmaf(lane_move<0x138>(1.0f, P), h, lane_move<0x138>(0.0f, H));
    if (p.marks && lane % (kMarkTokens / kLaneTokens) == 0 && t < end)
      p.marks[mark_row(start, b, t - start) * p.dim + c] = h;
#pragma unroll
    for (int e = 0; e < kLaneTokens; ++e) {
      h = __builtin_fmaf(a[e], h, u[e]);
      u[e] = h;
    }
    Raw8<D> o;
    o.from_float(u);
    o.template store<VEC>(out, p.o_st, t, end);
  }
  if (p.states && sub == 0 && lane == 0) p.states[slot * p.ss_slot + c] = carry;
}

// ---------------------------------------------------------------- channels in lanes

// For channels that lie side by side (rows of tokens): lane l takes V
// channels, wave w of a workgroup the rows [R w, R w + R) of each tile of
// NW * R tokens, and the tile's maps meet in LDS as above.
constexpr int kRowWaves = 8, kRowTokens = 8;

template <typename D, int V>
__global__ __launch_bounds__(kRowWaves * 64) void rec_fwd_rows_kernel(const RecFwdParams p) {
  using S = typename D::storage;
  using P_ = Pack<D, V>;
  constexpr int R = kRowTokens, NW = kRowWaves, kTile = R * NW;
  struct alignas(8 * V) Map { float P[V], H[V]; };
  __shared__ Map maps[2][NW][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t slabs = (uint32_t)((p.dim + 64 * V - 1) / (64 * V));
  const uint32_t wg = blockIdx.x;
  const int b = (int)(wg / slabs), slab = (int)(wg % slabs);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (slot == p.pad_slot_id) return;
  const int64_t start = p.qsl[b], end = p.qsl[b + 1];
  // lanes past the last channel read it and write nothing
  const int ch = (slab * 64 + lane) * V;
  const bool live = ch < p.dim;
  const int c = live ? ch : p.dim - V;
  const S* x = static_cast<const S*>(p.x) + c;  // may be out
  const S* ga = static_cast<const S*>(p.ga) + c;
  const S* gx = static_cast<const S*>(p.gx) + c;
  S* out = static_cast<S*>(p.out) + c;
  Decay d[V];
  float carry[V];
  const bool init = p.has_init && p.has_init[b] != 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    d[v] = make_decay(p.decay[c + v], p.scale);
    carry[v] = init ? p.states[slot * p.ss_slot + c + v] : 0.f;
  }
  P_ rx[R], ra[R], rg[R];
  auto fetch = [&](int64_t row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // past the sequence: its last row, unused
      const int64_t row = row0 + r < end ? row0 + r : end - 1;
      rx[r].load_nt(x + row * p.x_st);
      ra[r].load_nt(ga + row * p.ga_st);
      rg[r].load_nt(gx + row * p.gx_st);
    }
  };
  int64_t base = start;
  if (end > start) fetch(base + wave * R);
  for (int turn = 0; base < end; base += kTile, turn ^= 1) {
    const int64_t row0 = base + wave * R;
    float pl[R][V], hl[R][V];
    Map m;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m.P[v] = 1.f;
      m.H[v] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float xf[V], af[V], gf[V];
      rx[r].to_float(xf);
      ra[r].to_float(af);
      rg[r].to_float(gf);
      const bool in = row0 + r < end;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gates g = make_gates(af[v], gf[v], d[v]);
        const float a = in ? g.a : 1.f, u = in ? g.m * (g.i * xf[v]) : 0.f;
        m.H[v] = __builtin_fmaf(a, m.H[v], u);
        m.P[v] *= a;
        pl[r][v] = m.P[v];
        hl[r][v] = m.H[v];
      }
    }
    if (base + kTile < end) fetch(row0 + kTile);
    maps[turn][wave][lane] = m;
    if (p.marks && wave == 0 && live) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.marks[mark_row(start, b, base - start) * p.dim + c + v] = carry[v];
    }
    __syncthreads();
    float h[V];
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      const Map f = maps[turn][q][lane];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (q == wave) h[v] = carry[v];
        carry[v] = __builtin_fmaf(f.P[v], carry[v], f.H[v]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = __builtin_fmaf(pl[r][v], h[v], hl[r][v]);
      P_ o;
      o.from_float(y);
      if (live && row0 + r < end) o.store_nt(out + (row0 + r) * p.o_st);
    }
  }
  if (p.states && wave == 0 && live) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.states[slot * p.ss_slot + c + v] = carry[v];
  }
}

// ---------------------------------------------------------------- gradients

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

// Tokens in lanes, from the end of the sequence: lane l of a chunk takes
// tokens [8 (63 - l), 8 (63 - l) + 8), so that the gradient of the state,
// which runs against time, runs up the lanes.  The states come from the
// checkpoints: each row of 16 lanes (128 tokens) starts from its own, and
// only composes inside the row.  The gates are computed once per token.
template <typename D, bool VEC, int NW>
__global__ __launch_bounds__(NW > 4 ? NW * 64 : 256) void rec_bwd_kernel(const RecBwdParams p) {
  using S = typename D::storage;
  constexpr int kWaves = NW > 4 ? NW : 4;
  constexpr int kPairs = kWaves / NW;
  static_assert(kPairs == 1 || NW == 1, "a barrier is met by one pair only");
  __shared__ float2 maps[2][kPairs][NW];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int sub = wave % NW, mine = wave / NW;
  const int64_t pair = (int64_t)
      xcd_groups<8>(blockIdx.x, gridDim.x)
      * kPairs + mine;
  if (pair >= p.num_pairs) return;
  const int b = (int)(pair / p.dim), c = (int)(pair - (int64_t)b * p.dim);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (slot == p.pad_slot_id) {
    if (sub == 0 && lane == 0) p.partial[pair] = 0.f;
    return;
  }
  const int64_t start = p.qsl[b], end = p.qsl[b + 1];
  const Decay d = make_decay(p.decay[c], p.scale);
  float carry = p.dfinal ? p.dfinal[slot * p.df_slot + c] : 0.f;  // a_{t+1} dh_{t+1}
  const S* dout = static_cast<const S*>(p.dout) + c * p.do_sc;
  const S* x = static_cast<const S*>(p.x) + c * p.x_sc;
  const S* ga = static_cast<const S*>(p.ga) + c * p.ga_sc;
  const S* gx = static_cast<const S*>(p.gx) + c * p.gx_sc;
  S* dx = static_cast<S*>(p.dx) + c * p.dx_sc;
  S* dga = static_cast<S*>(p.dga) + c * p.dga_sc;
  S* dgx = static_cast<S*>(p.dgx) + c * p.dgx_sc;
  Raw8<D> rd, rx, ra, rg;
  float mark = 0.f;
  const int back = (63 - lane) * kLaneTokens;
  auto fetch = [&](int64_t base) {
    const int64_t t = base + back;
    if (base >= start) {
      rd.template load<VEC>(dout, p.do_st, t, p.total_T);
      rx.template load<VEC>(x, p.x_st, t, p.total_T);
      ra.template load<VEC>(ga, p.ga_st, t, p.total_T);
      rg.template load<VEC>(gx, p.gx_st, t, p.total_T);
      const int64_t row = (t - start) / 128 * 128;  // the first token of the row of lanes
      mark = start + row < end ? p.marks[mark_row(start, b, row) * p.dim + c] : 0.f;
    }
  };
  float acc = 0.f;
  const int64_t top = start + (end - 1 - start) / kChunkTokens * kChunkTokens;  // the last chunk
  if (end > start) fetch(top - sub * kChunkTokens);
  int turn = 0;
  for (int64_t high = top; end > start && high >= start; high -= NW * kChunkTokens, turn ^= 1) {
    const int64_t base = high - sub * kChunkTokens, t = base + back;
    const bool any = base >= start;
    float g[kLaneTokens], xf[kLaneTokens], a[kLaneTokens], r[kLaneTokens], i[kLaneTokens];
    float m[kLaneTokens], over[kLaneTokens];  // over: a i x / m
    float P = 1.f, H = 0.f, T = 0.f;
    if (any) {
      rd.to_float(g);
      rx.to_float(xf);
      ra.to_float(r);
      rg.to_float(i);
      const float h0 = mark;
      if (base + kChunkTokens > end) {
#pragma unroll
        for (int e = 0; e < kLaneTokens; ++e) {
          const bool in = t + e < end;
          g[e] = in ? g[e] : 0.f;
          xf[e] = in ? xf[e] : 0.f;
          r[e] = in ? r[e] : -INFINITY;  // r = 0: a = 1, u = 0, no part in a sum
          i[e] = in ? i[e] : 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e) {
        const GatesInv q = make_gates_inv(r[e], i[e], d);
        const float ix = q.i * xf[e];
        r[e] = q.r;
        i[e] = q.i;
        a[e] = q.a;
        m[e] = q.m;
        over[e] = q.a * q.inv_m * ix;
        H = __builtin_fmaf(q.a, H, q.m * ix);
        P *= q.a;
      }
      fetch(base - NW * kChunkTokens);
      // states before each token, less a i x / m
      float A = P;
      scan_row_down(P, H);
      float h = __builtin_fmaf(lane_move<0x101>(1.0f, P), h0, lane_move<0x101>(0.0f, H));
#pragma unroll
      for (int e = 0; e < kLaneTokens; ++e) {
        const float next = __builtin_fmaf(a[e], h, m[e] * (i[e] * xf[e]));
        over[e] = h - over[e];
        h = next;
      }
      // s -> a (dout + s), from the last token to the first
#pragma unroll
      for (int e = kLaneTokens - 1; e >= 0; --e) T = a[e] * (T + g[e]);
      P = A;
      scan_wave_up(P, T);
    }
    float s = carry;
    if constexpr (NW == 1) {
      carry = __builtin_fmaf(last_lane(P), carry, last_lane(T));
    } else {
      if (lane == 63) maps[turn][mine][sub] = make_float2(P, T);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        const float2 f = maps[turn][mine][q];
        if (q == sub) s = carry;
        carry = __builtin_fmaf(f.x, carry, f.y);
      }
    }
    if (!any) continue;
    s = __builtin_fmaf(lane_move<0x138>(1.0f, P), s, lane_move<0x138>(0.0f, T));
#pragma unroll
    for (int e = kLaneTokens - 1; e >= 0; --e) {
      const float dh = g[e] + s;
      s = a[e] * dh;
      const float vx = dh * (m[e] * i[e]);
      const float dlog = s * over[e];
      acc = __builtin_fmaf(dlog, r[e], acc);
      g[e] = vx;
      i[e] = vx * xf[e] * (1.f - i[e]);
      r[e] = -d.k * dlog * (r[e] * (1.f - r[e]));
    }
    Raw8<D> o;
    o.from_float(g);
    o.template store<VEC>(dx, p.dx_st, t, end);
    o.from_float(i);
    o.template store<VEC>(dgx, p.dgx_st, t, end);
    o.from_float(r);
    o.template store<VEC>(dga, p.dga_st, t, end);
  }
#pragma unroll
  for (int w = 32; w > 0; w >>= 1) acc += __shfl_xor(acc, w, 64);
  if constexpr (NW > 1) {
    __syncthreads();  // the last tile's maps have been read
    if (lane == 0) maps[0][0][sub].x = acc;
    __syncthreads();
    acc = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) acc += maps[0][0][q].x;
  }
  if (sub == 0 && lane == 0) {
    p.partial[pair] = acc;
    const bool init = p.has_init && p.has_init[b] != 0;
    if (p.dinitial) p.dinitial[slot * p.di_slot + c] = init ? carry : 0.f;
  }
}

// Channels in lanes, from the end: wave w takes the rows of a tile of 64
// tokens (one checkpoint) that are w * R from its end.  The forward maps and
// the backward ones, which share their factor, meet in LDS together.
constexpr int kRowBwdWaves = 16, kRowBwdTokens = 4;

template <typename D, int V>
__global__ __launch_bounds__(kRowBwdWaves * 64) void rec_bwd_rows_kernel(const RecBwdParams p) {
  using S = typename D::storage;
  using P_ = Pack<D, V>;
  constexpr int R = kRowBwdTokens, NW = kRowBwdWaves, kTile = R * NW;
  static_assert(kTile == kMarkTokens, "a tile starts at a checkpoint");
  __shared__ float mp[2][NW][V][64], mh[2][NW][V][64], mt[2][NW][V][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t slabs = (uint32_t)((p.dim + 64 * V - 1) / (64 * V));
  const uint32_t wg = blockIdx.x;
  const int b = (int)(wg / slabs), slab = (int)(wg % slabs);
  const int ch = (slab * 64 + lane) * V;
  const bool live = ch < p.dim;
  const int c = live ? ch : p.dim - V;
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (slot == p.pad_slot_id) {
    if (wave == 0 && live) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.partial[(int64_t)b * p.dim + c + v] = 0.f;
    }
    return;
  }
  const int64_t start = p.qsl[b], end = p.qsl[b + 1];
  const S* dout = static_cast<const S*>(p.dout) + c;
  const S* x = static_cast<const S*>(p.x) + c;
  const S* ga = static_cast<const S*>(p.ga) + c;
  const S* gx = static_cast<const S*>(p.gx) + c;
  S* dx = static_cast<S*>(p.dx) + c;
  S* dga = static_cast<S*>(p.dga) + c;
  S* dgx = static_cast<S*>(p.dgx) + c;
  Decay d[V];
  float carry[V], acc[V], mark[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    d[v] = make_decay(p.decay[c + v], p.scale);
    carry[v] = p.dfinal ? p.dfinal[slot * p.df_slot + c + v] : 0.f;
    acc[v] = mark[v] = 0.f;
  }
  P_ rd[R], rx[R], ra[R], rg[R];
  auto fetch = [&](int64_t base) {
    const int64_t row0 = base + (NW - 1 - wave) * R;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t row = row0 + q < end ? row0 + q : end - 1;
      rd[q].load_nt(dout + row * p.do_st);
      rx[q].load_nt(x + row * p.x_st);
      ra[q].load_nt(ga + row * p.ga_st);
      rg[q].load_nt(gx + row * p.gx_st);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) mark[v] = p.marks[mark_row(start, b, base - start) * p.dim + c + v];
  };
  int64_t base = start + (end - 1 - start) / kTile * kTile;
  if (end > start) fetch(base);
  for (int turn = 0; end > start && base >= start; base -= kTile, turn ^= 1) {
    const int64_t row0 = base + (NW - 1 - wave) * R;
    float g[R][V], xf[R][V], a[R][V], r[R][V], i[R][V], m[R][V], over[R][V];
    float P[V], H[V], T[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] = 1.f;
      H[v] = T[v] = 0.f;
      h[v] = mark[v];
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      rd[q].to_float(g[q]);
      rx[q].to_float(xf[q]);
      ra[q].to_float(r[q]);
      rg[q].to_float(i[q]);
      const bool in = row0 + q < end;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        g[q][v] = in ? g[q][v] : 0.f;
        xf[q][v] = in ? xf[q][v] : 0.f;
        r[q][v] = in ? r[q][v] : -INFINITY;  // r = 0: a = 1, u = 0, no part in a sum
        i[q][v] = in ? i[q][v] : 0.f;
        const GatesInv f = make_gates_inv(r[q][v], i[q][v], d[v]);
        const float ix = f.i * xf[q][v];
        r[q][v] = f.r;
        i[q][v] = f.i;
        a[q][v] = f.a;
        m[q][v] = f.m;
        over[q][v] = f.a * f.inv_m * ix;
        H[v] = __builtin_fmaf(f.a, H[v], f.m * ix);
        P[v] *= f.a;
      }
    }
    if (base > start) fetch(base - kTile);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int q = R - 1; q >= 0; --q) T[v] = a[q][v] * (T[v] + g[q][v]);
      mp[turn][wave][v][lane] = P[v];
      mh[turn][wave][v][lane] = H[v];
      mt[turn][wave][v][lane] = T[v];
    }
    __syncthreads();
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        if (q == wave) s[v] = carry[v];
        carry[v] = __builtin_fmaf(mp[turn][q][v][lane], carry[v], mt[turn][q][v][lane]);
      }
      for (int q = NW - 1; q > wave; --q)  // the rows before this wave's
        h[v] = __builtin_fmaf(mp[turn][q][v][lane], h[v], mh[turn][q][v][lane]);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const float next = __builtin_fmaf(a[q][v], h[v], m[q][v] * (i[q][v] * xf[q][v]));
        over[q][v] = h[v] - over[q][v];
        h[v] = next;
      }
    }
#pragma unroll
    for (int q = R - 1; q >= 0; --q) {
      float ox[V], oa[V], og[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float dh = g[q][v] + s[v];
        s[v] = a[q][v] * dh;
        ox[v] = dh * (m[q][v] * i[q][v]);
        const float dlog = s[v] * over[q][v];
        acc[v] = __builtin_fmaf(dlog, r[q][v], acc[v]);
        og[v] = ox[v] * xf[q][v] * (1.f - i[q][v]);
        oa[v] = -d[v].k * dlog * (r[q][v] * (1.f - r[q][v]));
      }
      if (live && row0 + q < end) {
        const int64_t row = row0 + q;
        P_ o;
        o.from_float(ox);
        o.store_nt(dx + row * p.dx_st);
        o.from_float(og);
        o.store_nt(dgx + row * p.dgx_st);
        o.from_float(oa);
        o.store_nt(dga + row * p.dga_st);
      }
    }
  }
  // ddecay's sum over the waves, in their order
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) mp[0][wave][v][lane] = acc[v];
  __syncthreads();
  if (wave != 0 || !live) return;
  const bool init = p.has_init && p.has_init[b] != 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) sum += mp[0][q][v][lane];
    p.partial[(int64_t)b * p.dim + c + v] = sum;
    if (p.dinitial) p.dinitial[slot * p.di_slot + c + v] = init ? carry[v] : 0.f;
  }
}

// ddecay[c] = -scale sigmoid(decay[c]) * the sequences' sums.
__global__ __launch_bounds__(kSumCols * kSumGroups) void rec_ddecay_kernel(
    const float* partial, const float* decay, float* ddecay, int32_t batch, int32_t dim,
    float scale) {
  column_sum(partial, batch, dim,
             [&](int64_t c, float v) { ddecay[c] = -scale * sigmoid(decay[c]) * v; });
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

template <typename D, bool VEC>
static void launch_fwd(int nw, const RecFwdParams& p, uint32_t grid, hipStream_t s) {
  switch (nw) {
    case 1: hipLaunchKernelGGL((rec_fwd_kernel<D, VEC, 1>), dim3(grid), dim3(256), 0, s, p); break;
    case 4: hipLaunchKernelGGL((rec_fwd_kernel<D, VEC, 4>), dim3(grid), dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((rec_fwd_kernel<D, VEC, 16>), dim3(grid), dim3(1024), 0, s, p); break;
  }
}

template <typename D, bool VEC>
static void launch_bwd(int nw, const RecBwdParams& p, uint32_t grid, hipStream_t s) {
  switch (nw) {
    case 1: hipLaunchKernelGGL((rec_bwd_kernel<D, VEC, 1>), dim3(grid), dim3(256), 0, s, p); break;
    case 4: hipLaunchKernelGGL((rec_bwd_kernel<D, VEC, 4>), dim3(grid), dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((rec_bwd_kernel<D, VEC, 16>), dim3(grid), dim3(1024), 0, s, p); break;
  }
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

// Whether a packed call runs with channels in lanes (every plane has its
// channels side by side).
static bool side_by_side(std::initializer_list<Plane> planes) {
  for (const Plane& a : planes)
    if (a.sc != 1) return false;
  return true;
}

// Vector lanes of V channels: every row starts on a multiple of V elements.
static bool row_lanes(std::initializer_list<Plane> planes, int64_t V) {
  for (const Plane& a : planes)
    if (a.nc % V != 0 || a.st % V != 0 || !aligned_to(a.p, V * a.es)) return false;
  return true;
}

// Vector lanes of eight tokens: tokens side by side, at any alignment.
static bool token_lanes(std::initializer_list<Plane> planes) {
  for (const Plane& a : planes)
    if (a.st != 1) return false;
  return true;
}

// Waves that walk one sequence together.
static int waves_per_pair(int64_t pairs, int64_t total_T, int32_t batch) {
  const int64_t mean = total_T / batch;
  if (pairs < 512 && mean >= 8 * kChunkTokens) return 16;
  if (pairs < 8192 && mean >= 2 * kChunkTokens) return 4;
  return 1;
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
  const auto planes = {px, pa, pg, po};
  if (side_by_side(planes) && dim > 1) {
    const bool two = row_lanes(planes, 2);
    const int64_t grid = batch * cdiv(dim, two ? 128 : 64);
    if (!valid_grid(grid, kRowWaves * 64))
      return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
    const dim3 g((uint32_t)grid), th(kRowWaves * 64);
    if (dtype == SCONV_BF16) {
      if (two) hipLaunchKernelGGL((rec_fwd_rows_kernel<Bf16, 2>), g, th, 0, stream, p);
      else hipLaunchKernelGGL((rec_fwd_rows_kernel<Bf16, 1>), g, th, 0, stream, p);
    } else {
      if (two) hipLaunchKernelGGL((rec_fwd_rows_kernel<F32, 2>), g, th, 0, stream, p);
      else hipLaunchKernelGGL((rec_fwd_rows_kernel<F32, 1>), g, th, 0, stream, p);
    }
    return check_launch(fn);
  }
  const bool vec = token_lanes(planes);
  const int nw = waves_per_pair(p.num_pairs, total_T, batch);
  const int64_t grid = nw == 1 ? cdiv(p.num_pairs, 4) : p.num_pairs;
  if (!valid_grid(grid, nw > 4 ? nw * 64 : 256))
    return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
  if (dtype == SCONV_BF16) {
    if (vec) launch_fwd<Bf16, true>(nw, p, (uint32_t)grid, stream);
    else launch_fwd<Bf16, false>(nw, p, (uint32_t)grid, stream);
  } else {
    if (vec) launch_fwd<F32, true>(nw, p, (uint32_t)grid, stream);
    else launch_fwd<F32, false>(nw, p, (uint32_t)grid, stream);
  }
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
  const auto planes = {in[0], in[1], in[2], in[3], ou[0], ou[1], ou[2]};
  if (batch > 0 && side_by_side(planes) && dim > 1) {
    const bool two = row_lanes(planes, 2);
    const int64_t grid = batch * cdiv(dim, two ? 128 : 64);
    if (!valid_grid(grid, kRowBwdWaves * 64))
      return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
    const dim3 g((uint32_t)grid), th(kRowBwdWaves * 64);
    if (dtype == SCONV_BF16) {
      if (two) hipLaunchKernelGGL((rec_bwd_rows_kernel<Bf16, 2>), g, th, 0, stream, p);
      else hipLaunchKernelGGL((rec_bwd_rows_kernel<Bf16, 1>), g, th, 0, stream, p);
    } else {
      if (two) hipLaunchKernelGGL((rec_bwd_rows_kernel<F32, 2>), g, th, 0, stream, p);
      else hipLaunchKernelGGL((rec_bwd_rows_kernel<F32, 1>), g, th, 0, stream, p);
    }
    if (const int rc = check_launch(fn)) return rc;
  } else if (batch > 0) {
    const bool vec = token_lanes(planes);
    const int nw = waves_per_pair(p.num_pairs, total_T, batch);
    const int64_t grid = nw == 1 ? cdiv(p.num_pairs, 4) : p.num_pairs;
    if (!valid_grid(grid, nw > 4 ? nw * 64 : 256))
      return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
    if (dtype == SCONV_BF16) {
      if (vec) launch_bwd<Bf16, true>(nw, p, (uint32_t)grid, stream);
      else launch_bwd<Bf16, false>(nw, p, (uint32_t)grid, stream);
    } else {
      if (vec) launch_bwd<F32, true>(nw, p, (uint32_t)grid, stream);
      else launch_bwd<F32, false>(nw, p, (uint32_t)grid, stream);
    }
    if (const int rc = check_launch(fn)) return rc;
  }
  hipLaunchKernelGGL(rec_ddecay_kernel, dim3((uint32_t)cdiv(dim, kSumCols)),
                     dim3(kSumCols * kSumGroups), 0, stream, workspace, decay, ddecay, batch, dim, decay_scale);
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
