// gated_recurrence.hip -- gated linear recurrence over packed
// variable-length sequences with a slot-indexed state pool (prefill), its
// gradients, and its one-token decode step, for gfx950.
//
// The recurrence is the layer step behind the short conv: it takes the
// conv's packing (query_start_loc), state slots and layouts.
#include <initializer_list>
#include <type_traits>

#include "column_sum.h"
#include "plane_host.h"
#include "recurrence_device.h"
#include "row_lanes.h"

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
  float *maps, *saved;  // segments: [segments, dim, 2] and [segments, dim]
  int64_t x_sc, x_st, ga_sc, ga_st, gx_sc, gx_st, o_sc, o_st, ss_slot, total_T, num_pairs;
  int32_t seg_rows;  // rows of a segment
  int32_t sorted;    // the longest sequences first
  uint32_t pad_lds;  // unused LDS of a workgroup (host: fewer on a CU)
  float scale;
  int32_t batch, dim, pad_slot_id;
};

struct RecBwdParams {
  const void *dout, *x, *ga, *gx;
  const float *decay, *marks;
  const int32_t* qsl;
  const int32_t* cache_indices;
  const uint8_t* has_init;
  const float* dfinal;
  float* dinitial;
  void *dx, *dga, *dgx;
  float* partial;  // [batch or segments, dim] sums over tokens of r * dlog a
  float *maps, *saved;  // as the forward's
  int64_t do_sc, do_st, x_sc, x_st, ga_sc, ga_st, gx_sc, gx_st;
  int64_t dx_sc, dx_st, dga_sc, dga_st, dgx_sc, dgx_st;
  int64_t df_slot, di_slot, total_T, num_pairs;
  int32_t seg_rows, sorted;
  float scale;
  int32_t batch, dim, pad_slot_id;
};

// The checkpoint row of sequence b's token start + rel (rel a multiple of
// 32): rows of later sequences lie behind it, since a sequence of L tokens has
// ceil(L / 32) of them and ends less than 32 ceil(L / 32) after its start.
__device__ __forceinline__ int64_t mark_row(int64_t start, int b, int64_t rel) {
  return start / kMarkTokens + b + rel / kMarkTokens;
}

// ---------------------------------------------------------------- tokens in lanes

// A wave takes a chunk of 512 tokens of one channel, counted from the
// sequence's start, lane l the tokens [8 l, 8 l + 8) of it.  The
// recurrence is a composition of maps h -> a h + u: a lane composes its
// eight, the wave its lanes (six DPP steps), and NW waves that walk one
// sequence together exchange their chunks' maps through LDS, so that no
// state ever waits for another workgroup and every input is read once:
// 8 x 4096 x 8192 bf16 363 us, 5.9 TB/s; 35 vector instructions an element.
// Tokens past the sequence are the identity (a = 1, u = 0).
template <typename D, bool VEC, int NW>
__global__ __launch_bounds__(NW > 4 ? NW * 64 : 256) void rec_fwd_kernel(const RecFwdParams p) {
  using S = typename D::storage;
  constexpr int N = kLaneTokens, kWaves = NW > 4 ? NW : 4;
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
    const int64_t t = base + lane * N;
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
    const int64_t t = base + lane * N;
    float a[N], u[N];
    float P = 1.f, H = 0.f;
    const bool any = base < end;
    if (any) {
      // the last chunk: this lane's tokens from `n` on are not the sequence's
      const int n = t + N <= end ? N : t < end ? (int)(end - t) : 0;
      auto gates = [&](auto edge) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const Gates g = make_gates(ra.get(e), rg.get(e), d);
          const bool in = !decltype(edge)::value || e < n;
          a[e] = in ? g.a : 1.f;
          u[e] = in ? g.m * (g.i * rx.get(e)) : 0.f;
          H = __builtin_fmaf(a[e], H, u[e]);
          P *= a[e];
        }
      };
      if (base + kChunkTokens <= end) gates(std::false_type());
      else gates(std::true_type());
      in_order();
      fetch(base + NW * kChunkTokens);
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
    if (p.marks && lane % (kMarkTokens / N) == 0 && t < end)
      p.marks[mark_row(start, b, t - start) * p.dim + c] = h;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      h = __builtin_fmaf(a[e], h, u[e]);
      u[e] = h;
    }
    Raw8<D> o;
    o.from_float(u);
    o.template store<VEC>(out, p.o_st, t, end);
  }
  if (p.states && sub == 0 && lane == 0) p.states[slot * p.ss_slot + c] = carry;
}

// The gradients, tokens in lanes, from the end of the sequence: lane l of a
// chunk takes tokens [8 (63 - l), 8 (63 - l) + 8), so that the gradient of
// the state, which runs against time, runs up the lanes.  The states come
// from the checkpoints: each row of 16 lanes (128 tokens) starts from its
// own, and only composes inside the row.  The gates are computed once.
// 63 vector instructions an element, and bytes: 1 x 65536 x 1024 bf16 192 us
// (4.9 TB/s of 14 bytes an element).
template <typename D, bool VEC, int NW>
__global__ __launch_bounds__(NW > 4 ? NW * 64 : 256, VEC && NW == 1 && sizeof(typename D::storage) == 2 ? 4 : 1)
void rec_bwd_kernel(const RecBwdParams p) {
  using S = typename D::storage;
  constexpr int N = kLaneTokens, kWaves = NW > 4 ? NW : 4;
  constexpr int kPairs = kWaves / NW;
  static_assert(kPairs == 1 || NW == 1, "a barrier is met by one pair only");
  __shared__ float2 maps[2][kPairs][NW];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int sub = wave % NW, mine = wave / NW;
  const int64_t pair = (int64_t)xcd_groups<8>(blockIdx.x, gridDim.x) * kPairs + mine;
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
  const int back = (63 - lane) * N;
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
    float g[N], xf[N], a[N], r[N], i[N], m[N], over[N];  // over: a i x / m
    float P = 1.f, H = 0.f, T = 0.f, h0 = 0.f;
    if (any) {
      const int n = t + N <= end ? N : t < end ? (int)(end - t) : 0;
      h0 = mark;
      auto gates = [&](auto edge) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const bool in = !decltype(edge)::value || e < n;
          g[e] = in ? rd.get(e) : 0.f;
          xf[e] = in ? rx.get(e) : 0.f;
          // r = 0 past the end: a = 1, u = 0, no part in a sum
          const GatesInv q = make_gates_inv(in ? ra.get(e) : -INFINITY, in ? rg.get(e) : 0.f, d);
          const float ix = q.i * xf[e];
          r[e] = q.r;
          i[e] = q.i;
          a[e] = q.a;
          m[e] = q.m;
          over[e] = q.a * q.inv_m * ix;
          H = __builtin_fmaf(q.a, H, q.m * ix);
          P *= q.a;
        }
      };
      if (base + kChunkTokens <= end) gates(std::false_type());
      else gates(std::true_type());
      in_order();
      fetch(base - NW * kChunkTokens);
      // states before each token, less a i x / m
      const float A = P;
      scan_row_down(P, H);
      float h = __builtin_fmaf(lane_move<0x101>(1.0f, P), h0, lane_move<0x101>(0.0f, H));
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float next = __builtin_fmaf(a[e], h, m[e] * (i[e] * xf[e]));
        over[e] = h - over[e];
        h = next;
      }
      // s -> a (dout + s), from the last token to the first
#pragma unroll
      for (int e = N - 1; e >= 0; --e) T = a[e] * (T + g[e]);
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
    for (int e = N - 1; e >= 0; --e) {
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

// ---------------------------------------------------------------- channels in lanes

// For channels that lie side by side (rows of tokens): lane l takes V
// channels, wave w of a workgroup R rows of each tile of NW * R = 64 tokens
// (counted from the sequence's start, so that a tile starts at a checkpoint),
// and the tile's maps meet in LDS.
//
// A workgroup takes one sequence where they are many, and else (SEG) a
// segment of rows of the flat token axis, whatever sequences it meets: the
// tiles that start in it.  Then a launch before has composed each segment's
// maps of the one sequence that goes on behind it, and a workgroup composes
// the segments before its own; a sequence that starts in a segment has its
// initial state folded into that map, so a composition starts from zero.
// The inputs are read twice then (14 bytes an element in bf16, not 8).
constexpr int kTile = 64;

// First token at or after row `at` that starts a tile of the sequence.
__device__ __forceinline__ int tile_start(int start, int at) {
  return at <= start ? start : start + (at - start + kTile - 1) / kTile * kTile;
}

// The part of a sequence whose tiles start in rows [lo, hi).
struct Part {
  int start, end, from, to;
  __device__ __forceinline__ Part(const int32_t* qsl, int b, int lo, int hi) {
    start = qsl[b];
    end = qsl[b + 1];
    from = tile_start(start, lo);
    to = tile_start(start, hi);
    to = to < end ? to : end;
  }
};

// Composes the maps of segments [first, last) in steps of `by` (1 or -1)
// from `first`, all waves of the workgroup together.
template <int V, int NW, typename M>
__device__ __forceinline__ void compose_segments(const float* seg_maps, int64_t dim, int c,
                                                 int first, int count, int by, int lane,
                                                 int wave, M (&maps)[NW][64], float (&h)[V]) {
  const int per = (count + NW - 1) / NW;
  const int j0 = wave * per, j1 = j0 + per < count ? j0 + per : count;
  M m;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    m.P[v] = 1.f;
    m.H[v] = 0.f;
  }
#pragma unroll 8
  for (int j = j0; j < j1; ++j) {
    const float* q = seg_maps + ((int64_t)(first + by * j) * dim + c) * 2;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m.H[v] = __builtin_fmaf(q[2 * v], m.H[v], q[2 * v + 1]);
      m.P[v] *= q[2 * v];
    }
  }
  maps[wave][lane] = m;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const M f = maps[w][lane];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(f.P[v], h[v], f.H[v]);
  }
  __syncthreads();
}

template <int V>
struct alignas(8 * V) RowMap { float P[V], H[V]; };

constexpr int kFwdWaves = 8;

template <typename D, int V, bool SEG>
__global__ __launch_bounds__(kFwdWaves * 64) void rec_fwd_rows_kernel(const RecFwdParams p) {
  using S = typename D::storage;
  using P_ = Pack<D, V>;
  constexpr int NW = kFwdWaves, R = kTile / NW;
  // Tiles of loads in flight: a long sequence alone on its CUs waits for them
  // (16 ragged x 4096: 154 against 163 us); where many segments share the
  // CUs, the registers are worth more (1 x 32768 x 1024: 102, with two 112).
  constexpr int kAhead = SEG ? 1 : 2;
  __shared__ RowMap<V> maps[2][NW][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t slabs = (uint32_t)((p.dim + 64 * V - 1) / (64 * V));
  const int unit = (int)(blockIdx.x / slabs);  // sequence or segment
  // lanes past the last channel read it and write nothing
  const int ch = (int)((blockIdx.x % slabs) * 64 + lane) * V;
  const bool live = ch < p.dim;
  const int c = live ? ch : p.dim - V;
  const uint32_t off = (uint32_t)c * (uint32_t)sizeof(S);
  const int total = (int)p.total_T, lo = SEG ? unit * p.seg_rows : 0;
  const bool last = !SEG || total - lo <= p.seg_rows;
  const int hi = last ? total : lo + p.seg_rows;
  const S* x = static_cast<const S*>(p.x);  // may be out
  const S* ga = static_cast<const S*>(p.ga);
  const S* gx = static_cast<const S*>(p.gx);
  S* out = static_cast<S*>(p.out);
  Decay d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = make_decay(p.decay[c + v], p.scale);
  int turn = 0;
  const int b0 = SEG        ? first_sequence(p.qsl, p.batch, lo)
                 : p.sorted ? by_length(p.qsl, p.batch, unit)
                            : unit;
  const int b1 = SEG ? p.batch : b0 + 1;
  for (int b = b0; b < b1; ++b) {
    const Part s(p.qsl, b, lo, hi);
    if (SEG && s.start >= hi && !(last && p.states)) break;  // nothing to keep of an empty one
    const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
    const bool opens = s.start >= lo;  // its first token, or its place if it has none
    if (slot == p.pad_slot_id || (s.from >= s.to && !(opens && s.start == s.end))) continue;
    float carry[V];
    if (!SEG || opens) {
      const bool init = p.has_init && p.has_init[b] != 0;
      // a sequence that goes on: its slot may hold its last state already
      const float* from = SEG && s.to < s.end ? p.saved + (int64_t)unit * p.dim : p.states + slot * p.ss_slot;
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = init ? from[c + v] : 0.f;
    } else {
      const int first = s.start / p.seg_rows;
      compose_segments<V, NW>(p.maps, p.dim, c, first, unit - first, 1, lane, wave, maps[turn], carry);
    }
    P_ rx[kAhead][R], ra[kAhead][R], rg[kAhead][R];
    auto fetch = [&](auto which, int base) {
      constexpr int k = decltype(which)::value;
      const int row0 = base + wave * R;
      load_rows(rx[k], x, p.x_st, row0, s.end, off);
      load_rows(ra[k], ga, p.ga_st, row0, s.end, off);
      load_rows(rg[k], gx, p.gx_st, row0, s.end, off);
    };
    auto tile = [&](auto which, int base) {
      constexpr int k = decltype(which)::value;
      const int row0 = base + wave * R;
      float pl[R][V], hl[R][V];
      RowMap<V> m;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        m.P[v] = 1.f;
        m.H[v] = 0.f;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float xf[V], af[V], gf[V];
        rx[k][r].to_float(xf);
        ra[k][r].to_float(af);
        rg[k][r].to_float(gf);
        const bool in = row0 + r < s.end;
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
      maps[turn][wave][lane] = m;
      if (base + kAhead * kTile < s.to) fetch(which, base + kAhead * kTile);
      __syncthreads();
      float h[V];
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        const RowMap<V> f = maps[turn][q][lane];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (q == wave) h[v] = carry[v];
          carry[v] = __builtin_fmaf(f.P[v], carry[v], f.H[v]);
        }
      }
      const uint32_t at = lane_offset(off);
      if (p.marks && wave * R % kMarkTokens == 0 && live && row0 < s.end) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          p.marks[mark_row(s.start, b, row0 - s.start) * p.dim + c + v] = h[v];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = __builtin_fmaf(pl[r][v], h[v], hl[r][v]);
        P_ o;
        o.from_float(y);
        if (live && row0 + r < s.end) o.store_nt(in_row(out + (int64_t)(row0 + r) * p.o_st, at));
      }
      turn ^= 1;
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, kAhead - 1> odd;
    if (s.from < s.to) fetch(even, s.from);
    if (kAhead == 2 && s.from + kTile < s.to) fetch(odd, s.from + kTile);
    for (int base = s.from; base < s.to; base += kAhead * kTile) {
      tile(even, base);
      if (kAhead == 2 && base + kTile < s.to) tile(odd, base + kTile);
    }
    if (p.states && s.to == s.end && wave == 0 && live) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.states[slot * p.ss_slot + c + v] = carry[v];
    }
  }
}

// Rows [from, to) cut into one run a wave, walked R rows at a time.
constexpr int kMapWaves = 8, kMapRows = 8;

// The map of the one sequence that goes on behind each segment, over its
// tiles in the segment.
template <typename D, int V>
__global__ __launch_bounds__(kMapWaves * 64) void rec_fwd_map_kernel(const RecFwdParams p) {
  using S = typename D::storage;
  using P_ = Pack<D, V>;
  constexpr int NW = kMapWaves, R = kMapRows;
  __shared__ RowMap<V> maps[NW][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t slabs = (uint32_t)((p.dim + 64 * V - 1) / (64 * V));
  const int unit = (int)(blockIdx.x / slabs), total = (int)p.total_T, lo = unit * p.seg_rows;
  const int hi = total - lo <= p.seg_rows ? total : lo + p.seg_rows;
  const int ch = (int)((blockIdx.x % slabs) * 64 + lane) * V;
  const bool live = ch < p.dim;
  const int c = live ? ch : p.dim - V;
  const uint32_t off = (uint32_t)c * (uint32_t)sizeof(S);
  const int b = first_sequence(p.qsl, p.batch, hi + 1);  // the first that ends behind hi
  if (b >= p.batch) return;
  const Part s(p.qsl, b, lo, hi);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (s.start >= hi || s.to >= s.end || slot == p.pad_slot_id) return;
  const S* x = static_cast<const S*>(p.x);
  const S* ga = static_cast<const S*>(p.ga);
  const S* gx = static_cast<const S*>(p.gx);
  Decay d[V];
  RowMap<V> m;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    d[v] = make_decay(p.decay[c + v], p.scale);
    m.P[v] = 1.f;
    m.H[v] = 0.f;
  }
  const int per = (s.to - s.from + NW - 1) / NW;
  const int from = s.from + wave * per, to = from + per < s.to ? from + per : s.to;
  P_ rx[R], ra[R], rg[R];
  auto fetch = [&](int row0) {
    load_rows(rx, x, p.x_st, row0, to, off);
    load_rows(ra, ga, p.ga_st, row0, to, off);
    load_rows(rg, gx, p.gx_st, row0, to, off);
  };
  if (from < to) fetch(from);
  for (int row0 = from; row0 < to; row0 += R) {
    P_ cx[R], ca[R], cg[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      cx[r] = rx[r];
      ca[r] = ra[r];
      cg[r] = rg[r];
    }
    if (row0 + R < to) fetch(row0 + R);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float xf[V], af[V], gf[V];
      cx[r].to_float(xf);
      ca[r].to_float(af);
      cg[r].to_float(gf);
      const bool in = row0 + r < to;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gates g = make_gates(af[v], gf[v], d[v]);
        m.H[v] = __builtin_fmaf(in ? g.a : 1.f, m.H[v], in ? g.m * (g.i * xf[v]) : 0.f);
        m.P[v] *= in ? g.a : 1.f;
      }
    }
  }
  maps[wave][lane] = m;
  __syncthreads();
  if (wave != 0 || !live) return;
  const bool opens = s.start >= lo, init = opens && p.has_init && p.has_init[b] != 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float P = 1.f, H = 0.f;
    if (opens) {
      P = 0.f;
      H = init ? p.states[slot * p.ss_slot + c + v] : 0.f;
      p.saved[(int64_t)unit * p.dim + c + v] = H;
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      H = __builtin_fmaf(maps[w][lane].P[v], H, maps[w][lane].H[v]);
      P *= maps[w][lane].P[v];
    }
    p.maps[((int64_t)unit * p.dim + c + v) * 2] = P;
    p.maps[((int64_t)unit * p.dim + c + v) * 2 + 1] = H;
  }
}

// The gradients, from the end: wave w takes the R rows of a tile that are
// w R from its end.  The forward maps and the backward ones, which share
// their factor, meet in LDS together.
// Tiles of 64 tokens (eight waves) for whole sequences, whose chain of tiles
// is what they wait for; of 32 (four waves) for segments, so that three
// workgroups share a CU where eight waves leave room for one (8000 x 2048 bf16,
// forward and gradients: 134 against 147 us; 33 ragged x 1001 fp32: 162 and 137).
template <bool SEG>
constexpr int kBwdWaves = SEG ? 4 : 8;

template <typename D, int V, bool SEG>
__global__ __launch_bounds__(kBwdWaves<SEG> * 64) void rec_bwd_rows_kernel(const RecBwdParams p) {
  using S = typename D::storage;
  using P_ = Pack<D, V>;
  constexpr int NW = kBwdWaves<SEG>, R = 8, kBwdTile = NW * R;
  static_assert(kBwdTile % kMarkTokens == 0, "a tile starts at a checkpoint");
  __shared__ RowMap<V> maps[2][NW][64];  // s -> P s + H
  __shared__ float mh[2][NW][V][64];     // h -> P h + mh
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t slabs = (uint32_t)((p.dim + 64 * V - 1) / (64 * V));
  const int unit = (int)(blockIdx.x / slabs);
  const int ch = (int)((blockIdx.x % slabs) * 64 + lane) * V;
  const bool live = ch < p.dim;
  const int c = live ? ch : p.dim - V;
  const uint32_t off = (uint32_t)c * (uint32_t)sizeof(S);
  const int total = (int)p.total_T, lo = SEG ? unit * p.seg_rows : 0;
  const bool last = !SEG || total - lo <= p.seg_rows;
  const int hi = last ? total : lo + p.seg_rows;
  const S* dout = static_cast<const S*>(p.dout);
  const S* x = static_cast<const S*>(p.x);
  const S* ga = static_cast<const S*>(p.ga);
  const S* gx = static_cast<const S*>(p.gx);
  S* dx = static_cast<S*>(p.dx);
  S* dga = static_cast<S*>(p.dga);
  S* dgx = static_cast<S*>(p.dgx);
  Decay d[V];
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    d[v] = make_decay(p.decay[c + v], p.scale);
    acc[v] = 0.f;
  }
  int turn = 0;
  const int b0 = SEG        ? first_sequence(p.qsl, p.batch, lo)
                 : p.sorted ? by_length(p.qsl, p.batch, unit)
                            : unit;
  const int b1 = SEG ? p.batch : b0 + 1;
  for (int b = b0; b < b1; ++b) {
    const Part q(p.qsl, b, lo, hi);
    if (SEG && q.start >= hi && !(last && p.dinitial)) break;
    const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
    const bool opens = q.start >= lo;
    if (slot == p.pad_slot_id || (q.from >= q.to && !(opens && q.start == q.end))) continue;
    float carry[V];
    if (!SEG || q.to == q.end) {
      // a sequence that began before: dfinal's slot may hold its dinitial already
      const float* from = SEG && !opens ? p.saved + (int64_t)unit * p.dim : p.dfinal + slot * p.df_slot;
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = p.dfinal ? from[c + v] : 0.f;
    } else {
      // from the segment of the last tile down to the next one
      const int top = (q.start + (q.end - 1 - q.start) / kTile * kTile) / p.seg_rows;
      compose_segments<V, NW>(p.maps, p.dim, c, top, top - unit, -1, lane, wave, maps[turn], carry);
    }
    P_ rd[R], rx[R], ra[R], rg[R];
    float mark[V];
    auto fetch = [&](int base) {
      const int row0 = base + (NW - 1 - wave) * R;
      load_rows(rd, dout, p.do_st, row0, q.end, off);
      load_rows(rx, x, p.x_st, row0, q.end, off);
      load_rows(ra, ga, p.ga_st, row0, q.end, off);
      load_rows(rg, gx, p.gx_st, row0, q.end, off);
#pragma unroll
      for (int v = 0; v < V; ++v) mark[v] = p.marks[mark_row(q.start, b, base - q.start) * p.dim + c + v];
    };
    int base = q.start + (q.to - 1 - q.start) / kBwdTile * kBwdTile;
    if (q.to > q.from) fetch(base);
    for (; q.to > q.from && base >= q.from; base -= kBwdTile, turn ^= 1) {
      const int row0 = base + (NW - 1 - wave) * R;
      float g[R][V], xf[R][V], a[R][V], r[R][V], i[R][V], m[R][V], over[R][V];
      float P[V], H[V], T[V], h[V], s[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        P[v] = 1.f;
        H[v] = T[v] = 0.f;
        h[v] = mark[v];
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        rd[k].to_float(g[k]);
        rx[k].to_float(xf[k]);
        ra[k].to_float(r[k]);
        rg[k].to_float(i[k]);
        const bool in = row0 + k < q.end;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          g[k][v] = in ? g[k][v] : 0.f;
          xf[k][v] = in ? xf[k][v] : 0.f;
          // r = 0 past the end: a = 1, u = 0, no part in a sum
          const GatesInv f = make_gates_inv(in ? r[k][v] : -INFINITY, in ? i[k][v] : 0.f, d[v]);
          const float ix = f.i * xf[k][v];
          r[k][v] = f.r;
          i[k][v] = f.i;
          a[k][v] = f.a;
          m[k][v] = f.m;
          over[k][v] = f.a * f.inv_m * ix;
          H[v] = __builtin_fmaf(f.a, H[v], f.m * ix);
          P[v] *= f.a;
        }
      }
      RowMap<V> f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = R - 1; k >= 0; --k) T[v] = a[k][v] * (T[v] + g[k][v]);
        f.P[v] = P[v];
        f.H[v] = T[v];
        mh[turn][wave][v][lane] = H[v];
      }
      maps[turn][wave][lane] = f;
      if (base > q.from) fetch(base - kBwdTile);
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        f = maps[turn][w][lane];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (w == wave) s[v] = carry[v];
          carry[v] = __builtin_fmaf(f.P[v], carry[v], f.H[v]);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        for (int w = NW - 1; w > wave; --w)  // the rows before this wave's
          h[v] = __builtin_fmaf(maps[turn][w][lane].P[v], h[v], mh[turn][w][v][lane]);
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const float next = __builtin_fmaf(a[k][v], h[v], m[k][v] * (i[k][v] * xf[k][v]));
          over[k][v] = h[v] - over[k][v];
          h[v] = next;
        }
      }
      const uint32_t at = lane_offset(off);
      // ddecay's terms of a tile first, then the tiles: T / 64 + 8 additions
      // behind one another, not T / 8
      float part[V];
#pragma unroll
      for (int v = 0; v < V; ++v) part[v] = 0.f;
#pragma unroll
      for (int k = R - 1; k >= 0; --k) {
        float ox[V], oa[V], og[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float dh = g[k][v] + s[v];
          s[v] = a[k][v] * dh;
          ox[v] = dh * (m[k][v] * i[k][v]);
          const float dlog = s[v] * over[k][v];
          part[v] = __builtin_fmaf(dlog, r[k][v], part[v]);
          og[v] = ox[v] * xf[k][v] * (1.f - i[k][v]);
          oa[v] = -d[v].k * dlog * (r[k][v] * (1.f - r[k][v]));
        }
        if (live && row0 + k < q.end) {
          const int64_t row = row0 + k;
          P_ o;
          o.from_float(ox);
          o.store_nt(in_row(dx + row * p.dx_st, at));
          o.from_float(og);
          o.store_nt(in_row(dgx + row * p.dgx_st, at));
          o.from_float(oa);
          o.store_nt(in_row(dga + row * p.dga_st, at));
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += part[v];
    }
    if (p.dinitial && opens && wave == 0 && live) {
      const bool init = p.has_init && p.has_init[b] != 0;
#pragma unroll
      for (int v = 0; v < V; ++v) p.dinitial[slot * p.di_slot + c + v] = init ? carry[v] : 0.f;
    }
  }
  // ddecay's sum over the waves, in their order
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) mh[0][wave][v][lane] = acc[v];
  __syncthreads();
  if (wave != 0 || !live) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += mh[0][w][v][lane];
    p.partial[(int64_t)unit * p.dim + c + v] = sum;  // in this launch's order of units
  }
}

// The backward map of the one sequence that began before each segment, over
// its tiles in the segment, from the last to the first: s -> a (dout + s).
template <typename D, int V>
__global__ __launch_bounds__(kMapWaves * 64) void rec_bwd_map_kernel(const RecBwdParams p) {
  using S = typename D::storage;
  using P_ = Pack<D, V>;
  constexpr int NW = kMapWaves, R = kMapRows;
  __shared__ RowMap<V> maps[NW][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t slabs = (uint32_t)((p.dim + 64 * V - 1) / (64 * V));
  const int unit = (int)(blockIdx.x / slabs), total = (int)p.total_T, lo = unit * p.seg_rows;
  const int hi = total - lo <= p.seg_rows ? total : lo + p.seg_rows;
  const int ch = (int)((blockIdx.x % slabs) * 64 + lane) * V;
  const bool live = ch < p.dim;
  const int c = live ? ch : p.dim - V;
  const uint32_t off = (uint32_t)c * (uint32_t)sizeof(S);
  const int b = first_sequence(p.qsl, p.batch, lo + 1);  // the first that ends behind lo
  if (b >= p.batch) return;
  const Part s(p.qsl, b, lo, hi);
  const int64_t slot = p.cache_indices ? (int64_t)p.cache_indices[b] : (int64_t)b;
  if (s.start >= lo || s.from >= s.to || slot == p.pad_slot_id) return;
  const S* dout = static_cast<const S*>(p.dout);
  const S* ga = static_cast<const S*>(p.ga);
  Decay d[V];
  RowMap<V> m;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    d[v] = make_decay(p.decay[c + v], p.scale);
    m.P[v] = 1.f;
    m.H[v] = 0.f;
  }
  // wave 0 has the last run
  const int per = (s.to - s.from + NW - 1) / NW;
  const int from = s.from + (NW - 1 - wave) * per, to = from + per < s.to ? from + per : s.to;
  P_ rd[R], ra[R];
  // groups of R rows, the last first; the group at `from` may reach behind `to`
  auto fetch = [&](int row0) {
    load_rows(rd, dout, p.do_st, row0, to, off);
    load_rows(ra, ga, p.ga_st, row0, to, off);
  };
  const int top = from + (to - 1 - from) / R * R;
  if (from < to) fetch(top);
  for (int row0 = top; from < to && row0 >= from; row0 -= R) {
    P_ cd[R], ca[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      cd[r] = rd[r];
      ca[r] = ra[r];
    }
    if (row0 - R >= from) fetch(row0 - R);
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float df[V], af[V];
      cd[r].to_float(df);
      ca[r].to_float(af);
      const bool in = row0 + r < to;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float a = __builtin_amdgcn_exp2f(d[v].k_log2 * sigmoid(af[v]));
        m.H[v] = in ? a * (m.H[v] + df[v]) : m.H[v];
        m.P[v] *= in ? a : 1.f;
      }
    }
  }
  maps[wave][lane] = m;
  __syncthreads();
  if (wave != 0 || !live) return;
  const bool ends = s.to == s.end;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float P = 1.f, H = 0.f;
    if (ends) {
      P = 0.f;
      H = p.dfinal ? p.dfinal[slot * p.df_slot + c + v] : 0.f;
      p.saved[(int64_t)unit * p.dim + c + v] = H;
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      H = __builtin_fmaf(maps[w][lane].P[v], H, maps[w][lane].H[v]);
      P *= maps[w][lane].P[v];
    }
    p.maps[((int64_t)unit * p.dim + c + v) * 2] = P;
    p.maps[((int64_t)unit * p.dim + c + v) * 2 + 1] = H;
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

// One token: a lane a channel of one sequence.  The largest sizes are bound by
// bytes (511 x 4095 fp32: 11 us through a caller's loop, 4.5 TB/s), the smallest by
// latency (8 x 8192 bf16: 2.7 us).
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

// Unused LDS that leaves room for three workgroups of a CU (of eight) where
// waves walk long sequences: more of them at once read from too many places
// (8 x 4096 x 8192 bf16: 369 us with three, 400 with four, 465 with all;
// 16 sequences of 1088 tokens: 128 us with all, 154 with three).
constexpr uint32_t kLongPadLds = 53000;
constexpr int64_t kLongTokens = 2048;
// The same for a whole sequence in rows: two of three (16 ragged sequences x
// 4096: 163 against 170 us, one alone 182).
constexpr uint32_t kRowsPadLds = 60000;

template <typename D, bool VEC>
static void launch_fwd(int nw, const RecFwdParams& p, uint32_t grid, hipStream_t s) {
  switch (nw) {
    case 1: hipLaunchKernelGGL((rec_fwd_kernel<D, VEC, 1>), dim3(grid), dim3(256), p.pad_lds, s, p); break;
    case 4: hipLaunchKernelGGL((rec_fwd_kernel<D, VEC, 4>), dim3(grid), dim3(256), 0, s, p); break;
    default:
      if constexpr (VEC)
        hipLaunchKernelGGL((rec_fwd_kernel<D, VEC, 16>), dim3(grid), dim3(1024), 0, s, p);
      break;
  }
}

template <typename D, bool VEC>
static void launch_bwd(int nw, const RecBwdParams& p, uint32_t grid, hipStream_t s) {
  switch (nw) {
    case 1: hipLaunchKernelGGL((rec_bwd_kernel<D, VEC, 1>), dim3(grid), dim3(256), 0, s, p); break;
    case 4: hipLaunchKernelGGL((rec_bwd_kernel<D, VEC, 4>), dim3(grid), dim3(256), 0, s, p); break;
    default:
      if constexpr (VEC)
        hipLaunchKernelGGL((rec_bwd_kernel<D, VEC, 8>), dim3(grid), dim3(512), 0, s, p);
      break;
  }
}

template <typename D, int V>
static void launch_fwd_rows(const RecFwdParams& p, uint32_t grid, hipStream_t s) {
  const dim3 g(grid), th(kFwdWaves * 64), tm(kMapWaves * 64);
  if (p.seg_rows) {
    hipLaunchKernelGGL((rec_fwd_map_kernel<D, V>), g, tm, 0, s, p);
    hipLaunchKernelGGL((rec_fwd_rows_kernel<D, V, true>), g, th, 0, s, p);
  } else if constexpr (V == 1) {
    hipLaunchKernelGGL((rec_fwd_rows_kernel<D, 1, false>), g, th, p.sorted ? kRowsPadLds : 0, s, p);
  }
}

// One channel a lane: the rows of seven planes leave no registers for two.
template <typename D>
static void launch_bwd_rows(const RecBwdParams& p, uint32_t grid, hipStream_t s) {
  const dim3 g(grid), tm(kMapWaves * 64);
  if (p.seg_rows) {
    hipLaunchKernelGGL((rec_bwd_map_kernel<D, 1>), g, tm, 0, s, p);
    hipLaunchKernelGGL((rec_bwd_rows_kernel<D, 1, true>), g, dim3(kBwdWaves<true> * 64), 0, s, p);
  } else {
    hipLaunchKernelGGL((rec_bwd_rows_kernel<D, 1, false>), g, dim3(kBwdWaves<false> * 64), 0, s, p);
  }
}

// ---------------------------------------------------------------- host

// Checks shared by the two packed entry points; `fn` names the caller.
static int rec_check(const char* fn, int32_t batch, int32_t dim, int64_t total_T, int32_t dtype,
                     float scale) {
  if (batch < 0 || dim < 0 || total_T < 0)
    return fail(SCONV_ERR_INVALID, "%s: batch, dim and total_T must be >= 0", fn);
  if (total_T > INT32_MAX - 4096)  // token numbers are int32, as the offsets
    return fail(SCONV_ERR_UNSUPPORTED, "%s: total_T too large", fn);
  if (dim > 1 << 28)  // a lane's byte offset in a row is 32 bits
    return fail(SCONV_ERR_UNSUPPORTED, "%s: dim too large", fn);
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

// Whether workgroups of whole sequences in rows take the longest ones first (and
// leave each CU two of them): few sequences, of a few tiles and more, since the
// order costs a round trip.  Forward + gradients, us, in order of length and as
// they come, three draws of lengths each: 33 of 248 tokens x 1001 fp32 128, 117, 152 and
// 113, 111, 155 (equal lengths: 120 and 116); 40 of 200 x 1024 bf16 86, 141, 102 and 107,
// 140, 99; 33 of 300 x 1001 fp32 182, 132, 123 and 199, 151, 141; 60 of 300 x 2048 bf16
// 258, 256, 258 and 263, 284, 271; 40 of 400 x 2048 bf16 323, 204, 235 and 389, 241, 325.
static bool longest_first(int64_t total_T, int32_t batch) {
  return batch > 1 && batch <= 64 && total_T / batch >= 4 * kTile;
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

// Waves that walk one sequence together, at most `most`: more of them where
// few (sequence, channel) pairs have chunks enough.  Measured, prefill and
// forward + gradients in us, bf16: sixteen (eight) waves and four: 1 x 65536 x 256 30,
// 76 and 38, 94; x 512 53, 145 and 53, 158; x 700 81, 215 and 81, 207; 1 x 4096 x 400 the
// same.  Four waves and one: 1 x 8192 x 512 10, 30 and 19, 47; 2 x 1024 x 1024 8.8, 29.7
// and 9.5, 31.9; 8 x 600 x 512 12.3, 39 and 9.7, 33; 4096 pairs of 1024 tokens 11.9,
// 36 and 9.9, 30 (fp32 13.6, 40 and 14.0, 39), of 1500 14.5, 45 and 13.7, 33 (18.9, 60 and
// 19.7, 61), of 2048 14.5, 43 and 15.6, 39 (26.5, 72 and 28.3, 79), of 8192 57, 143 and 65,
// 153; 8192 pairs of 4096 tokens 52, 142 and 45, 134.
static int waves_per_pair(int64_t pairs, int64_t total_T, int32_t batch, int most) {
  const int64_t mean = total_T / batch;
  if (most > 4 && pairs < 512 && mean >= 8 * kChunkTokens) return most;
  if (pairs < 8192 && mean >= (pairs < 4096 ? 2 : 4) * kChunkTokens) return 4;
  return 1;
}

// Rows of a segment of the flat token axis for calls whose channels lie side
// by side, or 0: a workgroup takes a whole sequence.
// Segments cost a second read of the inputs, and pay where whole sequences
// are too few workgroups, or too uneven ones, and long enough to be cut.
// Measured, prefill, in segments and without, by the lengths drawn: 8 ragged x
// 17409 x 4096 bf16 (512 workgroups) 203..216 and 150..383 us, of equal lengths 189 and
// 130; 9 (576) 204..214 and 150..200; 11 to 16 (704 to 1024) 202..216 and 131..194; 16 of equal
// lengths 123 and 130; 33 of 248 tokens x 1001 fp32 (528) 57 and 41..61; 16 of 256 x 1024
// bf16 (256) 26 and 36; 40 of 125 x 256 bf16 26..30 and 18..26; 1 x 32768 x 1024 102 and
// 1727.  2048 segments' workgroups instead of 1024 were no faster (108 us for the last).
static int64_t segment_rows(int64_t total_T, int32_t batch, int32_t dim) {
  const int64_t slabs = cdiv(dim, 64);
  if (batch == 0 || dim == 0 || total_T / batch < 200 || batch * slabs > 512) return 0;
  const int64_t segments = cdiv(1024, slabs);
  const int64_t rows = cdiv(cdiv(total_T, segments), kTile) * kTile;
  return rows < 2 * kTile ? 2 * kTile : rows;
}

// Floats of workspace: the segments' maps and saved states, and the parts of
// ddecay (backward).
static void rec_workspace(int64_t total_T, int32_t batch, int32_t dim, int64_t* fwd, int64_t* bwd) {
  const int64_t rows = segment_rows(total_T, batch, dim);
  const int64_t n = rows ? cdiv(total_T, rows) : 0;
  *fwd = 3 * n * dim;
  *bwd = 3 * n * dim + (n > batch ? n : batch) * dim;
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

extern "C" int gated_linear_recurrence_workspace(int64_t total_T, int32_t batch, int32_t dim,
                                                 int64_t* fwd_floats, int64_t* bwd_floats) {
  using namespace sconv;
  clear_error();
  const char* fn = "gated_linear_recurrence_workspace";
  if (total_T < 0 || batch < 0 || dim < 0 || !fwd_floats || !bwd_floats)
    return fail(SCONV_ERR_INVALID, "%s: sizes must be >= 0, results not NULL", fn);
  rec_workspace(total_T, batch, dim, fwd_floats, bwd_floats);
  return SCONV_OK;
}

extern "C" int gated_linear_recurrence_varlen_fwd(
    const void* x, int64_t x_stride_c, int64_t x_stride_t, const void* gate_a,
    int64_t ga_stride_c, int64_t ga_stride_t, const void* gate_x, int64_t gx_stride_c,
    int64_t gx_stride_t, const float* decay, float decay_scale, float* states, int64_t num_slots,
    int64_t st_stride_slot, const int32_t* query_start_loc, int32_t batch,
    const int32_t* cache_indices, const uint8_t* has_initial_state, void* out,
    int64_t out_stride_c, int64_t out_stride_t, float* checkpoints, int64_t checkpoint_rows,
    float* workspace, int64_t workspace_floats, int32_t dim, int64_t total_T, int32_t dtype,
    int32_t pad_slot_id, hipStream_t stream) {
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
  int64_t need = 0, bwd_need = 0;
  rec_workspace(total_T, batch, dim, &need, &bwd_need);
  const int64_t wb = workspace ? need * 4 : 0;
  if (workspace && workspace_floats < need)
    return fail(SCONV_ERR_INVALID, "%s: workspace holds %lld floats, %lld needed", fn,
                (long long)workspace_floats, (long long)need);
  const int64_t db = (int64_t)dim * 4;
  if (overlap(decay, db, out, po.bytes()) || overlap(decay, db, states, sb) ||
      overlap(decay, db, checkpoints, mb) || overlap(decay, db, workspace, wb))
    return fail(SCONV_ERR_INVALID, "%s: an output overlaps decay", fn);
  if (overlap(workspace, wb, x, px.bytes()) || overlap(workspace, wb, gate_a, pa.bytes()) ||
      overlap(workspace, wb, gate_x, pg.bytes()) || overlap(workspace, wb, out, po.bytes()) ||
      overlap(workspace, wb, states, sb) || overlap(workspace, wb, checkpoints, mb))
    return fail(SCONV_ERR_INVALID, "%s: workspace overlaps another buffer", fn);
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
    p.seg_rows = workspace ? (int32_t)segment_rows(total_T, batch, dim) : 0;
    // Two channels a lane halve the segments' instructions (bf16: 102 against
    // 108 us for 1 x 32768 x 1024; fp32 loses a workgroup a CU to their
    // registers, 34 us against 38 for 40000 x 100); a whole sequence is walked
    // sooner by twice the workgroups (203 -> 154 us for the 16).
    const bool two = p.seg_rows && dtype == SCONV_BF16 && row_lanes(planes, 2);
    const int64_t slabs = cdiv(dim, two ? 128 : 64);
    p.sorted = longest_first(total_T, batch);
    const int64_t segments = p.seg_rows ? cdiv(total_T, p.seg_rows) : 0;
    p.maps = workspace;
    p.saved = workspace + 2 * segments * dim;
    const int64_t grid = (segments ? segments : batch) * slabs;
    if (!valid_grid(grid, kFwdWaves * 64))
      return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
    if (dtype == SCONV_BF16) {
      if (two) launch_fwd_rows<Bf16, 2>(p, (uint32_t)grid, stream);
      else launch_fwd_rows<Bf16, 1>(p, (uint32_t)grid, stream);
    } else {
      launch_fwd_rows<F32, 1>(p, (uint32_t)grid, stream);
    }
    return check_launch(fn);
  }
  const bool vec = token_lanes(planes);
  const int nw = waves_per_pair(p.num_pairs, total_T, batch, vec ? 16 : 4);
  p.pad_lds = total_T / batch >= kLongTokens ? kLongPadLds : 0;
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
  int64_t fwd_need = 0, need = 0;
  rec_workspace(total_T, batch, dim, &fwd_need, &need);
  if (workspace_floats < need)
    return fail(SCONV_ERR_INVALID, "%s: workspace holds %lld floats, %lld needed", fn,
                (long long)workspace_floats, (long long)need);
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
      {dinitial_states, dib}, {ddecay, (int64_t)dim * 4}, {workspace, need * 4}};
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
        overlap(ou[i].p, ou[i].bytes(), decay, (int64_t)dim * 4) ||
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
  int64_t parts = batch;
  if (batch > 0 && side_by_side(planes) && dim > 1) {
    p.seg_rows = (int32_t)segment_rows(total_T, batch, dim);
    p.sorted = longest_first(total_T, batch);
    const int64_t segments = p.seg_rows ? cdiv(total_T, p.seg_rows) : 0;
    parts = segments ? segments : batch;
    p.maps = workspace;
    p.saved = workspace + 2 * segments * dim;
    p.partial = workspace + 3 * segments * dim;
    const int64_t grid = parts * cdiv(dim, 64);
    if (!valid_grid(grid, kMapWaves * 64))
      return fail(SCONV_ERR_UNSUPPORTED, "%s: batch * dim too large", fn);
    if (dtype == SCONV_BF16) launch_bwd_rows<Bf16>(p, (uint32_t)grid, stream);
    else launch_bwd_rows<F32>(p, (uint32_t)grid, stream);
    if (const int rc = check_launch(fn)) return rc;
  } else if (batch > 0) {
    const bool vec = token_lanes(planes);
    const int nw = waves_per_pair(p.num_pairs, total_T, batch, vec ? 8 : 4);
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
                     dim3(kSumCols * kSumGroups), 0, stream, p.partial, decay, ddecay,
                     (int32_t)parts, dim, decay_scale);
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
  if (overlap(decay, (int64_t)dim * 4, out, po.bytes()) ||
      overlap(decay, (int64_t)dim * 4, states, sb))
    return fail(SCONV_ERR_INVALID, "%s: an output overlaps decay", fn);
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
