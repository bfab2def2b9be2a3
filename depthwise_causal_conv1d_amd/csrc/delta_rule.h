// delta_rule.h -- what the kernels of the gated delta rule share: parameters,
// the chunks of packed sequences, and matrix tiles with their products.
//
// Per value head, with S a K x V matrix in fp32:
//   S' = e^g S,  u = beta (v - S'^T k),  S = S' + k u^T,  out = scale S^T q
//
// In a chunk of C tokens that starts at the state S0, with G the running sum
// of g and e_ij = e^(G_i - G_j):
//   A_ij = beta_i e_ij k_i.k_j (i > j),  T = (I + A)^-1 = I + N
//   R = beta (V - e^G (K S0)),  U = R + N R
//   P_ij = scale e_ij q_i.k_j (i >= j),  O = scale e^G (Q S0) + P U
//   S1 = e^(G_C) S0 + K^T (e^(G_C - G) U)
// The columns of S, V, R, U and O never meet, so a wave owns 16 of them, keeps
// its part of S in registers over a whole sequence and needs no other wave.
//
// Products run on the matrix cores in 16 x 16 tiles.  An accumulator tile
// holds column lane % 16, rows 4 (lane / 16) + 0..3; an operand wants, per
// lane, 8 entries of the 32 that a product sums over.  Both operands may take
// those 32 in any common order, so two accumulator tiles one above the other
// are an operand as they lie: entry (h, e) of lane group g is row
// 16 h + 4 g + e.  What R, U and S need as operands therefore never leaves
// the registers; K and Q are laid out in LDS in that order.
//
// bf16 inputs: q, k, v are exact operands.  What is computed in fp32 enters
// beside them as the sum of three bf16 parts, all 24 bits (S, what is added to a
// state), and beside each other (R, U, N, P) as the sum of two fp16 parts of the
// value times a power of two that brings the largest of its tile or column to 2^14:
// 22 bits, down to 2^-17 of that largest.  Three products of such parts take what
// three of two bf16 parts do, which hold 16 bits and are left where only bf16 dq and dk
// come of them.  Sums are fp32.  fp32 inputs: fp32 matrix instructions, nothing is split.
#pragma once

#include <type_traits>

#include "plane_host.h"
#include "sconv_device.h"

namespace sconv {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kDeltaMaxK = 128;

// Tokens of a chunk, and of the distance between checkpoints: fp32 halves it,
// so that a chunk's operands take the same LDS.
template <typename D> constexpr int kDeltaChunk = sizeof(typename D::storage) == 2 ? 64 : 32;
inline int delta_chunk(int32_t dtype) { return dtype == SCONV_BF16 ? 64 : 32; }

struct DeltaParams {
  const void *q, *k, *v, *g, *beta;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, g_t, g_h, b_t, b_h;
  const int32_t *qsl, *slots;
  const uint8_t* has;
  int32_t batch, pad, heads, group, K, V;  // heads: value heads; group: of one key head
  float scale;
  int32_t gates_f32, qk_vec, v_vec;
  int32_t spread;  // of a walk's workgroups, by delta_walk_grid
  // operands of every chunk: frags (2 KB each), then vectors
  char* frags;
  float* vectors;
};

// ---------------------------------------------------------------- chunks

// Chunk i of sequence b has row start_b / C + b + i in every per-chunk buffer.
inline int64_t delta_rows(int64_t total_T, int32_t batch, int C) { return cdiv(total_T, C) + batch; }

struct DeltaChunk {
  int32_t b, t0, len;  // len == 0: no chunk has this row
};

template <int C>
__device__ __forceinline__ DeltaChunk delta_find(const DeltaParams& p, int32_t row) {
  int32_t lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (p.qsl[mid] / C + mid <= row) lo = mid; else hi = mid;
  }
  const int32_t start = p.qsl[lo], i = row - (start / C + lo);
  DeltaChunk c = {lo, start + i * C, 0};
  const int32_t left = p.qsl[lo + 1] - c.t0;
  if (i >= 0 && left > 0 && !(p.slots && p.slots[lo] == p.pad)) c.len = left < C ? left : C;
  return c;
}

// Operand pieces (frags) of a C x C triangle: 16 rows x 32 columns each.
// Lower triangle: rows of tile r meet columns of step s <= r / 2; upper: s >= r / 2.
template <int C> constexpr int kDeltaFrags = C == 64 ? 6 : 2;
constexpr int kFragBytes = 2048;
template <int C> __host__ __device__ constexpr int lower_frag(int r, int s) {
  return r < 2 ? r : 2 * (r - 1) + s;
}
template <int C> __host__ __device__ constexpr int upper_frag(int r, int s) {
  return C == 32 ? r : r < 2 ? 2 * r + s : r + 2;
}
// Per chunk: e^G, e^(G_C - G), beta; sixteen factors, by which a triangle's tiles are
// to be multiplied (N's and P's of a row of tiles, or N^T's of a row and P^T's of a
// step of columns, four each; for gradients then N's); for gradients G as a sum of
// two floats.  fp32 triangles have no factors.
template <int C> constexpr int kDeltaVectors = 5 * C + 16;
template <int C> constexpr int kDeltaFactors = 3 * C;
template <int C> constexpr int kDeltaSums = 3 * C + 16;
constexpr int kFactorsN = 8;
// What a walk takes of these.
template <typename D, int C> constexpr int kWalkVectors = sizeof(typename D::storage) == 2 ? 3 * C + 8 : 3 * C;

// States of a chunk (checkpoints, and their gradients) lie as accumulator
// tiles: per row and value head ceil(V / 16) x ceil(K / 16) tiles of 1 KB, a
// lane's four rows of its column in 16 bytes, zeros behind K and V.
__host__ __device__ constexpr int32_t tiles16(int32_t n) { return (n + 15) / 16; }
__host__ __device__ constexpr int64_t delta_state_floats(int32_t K, int32_t V) {
  return (int64_t)tiles16(K) * tiles16(V) * 256;
}

// ---------------------------------------------------------------- operands

// The larger value of the four groups of 16 lanes, for each lane of a group.
__device__ __forceinline__ float groups_max(float v) {
  uint32_t b = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const float m = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
  b = __float_as_uint(m);
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
__device__ __forceinline__ float max4(const f32x4& a, float m) {
  return fmaxf(fmaxf(fmaxf(m, fabsf(a[0])), fmaxf(fabsf(a[1]), fabsf(a[2]))), fabsf(a[3]));
}
// A power of two that brings `most` to [2^14, 2^15) (a value below 2^-111 less
// far), and 1 / it.  An infinite value leaves nothing of those beside it: NaN for all.
struct Pow2 {
  float up, down;
  explicit __device__ __forceinline__ Pow2(float most) {
    const uint32_t b = min(268u - (__float_as_uint(most) >> 23), 253u);
    up = __uint_as_float(b << 23) + (most - most), down = __uint_as_float((254u - b) << 23);
  }
};

template <typename D> struct Tile;

template <> struct Tile<Bf16> {
  using S = uint16_t;
  struct Exact { bf16x8 v; };
  struct Split { bf16x8 hi, lo; };
  struct Fine { bf16x8 hi, mid, lo; };
  struct Pair { f16x8 hi, lo; };
  struct Half { f16x8 v; };
  static constexpr bool kScaled = true;

  static __device__ __forceinline__ Pair pair(const f32x4& a, const f32x4& b, float up) {
    Pair o;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const f32x2 x = (e < 4 ? (f32x2){a[e], a[e + 1]} : (f32x2){b[e - 4], b[e - 3]}) * up;
      const f16x2 h = __builtin_convertvector(x, f16x2);
      const f16x2 l = __builtin_convertvector(x - __builtin_convertvector(h, f32x2), f16x2);
      o.hi[e] = h[0], o.hi[e + 1] = h[1];
      o.lo[e] = l[0], o.lo[e + 1] = l[1];
    }
    return o;
  }
  static __device__ __forceinline__ Half as_half(const Exact& a) { return {__builtin_bit_cast(f16x8, a.v)}; }
  static __device__ __forceinline__ Pair as_pair(const Exact& hi, const Exact& lo) {
    return {__builtin_bit_cast(f16x8, hi.v), __builtin_bit_cast(f16x8, lo.v)};
  }
  // The larger sizes of eight entries and of `most` (pairs of them).
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ u16x2 larger(const Exact& x, u16x2 most) {
    typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
    const u16x8 w = __builtin_bit_cast(u16x8, __builtin_bit_cast(u32x4, x.v) & 0x7FFF7FFFu);
    return __builtin_elementwise_max(__builtin_elementwise_max(__builtin_elementwise_max(w.s01, w.s23), most),
                                     __builtin_elementwise_max(w.s45, w.s67));
  }
  // Eight entries times a power of two as fp16, which has their 8 bits.
  static __device__ __forceinline__ Exact scaled(const Exact& x, float up) {
    f32x4 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = value(x, e), b[e] = value(x, e + 4);
    return {__builtin_bit_cast(bf16x8, half(a, b, up).v)};
  }
  // One entry of a pair in storage, and back.
  static __device__ __forceinline__ void put_pair(uint16_t& hi, uint16_t& lo, float x) {
    const _Float16 h = (_Float16)x;
    hi = __builtin_bit_cast(uint16_t, h);
    lo = __builtin_bit_cast(uint16_t, (_Float16)(x - (float)h));
  }
  static __device__ __forceinline__ float value(const Pair& a, int e) { return (float)a.hi[e] + (float)a.lo[e]; }
  // of values of 8 bits
  static __device__ __forceinline__ Half half(const f32x4& a, const f32x4& b, float up) {
    Half o;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const f32x2 x = (e < 4 ? (f32x2){a[e], a[e + 1]} : (f32x2){b[e - 4], b[e - 3]}) * up;
      const f16x2 h = __builtin_convertvector(x, f16x2);
      o.v[e] = h[0], o.v[e + 1] = h[1];
    }
    return o;
  }
  static __device__ __forceinline__ Fine fine(const f32x4& a, const f32x4& b) {
    Fine o;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      f32x2 x = e < 4 ? (f32x2){a[e], a[e + 1]} : (f32x2){b[e - 4], b[e - 3]};
      bf16x2 part[3];
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        part[n] = __builtin_convertvector(x, bf16x2);
        const uint32_t w = __builtin_bit_cast(uint32_t, part[n]);
        x = (f32x2){x[0] - __uint_as_float(w << 16), x[1] - __uint_as_float(w & 0xFFFF0000u)};
      }
      o.hi[e] = part[0][0], o.hi[e + 1] = part[0][1];
      o.mid[e] = part[1][0], o.mid[e + 1] = part[1][1];
      o.lo[e] = part[2][0], o.lo[e + 1] = part[2][1];
    }
    return o;
  }
  // A product's instructions one by one, the small parts first, so that a
  // caller can let those of several tiles alternate: one that waits for the
  // last one's sum leaves the matrix core idle.
  static constexpr int kExactFine = 3, kSplitExact = 2, kPairPair = 3, kPairHalf = 2, kHalfPair = 2;
  template <int P> static __device__ __forceinline__ f32x4 part(const Split& a, const Exact& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(P == 0 ? a.lo : a.hi, b.v, c, 0, 0, 0);
  }
  // the product of the two small parts is below what the parts leave out
  template <int P> static __device__ __forceinline__ f32x4 part(const Pair& a, const Pair& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(P == 0 ? a.lo : a.hi, P == 1 ? b.lo : b.hi, c, 0, 0, 0);
  }
  template <int P> static __device__ __forceinline__ f32x4 part(const Pair& a, const Half& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(P == 0 ? a.lo : a.hi, b.v, c, 0, 0, 0);
  }
  template <int P> static __device__ __forceinline__ f32x4 part(const Half& a, const Pair& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v, P == 0 ? b.lo : b.hi, c, 0, 0, 0);
  }
  template <int P> static __device__ __forceinline__ f32x4 part(const Exact& a, const Fine& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, P == 0 ? b.lo : P == 1 ? b.mid : b.hi, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mul(const Exact& a, const Exact& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
  }
  // by whole words: a bit cast of one entry of a vector has come out as that of its first
  static __device__ __forceinline__ float value(const Exact& a, int e) {
    const uint32_t w = __builtin_bit_cast(u32x4, a.v)[e / 2];
    return __uint_as_float(e % 2 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ uint16_t raw(const Exact& a, int e) {
    return (uint16_t)(__builtin_bit_cast(u32x4, a.v)[e / 2] >> (16 * (e % 2)));
  }
  static __device__ __forceinline__ Exact join(const uint16_t (&a)[8]) {
    struct W { uint16_t e[8]; } w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w.e[e] = a[e];
    return {__builtin_bit_cast(bf16x8, w)};
  }
  // A frag as it lies in memory: 64 lanes x 16 bytes of the high parts, then the low ones.
  static __device__ __forceinline__ void put(char* frag, int lane, const Pair& s) {
    *reinterpret_cast<u32x4*>(frag + lane * 16) = __builtin_bit_cast(u32x4, s.hi);
    *reinterpret_cast<u32x4*>(frag + 1024 + lane * 16) = __builtin_bit_cast(u32x4, s.lo);
  }
  static __device__ __forceinline__ Pair get(const char* frag, int lane) {
    return {__builtin_bit_cast(f16x8, *reinterpret_cast<const u32x4*>(frag + lane * 16)),
            __builtin_bit_cast(f16x8, *reinterpret_cast<const u32x4*>(frag + 1024 + lane * 16))};
  }
};

template <> struct Tile<F32> {
  using S = float;
  struct Exact { f32x4 a, b; };
  using Split = Exact;
  using Fine = Exact;
  using Pair = Exact;
  using Half = Exact;
  static constexpr bool kScaled = false;

  static constexpr int kExactFine = 8, kSplitExact = 8, kPairPair = 8, kPairHalf = 8, kHalfPair = 8;
  template <int P> static __device__ __forceinline__ f32x4 part(const Exact& a, const Exact& b, f32x4 c) {
    if constexpr (P < 4) return __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[P], b.a[P], c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[P - 4], b.b[P - 4], c, 0, 0, 0);
  }
  static __device__ __forceinline__ Fine fine(const f32x4& a, const f32x4& b) { return {a, b}; }
  static __device__ __forceinline__ Pair pair(const f32x4& a, const f32x4& b, float) { return {a, b}; }
  static __device__ __forceinline__ Half half(const f32x4& a, const f32x4& b, float) { return {a, b}; }
  static __device__ __forceinline__ Half as_half(const Exact& a) { return a; }
  static __device__ __forceinline__ f32x4 mul(const Exact& a, const Exact& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[e], b.a[e], c, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[e], b.b[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ float value(const Exact& a, int e) {
    return e < 4 ? a.a[e] : a.b[e - 4];
  }
  static __device__ __forceinline__ float raw(const Exact& a, int e) { return value(a, e); }
  static __device__ __forceinline__ Exact join(const float (&a)[8]) {
    return {{a[0], a[1], a[2], a[3]}, {a[4], a[5], a[6], a[7]}};
  }
  static __device__ __forceinline__ void put(char* frag, int lane, const Split& s) {
    *reinterpret_cast<f32x4*>(frag + lane * 16) = s.a;
    *reinterpret_cast<f32x4*>(frag + 1024 + lane * 16) = s.b;
  }
  static __device__ __forceinline__ Split get(const char* frag, int lane) {
    return {*reinterpret_cast<const f32x4*>(frag + lane * 16),
            *reinterpret_cast<const f32x4*>(frag + 1024 + lane * 16)};
  }
};

// 8 consecutive entries of row t from c0 on; VEC: rows of 16-byte vectors.
// Every lane loads from some place inside rows 0 .. T - 1 (T > 0) and columns
// 0 .. W - 1, and drops by mask8 what it should not see when it uses it: a load
// under a condition, or a select behind it, waits for the data there (a chunk
// of the walk took 14 and 10 us so).
template <typename D, bool VEC>
__device__ __forceinline__ typename Tile<D>::Exact load8(const typename D::storage* m, int64_t ld, int t,
                                                         int T, int c0, int W) {
  const typename D::storage* row = m + (t < T ? t : T - 1) * ld;
  if constexpr (VEC) {
    const typename D::storage* at = row + (c0 < W ? c0 : 0);
    if constexpr (sizeof(typename D::storage) == 2)
      return {__builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(at))};
    else
      return {*reinterpret_cast<const f32x4*>(at),
              *reinterpret_cast<const f32x4*>(row + (c0 + 4 < W ? c0 + 4 : 0))};
  } else {
    typename D::storage w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = row[c0 + e < W ? c0 + e : W - 1];
    return Tile<D>::join(w);
  }
}

// The first n entries, zeros behind them.
template <typename D>
__device__ __forceinline__ typename Tile<D>::Exact mask8(typename Tile<D>::Exact x, int n) {
  if constexpr (sizeof(typename D::storage) == 2) {
    u32x4 w = __builtin_bit_cast(u32x4, x.v);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = n > 2 * e + 1 ? w[e] : n > 2 * e ? w[e] & 0xFFFFu : 0u;
    return {__builtin_bit_cast(bf16x8, w)};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x.a[e] = n > e ? x.a[e] : 0.f, x.b[e] = n > e + 4 ? x.b[e] : 0.f;
    return x;
  }
}

// 8 entries to columns c0.. of a row, those before W.
template <typename D>
__device__ __forceinline__ void put_row8(typename D::storage* row, int c0, int W, bool vec,
                                         const typename Tile<D>::Exact& x) {
  if (vec) {
    if constexpr (sizeof(typename D::storage) == 2) {
      if (c0 < W) *reinterpret_cast<u32x4*>(row + c0) = __builtin_bit_cast(u32x4, x.v);
    } else {
      if (c0 < W) *reinterpret_cast<f32x4*>(row + c0) = x.a;
      if (c0 + 4 < W) *reinterpret_cast<f32x4*>(row + c0 + 4) = x.b;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c0 + e < W) row[c0 + e] = Tile<D>::raw(x, e);
}

// A matrix of W columns (a multiple of 32) in LDS, one row a token.  bf16 rows
// keep, inside every 32 columns, the order of an operand (16 h + 4 g + e at
// 8 g + 4 h + e), so that a lane's 8 entries are one 16-byte read.  The pad
// of 32 bytes was the best of 0 to 128 for 16-byte and transposed reads together
// (timed alone; at 16 bytes half the LDS time of a walk was conflicts).
template <typename D, int W> struct LdsRows {
  using S = typename D::storage;
  static constexpr int kPad = sizeof(S) == 2 ? 16 : 4;
  static constexpr int LD = W + kPad;

  // where column c lies in a row
  static __device__ __forceinline__ int pos(int c) {
    if constexpr (sizeof(S) == 2) return (c & ~31) + ((c >> 2) & 3) * 8 + ((c >> 4) & 1) * 4 + (c & 3);
    return c;
  }
  // 8 consecutive columns c0.. (a multiple of 8) of row t
  static __device__ __forceinline__ void put8(S* m, int t, int c0, const typename Tile<D>::Exact& x) {
    if constexpr (sizeof(S) == 2) {
      const u32x4 w = __builtin_bit_cast(u32x4, x.v);
      S* at = m + t * LD + pos(c0);
      *reinterpret_cast<u32x2*>(at) = (u32x2){w[0], w[1]};
      *reinterpret_cast<u32x2*>(at + 8) = (u32x2){w[2], w[3]};
    } else {
      *reinterpret_cast<f32x4*>(m + t * LD + c0) = x.a;
      *reinterpret_cast<f32x4*>(m + t * LD + c0 + 4) = x.b;
    }
  }
  static __device__ __forceinline__ typename Tile<D>::Exact get8(const S* m, int t, int c0) {
    const S* at = m + t * LD + pos(c0);
    if constexpr (sizeof(S) == 2) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(at), y = *reinterpret_cast<const u32x2*>(at + 8);
      return {__builtin_bit_cast(bf16x8, (u32x4){x[0], x[1], y[0], y[1]})};
    } else {
      return {*reinterpret_cast<const f32x4*>(at), *reinterpret_cast<const f32x4*>(at + 4)};
    }
  }
  // operand whose rows are tokens t0 + lane % 16, summed over columns c0 .. c0 + 31
  static __device__ __forceinline__ typename Tile<D>::Exact rows(const S* m, int t0, int c0, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (sizeof(S) == 2)
      return {__builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(m + (t0 + r) * LD + c0 + 8 * g))};
    else
      return {*reinterpret_cast<const f32x4*>(m + (t0 + r) * LD + c0 + 4 * g),
              *reinterpret_cast<const f32x4*>(m + (t0 + r) * LD + c0 + 16 + 4 * g)};
  }
  // operand whose rows are columns c0 + lane % 16, summed over tokens t0 .. t0 + 31
  static __device__ __forceinline__ typename Tile<D>::Exact cols(const S* m, int t0, int c0, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (sizeof(S) == 2) {
      // 16 lanes read 4 tokens x 16 columns; each gets its column's 4 tokens
      const int col = (c0 & ~31) + (r & 3) * 8 + ((c0 >> 4) & 1) * 4;
      const S* at = m + (t0 + 4 * g + (r >> 2)) * LD + col;
      typedef __attribute__((address_space(3))) s16x4* lds4;
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)at);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + 16 * LD));
      return {__builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7))};
    } else {
      const S* at = m + (t0 + 4 * g) * LD + c0 + r;
      return {{at[0], at[LD], at[2 * LD], at[3 * LD]},
              {at[16 * LD], at[17 * LD], at[18 * LD], at[19 * LD]}};
    }
  }
};

// f(0), .. f(N - 1) with constants.
template <int N, int I = 0, typename F> __device__ __forceinline__ void each_part(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    each_part<N, I + 1>(f);
  }
}

// What is above stays above in the instruction stream: loads ahead of the
// products that cover their latency.  Left to itself the compiler puts each
// load right before its use, to save registers (a chunk of the walk took 20000
// cycles so, with 2400 of matrix instructions).
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ float delta_gate(const DeltaParams& p, const void* t, int64_t at) {
  return p.gates_f32 ? static_cast<const float*>(t)[at]
                     : bf16_bits_to_float(static_cast<const uint16_t*>(t)[at]);
}
// A g that is certain to close the state becomes a number whose sums stay
// finite (e^-200 is zero in fp32); NaN stays.
__device__ __forceinline__ float delta_bound(float g) { return g < -200.f ? -200.f : g; }

__device__ __forceinline__ f32x4 zero4() { return (f32x4){0.f, 0.f, 0.f, 0.f}; }
__device__ __forceinline__ f32x4 lds4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// One value of a row in the inputs' type.
template <typename D>
__device__ __forceinline__ typename D::storage delta_round(float v) {
  if constexpr (sizeof(typename D::storage) == 2)
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    return v;
}

}  // namespace sconv
