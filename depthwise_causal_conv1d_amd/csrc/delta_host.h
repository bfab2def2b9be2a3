// delta_host.h -- host-side checks shared by the gated delta rule's entry
// points.
#pragma once

#include <initializer_list>

#include "delta_rule.h"

namespace sconv {

struct DeltaCall {
  const char* what;
  int64_t tokens;
  int32_t batch, key_heads, heads, K, V, dtype, gate_dtype;
};

// Workspace in floats: vectors first, then frags (16-byte pieces), then for
// gradients dR's tiles and the states' gradients.
struct DeltaSpace {
  int64_t vectors, fwd, bwd, bwd_rows, bwd_states;
};

inline DeltaSpace delta_space(int64_t total_T, int32_t batch, int32_t heads, int32_t K, int32_t V,
                              int32_t dtype) {
  const int C = delta_chunk(dtype), nf = C == 64 ? kDeltaFrags<64> : kDeltaFrags<32>;
  const int64_t n = delta_rows(total_T, batch, C) * heads;
  DeltaSpace s;
  s.vectors = n * (5 * C + 16);
  s.fwd = s.vectors + n * 2 * nf * (kFragBytes / 4);
  s.bwd_rows = s.vectors + n * 3 * nf * (kFragBytes / 4);
  s.bwd_states = s.bwd_rows + n * C * tiles16(V) * 16;
  s.bwd = s.bwd_states + n * delta_state_floats(K, V);
  return s;
}

inline int delta_sizes(const DeltaCall& c) {
  if (c.tokens < 0 || c.batch < 0 || c.key_heads < 0 || c.heads < 0 || c.K < 0 || c.V < 0)
    return fail(SCONV_ERR_INVALID, "%s: negative size", c.what);
  if (!valid_dtype(c.dtype)) return fail(SCONV_ERR_INVALID, "%s: unknown dtype", c.what);
  if (c.gate_dtype != SCONV_F32 && c.gate_dtype != c.dtype)
    return fail(SCONV_ERR_INVALID, "%s: g and beta are fp32 or of the inputs' type", c.what);
  if (c.heads > 0 && (c.key_heads < 1 || c.heads % c.key_heads))
    return fail(SCONV_ERR_INVALID, "%s: %d value heads do not share %d key heads evenly", c.what,
                c.heads, c.key_heads);
  if (c.K < 1 && c.heads > 0 && c.V > 0)
    return fail(SCONV_ERR_INVALID, "%s: K must be positive", c.what);
  if (c.K > kDeltaMaxK)
    return fail(SCONV_ERR_UNSUPPORTED, "%s: key heads of %d channels (at most %d)", c.what, c.K,
                kDeltaMaxK);
  // chunks, heads and sequences are grid dimensions, of at most 512 threads each
  if (c.tokens > INT32_MAX - 4097 || c.V > (1 << 20) || c.heads > 65535 || c.batch > 65535 ||
      !valid_grid(delta_rows(c.tokens, c.batch, 32) + 1, 512))
    return fail(SCONV_ERR_UNSUPPORTED, "%s: too many tokens, sequences, heads or channels", c.what);
  return SCONV_OK;
}

// Memory that a call touches: `bytes` from p on, in runs `step` bytes apart
// (step 0: one run).
struct DeltaBuffer {
  const void* p;
  int64_t bytes, run, step;
};

inline DeltaBuffer delta_block(const void* p, int64_t bytes) { return {p, bytes, bytes, 0}; }

// A [tokens, heads, width] tensor, channels contiguous.
inline DeltaBuffer delta_tensor(const void* p, int64_t st, int64_t sh, int64_t tokens,
                                int64_t heads, int64_t width, int64_t es) {
  if (!tokens || !heads || !width) return delta_block(p, 0);
  const int64_t row = (heads - 1) * sh + width, all = (tokens - 1) * st + row;
  const int64_t head = (tokens - 1) * st + width;
  if (tokens > 1 && st >= row) return {p, all * es, row * es, st * es};
  if (heads > 1 && sh >= head) return {p, all * es, head * es, sh * es};
  return delta_block(p, all * es);
}

// Tensors whose rows lie between each other's (columns of one wider matrix) do not overlap.
inline bool delta_overlap(const DeltaBuffer& a, const DeltaBuffer& b) {
  if (!overlap(a.p, a.bytes, b.p, b.bytes)) return false;
  if (!a.step || a.step != b.step) return true;
  int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p) % a.step;
  if (d < 0) d += a.step;
  return d < a.run || a.step - d < b.run;
}

// Rows of whole 16-byte vectors of n elements, a chunk's rows within 2^31 bytes.
inline bool delta_vec(const void* t, int64_t st, int64_t sh, int64_t width, int64_t n) {
  return aligned16(t) && st % n == 0 && sh % n == 0 && width % n == 0 && st < (1 << 22);
}

inline int delta_inputs(const DeltaCall& c, DeltaParams& p, const void* q, int64_t q_t, int64_t q_h,
                        const void* k, int64_t k_t, int64_t k_h, const void* v, int64_t v_t,
                        int64_t v_h, const void* g, int64_t g_t, int64_t g_h, const void* beta,
                        int64_t b_t, int64_t b_h, float scale) {
  if (!(scale - scale == 0.f)) return fail(SCONV_ERR_INVALID, "%s: scale is not finite", c.what);
  if (c.tokens > 0 && (!q || !k || !v || !g || !beta))
    return fail(SCONV_ERR_INVALID, "%s: NULL input", c.what);
  for (int64_t s : {q_t, q_h, k_t, k_h, v_t, v_h, g_t, g_h, b_t, b_h})
    if (s < 0) return fail(SCONV_ERR_INVALID, "%s: negative stride", c.what);
  p.q = q, p.k = k, p.v = v, p.g = g, p.beta = beta;
  p.q_t = q_t, p.q_h = q_h, p.k_t = k_t, p.k_h = k_h, p.v_t = v_t, p.v_h = v_h;
  p.g_t = g_t, p.g_h = g_h, p.b_t = b_t, p.b_h = b_h;
  p.batch = c.batch, p.heads = c.heads, p.K = c.K, p.V = c.V;
  p.group = c.heads / c.key_heads;
  p.scale = scale;
  p.gates_f32 = c.gate_dtype == SCONV_F32;
  // rows that start and end on 16 bytes load as vectors
  const int64_t n = 16 / elem_size(c.dtype);
  p.qk_vec = delta_vec(q, q_t, q_h, c.K, n) && delta_vec(k, k_t, k_h, c.K, n);
  p.v_vec = delta_vec(v, v_t, v_h, c.V, n);
  return SCONV_OK;
}

// Whether a workgroup of a walk has eight waves on 128 columns and no loaders
// (else four on 64, and four loaders): it reads half as much LDS a product, on
// half as many CUs.  Where the narrow ones all have a CU of 256 at once they win
// (all of forward, 4 x 2048 tokens, 32 heads of 128 x 128 bf16: 176 us, wide 238),
// beyond that the wide ones (5 x 2048: 240 us, narrow 269; 8 x 4096: 573 and 627; of 64
// x 128: 427 and 466), but for the few calls of which a little over 256 are wide (9 x
// 2048 of 64 x 128, 288 of them: 342 and 309).  Products of 32-bit tiles take the
// same time either way (320 narrow workgroups: 329 us, wide 359; 512: 339 and 336),
// so they have the narrow form only.
inline bool delta_wide(const DeltaParams& p) {
  return p.V > 64 && (int64_t)p.batch * p.heads * ((p.V + 63) / 64) > 256;
}

// Workgroups of a walk with `cols` blocks of columns.  Those of one sequence
// and key head read the same K and Q, so they take one XCD's cache: numbers 8
// apart, where that gives the XCDs even shares and they have 16 workgroups each (the
// call of 8 x 4096 tokens, two value heads a key head: 585 us, in plain order 589; 3 x
// 4096 of 128 x 256: 242 and 246).  With fewer nothing is gained (1 x 8192 x 16 heads:
// 414 either way), and with fewer pairs than XCDs the others idle (1 x 4096, 16 value
// heads of one key head: 229 and 214; 4 of 8 x 256 columns: 214 and 211).
inline dim3 delta_walk_grid(DeltaParams& p, int32_t cols) {
  const int64_t pairs = (int64_t)p.batch * (p.heads / p.group), n = (int64_t)p.group * cols;
  const int64_t each = cdiv(pairs, 8);
  p.spread = pairs * n >= 128 && 8 * each <= pairs + pairs / 4 ? 8 : 1;
  return dim3((uint32_t)(cdiv(pairs, p.spread) * p.spread * n));
}

// Whether the walks' and the preparation's grids are one launch each.
inline int delta_grids(const DeltaCall& c) {
  if (c.heads == 0) return SCONV_OK;
  const int64_t group = c.heads / c.key_heads, pairs = ((int64_t)c.batch * c.key_heads + 7) / 8 * 8;
  const int64_t rows = (delta_rows(c.tokens, c.batch, 32) + 7) / 8 * 8;
  if (pairs * group * cdiv(c.V, 64) * 512 >= (int64_t)1 << 32 || rows * group * 64 >= (int64_t)1 << 32)
    return fail(SCONV_ERR_UNSUPPORTED, "%s: too many tokens, sequences, heads or channels", c.what);
  return SCONV_OK;
}

inline void delta_packing(DeltaParams& p, const int32_t* qsl, const int32_t* slots, const uint8_t* has,
                          int32_t pad) {
  p.qsl = qsl, p.slots = slots, p.has = has, p.pad = pad;
}

// An fp32 [num_slots, heads, K, V] pool, dense but for the slots.
inline int delta_pool(const DeltaCall& c, const void* pool, int64_t slots, int64_t stride,
                      bool indexed, const char* name, DeltaBuffer* out) {
  *out = delta_block(pool, 0);
  if (!pool) return SCONV_OK;
  const int64_t one = (int64_t)c.heads * c.K * c.V;
  if (slots < 0 || (slots > 1 && stride < one))
    return fail(SCONV_ERR_INVALID, "%s: %s: slots overlap", c.what, name);
  if (!indexed && slots < c.batch)
    return fail(SCONV_ERR_INVALID, "%s: %s has %lld slots, needs %d", c.what, name,
                (long long)slots, c.batch);
  *out = delta_block(pool, slots ? ((slots - 1) * stride + one) * 4 : 0);
  return SCONV_OK;
}

// An output [tokens, heads, width]: no two elements in one place.
inline int delta_output(const DeltaCall& c, const void* t, int64_t st, int64_t sh, int64_t heads,
                        int64_t width, const char* name, DeltaBuffer* out, int64_t es = 0) {
  es = es ? es : elem_size(c.dtype);
  *out = delta_block(t, 0);
  if (c.tokens == 0) return SCONV_OK;
  if (!t) return fail(SCONV_ERR_INVALID, "%s: NULL %s", c.what, name);
  if (st < 0 || sh < 0) return fail(SCONV_ERR_INVALID, "%s: negative stride", c.what);
  const bool rows = heads == 1 || (sh >= width && (c.tokens == 1 || st >= (heads - 1) * sh + width));
  const bool planes = c.tokens == 1 || (st >= width && (heads == 1 || sh >= (c.tokens - 1) * st + width));
  if (heads == 1 ? !planes : !(rows || planes))
    return fail(SCONV_ERR_INVALID, "%s: elements of %s share memory", c.what, name);
  *out = delta_tensor(t, st, sh, c.tokens, heads, width, es);
  return SCONV_OK;
}

// Outputs overlap neither each other nor an input (the first may be v itself).
inline int delta_disjoint(const DeltaCall& c, const DeltaParams& p,
                          std::initializer_list<DeltaBuffer> outs, bool first_is_v = false) {
  const int64_t es = elem_size(c.dtype), gs = elem_size(c.gate_dtype);
  const DeltaBuffer ins[] = {delta_tensor(p.v, p.v_t, p.v_h, c.tokens, c.heads, c.V, es),
                             delta_tensor(p.q, p.q_t, p.q_h, c.tokens, c.key_heads, c.K, es),
                             delta_tensor(p.k, p.k_t, p.k_h, c.tokens, c.key_heads, c.K, es),
                             delta_tensor(p.g, p.g_t, p.g_h, c.tokens, c.heads, 1, gs),
                             delta_tensor(p.beta, p.b_t, p.b_h, c.tokens, c.heads, 1, gs)};
  const DeltaBuffer* o = outs.begin();
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = 0; j < i; ++j)
      if (delta_overlap(o[i], o[j]))
        return fail(SCONV_ERR_INVALID, "%s: outputs, states or workspace overlap", c.what);
    for (int j = 0; j < 5; ++j) {
      if (i == 0 && j == 0 && first_is_v) continue;
      if (delta_overlap(o[i], ins[j]))
        return fail(SCONV_ERR_INVALID, "%s: an output overlaps an input", c.what);
    }
  }
  return SCONV_OK;
}

}  // namespace sconv
