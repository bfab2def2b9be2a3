// paged_metadata.hip -- block tables, slots and per-token metadata of a step
// from its requests' lengths.
//
// Two running sums over the requests (tokens, and blocks that a table lacks)
// decide everything; the rest is a search per token.  Up to kMetaReqs
// requests every workgroup makes both sums for itself in LDS: a few loads a
// thread, against a second launch that would wait for the first.  Launches one
// after another in a graph, one (two): 256 requests of one token 4.3 us (6.0), 64
// of 256 tokens 4.2 (7.0), 1000 of 65 6.3 (10.5), 1000 of 4096 85 (330), 2000 of 512 64
// (80), 4096 of 16 14.3 (18.1), of 64 34 (31), of 512 234 (181).  Latency bounds the
// small ones (1000 requests' 65 tokens are 2 MB, 0.4 us).  Thousands of requests are
// bound by their sums, which every workgroup of the one launch makes again; two make
// them once, but their one workgroup of sums also fills every table, which takes longer
// for all but the most.
#include "sconv_device.h"
#include "sconv_host.h"

namespace sconv {

struct PagedMeta {
  const int32_t *query, *context, *free;
  int32_t *table, *qsl, *seq_idx, *query_start, *used;
  int64_t *positions, *slots;
  int64_t num_free, bt_rs, padded;
  int32_t reqs, max_blocks, block;
};

constexpr int kPagedThreads = 256;
constexpr int kMetaReqs = 4096;  // requests of the one-launch form: 32 KB of LDS

__device__ __forceinline__ int32_t request_len(const int32_t* lens, int32_t r) {
  const int32_t n = lens[r];
  return n > 0 ? n : 0;
}
__device__ __forceinline__ uint32_t blocks_of(uint32_t tokens, uint32_t block) {
  return (tokens + block - 1) / block;
}
// Blocks that request r has, and lacks for this step.
__device__ __forceinline__ uint2 request_blocks(const PagedMeta& p, int32_t r, uint32_t len) {
  const uint32_t c = request_len(p.context, r), have = blocks_of(c, p.block);
  return make_uint2(have, blocks_of(c + len, p.block) - have);
}

// Sums of (a, b) over the threads before this one, and over all.
template <int THREADS>
__device__ __forceinline__ void scan_pairs(uint32_t& a, uint32_t& b, uint2* waves, uint2& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t a0 = a, b0 = b;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t x = __shfl_up(a, d, 64), y = __shfl_up(b, d, 64);
    if (lane >= d) a += x, b += y;
  }
  if (lane == 63) waves[wave] = make_uint2(a, b);
  __syncthreads();
  uint2 before = make_uint2(0, 0);
  all = make_uint2(0, 0);
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w == wave) before = all;
    all.x += waves[w].x, all.y += waves[w].y;
  }
  a += before.x - a0;
  b += before.y - b0;
  __syncthreads();
}

// Largest r in [0, n) with sums[r] <= x.
__device__ __forceinline__ int32_t find_sum(const uint32_t* sums, int32_t n, uint32_t x) {
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The i-th block taken from the free list, or -1 where the list has ended.
__device__ __forceinline__ int32_t free_block(const PagedMeta& p, uint32_t i) {
  return i < p.num_free ? p.free[i] : -1;
}

__device__ __forceinline__ void put_token(const PagedMeta& p, int64_t t, int32_t r, uint32_t start,
                                          int64_t pos, int64_t slot) {
  if (p.seq_idx) p.seq_idx[t] = r;
  if (p.query_start) p.query_start[t] = (int32_t)start;
  p.positions[t] = pos;
  p.slots[t] = slot;
}

__device__ __forceinline__ int64_t slot_of(const PagedMeta& p, int32_t id, uint32_t pos) {
  return id < 0 ? -1 : (int64_t)id * p.block + pos % (uint32_t)p.block;
}

__global__ __launch_bounds__(kPagedThreads) void paged_metadata_kernel(PagedMeta p) {
  __shared__ uint32_t tok[kMetaReqs + 1], blk[kMetaReqs + 1];
  __shared__ uint2 waves[kPagedThreads / 64];
  const int per = (p.reqs + kPagedThreads - 1) / kPagedThreads;
  const int lo = min((int)threadIdx.x * per, p.reqs), hi = min(lo + per, p.reqs);
  uint32_t a = 0, b = 0;
  for (int r = lo; r < hi; ++r) {
    const uint32_t len = request_len(p.query, r);
    a += len;
    b += request_blocks(p, r, len).y;
  }
  uint2 all;
  scan_pairs<kPagedThreads>(a, b, waves, all);
  for (int r = lo; r < hi; ++r) {
    const uint32_t len = request_len(p.query, r);
    tok[r] = a, blk[r] = b;
    if (blockIdx.x == 0) p.qsl[r] = (int32_t)a;
    a += len;
    b += request_blocks(p, r, len).y;
  }
  if (threadIdx.x == 0) {
    tok[p.reqs] = all.x, blk[p.reqs] = all.y;
    if (blockIdx.x == 0) {
      p.qsl[p.reqs] = (int32_t)all.x;
      if (p.used) *p.used = (int32_t)all.y;
    }
  }
  __syncthreads();
  const int64_t at = (int64_t)blockIdx.x * kPagedThreads + threadIdx.x;
  // new entries of the tables
  for (int64_t i = at; i < all.y; i += (int64_t)gridDim.x * kPagedThreads) {
    const int32_t r = find_sum(blk, p.reqs, (uint32_t)i);
    const uint32_t j = request_blocks(p, r, 0).x + ((uint32_t)i - blk[r]);
    if (j < (uint32_t)p.max_blocks) p.table[r * p.bt_rs + j] = free_block(p, (uint32_t)i);
  }
  if (at >= p.padded) return;
  if (at >= all.x) return put_token(p, at, 0, 0, 0, -1);
  const int32_t r = find_sum(tok, p.reqs, (uint32_t)at);
  const uint32_t have = request_blocks(p, r, 0).x;
  const uint32_t pos = request_len(p.context, r) + ((uint32_t)at - tok[r]), j = pos / (uint32_t)p.block;
  int32_t id = -1;
  if (j < (uint32_t)p.max_blocks)
    id = j < have ? p.table[r * p.bt_rs + j] : free_block(p, blk[r] + (j - have));
  put_token(p, at, r, tok[r], pos, slot_of(p, id, pos));
}

// More requests: one workgroup makes the sums tile by tile and fills the
// tables, then a second launch finds every token's request in the offsets.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void paged_sums_kernel(PagedMeta p) {
  __shared__ uint32_t blk[kSumThreads];
  __shared__ uint2 waves[kSumThreads / 64];
  uint2 done = make_uint2(0, 0);
  for (int32_t r0 = 0; r0 < p.reqs; r0 += kSumThreads) {
    const int32_t r = r0 + threadIdx.x, n = min(kSumThreads, p.reqs - r0);
    uint32_t a = 0, b = 0;
    if (r < p.reqs) {
      a = request_len(p.query, r);
      b = request_blocks(p, r, a).y;
    }
    uint2 all;
    scan_pairs<kSumThreads>(a, b, waves, all);
    blk[threadIdx.x] = b;
    if (r < p.reqs) p.qsl[r] = (int32_t)(done.x + a);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < all.y; i += kSumThreads) {
      const int32_t q = find_sum(blk, n, i);
      const uint32_t j = request_blocks(p, r0 + q, 0).x + (i - blk[q]);
      if (j < (uint32_t)p.max_blocks) p.table[(r0 + q) * p.bt_rs + j] = free_block(p, done.y + i);
    }
    done.x += all.x, done.y += all.y;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.qsl[p.reqs] = (int32_t)done.x;
    if (p.used) *p.used = (int32_t)done.y;
  }
}

__global__ __launch_bounds__(kPagedThreads) void paged_tokens_kernel(PagedMeta p) {
  const int64_t t = (int64_t)blockIdx.x * kPagedThreads + threadIdx.x;
  if (t >= p.padded) return;
  const uint32_t* qsl = reinterpret_cast<const uint32_t*>(p.qsl);
  if (t >= qsl[p.reqs]) return put_token(p, t, 0, 0, 0, -1);
  const int32_t r = find_sum(qsl, p.reqs, (uint32_t)t);
  const uint32_t pos = request_len(p.context, r) + ((uint32_t)t - qsl[r]), j = pos / (uint32_t)p.block;
  const int32_t id = j < (uint32_t)p.max_blocks ? p.table[r * p.bt_rs + j] : -1;
  put_token(p, t, r, qsl[r], pos, slot_of(p, id, pos));
}

}  // namespace sconv

extern "C" int sconv_paged_metadata(const int32_t* query_lens, const int32_t* context_lens,
                                    int32_t num_reqs, const int32_t* free_blocks, int64_t num_free,
                                    int32_t* block_table, int64_t bt_row_stride, int32_t max_blocks,
                                    int32_t block_size, int32_t* query_start_loc,
                                    int64_t num_padded_tokens, int32_t* seq_idx_out,
                                    int32_t* query_start_out, int64_t* positions_out,
                                    int64_t* slot_mapping_out, int32_t* blocks_used,
                                    hipStream_t stream) {
  using namespace sconv;
  clear_error();
  const char* fn = "sconv_paged_metadata";
  if (num_reqs < 0 || num_free < 0 || max_blocks < 0 || num_padded_tokens < 0)
    return fail(SCONV_ERR_INVALID, "%s: negative size", fn);
  if (block_size < 1) return fail(SCONV_ERR_INVALID, "%s: block_size must be positive", fn);
  if (num_reqs > 1 && bt_row_stride < max_blocks)
    return fail(SCONV_ERR_INVALID, "%s: rows of block_table overlap", fn);
  if (!query_start_loc || (num_reqs > 0 && (!query_lens || !context_lens)) ||
      (num_reqs > 0 && max_blocks > 0 && !block_table) || (num_free > 0 && !free_blocks) ||
      (num_padded_tokens > 0 && (!positions_out || !slot_mapping_out)))
    return fail(SCONV_ERR_INVALID, "%s: NULL pointer", fn);
  const int64_t n = num_padded_tokens, r4 = (int64_t)num_reqs * 4;
  const struct { const void* p; int64_t n; } b[10] = {
      {block_table, num_reqs ? ((num_reqs - 1) * bt_row_stride + max_blocks) * 4 : 0},
      {query_start_loc, r4 + 4}, {seq_idx_out, seq_idx_out ? n * 4 : 0},
      {query_start_out, query_start_out ? n * 4 : 0}, {positions_out, n * 8},
      {slot_mapping_out, n * 8}, {blocks_used, blocks_used ? 4 : 0},
      {query_lens, r4}, {context_lens, r4}, {free_blocks, num_free * 4}};
  for (int i = 0; i < 7; ++i)
    for (int j = i + 1; j < 10; ++j)
      if (overlap(b[i].p, b[i].n, b[j].p, b[j].n))
        return fail(SCONV_ERR_INVALID, "%s: an output overlaps another buffer", fn);
  const int64_t groups = n > 0 ? cdiv(n, kPagedThreads) : 1;
  if (groups >= (int64_t)1 << 24) return fail(SCONV_ERR_UNSUPPORTED, "%s: too many tokens", fn);
  const PagedMeta p = {query_lens, context_lens, free_blocks, block_table, query_start_loc,
                       seq_idx_out, query_start_out, blocks_used, positions_out, slot_mapping_out,
                       num_free, bt_row_stride, n, num_reqs, max_blocks, block_size};
  if (num_reqs <= kMetaReqs) {
    hipLaunchKernelGGL(paged_metadata_kernel, dim3((uint32_t)groups), dim3(kPagedThreads), 0, stream, p);
    return check_launch(fn);
  }
  hipLaunchKernelGGL(paged_sums_kernel, dim3(1), dim3(kSumThreads), 0, stream, p);
  if (const int rc = check_launch(fn)) return rc;
  if (n == 0) return SCONV_OK;
  hipLaunchKernelGGL(paged_tokens_kernel, dim3((uint32_t)groups), dim3(kPagedThreads), 0, stream, p);
  return check_launch(fn);
}
