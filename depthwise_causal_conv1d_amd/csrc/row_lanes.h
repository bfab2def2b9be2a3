// row_lanes.h -- channels in lanes: addresses and loads of rows of tokens,
// shared by the gated linear recurrence and the conv's gradients.
#pragma once

#include <type_traits>

#include "sconv_device.h"

namespace sconv {

// A lane's vector of one row: a uniform row and a 32-bit byte offset, which
// is what the addressing mode takes.
template <typename S>
__device__ __forceinline__ S* in_row(S* row, uint32_t bytes) {
  typedef std::conditional_t<std::is_const_v<S>, const char, char> B;
  return reinterpret_cast<S*>(reinterpret_cast<B*>(row) + bytes);
}

// Hides where a lane's byte offset comes from: a 64-bit copy made once ahead
// of a loop would keep the addressing mode from taking the 32-bit one.
__device__ __forceinline__ uint32_t lane_offset(uint32_t bytes) {
  asm("" : "+v"(bytes));
  return bytes;
}

// R rows [row0, row0 + R) of a plane, rows from `end` on read as row end - 1
// (unused).  Ordinary loads: streaming ones read lines that two workgroups
// share twice (8191 x 1001 fp32, forward and gradients: 176 against 134 us);
// where rows are whole lines they gain 2% (16 ragged sequences x 4096 bf16,
// prefill: 148 against 152 us).
template <typename P, int R, typename S>
__device__ __forceinline__ void load_rows(P (&v)[R], const S* plane, int64_t stride, int row0,
                                          int end, uint32_t bytes) {
  const int n = end - row0;
  const S* q = plane + (n > 0 ? row0 : end - 1) * stride;
  bytes = lane_offset(bytes);
  // (No second path for whole tiles: a branch between a load and its use makes
  // the loads wait where the paths meet, 220 against 152 us.)
#pragma unroll
  for (int r = 0; r < R; ++r) {
    v[r].load(in_row(q, bytes));
    q += r + 1 < n ? stride : 0;
  }
}

}  // namespace sconv
