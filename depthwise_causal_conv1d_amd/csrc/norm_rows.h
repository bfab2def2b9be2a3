// norm_rows.h -- what the norms of rows share: sums over lanes, how a row is
// spread over threads, and when it loads in whole vectors.
#pragma once

#include <initializer_list>
#include <type_traits>

#include "plane_host.h"
#include "sconv_device.h"

namespace sconv {

constexpr int kNormThreads = 256;

// v combined over groups of N consecutive lanes (a power of two); every lane
// gets the result.  Up to 16 lanes by DPP moves inside a row.
template <int N, typename T, typename F>
__device__ __forceinline__ T lanes_reduce(T v, F&& f) {
  auto step = [&](auto ctrl) {
    constexpr int C = decltype(ctrl)::value;
    const int m = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), C, 0xF, 0xF, true);
    v = f(v, __builtin_bit_cast(T, m));
  };
  if constexpr (N >= 2) step(std::integral_constant<int, 0xB1>());   // lanes 1 0 3 2
  if constexpr (N >= 4) step(std::integral_constant<int, 0x4E>());   // lanes 2 3 0 1
  if constexpr (N >= 8) step(std::integral_constant<int, 0x141>());  // half rows mirrored
  if constexpr (N >= 16) step(std::integral_constant<int, 0x140>()); // rows mirrored
  if constexpr (N >= 32) v = f(v, __shfl_xor(v, 16, 64));
  if constexpr (N >= 64) v = f(v, __shfl_xor(v, 32, 64));
  return v;
}

struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// Sum over the workgroup; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = lanes_reduce<64>(v, Add());
  const int wave = threadIdx.x >> 6, n = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) lds[wave] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < n; ++i) t += lds[i];
  __syncthreads();
  return t;
}

// How many vectors of a row T threads hold: the smallest instance that
// covers dim, 0 if none does.
static int norm_vectors(int32_t dim, int V, int T) {
  const int64_t need = cdiv(dim, (int64_t)V * T);
  if (V > 1) return need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : 0;
  return need <= 4 ? 4 : need <= 16 ? 16 : need <= 32 ? 32 : 0;
}

// Threads of a row: a wave where it holds the row in two vectors a lane (16
// single elements), which spares the barriers; else four waves, however many
// the rows: with a wave for rows of four and eight vectors, 17408 x 4096 bf16 to
// 8 bits takes 102 us (four waves 90), 4096 x 4096 30 (24), 17408 x 2048 fp32 97 (83).
static int norm_threads(int32_t dim, int V) {
  return cdiv(dim, (int64_t)V * 64) <= (V > 1 ? 2 : 16) ? 64 : 256;
}

// Every row starts on a multiple of V elements, and holds whole vectors.
static bool norm_vec(std::initializer_list<Plane> planes, int64_t V) {
  for (const Plane& a : planes)
    if (!a.empty() && (a.nc % V != 0 || (a.nt > 1 && a.st % V != 0) || !aligned_to(a.p, V * a.es)))
      return false;
  return true;
}

}  // namespace sconv
