// Exchanges and reductions between the lanes of a wave (gfx950), shared by the
// kernels that reduce rows.  Internal interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dgmi {

// The value of the lane at the other end of a butterfly step: within 2, 4, 8
// and 16 lanes by DPP (no shared memory), then across rows of 16 and halves.
template <int STEP>
__device__ __forceinline__ int other(int v) {
  if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true);        // quad 1 0 3 2
  else if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true);   // quad 2 3 0 1
  else if constexpr (STEP == 4) return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true);  // mirror of 8
  else if constexpr (STEP == 8) return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, true);  // mirror of 16
  else if constexpr (STEP == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? r[0] : r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32) ? r[0] : r[1];
  }
}
template <int STEP>
__device__ __forceinline__ uint32_t other(uint32_t v) { return (uint32_t)other<STEP>((int)v); }
template <int STEP>
__device__ __forceinline__ float other(float v) { return __int_as_float(other<STEP>(__float_as_int(v))); }

// Reductions over the N lanes of a token; every lane gets the result.
template <int N, typename T, typename F>
__device__ __forceinline__ T lanes_reduce(T v, F f) {
  if constexpr (N >= 2) v = f(v, other<1>(v));
  if constexpr (N >= 4) v = f(v, other<2>(v));
  if constexpr (N >= 8) v = f(v, other<4>(v));
  if constexpr (N >= 16) v = f(v, other<8>(v));
  // (a swap of two copies leaves both values of a pair in every lane)
  if constexpr (N >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(int, v), __builtin_bit_cast(int, v), false, false);
    v = f(__builtin_bit_cast(T, (int)r[0]), __builtin_bit_cast(T, (int)r[1]));
  }
  if constexpr (N >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, v), __builtin_bit_cast(int, v), false, false);
    v = f(__builtin_bit_cast(T, (int)r[0]), __builtin_bit_cast(T, (int)r[1]));
  }
  return v;
}
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_reduce<N>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_reduce<N>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_reduce<N>(v, [](float a, float b) { return a + b; });
}

}  // namespace dgmi
