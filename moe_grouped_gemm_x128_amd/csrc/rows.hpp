// Rows taken eight elements a lane: loads, stores, sums over a row's lanes and
// the 1x128 FP8 cast of values in registers.  Internal interface.
#pragma once

#include "common.hpp"
#include "lanes.hpp"

namespace dgmi {

// Elements at .. at+7 of a row of n (fewer at its end: zeros); vec: the row
// starts on 16 bytes.
__device__ __forceinline__ void load8(const void* base, bool bf16, int64_t row, int at, int n, bool vec, float v[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  if (bf16) {
    const uint16_t* from = static_cast<const uint16_t*>(base) + row + at;
    if (vec && at + 8 <= n) {
      const i32x4 t = *reinterpret_cast<const i32x4*>(from);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float((uint32_t)t[e] << 16);
        v[2 * e + 1] = __uint_as_float((uint32_t)t[e] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < n) v[e] = bf16_to_f32(from[e]);
    }
  } else {
    const float* from = static_cast<const float*>(base) + row + at;
    if (vec && at + 8 <= n) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(from), b = *reinterpret_cast<const f32x4*>(from + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < n) v[e] = from[e];
    }
  }
}

__device__ __forceinline__ i32x4 round8(const float v[8]) {
  const i32x2 a = to_bf16x4_bits(f32x4{v[0], v[1], v[2], v[3]}), b = to_bf16x4_bits(f32x4{v[4], v[5], v[6], v[7]});
  return i32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ void store8(void* base, bool bf16, int64_t row, int at, int n, bool vec, const float v[8]) {
  if (at >= n) return;
  if (bf16) {
    uint16_t* to = static_cast<uint16_t*>(base) + row + at;
    const i32x4 w = round8(v);
    if (vec && at + 8 <= n) {
      *reinterpret_cast<i32x4*>(to) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < n) to[e] = (uint16_t)((uint32_t)w[e / 2] >> (16 * (e & 1)));
    }
  } else {
    float* to = static_cast<float*>(base) + row + at;
    if (vec && at + 8 <= n) {
      *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < n) to[e] = v[e];
    }
  }
}

// Sum over the NT lanes of a row; every lane gets it.  red: one float a wave.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = lanes_sum<NT < 64 ? NT : 64>(v);
  if constexpr (NT > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += red[w];
  }
  return v;
}

// encode4 of values that are at most 448 scales (and of some that are not finite, whose codes do not matter): without
// its clamp (6144 rows of 2048 through the activation 16.4 us for 17.3).  A quotient that rounds past 448 still rounds
// to 448's code.
__device__ __forceinline__ uint32_t encode4_in_range(const float v[4], Recip d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(quot(v[0], d), quot(v[1], d), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(quot(v[2], d), quot(v[3], d), w, true);
  return (uint32_t)w;
}

// The FP8 cast of a 128-element block held by 16 lanes, eight elements each
// (zeros past its end): the lane's codes, and the block's scale as every cast of
// the library forms it.  As in the append to the cache, values that are not
// finite become NaN codes and do not count for the scale.
__device__ __forceinline__ float cast_block8(const float v[8], int ue8m0, uint32_t& lo, uint32_t& hi) {
  float amax = 0.0f, odd = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    amax = fmaxf(amax, fabsf(v[e]));  // (passes over NaN)
    odd = __builtin_fmaf(v[e], 0.0f, odd);  // NaN if one of them is not finite
  }
  amax = lanes_max<16>(amax);
  if (amax == INFINITY) {  // (of all 16 lanes)
    amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]) < INFINITY ? fabsf(v[e]) : 0.0f);
    amax = lanes_max<16>(amax);
  }
  const float s = block_scale(amax, ue8m0);
  const Recip d = recip_of(s);
  lo = encode4_in_range(v, d);
  hi = encode4_in_range(v + 4, d);
  if (odd != odd) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!(fabsf(v[e]) < INFINITY)) lo |= 0x7fu << (8 * e);
      if (!(fabsf(v[4 + e]) < INFINITY)) hi |= 0x7fu << (8 * e);
    }
  }
  return s;
}

// Eight codes at at .. at+7 of a row of n; vec: the row starts on 8 bytes.
__device__ __forceinline__ void store_codes8(uint8_t* row, int at, int n, bool vec, uint32_t lo, uint32_t hi) {
  if (vec && at + 8 <= n) {
    *reinterpret_cast<i32x2*>(row + at) = i32x2{(int)lo, (int)hi};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < n) row[at + e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
  }
}

}  // namespace dgmi
