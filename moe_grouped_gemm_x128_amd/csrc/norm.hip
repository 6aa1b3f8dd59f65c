// Root-mean-square norm with the residual's addition and FP8 output, and its
// gradient, gfx950.
//
//   h   = x + residual, rounded to the residual's type (h = x without one)
//   r   = 1 / sqrt(mean(h^2) + eps)
//   y   = h r w                                     (FP32)
//   out   y rounded to BF16 or F32, and / or q, sf: the 1x128 FP8 cast of the
//         FP32 y (amax / 448 floored as the per-token cast does)
//   gradient of the sum h, with g = w dy and xh = h r:
//   dx  = dh + r (g - xh mean(g xh)),   dw = sum over rows of dy xh
//
// A row is held in registers by NT lanes, NI chunks of 8 elements each, chunk c
// of the row in lane c % NT: 16 lanes hold one 128-element block of the cast,
// whose maximum is reduced without shared memory.  Where squares leave FP32's
// range (their sum past it, or below 2^-100 with an eps there too) they are taken
// again of h 2^-72 or h 2^96: 16384 squares of values below 2^128 2^-72 stay below
// 2^126.
//
// What bounds it: memory.  Read once, written once: 16384 rows of 7168 with the
// residual, its sum and FP8 codes (826 MB) take 161 us, 5.1 TB/s; 65536 x 1024
// without them 41 us, 6.6 TB/s from the last cache.  The gradient waits for a row's
// sums before it stores; BF16 rows are kept packed and the next one is on its way
// meanwhile: 8192 x 4096 with its weight's gradient and grad_h 57 us over three sets of
// inputs (4.7 TB/s; 48 us where they stay in the last cache, 56 without the packing), 8192
// x 7168 97 us (4.9 TB/s; 114).  F32 rows, loaded when their turn comes,
// reach 5.2 TB/s.  The weight's gradient takes 5 to 7 us of that.

#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"

namespace dgmi {

namespace {

// The sum of squares s of a row has left FP32's range, or lost bits that eps does not cover: the row is taken again
// with this factor on its values.
__device__ __forceinline__ bool out_of_range(float s, float eps) { return !(s < INFINITY) || (s < 0x1p-100f && eps < 0x1p-100f); }
__device__ __forceinline__ float factor_of(float s) { return s < 0x1p-100f ? 0x1p96f : 0x1p-72f; }

// The sum m of dy w h, made in one exchange with that of the squares, has left FP32's range where g xh need not: past
// it, or so small that what the products lost below 2^-149 counts (with r up to 2^10 it is below 2^-122 in grad_x).
// It is then taken again of values that are normalised first, with their factor on g where the sum could overflow a
// second time (16384 products of at most 2^128 2^-24 2^7).
__device__ __forceinline__ bool products_out_of_range(float m, float mean, float r) {
  return !(fabsf(m) < INFINITY) || !(fabsf(mean) < INFINITY) || (fabsf(m) < 0x1p-112f && r > 0x1p10f);
}

// a + b as FP32 holds it, one bit aside where the sum is not exact: rounded to BF16 next, a sum halfway between two
// BF16 numbers goes to the side of the exact one.  (Two BF16 values need no such care: where FP32 cannot hold their sum,
// the smaller of them does not lead near a middle.)
__device__ __forceinline__ float sum_aside(float a, float b) {
  const float s = a + b, c = s - a;
  const float rest = (a - (s - c)) + (b - c);  // what the rounding left, exactly
  const uint32_t bits = __float_as_uint(s);
  if (!(fabsf(s) < INFINITY) || rest == 0.0f || (bits & 0xffff) != 0x8000) return s;
  return __uint_as_float((rest < 0.0f) == (s < 0.0f) ? bits + 1 : bits - 1);
}

template <int NT>
constexpr int rows_of() { return NT < 256 ? 256 / NT : 1; }  // rows a workgroup takes side by side

template <int NT, int NI>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rms_norm_kernel(const RmsNormArgs p) {
  __shared__ float red[NT / 64 + 1];
  const int lane = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * rows_of<NT>() + threadIdx.x / NT;
  if (row >= p.rows) return;  // (whole groups of NT lanes; NT > 64 has one row a workgroup)
  const int64_t i0 = row / p.heads, i1 = row % p.heads;
  float v[NI][8];
  const int64_t ox = i0 * p.sx_0 + i1 * p.sx_1;
#pragma unroll
  for (int i = 0; i < NI; ++i) load8(p.x, p.x_bf16, ox, (lane + i * NT) * 8, p.H, p.x_vec, v[i]);
  if (p.res != nullptr) {
    const int64_t orr = i0 * p.sr_0 + i1 * p.sr_1, oh = i0 * p.sh_0 + i1 * p.sh_1;
    float t[NI][8];
#pragma unroll
    for (int i = 0; i < NI; ++i) load8(p.res, p.r_bf16, orr, (lane + i * NT) * 8, p.H, p.r_vec, t[i]);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (p.r_bf16 && !p.x_bf16) {
        bool middle = false;  // is a sum, as FP32 holds it, halfway between two BF16 numbers?
#pragma unroll
        for (int e = 0; e < 8; ++e) middle |= (__float_as_uint(v[i][e] + t[i][e]) & 0xffff) == 0x8000;
        if (middle) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[i][e] = sum_aside(v[i][e], t[i][e]);
            t[i][e] = -0.0f;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += t[i][e];
      if (p.r_bf16) {  // the norm is of the sum as it is stored
        const i32x4 w = round8(v[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[i][2 * e] = __uint_as_float((uint32_t)w[e] << 16);
          v[i][2 * e + 1] = __uint_as_float((uint32_t)w[e] & 0xffff0000u);
        }
      }
      if (p.h != nullptr) store8(p.h, p.r_bf16, oh, (lane + i * NT) * 8, p.H, p.h_vec, v[i]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fmaf(v[i][e], v[i][e], s);
  s = row_sum<NT>(s, red);
  float k = 1.0f;
  if (out_of_range(s, p.eps)) {  // (the whole row takes this turn)
    k = factor_of(s);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += (v[i][e] * k) * (v[i][e] * k);
    s = row_sum<NT>(s, red);
  }
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(s, (float)p.H) + p.eps * k * k));
  const int64_t oy = i0 * p.sy_0 + i1 * p.sy_1, oq = i0 * p.sq_0 + i1 * p.sq_1, os = i0 * p.ss_0 + i1 * p.ss_1;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int at = (lane + i * NT) * 8;
    if (at - (lane & 15) * 8 >= p.H) continue;  // (of the 16 lanes of a block)
    float w[8];
    load8(p.w, p.w_bf16, 0, at, p.H, p.w_vec, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= (v[i][e] * k) * r;
    if (p.y != nullptr) store8(p.y, p.y_bf16, oy, at, p.H, p.y_vec, w);
    if (p.q == nullptr) continue;
    uint32_t lo, hi;
    const float sc = cast_block8(w, p.ue8m0, lo, hi);
    if (at >= p.H) continue;
    store_codes8(p.q + oq, at, p.H, p.q_vec, lo, hi);
    if ((lane & 15) == 0) p.sf[os + (at >> 7) * p.ss_k] = sc;
  }
}

// Eight BF16 values of a row as they are stored (zeros past its end); value e of them.
__device__ __forceinline__ i32x4 raw8(const void* base, int64_t row, int at, int n) {
  if (at >= n) return i32x4{0, 0, 0, 0};
  return *reinterpret_cast<const i32x4*>(static_cast<const uint16_t*>(base) + row + at);
}
__device__ __forceinline__ float raw_value(const i32x4& v, int e) {
  return __uint_as_float(e & 1 ? (uint32_t)v[e / 2] & 0xffff0000u : (uint32_t)v[e / 2] << 16);
}

// Rows blockIdx, + gridDim, ... of the gradient; the weight's sums stay in
// registers and leave as one row of partial sums a workgroup.  RAW: the inputs are
// BF16, their rows whole 16-byte words: they stay packed, and the next row's are
// loaded while this one's sums are made (16384 x 4096 83 us for 97, 65536 x 1024 87 for 97).
// (Two chunks of 64 lanes unpacked take 129 registers unbidden: 65536 x 1024 168 us for 109 with 128.)
template <int NT, int NI, bool RAW>
__global__ __launch_bounds__(NT < 256 ? 256 : NT, NT == 64 && NI == 2 && !RAW ? 4 : 1) void rms_norm_bwd_kernel(const RmsNormBwdArgs p) {
  constexpr int RW = rows_of<NT>();
  __shared__ float red[NT / 64 + 1];
  __shared__ float sums[2][2][NT / 64 + 1];
  __shared__ float part[RW > 1 ? RW * NT * NI * 8 : 1];
  const int lane = threadIdx.x % NT, slot = threadIdx.x / NT;
  float w[NI][8], dw[NI][8];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    load8(p.w, p.w_bf16, 0, (lane + i * NT) * 8, p.H, p.w_vec, w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * RW;
  int turn = 0;
  struct Row {
    i32x4 x[NI], dy[NI], dh[NI];
  };
  auto load_row = [&](int64_t row, Row& v) __attribute__((always_inline)) {
    const int64_t i0 = row / p.heads, i1 = row - i0 * p.heads;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = (lane + i * NT) * 8;
      v.x[i] = raw8(p.h, i0 * p.sh_0 + i1 * p.sh_1, at, p.H);
      v.dy[i] = raw8(p.dy, i0 * p.sg_0 + i1 * p.sg_1, at, p.H);
      v.dh[i] = raw8(p.dh, i0 * p.sd_0 + i1 * p.sd_1, at, p.dh != nullptr ? p.H : 0);
    }
  };
  Row ahead;
  const int64_t first = (int64_t)blockIdx.x * RW + slot;
  if (RAW && first < p.rows) load_row(first, ahead);
  for (int64_t row = first; row < p.rows; row += step, turn ^= 1) {
    const int64_t i0 = row / p.heads, i1 = row - i0 * p.heads;
    const int64_t oh = i0 * p.sh_0 + i1 * p.sh_1, og = i0 * p.sg_0 + i1 * p.sg_1;
    float xf[RAW ? 1 : NI][8], dyf[RAW ? 1 : NI][8];
    Row here;
    if constexpr (RAW) {
      here = ahead;
      if (row + step < p.rows) load_row(row + step, ahead);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        load8(p.h, p.h_bf16, oh, (lane + i * NT) * 8, p.H, p.h_vec, xf[i]);
        load8(p.dy, p.dy_bf16, og, (lane + i * NT) * 8, p.H, p.dy_vec, dyf[i]);
      }
    }
    auto x = [&](int i, int e) __attribute__((always_inline)) {
      if constexpr (RAW) return raw_value(here.x[i], e);
      else return xf[i][e];
    };
    auto dy = [&](int i, int e) __attribute__((always_inline)) {
      if constexpr (RAW) return raw_value(here.dy[i], e);
      else return dyf[i][e];
    };
    float s = 0.0f, m = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = __builtin_fmaf(x(i, e), x(i, e), s);
        m = __builtin_fmaf(dy(i, e) * w[i][e], x(i, e), m);
      }
    s = lanes_sum<NT < 64 ? NT : 64>(s);
    m = lanes_sum<NT < 64 ? NT : 64>(m);
    if constexpr (NT > 64) {
      // both sums in one exchange (a slot is written again two rows on, past a barrier that follows its reads)
      if ((threadIdx.x & 63) == 0) {
        sums[turn][0][threadIdx.x >> 6] = s;
        sums[turn][1][threadIdx.x >> 6] = m;
      }
      __syncthreads();
      s = m = 0.0f;
#pragma unroll
      for (int v = 0; v < NT / 64; ++v) {
        s += sums[turn][0][v];
        m += sums[turn][1][v];
      }
    }
    float k = 1.0f;
    if (out_of_range(s, p.eps)) {  // (the whole row takes this turn)
      k = factor_of(s);
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += (x(i, e) * k) * (x(i, e) * k);
      s = row_sum<NT>(s, red);
    }
    const float rk = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(s, (float)p.H) + p.eps * k * k));
    const float r = rk * k;                      // h r = (h k) rk
    float mean = __fdiv_rn(m * rk, (float)p.H);  // of g xh
    if (k != 1.0f || products_out_of_range(m, mean, rk)) {  // (the whole row, too)
      const float j = fabsf(m) < INFINITY ? 1.0f : 0x1p-24f;
      float rr = rk;
      asm volatile("" : "+v"(rr));  // (what follows from it is not kept for the outputs: there are no registers for it)
      m = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = __builtin_fmaf(dy(i, e) * w[i][e] * j, (x(i, e) * k) * rr, m);
      mean = __fdiv_rn(row_sum<NT>(m, red), (float)p.H) * (1.0f / j);
    }
    const int64_t od = i0 * p.sd_0 + i1 * p.sd_1, ox = i0 * p.sx_0 + i1 * p.sx_1;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = (lane + i * NT) * 8;
      float dx[8];
      if constexpr (RAW) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] = raw_value(here.dh[i], e);
      } else {
        load8(p.dh != nullptr ? p.dh : p.h, p.dh_bf16, od, at, p.dh != nullptr ? p.H : 0, p.dh_vec, dx);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (x(i, e) * k) * rk;
        dw[i][e] = __builtin_fmaf(dy(i, e), xh, dw[i][e]);
        dx[e] = __builtin_fmaf(r, __builtin_fmaf(-xh, mean, dy(i, e) * w[i][e]), dx[e]);
      }
      store8(p.dx, p.dx_bf16, ox, at, p.H, p.dx_vec, dx);
    }
  }
  if (p.part == nullptr) return;
  float* to = p.part + (int64_t)blockIdx.x * p.H;
  if constexpr (RW > 1) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) part[slot * NT * NI * 8 + (lane + i * NT) * 8 + e] = dw[i][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.H; c += 256) {
      float t = 0.0f;
      for (int o = 0; o < RW; ++o) t += part[o * NT * NI * 8 + c];
      to[c] = t;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((lane + i * NT) * 8 + e < p.H) to[(lane + i * NT) * 8 + e] = dw[i][e];
  }
}

// The weight's gradient from the partial rows, in their order: 32 columns a
// workgroup, 32 runs of partial rows side by side.
__global__ __launch_bounds__(1024) void rms_norm_bwd_weight_kernel(const float* part, int parts, int H, void* dw,
                                                                   int bf16) {
  __shared__ float sums[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  const int per = (parts + 31) / 32;
  float s = 0.0f;
  if (c < H) {
    const int end = min(parts, (run + 1) * per);
#pragma unroll 8
    for (int i = run * per; i < end; ++i) s += part[(int64_t)i * H + c];
  }
  sums[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run == 0 && c < H) {
    s = 0.0f;
    for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
    if (bf16) static_cast<uint16_t*>(dw)[c] = f32_to_bf16_rne(s);
    else static_cast<float*>(dw)[c] = s;
  }
}

// Lanes and chunks that hold a row of H: NT * NI * 8 >= H.  Forward: two chunks a lane past 2048 (16384 rows of 4096
// with residual and codes 89 us, 512 lanes of one chunk 108), three past 4096 (9887 x 5120 with codes 36 us, 512 lanes
// of two 44), 512 lanes of two past 6144 (8192 x 7168 84 us, 256 lanes of four 95, 1024 of one 125).
// The gradient has more to hold a chunk, and takes one up to 8192 (16384 x 4096, not packed, 97 us, 256 lanes of two
// 161; packed 82; 16384 x 7168 168 us, 512 of two 198).
template <bool BWD, class F>
hipError_t with_row_shape(int64_t H, F f) {
#define DGMI_ROW(NT_, NI_) \
  if (H <= (int64_t)NT_ * NI_ * 8) return f(std::integral_constant<int, NT_>{}, std::integral_constant<int, NI_>{})
  DGMI_ROW(16, 1);
  DGMI_ROW(32, 1);
  DGMI_ROW(64, 1);
  DGMI_ROW(64, 2);
  DGMI_ROW(256, 1);
  if constexpr (BWD) {
    DGMI_ROW(512, 1);
  } else {
    DGMI_ROW(256, 2);
    DGMI_ROW(256, 3);
  }
  if constexpr (BWD) {
    DGMI_ROW(1024, 1);
  } else {
    DGMI_ROW(512, 2);
  }
  DGMI_ROW(1024, 2);
#undef DGMI_ROW
  return hipErrorInvalidValue;
}

}  // namespace

// Rows of H that one launch takes: 2^32 threads less than a workgroup.
int64_t rms_norm_max_rows(int64_t H) {
  int64_t lanes = 1024;
  (void)with_row_shape<true>(H, [&](auto nt, auto) {
    lanes = decltype(nt)::value;
    return hipSuccess;
  });
  return ((int64_t(1) << 32) - 1024) / lanes;
}

// Partial rows of the weight's gradient: workgroups of the gradient kernel.  Of 256 lanes four to a compute unit (32768
// x 2048, not packed, 94 us, two 147, three 108, eight 98; packed 84), of 512 lanes two (8192 x 4096 43 us, three 47, four 48), of 1024 one
// (16384 x 7168 168 us, two 175; 4096 x 16384 121, two 132).
int64_t rms_norm_bwd_parts(int64_t rows, int64_t H) {
  const int64_t per = H <= 128 ? 16 : H <= 256 ? 8 : H <= 1024 ? 4 : 1;  // rows a workgroup takes side by side
  const int64_t groups = (rows + per - 1) / per;
  const int64_t most = H <= 2048 ? 1024 : H <= 4096 ? 512 : 256;
  return groups < most ? groups : most;
}

hipError_t launch_rms_norm(const RmsNormArgs& p, hipStream_t stream) {
  return with_row_shape<false>(p.H, [&](auto nt, auto ni) {
    constexpr int NT = decltype(nt)::value, NI = decltype(ni)::value;
    const int64_t blocks = (p.rows + rows_of<NT>() - 1) / rows_of<NT>();
    rms_norm_kernel<NT, NI><<<dim3((unsigned)blocks), dim3(NT < 256 ? 256 : NT), 0, stream>>>(p);
    return hipGetLastError();
  });
}

hipError_t launch_rms_norm_bwd(const RmsNormBwdArgs& p, hipStream_t stream) {
  const int64_t parts = rms_norm_bwd_parts(p.rows, p.H);
  const hipError_t e = parts == 0 ? hipSuccess : with_row_shape<true>(p.H, [&](auto nt, auto ni) {
    constexpr int NT = decltype(nt)::value, NI = decltype(ni)::value;
    const bool raw = p.h_bf16 && p.dy_bf16 && p.h_vec && p.dy_vec && p.H % 8 == 0 &&
                     (p.dh == nullptr || (p.dh_bf16 && p.dh_vec));
    const dim3 gr((unsigned)parts), b(NT < 256 ? 256 : NT);
    // (1024 lanes of two chunks: the packed rows spill; 64 of two with grad_h: 65536 x 1024 113 us for 108)
    if constexpr (NT <= 64 || NI == 1) {
      if (raw && (NI == 1 || p.dh == nullptr)) {
        rms_norm_bwd_kernel<NT, NI, true><<<gr, b, 0, stream>>>(p);
        return hipGetLastError();
      }
    }
    rms_norm_bwd_kernel<NT, NI, false><<<gr, b, 0, stream>>>(p);
    return hipGetLastError();
  });
  if (e != hipSuccess || p.dw == nullptr) return e;
  rms_norm_bwd_weight_kernel<<<dim3((unsigned)((p.H + 31) / 32)), dim3(1024), 0, stream>>>(p.part, (int)parts, p.H,
                                                                                          p.dw, p.dw_bf16);
  return hipGetLastError();
}

}  // namespace dgmi
