// The gated activation between an expert's two products, with FP8 output, and
// its gradient, gfx950.
//
//   g = x[.., :I], u = x[.., I:],  s = 1 / (1 + exp(-g))
//   y = w (g s) u         (w the row's weight, 1 without)
//   out: y rounded to BF16 or F32, and / or q, sf: the 1x128 FP8 cast of the FP32 y
//   gradient, with z = dy w:
//   dg = z u s (1 + g (1 - s)),  du = z g s,  dw = sum over the row of dy (g s) u
//
// Sixteen lanes take a 128-element block of a row, eight elements each.

#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"

namespace dgmi {

namespace {

// 1 / (1 + exp(-g)) within 4 u: exp(-g) = 2^n 2^f with n whole and f the rest of
// -g log2 e, formed with two FMAs so that no bit of it is lost.
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float L2E = 1.44269504088896340736f, L2E_LO = 1.92596299112661746887e-8f;
  const float t = __builtin_amdgcn_fmed3f(-g, -104.0f, 104.0f);
  const float n = __builtin_rintf(t * L2E);
  const float f = __builtin_fmaf(t, L2E_LO, __builtin_fmaf(t, L2E, -n));
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// Rows of group g that count: all, or masked_m[g] of them.
__device__ __forceinline__ int live_rows(const int32_t* masked, int g, int rows) {
  return masked == nullptr ? rows : min(max(masked[g], 0), rows);
}

__global__ __launch_bounds__(256) void swiglu_kernel(const SwigluArgs p) {
  const int sub = threadIdx.x & 15;
  const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);  // a block of a row
  const int blk = (int)(unit % p.blocks);
  const int64_t row = unit / p.blocks;
  const int g = (int)(row / p.R), r = (int)(row % p.R);
  if (g >= p.G || r >= live_rows(p.masked, g, p.R)) return;  // (whole groups of 16 lanes)
  const int at = blk * 128 + sub * 8;
  const int64_t ox = g * p.sx_g + r * p.sx_r;
  float a[8], b[8];
  load8(p.x, p.x_bf16, ox, at, p.I, p.x_vec, a);
  load8(p.x, p.x_bf16, ox + p.I, at, p.I, p.u_vec, b);
  const float w = p.w != nullptr ? p.w[row * p.sw] : 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = (a[e] * sigmoid(a[e])) * b[e] * w;
  if (p.y != nullptr) store8(p.y, p.y_bf16, g * p.sy_g + r * p.sy_r, at, p.I, p.y_vec, a);
  if (p.q == nullptr) return;
  uint32_t lo, hi;
  const float s = cast_block8(a, p.ue8m0, lo, hi);
  if (at >= p.I) return;
  store_codes8(p.q + g * p.sq_g + r * p.sq_r, at, p.I, p.q_vec, lo, hi);
  if (sub == 0) p.sf[g * p.ss_g + r * p.ss_r + blk * p.ss_k] = s;
}

// One row takes NT lanes.
template <int NT>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(const SwigluBwdArgs p) {
  __shared__ float red[4];
  const int lane = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * (256 / NT) + threadIdx.x / NT;
  const int g = (int)(row / p.R), r = (int)(row % p.R);
  if (g >= p.G || r >= live_rows(p.masked, g, p.R)) return;
  const int64_t ox = g * p.sx_g + r * p.sx_r, oy = g * p.sy_g + r * p.sy_r, od = g * p.sd_g + r * p.sd_r;
  const float w = p.w != nullptr ? p.w[row * p.sw] : 1.0f;
  float sum = 0.0f;
  for (int at = lane * 8; at < p.I; at += NT * 8) {
    float a[8], b[8], dy[8];
    load8(p.x, p.x_bf16, ox, at, p.I, p.x_vec, a);
    load8(p.x, p.x_bf16, ox + p.I, at, p.I, p.u_vec, b);
    load8(p.dy, p.dy_bf16, oy, at, p.I, p.dy_vec, dy);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sigmoid(a[e]), z = dy[e] * w, act = a[e] * s;
      sum = __builtin_fmaf(dy[e], act * b[e], sum);
      const float da = z * b[e] * (s * __builtin_fmaf(a[e], 1.0f - s, 1.0f));
      b[e] = z * act;
      a[e] = da;
    }
    store8(p.dx, p.dx_bf16, od, at, p.I, p.dx_vec, a);
    store8(p.dx, p.dx_bf16, od + p.I, at, p.I, p.du_vec, b);
  }
  if (p.dw == nullptr) return;
  sum = row_sum<NT>(sum, red);
  if (lane == 0) p.dw[row * p.sdw] = sum;
}

}  // namespace

int64_t swiglu_grid(int64_t rows, int64_t I) { return (rows * ((I + 127) / 128) + 15) / 16; }
int64_t swiglu_bwd_grid(int64_t rows, int64_t I) {
  const int64_t per = I <= 128 ? 16 : I <= 512 ? 4 : 1;
  return (rows + per - 1) / per;
}

hipError_t launch_swiglu(SwigluArgs p, hipStream_t stream) {
  p.blocks = (p.I + 127) / 128;
  swiglu_kernel<<<dim3((unsigned)swiglu_grid((int64_t)p.G * p.R, p.I)), dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwdArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)swiglu_bwd_grid((int64_t)p.G * p.R, p.I)), block(256);
  if (p.I <= 128) swiglu_bwd_kernel<16><<<grid, block, 0, stream>>>(p);
  else if (p.I <= 512) swiglu_bwd_kernel<64><<<grid, block, 0, stream>>>(p);
  else swiglu_bwd_kernel<256><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace dgmi
