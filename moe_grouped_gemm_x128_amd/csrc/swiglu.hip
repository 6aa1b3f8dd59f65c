// The gated activation between an expert's two products, with FP8 output, and
// its gradient, gfx950.
//
//   g = x[.., :I], u = x[.., I:],  s = 1 / (1 + exp(-g))
//   y = w (g s) u         (w the row's weight, 1 without)
//   out: y rounded to BF16 or F32, and / or q, sf: the 1x128 FP8 cast of the FP32 y
//   gradient, with z = dy w:
//   dg = z u s (1 + g (1 - s)),  du = z g s,  dw = sum over the row of dy (g s) u
//
// A row takes 16 to 256 lanes, eight elements each at a time; 16 lanes hold a
// 128-element block of the cast.
//
// What bounds it: memory for rows kept in BF16 (32749 x 2048, forward and gradient
// together 1.07 GB in 184 us, 5.8 TB/s); with the cast about 24 vector instructions an
// element, half the time of 6144 rows of 2048 (16.6 us, 3.8 TB/s), whose bytes fit the
// last cache.  A masked buffer that is mostly empty takes a workgroup for each of its
// rows all the same (32 x 4096 rows, 8 of them in use, 29 us; 32 x 256 6 us).

#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"

namespace dgmi {

namespace {

// 1 / (1 + exp(-g)) within 6 u for g from FAR up: exp(-g) = 2^x with x = -g log2 e, and what the
// rounding of x left over put back by an FMA.
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float L2E = 1.44269504088896340736f, L2E_LO = 1.92596299112661746887e-8f, LN2 = 0.693147180559945309417f;
  const float t = __builtin_amdgcn_fmed3f(-g, -104.0f, 88.0f);  // (2^x stays a number: past it the result is 0)
  const float x = t * L2E;
  const float rest = __builtin_fmaf(t, L2E_LO, __builtin_fmaf(t, L2E, -x)) * LN2;
  const float e = __builtin_amdgcn_exp2f(x);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, rest, e));
}

// Gates below FAR have sigmoids near and below 2^-126, which FP32 does not hold though their products with a large up
// or gradient may count: exp(g), taken as 2^192 times itself in FP32 and handed on in FP64.  Such gates are
// looked for in eight elements at once (6144 rows of 2048 with the cast 16.6 us for 16.1, in BF16 with the gradient
// none).
constexpr float FAR = -87.0f;
__device__ __forceinline__ double far_sigmoid(float g) {
  constexpr float L2E = 1.44269504088896340736f, L2E_LO = 1.92596299112661746887e-8f, LN2 = 0.693147180559945309417f;
  const float t = fmaxf(g, -230.0f);  // (2^-331: with what it may be multiplied by, nothing)
  float x = t * L2E;
  asm volatile("" : "+v"(x));  // (rounded here: fused with the sum below, it would not be the x of the rest)
  const float rest = __builtin_fmaf(t, L2E_LO, __builtin_fmaf(t, L2E, -x)) * LN2;
  const float e = __builtin_amdgcn_exp2f(x + 192.0f);
  return (double)__builtin_fmaf(e, rest, e) * 0x1p-192;
}
__device__ __forceinline__ bool any_far(const float g[8]) {
  uint32_t low = 0;  // (of negative numbers the lowest has the largest bits)
#pragma unroll
  for (int e = 0; e < 8; ++e) low = max(low, __float_as_uint(g[e]));
  return low > __float_as_uint(FAR);
}

// Rows of group g that count: all, or masked_m[g] of them.
__device__ __forceinline__ int live_rows(const int32_t* masked, int g, int rows) {
  return masked == nullptr ? rows : min(max(masked[g], 0), rows);
}

// Lanes of a row of I, eight elements each at a time: as many as one chunk a lane takes (two chunks a lane: 6144 rows
// of 2048 18.5 us for 16.0, 32768 of 512 17.8 for 16.8; half of the lanes idle: 16384 rows of 1024 27.1 for 16.4).
constexpr int fwd_lanes(int64_t I) { return I <= 128 ? 16 : I <= 256 ? 32 : I <= 512 ? 64 : I <= 1024 ? 128 : 256; }

template <int NT>
__global__ __launch_bounds__(256) void swiglu_kernel(const SwigluArgs p) {
  const int lane = threadIdx.x % NT;
  const uint32_t row = blockIdx.x * (256 / NT) + threadIdx.x / NT;
  if (row >= (uint32_t)(p.G * p.R)) return;  // (whole rows, as below)
  const int g = p.G == 1 ? 0 : (int)(row / (uint32_t)p.R), r = (int)(row - (uint32_t)g * p.R);
  if (r >= live_rows(p.masked, g, p.R)) return;
  const int64_t ox = g * p.sx_g + r * p.sx_r, oy = g * p.sy_g + r * p.sy_r;
  uint8_t* q = p.q + g * p.sq_g + r * p.sq_r;
  float* sf = p.sf + g * p.ss_g + r * p.ss_r;
  const float w = p.w != nullptr ? p.w[row * p.sw] : 1.0f;
  for (int from = 0; from < p.I; from += NT * 8) {
    const int at = from + lane * 8;
    float a[8], b[8];
    load8(p.x, p.x_bf16, ox, at, p.I, p.x_vec, a);
    load8(p.x, p.x_bf16, ox + p.I, at, p.I, p.u_vec, b);
    if (any_far(a)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!(a[e] < FAR)) continue;
        b[e] = (float)((double)a[e] * far_sigmoid(a[e]) * (double)b[e] * 0x1p-5);
        a[e] = 32.0f;  // (its sigmoid is 1)
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = (a[e] * sigmoid(a[e])) * b[e] * w;
    if (p.y != nullptr) store8(p.y, p.y_bf16, oy, at, p.I, p.y_vec, a);
    if (p.q == nullptr) continue;
    uint32_t lo, hi;
    const float s = cast_block8(a, p.ue8m0, lo, hi);
    if (at >= p.I) continue;
    store_codes8(q, at, p.I, p.q_vec, lo, hi);
    if ((lane & 15) == 0) sf[(at >> 7) * p.ss_k] = s;
  }
}

// One row takes NT lanes.
template <int NT>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(const SwigluBwdArgs p) {
  __shared__ float red[4];
  const int lane = threadIdx.x % NT;
  const uint32_t row = blockIdx.x * (256 / NT) + threadIdx.x / NT;
  if (row >= (uint32_t)(p.G * p.R)) return;
  const int g = p.G == 1 ? 0 : (int)(row / (uint32_t)p.R), r = (int)(row - (uint32_t)g * p.R);
  if (r >= live_rows(p.masked, g, p.R)) return;
  const int64_t ox = g * p.sx_g + r * p.sx_r, oy = g * p.sy_g + r * p.sy_r, od = g * p.sd_g + r * p.sd_r;
  const float w = p.w != nullptr ? p.w[row * p.sw] : 1.0f;
  float sum = 0.0f;
  for (int at = lane * 8; at < p.I; at += NT * 8) {
    float a[8], b[8], dy[8];
    load8(p.x, p.x_bf16, ox, at, p.I, p.x_vec, a);
    load8(p.x, p.x_bf16, ox + p.I, at, p.I, p.u_vec, b);
    load8(p.dy, p.dy_bf16, oy, at, p.I, p.dy_vec, dy);
    auto gradients = [&](auto far) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = dy[e] * w;
        if (decltype(far)::value && a[e] < FAR) {
          const double s = far_sigmoid(a[e]), act = a[e] * s;
          sum += (float)(dy[e] * act * b[e]);
          const double da = (double)z * b[e] * (s * (1.0 + a[e]));  // (1 - s is 1)
          b[e] = (float)(z * act);
          a[e] = (float)da;
        } else {
          const float s = sigmoid(a[e]), act = a[e] * s;
          sum = __builtin_fmaf(dy[e], act * b[e], sum);
          const float da = z * b[e] * (s * __builtin_fmaf(a[e], 1.0f - s, 1.0f));
          b[e] = z * act;
          a[e] = da;
        }
      }
    };
    if (any_far(a)) gradients(std::true_type{});
    else gradients(std::false_type{});
    store8(p.dx, p.dx_bf16, od, at, p.I, p.dx_vec, a);
    store8(p.dx, p.dx_bf16, od + p.I, at, p.I, p.du_vec, b);
  }
  if (p.dw == nullptr) return;
  sum = row_sum<NT>(sum, red);
  if (lane == 0) p.dw[row * p.sdw] = sum;
}

}  // namespace

int64_t swiglu_grid(int64_t rows, int64_t I) { return (rows * fwd_lanes(I) + 255) / 256; }
int64_t swiglu_bwd_grid(int64_t rows, int64_t I) {
  const int64_t per = I <= 128 ? 16 : I <= 512 ? 4 : 1;
  return (rows + per - 1) / per;
}

hipError_t launch_swiglu(const SwigluArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)swiglu_grid((int64_t)p.G * p.R, p.I)), block(256);
  switch (fwd_lanes(p.I)) {
    case 16: swiglu_kernel<16><<<grid, block, 0, stream>>>(p); break;
    case 32: swiglu_kernel<32><<<grid, block, 0, stream>>>(p); break;
    case 64: swiglu_kernel<64><<<grid, block, 0, stream>>>(p); break;
    case 128: swiglu_kernel<128><<<grid, block, 0, stream>>>(p); break;
    default: swiglu_kernel<256><<<grid, block, 0, stream>>>(p); break;
  }
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
