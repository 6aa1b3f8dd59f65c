// Expert routing of a mixture-of-experts layer, gfx950: from the router's
// logits to the table moe_dispatch_* reads (topk_idx) and the weights
// moe_combine reads (topk_weights), and the gradient of the logits.
//
//   scores      s = 1 / (1 + exp(-x))               (sigmoid)
//               s = exp(x - max x) / sum            (softmax)
//   choice      c = s + bias; softmax without bias: c = exp(x - max x), the
//               same order without the sum's rounding
//   eligible    an expert whose logit and bias are not -inf
//   groups      the E experts are n_group equal ranges; a group's score is
//               the sum of its group_top (1 or 2) best eligible choices; the
//               topk_group best groups stay
//   selection   the k best eligible choices of the groups that stay; ties go
//               to the lowest index, NaN ranks below every number; -1 where
//               fewer than k are eligible
//   weights     scale s_j; renormalised: scale s_j / (sum_j s_j + 1e-20)
//               (sigmoid), scale * softmax over the chosen logits (softmax)
//
// The backward takes the choice as given: with z_j = s of choice j, D = sum
// z_j + 1e-20 and g the gradient of the weights,
//   dz_j = scale g_j, renormalised scale (g_j - sum_i g_i z_i / D) / D,
//   sigmoid  dx_e = dz_e s_e (1 - s_e),
//   softmax  dx_e = s_e (dz_e - sum_j dz_j z_j),
//   softmax, renormalised: with q the softmax over the chosen logits,
//            dx_j = scale q_j (g_j - sum_i g_i q_i), and zero elsewhere.
//
// One wave per token.  Lane l holds the NE consecutive experts l * NE ...,
// so that among equal choices the lowest lane has the lowest index.

#include "common.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

constexpr int ROUTER_WAVES = 4;  // tokens per workgroup

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}
__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// A choice as an unsigned key of the same order: 0 is kept for experts that
// cannot be chosen, NaN is 1, -0 counts as +0.
__device__ __forceinline__ uint32_t choice_key(float c) {
  const uint32_t u = __float_as_uint(c + 0.0f);
  const uint32_t key = u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
  return c != c ? 1u : key;
}
__device__ __forceinline__ float key_choice(uint32_t key) {
  return key <= 1u ? __uint_as_float(0x7fc00000u) : __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float sigmoid_f32(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }

// The NE logits of a lane (experts e0 ...; -inf past the last one).
template <int NE>
__device__ __forceinline__ void load_logits(const void* base, int bf16, int64_t row, int e0, int E, float x[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    x[i] = -INFINITY;
    if (e0 + i < E)
      x[i] = bf16 ? bf16_to_f32(static_cast<const uint16_t*>(base)[row + e0 + i])
                  : static_cast<const float*>(base)[row + e0 + i];
  }
}

template <int NE>
__global__ __launch_bounds__(64 * ROUTER_WAVES) void moe_route_topk_kernel(const RouteTopkArgs p) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * ROUTER_WAVES + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int e0 = lane * NE;
  float x[NE], s[NE];
  load_logits<NE>(p.logits, p.bf16, (int64_t)t * p.sl, e0, p.E, x);
  float top = -INFINITY;  // softmax: the row's largest logit, 0 where there is none
  if (p.softmax) {
#pragma unroll
    for (int i = 0; i < NE; ++i) top = fmaxf(top, x[i]);
    top = wave_max_f32(top);
    if (top == -INFINITY) top = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) s[i] = p.softmax ? expf(x[i] - top) : sigmoid_f32(x[i]);
  // softmax without renormalisation, or with a bias on the scores: the sum
  float inv = 1.0f;
  if (p.softmax && (!p.renorm || p.bias != nullptr)) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) sum += s[i];
    sum = wave_sum_f32(sum);
    inv = sum;
  }
  uint32_t key[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    float c = s[i];
    bool ok = x[i] != -INFINITY;
    if (p.bias != nullptr && e0 + i < p.E) {
      const float b = p.bias[e0 + i];
      c = (p.softmax ? __fdiv_rn(c, inv) : c) + b;
      ok = ok && b != -INFINITY;
    }
    key[i] = ok ? choice_key(c) : 0u;
  }
  if (p.n_group > 1) {
    // score of each group, kept by the lane of the group's number
    uint32_t mine = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const int lo = g * p.group_size, hi = lo + p.group_size;
      uint32_t m1 = 0, m2 = 0;  // this lane's two best of the group
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const uint32_t v = (e0 + i >= lo && e0 + i < hi) ? key[i] : 0u;
        m2 = max(m2, min(m1, v));
        m1 = max(m1, v);
      }
      const uint32_t best = wave_max_u32(m1);
      uint32_t score = best;
      if (p.group_top == 2 && best != 0) {
        const uint64_t at = __ballot(m1 == best);
        const uint32_t second = wave_max_u32(lane == __ffsll((unsigned long long)at) - 1 ? m2 : m1);
        if (second != 0) score = choice_key(key_choice(best) + key_choice(second));
      }
      if (lane == g) mine = score;
    }
    uint64_t kept = 0;
    for (int r = 0; r < p.topk_group; ++r) {
      const uint32_t best = wave_max_u32(mine);
      if (best == 0) break;
      const int g = __ffsll((unsigned long long)__ballot(mine == best)) - 1;
      kept |= 1ull << g;
      if (lane == g) mine = 0;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int g = (e0 + i) / p.group_size;
      if (g >= 64 || !((kept >> g) & 1)) key[i] = 0;
    }
  }
  // selection: lane j keeps choice j
  int idx = -1;
  float z = 0.0f, xz = -INFINITY;
  for (int j = 0; j < p.k; ++j) {
    uint32_t m = 0;
    int at = 0;
    float ms = 0.0f, mx = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const bool more = key[i] > m;
      m = more ? key[i] : m;
      at = more ? i : at;
      ms = more ? s[i] : ms;
      mx = more ? x[i] : mx;
    }
    const uint32_t best = wave_max_u32(m);
    if (best == 0) break;
    const int w = __ffsll((unsigned long long)__ballot(m == best)) - 1;
    const int wi = __shfl(at, w, 64);
    const float ws = __shfl(ms, w, 64), wx = __shfl(mx, w, 64);
    if (lane == j) {
      idx = w * NE + wi;
      z = ws;
      xz = wx;
    }
    if (lane == w) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (i == at) key[i] = 0;
    }
  }
  float wgt;
  if (!p.softmax) {
    wgt = p.renorm ? __fdiv_rn(z, wave_sum_f32(z) + 1e-20f) : z;
  } else if (!p.renorm) {
    wgt = idx >= 0 ? __fdiv_rn(z, inv) : 0.0f;
  } else {
    const float m = wave_max_f32(xz);
    const float e = idx >= 0 ? expf(xz - m) : 0.0f;
    const float sum = wave_sum_f32(e);
    wgt = idx >= 0 ? __fdiv_rn(e, sum) : 0.0f;
    // NaN and +inf anywhere among softmax logits: no weight of the row is a number
    if (idx >= 0 && !(top < INFINITY)) wgt = __uint_as_float(0x7fc00000u);
  }
  if (lane < p.k) {
    p.idx[(int64_t)t * p.si + lane] = idx;
    p.w[(int64_t)t * p.sw + lane] = p.scale * wgt;
  }
}

template <int NE>
__global__ __launch_bounds__(64 * ROUTER_WAVES) void moe_route_topk_bwd_kernel(const RouteTopkBwdArgs p) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * ROUTER_WAVES + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int e0 = lane * NE;
  const int64_t row = (int64_t)t * p.sl;
  int idx = -1;
  float g = 0.0f, xz = -INFINITY;
  if (lane < p.k) {
    idx = p.idx[(int64_t)t * p.si + lane];
    if (idx < 0 || idx >= p.E) idx = -1;
  }
  if (idx >= 0) {
    g = p.scale * p.g[(int64_t)t * p.sg + lane];
    xz = p.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[row + idx])
                : static_cast<const float*>(p.logits)[row + idx];
  }
  float d = 0.0f;         // gradient of logit idx through choice `lane`
  float x[NE], sub = 0.0f;  // softmax scores of the row, and what each takes off
#pragma unroll
  for (int i = 0; i < NE; ++i) x[i] = 0.0f;
  if (!p.softmax) {
    const float z = idx >= 0 ? sigmoid_f32(xz) : 0.0f;
    float dz = g;
    if (p.renorm) {
      const float D = wave_sum_f32(z) + 1e-20f;
      dz = __fdiv_rn(g - __fdiv_rn(wave_sum_f32(g * z), D), D);
    }
    d = idx >= 0 ? dz * (z * (1.0f - z)) : 0.0f;
  } else if (p.renorm) {
    const float m = wave_max_f32(xz);
    const float e = idx >= 0 ? expf(xz - m) : 0.0f;
    const float sum = wave_sum_f32(e);
    const float q = idx >= 0 ? __fdiv_rn(e, sum) : 0.0f;
    d = q * (g - wave_sum_f32(g * q));
  } else {
    load_logits<NE>(p.logits, p.bf16, row, e0, p.E, x);
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) top = fmaxf(top, x[i]);
    top = wave_max_f32(top);
    if (top == -INFINITY) top = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      x[i] = expf(x[i] - top);
      sum += x[i];
    }
    sum = wave_sum_f32(sum);
    if (sum == 0.0f) sum = 1.0f;  // every logit -inf
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] = __fdiv_rn(x[i], sum);
    const float z = idx >= 0 ? __fdiv_rn(expf(xz - top), sum) : 0.0f;
    sub = wave_sum_f32(g * z);
    d = g * z;
  }
  // dx_e = (what choice j of expert e gives) - score * sub
  float dx[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) dx[i] = -(x[i] * sub);
  for (int j = 0; j < p.k; ++j) {
    const int ej = __shfl(idx, j, 64);
    const float dj = __shfl(d, j, 64);
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (ej == e0 + i) dx[i] += dj;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if (e0 + i >= p.E) continue;
    const int64_t at = (int64_t)t * p.so + e0 + i;
    if (p.out_bf16) static_cast<uint16_t*>(p.dlogits)[at] = f32_to_bf16_rne(dx[i]);
    else static_cast<float*>(p.dlogits)[at] = dx[i];
  }
}

}  // namespace

hipError_t launch_moe_route_topk(const RouteTopkArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + ROUTER_WAVES - 1) / ROUTER_WAVES)), block(64 * ROUTER_WAVES);
  if (p.E <= 64) moe_route_topk_kernel<1><<<grid, block, 0, stream>>>(p);
  else if (p.E <= 128) moe_route_topk_kernel<2><<<grid, block, 0, stream>>>(p);
  else if (p.E <= 256) moe_route_topk_kernel<4><<<grid, block, 0, stream>>>(p);
  else if (p.E <= 512) moe_route_topk_kernel<8><<<grid, block, 0, stream>>>(p);
  else moe_route_topk_kernel<16><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_moe_route_topk_bwd(const RouteTopkBwdArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + ROUTER_WAVES - 1) / ROUTER_WAVES)), block(64 * ROUTER_WAVES);
  if (p.E <= 64) moe_route_topk_bwd_kernel<1><<<grid, block, 0, stream>>>(p);
  else if (p.E <= 128) moe_route_topk_bwd_kernel<2><<<grid, block, 0, stream>>>(p);
  else if (p.E <= 256) moe_route_topk_bwd_kernel<4><<<grid, block, 0, stream>>>(p);
  else if (p.E <= 512) moe_route_topk_bwd_kernel<8><<<grid, block, 0, stream>>>(p);
  else moe_route_topk_bwd_kernel<16><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace dgmi
