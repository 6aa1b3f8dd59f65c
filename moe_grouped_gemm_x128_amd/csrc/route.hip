// Expert routing of a mixture-of-experts layer, gfx950: from the router's
// logits to the table moe_dispatch_* reads (topk_idx) and the weights
// moe_combine reads (topk_weights), and the gradient of the logits.
//
//   scores      s = 1 / (1 + exp(-x))               (sigmoid)
//               s = exp(x - max x) / sum            (softmax)
//   choice      c = s + bias; without a bias the logit itself: scores rise with
//               it, and in FP32 neighbours, scores near 1 and scores that
//               underflow would become equal
//   eligible    an expert whose logit and bias are not -inf
//   groups      the E experts are n_group equal ranges; a group's score is
//               its best eligible choice, or the sum of its two best s + bias
//               (softmax without a bias: of exp(x - max x)); the topk_group
//               best groups stay
//   selection   the k best eligible choices of the groups that stay; ties go
//               to the lowest index, NaN ranks below every number; -1 where
//               fewer than k are eligible
//   weights     scale s_j; renormalised: scale s_j / (sum_j s_j + 1e-20)
//               (sigmoid), scale * softmax over the chosen logits (softmax)
//
// The backward takes the choice as given: with z_j = s of choice j, D = sum
// z_j + 1e-20 and g the gradient of the weights,
//   dz_j = scale g_j, renormalised scale (g_j - sum_i g_i z_i / D) / D,
//   sigmoid  dx_e = dz_e s_e (1 - s_e), 1 - s_e as s(-x_e),
//   softmax  dx_e = s_e (dz_e - sum_j dz_j z_j),
//   softmax, renormalised: with q the softmax over the chosen logits,
//            dx_j = scale q_j (g_j - sum_i g_i q_i), and zero elsewhere.
//
// A token takes LT = 16, 32 or 64 lanes (four tokens, two or one to a wave); each group
// takes L of them, a power of two with n_group L <= LT, and a lane NE
// consecutive experts of its group.  So every group is a run of lanes that the
// first steps of one butterfly reduce for all groups at once, and among equal
// choices the lowest lane has the lowest index.  Selection takes one round a
// choice: the lane's best key, the butterfly, a ballot for the lowest lane that
// has it.
//
// What bounds it: a token's logits are read once (16384 x 256 FP32: 3.5 us at
// the copy rate), but the scores that a bias asks for (an accurate exponential
// and a division each) and the rounds are about 530 vector instructions of a wave
// per token of 256 experts: 16 us for 16384 tokens on 1024 SIMDs.  Without a bias
// only the chosen experts' scores are formed: 160 per token of 128 experts, 7.1 us
// for 16384 tokens, whose waves spend 54% of their cycles waiting, 20% waiting to
// issue and 26% issuing (each round hangs on the one before it).  One token takes
// 4.3 us, of which a launch is about 2.

#include "common.hpp"
#include "lanes.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

constexpr int ROUTER_WAVES = 4;  // waves per workgroup

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

// NE consecutive values from `at`, the first `n` of them (0 .. NE); the others
// are `rest`.  vec: rows start on 16 bytes and n is a whole number of 16-byte
// chunks.
template <int NE>
__device__ __forceinline__ void load_run(const void* base, bool bf16, int64_t at, int n, bool vec, float rest,
                                         float x[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) x[i] = rest;
  if (bf16) {
    const uint16_t* from = static_cast<const uint16_t*>(base) + at;
    if constexpr (NE >= 8) {
      if (vec) {
#pragma unroll
        for (int i = 0; i < NE; i += 8)
          if (i < n) {
            const i32x4 v = *reinterpret_cast<const i32x4*>(from + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[i + 2 * e] = __uint_as_float((uint32_t)v[e] << 16);
              x[i + 2 * e + 1] = __uint_as_float((uint32_t)v[e] & 0xffff0000u);
            }
          }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) x[i] = bf16_to_f32(from[i]);
  } else {
    const float* from = static_cast<const float*>(base) + at;
    if constexpr (NE >= 4) {
      if (vec) {
#pragma unroll
        for (int i = 0; i < NE; i += 4)
          if (i < n) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(from + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i + e] = v[e];
          }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) x[i] = from[i];
  }
}

// LDS written by a wave and read by the same wave.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int LT, int NE>
__global__ __launch_bounds__(64 * ROUTER_WAVES) void moe_route_topk_kernel(const RouteTopkArgs p) {
  constexpr int TOKENS = 64 * ROUTER_WAVES / LT;
  __shared__ int chosen[TOKENS][LT];  // expert of each choice
  const int tl = threadIdx.x / LT, lane = threadIdx.x % LT;  // token of the workgroup, lane of the token
  const int t = blockIdx.x * TOKENS + tl;
  const bool live = t < p.T;
  const int g = lane >> p.log_l;                              // this lane's group
  const int first = (lane & ((1 << p.log_l) - 1)) * NE;       // its experts in the group
  int n = p.group_size - first;
  n = n < 0 || g >= p.n_group || !live ? 0 : n > NE ? NE : n;
  const int e0 = g * p.group_size + first;
  float x[NE], b[NE];
  load_run<NE>(p.logits, p.bf16, (int64_t)t * p.sl + e0, n, p.vec, -INFINITY, x);
  if (p.bias != nullptr) load_run<NE>(p.bias, false, e0, n, p.vec_bias, 0.0f, b);
  float top = -INFINITY;  // softmax: the row's largest logit, 0 where there is none
  if (p.softmax) {
#pragma unroll
    for (int i = 0; i < NE; ++i) top = fmaxf(top, x[i]);
    top = lanes_max<LT>(top);
    if (top == -INFINITY) top = 0.0f;
  }
  // a logit's score; softmax: before the division by the sum
  const auto score_of = [&](float v) { return p.softmax ? expf(v - top) : sigmoid_f32(v); };
  uint32_t key[NE];
  float sum = 1.0f;  // softmax: the row's sum, where it is wanted
  if (p.bias != nullptr || (p.softmax && !p.renorm)) {
    float s[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) s[i] = score_of(x[i]);
    if (p.softmax) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) sum += s[i];
      sum = lanes_sum<LT>(sum);
    }
    if (p.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float c = (p.softmax ? __fdiv_rn(s[i], sum) : s[i]) + b[i];
        key[i] = x[i] != -INFINITY && b[i] != -INFINITY ? choice_key(c) : 0u;
      }
    }
  }
  if (p.bias == nullptr) {
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = x[i] != -INFINITY ? choice_key(x[i]) : 0u;
  }
  if (p.n_group > 1) {
    // the group's two best choices, in all of its lanes
    uint32_t m1 = 0, m2 = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      m2 = max(m2, min(m1, key[i]));
      m1 = max(m1, key[i]);
    }
    auto merge = [&](uint32_t o1, uint32_t o2) {
      m2 = max(max(m2, o2), min(m1, o1));
      m1 = max(m1, o1);
    };
    if (p.log_l >= 1) merge(other<1>(m1), other<1>(m2));
    if (p.log_l >= 2) merge(other<2>(m1), other<2>(m2));
    if (p.log_l >= 3) merge(other<4>(m1), other<4>(m2));
    if constexpr (LT >= 32)
      if (p.log_l >= 4) merge(other<8>(m1), other<8>(m2));
    if constexpr (LT >= 64)
      if (p.log_l >= 5) merge(other<16>(m1), other<16>(m2));
    uint32_t score = m1;
    if (p.group_top == 2 && m1 != 0) {
      // (without a bias the keys are those of logits)
      const float c1 = p.bias != nullptr ? key_choice(m1) : score_of(key_choice(m1));
      const float c2 = m2 == 0 ? 0.0f : p.bias != nullptr ? key_choice(m2) : score_of(key_choice(m2));
      score = choice_key(c1 + c2);
    }
    // the group stays if fewer than topk_group others are better
    int better = 0;
    const int row = (threadIdx.x & 63) - lane;  // first lane of the token
    for (int o = 0; o < p.n_group; ++o) {
      const uint32_t v = LT == 64 ? (uint32_t)__builtin_amdgcn_readlane((int)score, o << p.log_l)
                                  : (uint32_t)__builtin_amdgcn_ds_bpermute((row + (o << p.log_l)) * 4, (int)score);
      better += v > score || (v == score && o < g) ? 1 : 0;
    }
    if (better >= p.topk_group) {
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] = 0;
    }
  }
  // selection: one choice a round, its lane writes it down
  if (lane < p.k) chosen[tl][lane] = -1;
  wave_lds_fence();
  for (int j = 0; j < p.k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) m = max(m, key[i]);
    const uint32_t best = lanes_max<LT>(m);
    if (!__any(best != 0)) break;
    const uint64_t at = __ballot(m == best && best != 0);
    bool mine;  // the lowest lane of the token with the best key
    if constexpr (LT == 64) {
      mine = lane == __ffsll((unsigned long long)at) - 1;
    } else {
      const uint64_t part = at >> ((threadIdx.x & 63) - lane);
      mine = ((uint32_t)part & ((2u << lane) - 1)) == (1u << lane);
    }
    if (mine) {
      int i_best = 0;
#pragma unroll
      for (int i = NE - 1; i > 0; --i) i_best = key[i] == best ? i : i_best;
      i_best = key[0] == best ? 0 : i_best;
      chosen[tl][j] = e0 + i_best;
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] = i == i_best ? 0u : key[i];
    }
  }
  wave_lds_fence();
  const int idx = lane < p.k ? chosen[tl][lane] : -1;
  const bool got = idx >= 0;
  // the choice's logit, read once more: keeping every lane's logits and scores
  // at hand through the rounds costs more
  float z = 0.0f, xz = -INFINITY;
  if (got) {
    const int64_t at = (int64_t)t * p.sl + idx;
    xz = p.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[at]) : static_cast<const float*>(p.logits)[at];
    z = score_of(xz);
  }
  float wgt;
  if (!p.softmax) {
    const float d = p.renorm ? lanes_sum<LT>(z) + 1e-20f : 1.0f;
    wgt = p.renorm && got ? __fdiv_rn(z, d) : z;  // (0 where nothing was chosen, also beside a NaN)
  } else if (!p.renorm) {
    wgt = got ? __fdiv_rn(z, sum) : 0.0f;
  } else {
    const float m = lanes_max<LT>(xz);
    const float e = got ? expf(xz - m) : 0.0f;
    const float d = lanes_sum<LT>(e);
    wgt = got ? __fdiv_rn(e, d) : 0.0f;
    // +inf anywhere among softmax logits: no weight of the row is a number
    if (got && !(top < INFINITY)) wgt = __uint_as_float(0x7fc00000u);
  }
  if (lane < p.k && live) {
    p.idx[(int64_t)t * p.si + lane] = idx;
    p.w[(int64_t)t * p.sw + lane] = p.scale * wgt;
  }
}

// g less its mean under weights q of sum 1.  The mean goes off in two steps, r as
// it was rounded and then the mean of what is left: where one weight is nearly 1
// its g - mean is far below the spacing of g and would be lost in one.
template <int LT>
__device__ __forceinline__ float less_mean(float g, float q, float r) {
  const float left = g - r;
  return left - lanes_sum<LT>(left * q);
}

template <int LT, int NE>
__global__ __launch_bounds__(64 * ROUTER_WAVES) void moe_route_topk_bwd_kernel(const RouteTopkBwdArgs p) {
  constexpr int TOKENS = 64 * ROUTER_WAVES / LT;
  __shared__ int2 part[TOKENS][LT];  // {expert, gradient of its logit} of each choice
  const int tl = threadIdx.x / LT, lane = threadIdx.x % LT;
  const int t = blockIdx.x * TOKENS + tl;
  const bool live = t < p.T;
  const int e0 = lane * NE;
  int n = p.E - e0;
  n = n < 0 || !live ? 0 : n > NE ? NE : n;
  const int64_t row = (int64_t)t * p.sl;
  int idx = -1;
  float g = 0.0f, xz = -INFINITY;
  if (lane < p.k && live) {
    idx = p.idx[(int64_t)t * p.si + lane];
    if (idx < 0 || idx >= p.E) idx = -1;
  }
  if (idx >= 0) {
    g = p.scale * p.g[(int64_t)t * p.sg + lane];
    xz = p.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[row + idx])
                : static_cast<const float*>(p.logits)[row + idx];
  }
  float d = g;      // gradient of logit idx through choice `lane`; softmax weights as they are: of its score
  float x[NE], r = 0.0f;  // softmax scores of the row, and the mean of their gradients
  if (!p.softmax) {
    const float z = idx >= 0 ? sigmoid_f32(xz) : 0.0f;
    float dz = g;
    if (p.renorm) {
      // (the weights z / D add up to 1 - 1e-20 / D)
      const float D = lanes_sum<LT>(z) + 1e-20f, q = __fdiv_rn(z, D), mean = lanes_sum<LT>(g * q);
      dz = __fdiv_rn(less_mean<LT>(g, q, mean) + mean * __fdiv_rn(1e-20f, D), D);
    }
    // (1 - s(x) as s(-x): taken from the rounded s it would be 0 from logits of 17 on)
    d = idx >= 0 ? dz * (z * sigmoid_f32(-xz)) : 0.0f;
  } else if (p.renorm) {
    const float m = lanes_max<LT>(xz);
    const float e = idx >= 0 ? expf(xz - m) : 0.0f;
    const float sum = lanes_sum<LT>(e);
    const float q = idx >= 0 ? __fdiv_rn(e, sum) : 0.0f;
    d = q * less_mean<LT>(g, q, lanes_sum<LT>(g * q));
  } else {
    load_run<NE>(p.logits, p.bf16, row + e0, n, p.vec, -INFINITY, x);
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) top = fmaxf(top, x[i]);
    top = lanes_max<LT>(top);
    if (top == -INFINITY) top = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      x[i] = expf(x[i] - top);
      sum += x[i];
    }
    sum = lanes_sum<LT>(sum);
    if (sum == 0.0f) sum = 1.0f;  // every logit -inf
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] = __fdiv_rn(x[i], sum);
    const float z = idx >= 0 ? __fdiv_rn(expf(xz - top), sum) : 0.0f;
    r = lanes_sum<LT>(g * z);
  }
  if (lane < p.k) part[tl][lane] = int2{idx, __float_as_int(d)};
  wave_lds_fence();
  // what the choices of each expert give
  float dx[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) dx[i] = 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int2 c = part[tl][j];
    const int at = c.x - e0;
#pragma unroll
    for (int i = 0; i < NE; ++i) dx[i] += at == i ? __int_as_float(c.y) : 0.0f;
  }
  if (p.softmax && !p.renorm) {  // score * (its gradient less their mean), in two steps as above
    float left = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      dx[i] -= r;
      left += dx[i] * x[i];
    }
    left = lanes_sum<LT>(left);
#pragma unroll
    for (int i = 0; i < NE; ++i) dx[i] = x[i] * (dx[i] - left);
  }
  const int64_t out = (int64_t)t * p.so + e0;
  if (p.out_bf16) {
    uint16_t* to = static_cast<uint16_t*>(p.dlogits) + out;
    if constexpr (NE >= 4) {
      if (p.vec_out) {
#pragma unroll
        for (int i = 0; i < NE; i += 4)
          if (i < n) *reinterpret_cast<i32x2*>(to + i) = to_bf16x4_bits(f32x4{dx[i], dx[i + 1], dx[i + 2], dx[i + 3]});
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) to[i] = f32_to_bf16_rne(dx[i]);
  } else {
    float* to = static_cast<float*>(p.dlogits) + out;
    if constexpr (NE >= 4) {
      if (p.vec_out) {
#pragma unroll
        for (int i = 0; i < NE; i += 4)
          if (i < n) *reinterpret_cast<f32x4*>(to + i) = f32x4{dx[i], dx[i + 1], dx[i + 2], dx[i + 3]};
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) to[i] = dx[i];
  }
}

bool aligned16(const void* p, int64_t row_stride_bytes, int64_t rows) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || row_stride_bytes % 16 == 0);
}

// The smallest of 1, 2, 4, ... that holds v.
int pow2_up(int v) {
  int n = 1;
  while (n < v) n *= 2;
  return n;
}

}  // namespace

hipError_t launch_moe_route_topk(RouteTopkArgs p, hipStream_t stream) {
  const int es = p.bf16 ? 2 : 4;
  int lt = 64, ne = 0;
  auto place = [&](int lanes) {  // lanes of a group and experts of a lane
    if (p.k > lanes || p.n_group > lanes) return false;
    int log_l = 0;
    while ((p.n_group << (log_l + 1)) <= lanes) ++log_l;
    const int run = pow2_up((p.group_size + (1 << log_l) - 1) >> log_l);
    if (run > (lanes == 64 ? 32 : 16)) return false;
    p.log_l = log_l;
    ne = run;
    lt = lanes;
    return true;
  };
  // Few tokens: many lanes, whose rounds are the shortest; many: few lanes, of
  // which four or two tokens share an instruction.  Measured with 64 / 32 / 16
  // lanes, in us: 256 tokens, 256 experts with a bias (8 of them, 4 of 8 groups)
  // 5.4 / 6.8 / 10.3, 4096 tokens 7.9 / 7.6 / 9.2, 16384 tokens 19.6 / 17.1 / 16.0;
  // 128 experts without bias and groups 4.4 / 4.7 / 5.2, 5.6 / 5.0 / 5.1, 12.0 / 9.3
  // / 7.1.
  if (!(p.T > 8192 && place(16)) && !(p.T > 2048 && place(32))) place(64);
  const int chunk = 16 / es;
  p.vec = p.group_size % chunk == 0 && ne % chunk == 0 && aligned16(p.logits, p.sl * es, p.T);
  p.vec_bias = p.bias != nullptr && p.group_size % 4 == 0 && ne % 4 == 0 && aligned16(p.bias, 0, 1);
  const dim3 block(64 * ROUTER_WAVES);
  const dim3 grid((unsigned)(((int64_t)p.T * lt + block.x - 1) / block.x));
#define ROUTE_CASE(LT, NE) \
  if (lt == LT && ne == NE) moe_route_topk_kernel<LT, NE><<<grid, block, 0, stream>>>(p);
  ROUTE_CASE(16, 1) ROUTE_CASE(16, 2) ROUTE_CASE(16, 4) ROUTE_CASE(16, 8) ROUTE_CASE(16, 16)
  ROUTE_CASE(32, 1) ROUTE_CASE(32, 2) ROUTE_CASE(32, 4) ROUTE_CASE(32, 8) ROUTE_CASE(32, 16)
  ROUTE_CASE(64, 1) ROUTE_CASE(64, 2) ROUTE_CASE(64, 4) ROUTE_CASE(64, 8) ROUTE_CASE(64, 16) ROUTE_CASE(64, 32)
#undef ROUTE_CASE
  return hipGetLastError();
}

hipError_t launch_moe_route_topk_bwd(RouteTopkBwdArgs p, hipStream_t stream) {
  const int es = p.bf16 ? 2 : 4, oes = p.out_bf16 ? 2 : 4;
  // At most eight experts to a lane, so that a token's lanes write whole lines:
  // 16384 tokens with 64 / 32 / 16 lanes took 9.7 / 8.1 / 10.0 us for 256
  // experts, 7.6 / 6.1 / 5.6 us for 128, 6.9 / 5.3 / 4.5 us for 64.
  const int lt = p.k <= 16 && p.E <= 128 ? 16 : p.k <= 32 && p.E <= 256 ? 32 : 64;
  const int ne = pow2_up((p.E + lt - 1) / lt);
  p.vec = p.E % (16 / es) == 0 && ne % (16 / es) == 0 && aligned16(p.logits, p.sl * es, p.T);
  p.vec_out = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % (4 * oes) == 0 && (p.T <= 1 || p.so % 4 == 0);
  const dim3 block(64 * ROUTER_WAVES);
  const dim3 grid((unsigned)(((int64_t)p.T * lt + block.x - 1) / block.x));
#define ROUTE_CASE(LT, NE) \
  if (lt == LT && ne == NE) moe_route_topk_bwd_kernel<LT, NE><<<grid, block, 0, stream>>>(p);
  ROUTE_CASE(16, 1) ROUTE_CASE(16, 2) ROUTE_CASE(16, 4) ROUTE_CASE(16, 8)
  ROUTE_CASE(32, 1) ROUTE_CASE(32, 2) ROUTE_CASE(32, 4) ROUTE_CASE(32, 8)
  ROUTE_CASE(64, 1) ROUTE_CASE(64, 2) ROUTE_CASE(64, 4) ROUTE_CASE(64, 8) ROUTE_CASE(64, 16)
#undef ROUTE_CASE
  return hipGetLastError();
}

}  // namespace dgmi
