// Append of new tokens to a paged FP8 key/value cache, gfx950, with the
// position rotation applied on the way.
//
//   token t of sequence s (cu[s] <= t < cu[s+1]) has position
//   pos = start[s] + t - cu[s] and goes to slot pos % P of page
//   block_table[s][pos / P].
//   k (and q) are rotated, v is taken as it is: with c, s the cosine and
//   sine of (pos, j), each pair (x, y) -- elements (j, j + rot/2) of the
//   head, or (2j, 2j + 1) when interleaved -- becomes (x c - y s, y c + x s),
//   every product and sum rounded to FP32 on its own.
//   One scale per (page, head): a = max |value| over the page's new tokens
//   (floored at 1e-4), scale = a / 448 rounded up to a power of two.  A page
//   that already holds tokens keeps its scale if that is the larger one;
//   otherwise its older codes are re-encoded as e4m3(code * old / new),
//   which is exact while the result is a normal number (both powers of two).
//   code = e4m3(clamp(value / scale, -448, 448)), nearest even.  A value
//   that is not finite is stored as NaN and does not count for the maximum.
//
// The scale ties together all tokens of a page, so one workgroup owns a
// touched (page, head) of K or of V: it finds the maximum of the page's new
// tokens, then encodes them.  The rotation of q rides in the same launch.

#include "common.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

constexpr int APPEND_THREADS = 256;

// The sequence of token t (-1 if none): how many of cu[1 .. S-1] are <= t.
__device__ __forceinline__ int find_seq(const KvAppendArgs& p, int64_t t) {
  int n = 0;
  for (int base = 1; base < p.S; base += APPEND_THREADS) {
    const int j = base + threadIdx.x;
    n += __syncthreads_count(j < p.S && p.cu[j] <= t);
  }
  return (t >= p.cu[n] && t < p.cu[n + 1]) ? n : -1;
}

// Eight consecutive values of a row.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t at, float y[8]) {
  if constexpr (BF16) {
    const i32x4 v = *reinterpret_cast<const i32x4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __uint_as_float((uint32_t)v[i] << 16);
      y[2 * i + 1] = __uint_as_float((uint32_t)v[i] & 0xffff0000u);
    }
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + at);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = a[i];
      y[4 + i] = b[i];
    }
  }
}

// Elements d0 .. d0+7 of a head, rotated for position `pos` (row at `at`).
template <bool BF16>
__device__ __forceinline__ void load_rotated(const KvAppendArgs& p, const void* base, int64_t at, int d0, int64_t pos,
                                             float y[8]) {
  // (this file is compiled without contraction into FMAs)
  load8<BF16>(base, at + d0, y);
  if (d0 >= p.rot) return;  // (rot is 0 without a table)
  const int half = p.rot / 2;
  const float* row = p.cos_sin + pos * p.s_cs;
  if (p.interleaved) {
    const f32x4 c = *reinterpret_cast<const f32x4*>(row + d0 / 2);
    const f32x4 s = *reinterpret_cast<const f32x4*>(row + half + d0 / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1];
      const float ac = a * c[i], bs = b * s[i], bc = b * c[i], as = a * s[i];
      y[2 * i] = ac - bs;
      y[2 * i + 1] = bc + as;
    }
  } else {
    const bool first = d0 < half;
    const int j = first ? d0 : d0 - half;
    float o[8];
    load8<BF16>(base, at + (first ? d0 + half : d0 - half), o);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 c = *reinterpret_cast<const f32x4*>(row + j + 4 * h);
      const f32x4 s = *reinterpret_cast<const f32x4*>(row + half + j + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float yc = y[4 * h + i] * c[i], os = o[4 * h + i] * s[i];
        y[4 * h + i] = first ? yc - os : yc + os;
      }
    }
  }
}

// v / s clamped to +-448; NaN where v is not finite.
__device__ __forceinline__ float scaled(float v, Recip s) {
  const float q = fminf(fmaxf(quot(v, s), -448.0f), 448.0f);
  return fabsf(v) < INFINITY ? q : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ int pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

template <int D, bool BF16>
__global__ __launch_bounds__(APPEND_THREADS) void kv_append_kernel(const KvAppendArgs p) {
  __shared__ float red[APPEND_THREADS / 64];
  constexpr int C = D / 8;  // chunks of eight elements per head
  const int tid = threadIdx.x;

  if ((int64_t)blockIdx.x >= p.kv_blocks) {  // one token of q
    const int64_t t = (int64_t)blockIdx.x - p.kv_blocks;
    const int s = find_seq(p, t);
    if (s < 0) return;
    const int64_t pos = (int64_t)p.start[s] + t - p.cu[s];
    if (pos < 0 || p.start[s] < 0 || (p.rot > 0 && pos >= p.positions)) return;
    for (int c = tid; c < p.Hq * C; c += APPEND_THREADS) {
      const int h = c / C, d0 = c % C * 8;
      float y[8];
      load_rotated<BF16>(p, p.q, t * p.sq_t + h * p.sq_h, d0, pos, y);
      const i32x2 lo = to_bf16x4_bits(f32x4{y[0], y[1], y[2], y[3]}), hi = to_bf16x4_bits(f32x4{y[4], y[5], y[6], y[7]});
      *reinterpret_cast<i32x4*>(p.q_out + t * p.so_t + h * p.so_h + d0) = i32x4{lo[0], lo[1], hi[0], hi[1]};
    }
    return;
  }

  // slot of touched pages -> the sequence and its run of new tokens in one page
  const int h = (int)(blockIdx.x % p.Hkv);
  const bool is_v = (blockIdx.x / p.Hkv) & 1;
  const int64_t slot = blockIdx.x / (2 * p.Hkv);
  int s;
  int64_t first, pos;  // the run's first token and its position
  if (p.by_token) {
    s = find_seq(p, slot);
    if (s < 0) return;
    first = slot;
    pos = (int64_t)p.start[s] + slot - p.cu[s];
    if (slot != p.cu[s] && pos % p.P != 0) return;  // inside another slot's run
  } else {
    // sequence s has the slots cu[s] / P + 2s ... (at least as many as pages it can touch)
    s = 0;
    for (int base = 1; base < p.S; base += APPEND_THREADS) {
      const int j = base + tid;
      s += __syncthreads_count(j < p.S && (int64_t)p.cu[j] / p.P + 2 * (int64_t)j <= slot);
    }
    const int64_t nth = slot - ((int64_t)p.cu[s] / p.P + 2 * (int64_t)s);
    const int64_t begin = p.start[s], page = begin / p.P + nth;
    pos = nth == 0 ? begin : page * p.P;
    first = p.cu[s] + pos - begin;
    if (nth < 0 || first >= p.cu[s + 1]) return;
  }
  if (pos < 0 || p.start[s] < 0 || first < 0) return;
  const int64_t logical = pos / p.P;
  const int lo = (int)(pos % p.P);  // older tokens of the page
  if (logical >= p.max_pages) return;
  const int page = p.table[s * p.s_table + logical];
  if (page < 0 || page >= p.pages) return;
  int64_t last = (int64_t)p.cu[s + 1];
  if (last > p.T) last = p.T;
  int64_t count = last - first;
  if (count > p.P - lo) count = p.P - lo;
  if (p.rot > 0 && count > p.positions - pos) count = p.positions - pos;  // past the table: dropped
  if (count <= 0) return;

  const void* x = is_v ? p.v : p.k;
  const int64_t at0 = first * (is_v ? p.sv_t : p.sk_t) + h * (is_v ? p.sv_h : p.sk_h);
  const int64_t step = is_v ? p.sv_t : p.sk_t;
  uint8_t* rows = (is_v ? p.v_cache + page * p.svc_p + h * p.svc_h : p.k_cache + page * p.skc_p + h * p.skc_h);
  const int64_t row_step = is_v ? p.svc_t : p.skc_t;
  float* scale = is_v ? p.v_scale + page * p.svs_p + h * p.svs_h : p.k_scale + page * p.sks_p + h * p.sks_h;
  const float old = lo > 0 ? *scale : 0.0f;
  const int chunks = (int)count * C;

  float amax = 0.0f;
  for (int c = tid; c < chunks; c += APPEND_THREADS) {
    const int i = c / C, d0 = c % C * 8;
    float y[8];
    if (is_v) load8<BF16>(x, at0 + i * step + d0, y);
    else load_rotated<BF16>(p, x, at0 + i * step, d0, pos + i, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = fabsf(y[e]);
      amax = fmaxf(amax, a < INFINITY ? a : 0.0f);
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
  if ((tid & 63) == 0) red[tid >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < APPEND_THREADS / 64; ++w) amax = fmaxf(amax, red[w]);
  const float sc = fmaxf(block_scale(amax, 1), old);
  const Recip rs = recip_of(sc);
  if (lo > 0 && sc > old) {
    // older codes of the page, four at a time
    const float ratio = __fdiv_rn(old, sc);
    for (int c = tid; c < lo * (D / 4); c += APPEND_THREADS) {
      int* at = reinterpret_cast<int*>(rows + c / (D / 4) * row_step + c % (D / 4) * 4);
      const int w = *at;
      *at = pack4(__builtin_amdgcn_cvt_f32_fp8(w, 0) * ratio, __builtin_amdgcn_cvt_f32_fp8(w, 1) * ratio,
                  __builtin_amdgcn_cvt_f32_fp8(w, 2) * ratio, __builtin_amdgcn_cvt_f32_fp8(w, 3) * ratio);
    }
  }
  for (int c = tid; c < chunks; c += APPEND_THREADS) {
    const int i = c / C, d0 = c % C * 8;
    float y[8];
    if (is_v) load8<BF16>(x, at0 + i * step + d0, y);
    else load_rotated<BF16>(p, x, at0 + i * step, d0, pos + i, y);
    *reinterpret_cast<i32x2*>(rows + (lo + i) * row_step + d0) =
        i32x2{pack4(scaled(y[0], rs), scaled(y[1], rs), scaled(y[2], rs), scaled(y[3], rs)),
              pack4(scaled(y[4], rs), scaled(y[5], rs), scaled(y[6], rs), scaled(y[7], rs))};
  }
  if (tid == 0) *scale = sc;
}

template <int D>
hipError_t launch_append(const KvAppendArgs& p, int64_t grid, hipStream_t stream) {
  if (p.bf16) kv_append_kernel<D, true><<<dim3((unsigned)grid), dim3(APPEND_THREADS), 0, stream>>>(p);
  else kv_append_kernel<D, false><<<dim3((unsigned)grid), dim3(APPEND_THREADS), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

// Workgroups of the launch: 2 * Hkv for each slot of touched pages, and one
// for each token of q.  A token touches one page, and T tokens of S sequences
// at most T / P + 2 S: whichever is fewer.
int64_t kv_append_grid(int64_t T, int64_t S, int64_t P, int64_t Hkv, bool q, int64_t* kv_blocks, int* by_token) {
  const int64_t by_page = T / P + 2 * S;
  *by_token = T <= by_page;
  *kv_blocks = (*by_token ? T : by_page) * 2 * Hkv;
  return *kv_blocks + (q ? T : 0);
}

hipError_t launch_kv_append(KvAppendArgs p, hipStream_t stream) {
  const int64_t grid = kv_append_grid(p.T, p.S, p.P, p.Hkv, p.q != nullptr, &p.kv_blocks, &p.by_token);
  if (p.D == 64) return launch_append<64>(p, grid, stream);
  if (p.D == 128) return launch_append<128>(p, grid, stream);
  return launch_append<256>(p, grid, stream);
}

}  // namespace dgmi
