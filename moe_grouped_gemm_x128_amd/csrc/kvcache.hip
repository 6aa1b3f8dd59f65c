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
// touched page of a head's K or V (a "kind": 2 Hkv of them): it finds the
// maximum of the page's new tokens, which it keeps in registers, then encodes
// them.  A thread works on items of 16 elements that hold both members of
// their pairs.  Where a page gets a few tokens (decode), D / 16 lanes take a
// kind and a workgroup takes several kinds, which share the search for the
// sequence.  The rotation of q rides in the same launch.
//
// What bounds it: with many tokens the copy, 30,636 BF16 tokens of six prompts
// (8 KV heads and 32 heads of q, D = 128) take 146 us for 706 MB, 4.84 TB/s, the
// rate of a large copy; with one token a sequence the chain from the lengths
// over the page table to the page, then to its scale: 256 sequences 6.1 us, one
// 4.7 us, where an empty launch takes about 2.

#include "common.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

constexpr int APPEND_THREADS = 256;

// Tokens of a page that D / 16 lanes take by themselves.  Two serve a single
// token and a short draft; with four the registers of every variant go from 94
// to 109 and 30,636 tokens of six prompts take 154 us for 146.
constexpr int FEW = 2;

struct Seq {
  int s, cu0, cu1, start;
};

// The sequence that holds token (or page slot) `at`, found by all threads
// side by side; false if there is none.  Sequence j owns the tokens cu[j] ..
// cu[j+1]-1, or the page slots cu[j] / P + 2 j .. (as many as pages it can
// touch at least).
template <bool PAGES>
__device__ __forceinline__ bool find_seq(const KvAppendArgs& p, int64_t at, Seq* lds, Seq& q) {
  for (int base = 0; base < p.S; base += APPEND_THREADS) {
    const int j = base + threadIdx.x;
    bool mine = false;
    if (j < p.S) {
      const int c0 = p.cu[j], c1 = p.cu[j + 1], st = p.start[j];
      if constexpr (PAGES)
        mine = at >= (int64_t)(c0 >> p.log_p) + 2 * (int64_t)j && at < (int64_t)(c1 >> p.log_p) + 2 * (int64_t)j + 2;
      else
        mine = at >= c0 && at < c1;
      if (mine) *lds = Seq{j, c0, c1, st};
    }
    if (__syncthreads_or(mine)) {
      q = *lds;
      return true;
    }
  }
  return false;
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

// Item m of a head's D / 16: elements a .. a+7 and b .. b+7, which hold both
// members of their pairs.
struct ItemAt {
  int a, b;
};
__device__ __forceinline__ ItemAt item_at(const KvAppendArgs& p, int m) {
  const bool halves = !p.interleaved && 16 * m < p.rot;
  return halves ? ItemAt{8 * m, 8 * m + p.rot / 2} : ItemAt{16 * m, 16 * m + 8};
}

template <bool BF16>
__device__ __forceinline__ void load_item(const void* base, int64_t row, ItemAt it, float y[16]) {
  load8<BF16>(base, row + it.a, y);
  load8<BF16>(base, row + it.b, y + 8);
}

// Rotation of an item for position pos.  (This file is compiled without
// contraction into FMAs: every product and sum is rounded on its own.)
__device__ __forceinline__ void rotate_item(const KvAppendArgs& p, int m, int64_t pos, float y[16]) {
  if (16 * m >= p.rot) return;  // (rot is 0 without a table)
  const float* row = p.cos_sin + pos * p.s_cs + 8 * m;
  float c[8], s[8];
  load8<false>(row, 0, c);
  load8<false>(row, p.rot / 2, s);
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1];
      const float ac = a * c[i], bs = b * s[i], bc = b * c[i], as = a * s[i];
      y[2 * i] = ac - bs;
      y[2 * i + 1] = bc + as;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = y[i], b = y[8 + i];
      const float ac = a * c[i], bs = b * s[i], bc = b * c[i], as = a * s[i];
      y[i] = ac - bs;
      y[8 + i] = bc + as;
    }
  }
}

__device__ __forceinline__ float item_amax(const float y[16], float amax) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float a = fabsf(y[e]);
    amax = fmaxf(amax, a < INFINITY ? a : 0.0f);
  }
  return amax;
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

__device__ __forceinline__ void store_item(uint8_t* row, ItemAt it, const float y[16], Recip rs) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* v = y + 8 * h;
    *reinterpret_cast<i32x2*>(row + (h ? it.b : it.a)) =
        i32x2{pack4(scaled(v[0], rs), scaled(v[1], rs), scaled(v[2], rs), scaled(v[3], rs)),
              pack4(scaled(v[4], rs), scaled(v[5], rs), scaled(v[6], rs), scaled(v[7], rs))};
  }
}

// The `lo` older tokens of a page re-encoded for a scale that grew, 16 codes
// at a time by `lanes` threads.
template <int D>
__device__ __forceinline__ void re_encode(uint8_t* rows, int64_t step, int lo, float ratio, int lane, int lanes) {
  for (int c = lane; c < lo * (D / 16); c += lanes) {
    i32x4* at = reinterpret_cast<i32x4*>(rows + c / (D / 16) * step + c % (D / 16) * 16);
    i32x4 w = *at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack4(__builtin_amdgcn_cvt_f32_fp8(w[i], 0) * ratio, __builtin_amdgcn_cvt_f32_fp8(w[i], 1) * ratio,
                   __builtin_amdgcn_cvt_f32_fp8(w[i], 2) * ratio, __builtin_amdgcn_cvt_f32_fp8(w[i], 3) * ratio);
    *at = w;
  }
}

// One kind: a head's K or V.
struct Kind {
  const void* x;
  int64_t at, step;      // element of the first token's row, and between tokens
  uint8_t* rows;         // the page's rows of the head
  int64_t row_step;
  float* scale;
  bool is_v;
};
__device__ __forceinline__ Kind kind_of(const KvAppendArgs& p, int kind, int64_t first, int64_t page) {
  const int h = kind >> 1;
  if (kind & 1)
    return Kind{p.v, first * p.sv_t + h * p.sv_h, p.sv_t, p.v_cache + page * p.svc_p + h * p.svc_h, p.svc_t,
                p.v_scale + page * p.svs_p + h * p.svs_h, true};
  return Kind{p.k, first * p.sk_t + h * p.sk_h, p.sk_t, p.k_cache + page * p.skc_p + h * p.skc_h, p.skc_t,
              p.k_scale + page * p.sks_p + h * p.sks_h, false};
}

// IT: items a thread keeps where a whole workgroup takes a kind (P D / 16 / 256).
template <int D, bool BF16, int IT>
__global__ __launch_bounds__(APPEND_THREADS) void kv_append_kernel(const KvAppendArgs p) {
  constexpr int C = D / 16;  // items of a head
  __shared__ float red[APPEND_THREADS / 64];
  __shared__ Seq found;
  const int tid = threadIdx.x;
  const int m = tid % C;     // this thread's item of every head it works on
  const ItemAt it = item_at(p, m);
  Seq q;

  if ((int64_t)blockIdx.x >= p.kv_blocks) {  // some tokens of q
    const int64_t t0 = ((int64_t)blockIdx.x - p.kv_blocks) * p.q_tokens;
    bool any = false;  // (q is the sequence of token t once one has been found)
    for (int i = 0; i < p.q_tokens; ++i) {
      const int64_t t = t0 + i;
      if (t >= p.T) return;
      if (!any || t < q.cu0 || t >= q.cu1) {
        if (i > 0) __syncthreads();  // the last one found has been read
        any = find_seq<false>(p, t, &found, q);
        if (!any) continue;
      }
      const int64_t pos = (int64_t)q.start + t - q.cu0;
      if (q.start < 0 || (p.rot > 0 && pos >= p.positions)) continue;
      for (int h = tid / C; h < p.Hq; h += APPEND_THREADS / C) {
        float y[16];
        load_item<BF16>(p.q, t * p.sq_t + h * p.sq_h, it, y);
        rotate_item(p, m, pos, y);
        uint16_t* to = p.q_out + t * p.so_t + h * p.so_h;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float* v = y + 8 * c;
          const i32x2 lo = to_bf16x4_bits(f32x4{v[0], v[1], v[2], v[3]}), hi = to_bf16x4_bits(f32x4{v[4], v[5], v[6], v[7]});
          *reinterpret_cast<i32x4*>(to + (c ? it.b : it.a)) = i32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      }
    }
    return;
  }

  // slot of touched pages -> the sequence and its run of new tokens in one page
  const int kind0 = (int)(blockIdx.x % p.kind_blocks) * p.kinds;
  const int64_t slot = blockIdx.x / p.kind_blocks;
  int64_t first, pos;  // the run's first token and its position
  if (p.by_token) {
    if (!find_seq<false>(p, slot, &found, q)) return;
    first = slot;
    pos = (int64_t)q.start + slot - q.cu0;
    if (slot != q.cu0 && (pos & (p.P - 1)) != 0) return;  // inside another slot's run
  } else {
    if (!find_seq<true>(p, slot, &found, q)) return;
    const int64_t nth = slot - ((int64_t)(q.cu0 >> p.log_p) + 2 * (int64_t)q.s);
    pos = nth == 0 ? q.start : ((q.start >> p.log_p) + nth) * (int64_t)p.P;
    first = q.cu0 + pos - q.start;
    if (first >= q.cu1) return;
  }
  if (q.start < 0 || first < 0) return;
  const int64_t logical = pos >> p.log_p;
  const int lo = (int)(pos & (p.P - 1));  // older tokens of the page
  if (logical >= p.max_pages) return;
  const int page = p.table[q.s * p.s_table + logical];
  if (page < 0 || page >= p.pages) return;
  int64_t last = q.cu1 < p.T ? q.cu1 : p.T, left = last - first;
  if (left > p.P - lo) left = p.P - lo;
  if (p.rot > 0 && left > p.positions - pos) left = p.positions - pos;  // past the table: dropped
  if (left <= 0) return;
  const int count = (int)left;

  if (count <= FEW) {
    const int kind = kind0 + tid / C;
    if (tid / C >= p.kinds || kind >= 2 * p.Hkv) return;
    const Kind k = kind_of(p, kind, first, page);
    const float old = lo > 0 ? *k.scale : 0.0f;
    float y[FEW][16], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < FEW; ++i)
      if (i < count) load_item<BF16>(k.x, k.at + i * k.step, it, y[i]);
#pragma unroll
    for (int i = 0; i < FEW; ++i)
      if (i < count) {
        if (!k.is_v) rotate_item(p, m, pos + i, y[i]);
        amax = item_amax(y[i], amax);
      }
#pragma unroll
    for (int off = 1; off < C; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    const float sc = fmaxf(block_scale(amax, 1), old);
    const Recip rs = recip_of(sc);
    if (lo > 0 && sc > old) re_encode<D>(k.rows, k.row_step, lo, __fdiv_rn(old, sc), m, C);
#pragma unroll
    for (int i = 0; i < FEW; ++i)
      if (i < count) store_item(k.rows + (lo + i) * k.row_step, it, y[i], rs);
    if (m == 0) *k.scale = sc;  // (after every lane of the kind has read the old one: they run together)
    return;
  }

  for (int kind = kind0; kind < kind0 + p.kinds && kind < 2 * p.Hkv; ++kind) {
    const Kind k = kind_of(p, kind, first, page);
    const float old = lo > 0 ? *k.scale : 0.0f;
    float y[IT][16], amax = 0.0f;
    const int r0 = tid / C;
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int i = r0 + j * (APPEND_THREADS / C);
      if (i < count) load_item<BF16>(k.x, k.at + i * k.step, it, y[j]);
    }
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int i = r0 + j * (APPEND_THREADS / C);
      if (i < count) {
        if (!k.is_v) rotate_item(p, m, pos + i, y[j]);
        amax = item_amax(y[j], amax);
      }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    if (kind > kind0) __syncthreads();  // the last kind's maxima have been read
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < APPEND_THREADS / 64; ++w) amax = fmaxf(amax, red[w]);
    const float sc = fmaxf(block_scale(amax, 1), old);
    const Recip rs = recip_of(sc);
    if (lo > 0 && sc > old) re_encode<D>(k.rows, k.row_step, lo, __fdiv_rn(old, sc), tid, APPEND_THREADS);
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int i = r0 + j * (APPEND_THREADS / C);
      if (i < count) store_item(k.rows + (lo + i) * k.row_step, it, y[j], rs);
    }
    if (tid == 0) *k.scale = sc;
  }
}

template <int D, int IT>
hipError_t launch_append(const KvAppendArgs& p, int64_t grid, hipStream_t stream) {
  if (p.bf16) kv_append_kernel<D, true, IT><<<dim3((unsigned)grid), dim3(APPEND_THREADS), 0, stream>>>(p);
  else kv_append_kernel<D, false, IT><<<dim3((unsigned)grid), dim3(APPEND_THREADS), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

// The launch: a pure function of the sizes.  A token touches one page, and T
// tokens of S sequences at most T / P + 2 S: whichever is fewer is the count of
// page slots.  With a slot per token the pages get few tokens: a workgroup
// takes as many kinds as keep the grid near 1024 (all of them resident at
// once), with a slot per page one.  q goes a token to a workgroup, four where
// there are enough to fill the machine.
KvAppendPlan kv_append_plan(int64_t T, int64_t S, int64_t P, int64_t Hkv, int64_t D, bool q) {
  KvAppendPlan a;
  const int64_t by_page = T / P + 2 * S;
  a.by_token = T <= by_page;
  a.kinds = 1;
  if (a.by_token)
    while (a.kinds < 2 * Hkv && a.kinds < APPEND_THREADS / (D / 16) && T * 2 * Hkv > 1024 * a.kinds) a.kinds *= 2;
  a.kind_blocks = (2 * Hkv + a.kinds - 1) / a.kinds;
  a.kv_blocks = (a.by_token ? T : by_page) * a.kind_blocks;
  a.q_tokens = T >= 4096 ? 4 : 1;
  a.grid = a.kv_blocks + (q ? (T + a.q_tokens - 1) / a.q_tokens : 0);
  return a;
}

hipError_t launch_kv_append(KvAppendArgs p, hipStream_t stream) {
  const KvAppendPlan a = kv_append_plan(p.T, p.S, p.P, p.Hkv, p.D, p.q != nullptr);
  p.kv_blocks = a.kv_blocks;
  p.kind_blocks = (int32_t)a.kind_blocks;
  p.kinds = (int32_t)a.kinds;
  p.q_tokens = (int32_t)a.q_tokens;
  p.by_token = a.by_token;
  p.log_p = __builtin_ctz(p.P);
  const int it = p.P * p.D / 16 / APPEND_THREADS;
#define APPEND_CASE(D_, IT) \
  if (p.D == D_ && (it > 1 ? it : 1) == IT) return launch_append<D_, IT>(p, a.grid, stream);
  APPEND_CASE(64, 1) APPEND_CASE(64, 2)
  APPEND_CASE(128, 1) APPEND_CASE(128, 2) APPEND_CASE(128, 4)
  APPEND_CASE(256, 1) APPEND_CASE(256, 2) APPEND_CASE(256, 4) APPEND_CASE(256, 8)
#undef APPEND_CASE
  return hipErrorInvalidValue;
}

}  // namespace dgmi
