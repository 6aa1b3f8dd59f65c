// Attention of a few query tokens per sequence over a paged FP8 key/value
// cache, gfx950.
//
//   query i (of n) of sequence s stands at position pos = len[s] - n + i and
//   sees the positions max(0, pos - window + 1) .. pos (window 0: all)
//   x_t = scale (q . k_t),  o = sum_t exp(x_t - m) v_t / sum_t exp(x_t - m),
//   lse = m + log sum_t exp(x_t - m); a query that sees nothing gives o = 0,
//   lse = -inf.
//   k_t, v_t = E4M3 code times the scale of (page, head).
//
// The g = Hq / Hkv query heads that share a KV head, times the n queries, are
// the rows of a matrix product over the cache: 16 rows go through the matrix
// cores at once, so every code is read once for all of them.  Both products
// are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that
//   - a lane holds the scores of one row, for four consecutive tokens of a
//     16-token tile, which is where the second product wants its P: nothing
//     passes through shared memory, and the running maximum and sum of a row
//     are scalars of the lane;
//   - the token order inside a product is free as long as P and V agree, so a
//     lane takes tokens 4 (l / 16) + {0..3} of two tiles, reads D / 16
//     consecutive bytes of each, and turns the 8 x D/16 bytes round in its
//     own registers (one byte permute and two conversions per four codes);
//   - the head's elements are free in the first product: a lane reads 16
//     consecutive bytes of every 64 of a token's key, so that a load takes
//     whole 64-byte pieces.
// E4M3 is exact in BF16 and in FP16.  Keys meet the BF16 queries in BF16.
// The weights P are rounded to FP16 (11 bits; rounding them to BF16 would add
// as much error again as the BF16 output has); to keep them in FP16's range
// the scale of V is taken into the exponent: with y_t = x_t log2 e + log2 sv_t,
//   o = sum_t 2^(y_t - M) code_t / sum_t 2^(y_t - M) / sv_t,  M = max y,
// and P is held times 2^14, so that weights down to 2^-28 of the largest are
// normal numbers and those below 2^-39 vanish.  (More bits would cost the matrix
// cores' rate for FP16; against 64 bits the BF16 output is off by 1.658e-3 of
// itself, with FP32 weights by 1.654e-3.)
// Sums, maxima and the output stay in FP32.
//
// Work is cut along the cache by device-side lengths: the 32-token tiles of
// all (sequence, KV head, row tile) units form one line, and each workgroup
// takes an equal share of it, a few units' ends or a piece of one.  A unit that
// lies in one share is finished there; pieces are written to the workspace
// (FP32 sums, maximum, output) and joined by a second kernel in the order of
// the cache, whichever workgroup ran first.
//
// What bounds it: for the 16 rows of a wave a tile costs about 220 vector and
// 80 scalar instructions (D = 128), 0.68 us to a wave alone; four waves on
// each of two workgroups a compute unit keep 64 KiB of codes on their way there
// and reach what HBM gives to reads: 128 sequences of 1 to 8192 tokens (8 KV
// heads, D = 128, 1.09 GB) 193 us, 5.6 TB/s; 4 of 60,000 to 131,071 (4 heads, 410
// MB) 68 us, 6.0 TB/s.  Calls with little to read are bound by what each share
// spends before and after its tiles, 3 and 2 us, the first tile's 2 to 5 us of
// latency, and the join's launch, 4 to 6 us: 32 sequences, window 2048, four
// queries of 8 heads each over 2 KV heads, D = 256 (65 MB): 23 + 4.2 us; one
// sequence of 777 tokens, not cut: 10.0 us.

#include "common.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int CUS = 256;
constexpr int ATTN_WAVES = 4;
constexpr int ATTN_THREADS = 64 * ATTN_WAVES;
// Waves per SIMD that the registers are held to: the output takes D / 4 MT
// registers of a lane, the queries D / 8 MT, a tile's codes D / 4.
constexpr int WAVES_PER_SIMD(int D, int MT) { return D * MT <= 128 ? 3 : 2; }
constexpr int FEW_TILES = 32;
constexpr float P_GAIN = 16384.0f, P_GAIN_LOG2 = 14.0f;  // weights are held times 2^14 in FP16
constexpr float ON_GRID = 192.0f;  // added and taken off: leaves a multiple of 2^-16
constexpr float FAR = 65536.0f;    // of a maximum in base 2: from here on exponents are rounded before the maximum goes off
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

// Four E4M3 codes -> four BF16 values in two words.
__device__ __forceinline__ i32x2 fp8x4_to_bf16(int w) {
  return i32x2{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
}

// Uniform loads of what this kernel never writes, through the scalar path.
typedef const __attribute__((address_space(4))) int32_t* const_i32;
typedef const __attribute__((address_space(4))) float* const_f32;
__device__ __forceinline__ int uniform_load(const int32_t* p) { return *(const_i32)(uintptr_t)p; }
__device__ __forceinline__ float uniform_load(const float* p) { return *(const_f32)(uintptr_t)p; }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A barrier for what passes through shared memory alone: loads and stores of
// global memory go on meanwhile.
__device__ __forceinline__ void local_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The kernel's arguments, to be fetched where they are used.
__device__ __forceinline__ const PagedAttnArgs& arguments() {
  auto p = (const __attribute__((address_space(4))) PagedAttnArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const PagedAttnArgs*)p;
}

// Tiles of 32 positions that the queries of sequence s look at: [begin, end).
// A sequence whose queries see nothing has one tile (of masked positions), so
// that every unit is somebody's work.
struct Span {
  int len, begin, end;
};
__device__ __forceinline__ Span span_of(const PagedAttnArgs& p, int len) {
  const int64_t cap = (int64_t)p.max_pages * p.P;
  if (len > cap) len = (int)cap;
  if (len < 0 || p.pages == 0) len = 0;
  int lo = 0;
  if (p.window > 0) {
    const int64_t first = (int64_t)len - p.n - p.window + 1;
    lo = first > 0 ? (int)first : 0;
  }
  const int begin = lo / 32, end = (len + 31) / 32;
  return Span{len, begin, end > begin ? end : begin + 1};
}

// Inclusive prefix sum over the wave's lanes: within rows of 16 by DPP shifts,
// then the rows' last lanes passed on.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row shift right by 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  const int r0 = __builtin_amdgcn_readlane(v, 15), r1 = __builtin_amdgcn_readlane(v, 31), r2 = __builtin_amdgcn_readlane(v, 47);
  const int row = (threadIdx.x >> 4) & 3;
  return v + (row > 0 ? r0 : 0) + (row > 1 ? r1 : 0) + (row > 2 ? r2 : 0);
}

// Inclusive prefix sum of v over the workgroup; *all gets the total.
__device__ __forceinline__ int line_scan(int v, int* red, int* all) {
  const int wave = threadIdx.x >> 6;
  v = wave_scan(v);
  __syncthreads();  // the last scan's sums have been read
  if ((threadIdx.x & 63) == 63) red[wave] = v;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < ATTN_WAVES; ++w) {
    v += w < wave ? red[w] : 0;
    total += red[w];
  }
  *all = uniform(total);
  return v;
}

__device__ __forceinline__ int padded(int tiles, int pad) { return (tiles + pad - 1) / pad * pad; }

// Places of sequence s on the line of all units' tiles (the line is below
// 2^31): a unit's tiles, rounded up to a multiple of pad.
__device__ __forceinline__ int line_tiles(const PagedAttnArgs& p, int s, int pad, int* len) {
  *len = s < p.S ? p.lens[s] : 0;
  const Span sp = span_of(p, *len);
  return s < p.S ? padded(sp.end - sp.begin, pad) * p.units : 0;
}

// This workgroup's part [at, end) of the line, the sequence in which it begins
// and the places before that one; pad as above.
struct Share {
  int size, pad, at, end, before, s, len;
};

// A share's size: an equal part of all tiles for two workgroups of every
// compute unit, or for one where that is at most FEW_TILES, as a share costs its
// start and the join of its part whatever its size.  Two / one, in us: 8 units
// of up to 256 tiles, D = 256 and 32 rows 21.8 / 19.5; 6 units of up to 940
// tiles, D = 256 25.4 / 22.8; 8 units of 256 tiles, D = 128 13.1 / 14.3.
__device__ __forceinline__ void share_size(const PagedAttnArgs& p, int total, Share& o) {
  const int one = (int)(((uint32_t)total + p.cuts_one - 1) / p.cuts_one);
  int n = (int)(((uint32_t)total + p.cuts - 1) / p.cuts);
  if (one <= FEW_TILES) n = one;
  o.size = uniform((n + p.min_share - 1) & -p.min_share);  // as many tiles for each stream of waves
  o.pad = p.whole ? o.size : 1;  // (whole: no share reaches past its unit)
}
// false: it begins past the line's end.
__device__ __forceinline__ bool share_place(int total, Share& o) {
  const int64_t at = (int64_t)blockIdx.x * o.size;
  if (at >= total) return false;
  o.at = (int)at;
  o.end = at + o.size < total ? o.at + o.size : total;
  return true;
}

// false: nothing for this workgroup.
__device__ __forceinline__ bool line_share(const PagedAttnArgs& p, int* red, int* found, Share& o) {
  int len, total;
  if (p.S <= 64) {  // a lane a sequence, every wave by itself
    const int lane = threadIdx.x & 63;
    int mine = line_tiles(p, lane, 1, &len);
    int upto = wave_scan(mine);
    share_size(p, __builtin_amdgcn_readlane(upto, 63), o);
    if (o.pad > 1) {
      mine = line_tiles(p, lane, o.pad, &len);
      upto = wave_scan(mine);
    }
    if (!share_place(__builtin_amdgcn_readlane(upto, 63), o)) return false;
    o.s = __builtin_ctzll(__ballot(o.at < upto));  // the first one that ends past it
    o.before = __builtin_amdgcn_readlane(upto - mine, o.s);
    o.len = __builtin_amdgcn_readlane(len, o.s);
    return true;
  }
  int mine, upto;
  const auto scan_all = [&](int pad) {  // (mine, upto: of the first ATTN_THREADS sequences)
    mine = line_tiles(p, threadIdx.x, pad, &len);
    upto = line_scan(mine, red, &total);
    for (int base = ATTN_THREADS; base < p.S; base += ATTN_THREADS) {
      int l, all;
      line_scan(line_tiles(p, base + threadIdx.x, pad, &l), red, &all);
      total += all;
    }
  };
  scan_all(1);
  share_size(p, total, o);
  if (o.pad > 1) scan_all(o.pad);
  if (!share_place(total, o)) return false;
  int before = 0;
  for (int base = 0;; base += ATTN_THREADS) {
    if (p.S > ATTN_THREADS) {
      int all;
      mine = line_tiles(p, base + threadIdx.x, o.pad, &len);
      upto = before + line_scan(mine, red, &all);
      before += all;
    }
    if (o.at >= upto - mine && o.at < upto) {
      found[0] = base + threadIdx.x;
      found[1] = upto - mine;
      found[2] = len;
    }
    if (p.S <= ATTN_THREADS || o.at < before) break;
  }
  __syncthreads();
  o.s = uniform(found[0]);
  o.before = uniform(found[1]);
  o.len = uniform(found[2]);
  return true;
}

// A head's place in the caches, for one sequence.
struct Heads {
  const int32_t* table;
  const uint8_t *k, *v;      // of page 0, token 0
  const float *ks, *vs;
  int len;
};

// The pages of a tile's two 16-token halves as the table has them, -1 past
// the end.  P16: a page holds 16 tokens; else the second half's is the first's.
struct Pages {
  int id0, id1;
};
template <bool P16>
__device__ __forceinline__ void find_pages(const PagedAttnArgs& p, const Heads& hd, int t, bool wanted, Pages& x) {
  x.id0 = x.id1 = -1;
  if (wanted && t * 32 < hd.len) x.id0 = uniform_load(hd.table + ((t * 32) >> p.log_p));
  if (P16 && wanted && t * 32 + 16 < hd.len) x.id1 = uniform_load(hd.table + 2 * t + 1);
}

// Half u's page; page 0 is read where it takes no part (ok: it does).
template <bool P16>
__device__ __forceinline__ int page_of(const PagedAttnArgs& p, const Pages& x, int u, bool* ok) {
  const int id = P16 && u == 1 ? x.id1 : x.id0;
  *ok = id >= 0 && id < p.pages;
  return *ok ? id : 0;
}
// One page's place: strides are below 2^32 bytes, a page's tokens within 2^31.
__device__ __forceinline__ uint64_t page_offset(int page, uint32_t stride) { return (uint64_t)(uint32_t)page * stride; }

// Where half u's codes begin.
template <bool P16>
__device__ __forceinline__ const uint8_t* half_at(const PagedAttnArgs& p, const uint8_t* base, uint32_t page_step, uint32_t step,
                                                  int t, const Pages& x, int u) {
  bool ok;
  const uint32_t slot = P16 ? 0 : ((t * 32) & (p.P - 1)) + 16 * u;
  return base + page_offset(page_of<P16>(p, x, u, &ok), page_step) + slot * step;
}

// The scales of a tile's halves as they are stored.  ok: the half takes part --
// its page is there, and where it has a page of its own some row of the wave
// sees into it ([lo, hi]): the scales of a page that no row sees may be anything.
struct Scales {
  int ks[2], vs[2];
  bool ok[2];
};
template <bool P16>
__device__ __forceinline__ void load_scales(const PagedAttnArgs& p, const Heads& hd, const Pages& pages, int t, int lo, int hi,
                                            Scales& x) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (!P16 && u == 1) {
      x.ks[1] = x.ks[0];
      x.vs[1] = x.vs[0];
      x.ok[1] = x.ok[0];
      break;
    }
    const int page = page_of<P16>(p, pages, u, &x.ok[u]);
    x.ks[u] = uniform_load(reinterpret_cast<const int32_t*>(reinterpret_cast<const uint8_t*>(hd.ks) + page_offset(page, p.sks_p)));
    x.vs[u] = uniform_load(reinterpret_cast<const int32_t*>(reinterpret_cast<const uint8_t*>(hd.vs) + page_offset(page, p.svs_p)));
    if (P16) x.ok[u] = x.ok[u] && t * 32 + 16 * u + 15 >= lo && t * 32 + 16 * u <= hi;
  }
}

// A tile's codes in registers.
template <int D>
struct Tile {
  int k[2][D / 16];     // D / 4 bytes of a token in each half, 16 of every 64
  int v[2][4][D / 64];  // D / 16 bytes of four tokens in each half
};

// ONCE: no other wave reads these codes and no cache will hold them until the
// next call, so they are loaded past the caches (non-temporal).
template <bool ONCE, typename T>
__device__ __forceinline__ T load_codes(const uint8_t* at) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const T*>(at));
  else return *reinterpret_cast<const T*>(at);
}

// lane: this lane's offset inside a 16-token half.  (Kept opaque, so that the
// loads take a scalar base and a 32-bit offset.)
template <int D, bool ONCE, bool P16>
__device__ __forceinline__ void load_k(const PagedAttnArgs& p, const Heads& hd, int t, const Pages& pages, uint32_t lane,
                                       Tile<D>& x) {
  asm volatile("" : "+v"(lane));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* kp = half_at<P16>(p, hd.k, p.skc_p, p.skc_t, t, pages, u);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const i32x4 v = load_codes<ONCE, i32x4>(kp + lane + 64 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) x.k[u][4 * j + e] = v[e];
    }
  }
}

template <int D, bool ONCE, bool P16>
__device__ __forceinline__ void load_v(const PagedAttnArgs& p, const Heads& hd, int t, const Pages& pages, uint32_t lane,
                                       Tile<D>& x) {
  constexpr int VB = D / 16;
  uint32_t off[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    off[e] = lane + e * p.svc_t;
    asm volatile("" : "+v"(off[e]));
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* vp = half_at<P16>(p, hd.v, p.svc_p, p.svc_t, t, pages, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* row = vp + off[e];
      if constexpr (VB == 4) {
        x.v[u][e][0] = load_codes<ONCE, int>(row);
      } else if constexpr (VB == 8) {
        const i32x2 v = load_codes<ONCE, i32x2>(row);
        x.v[u][e][0] = v[0];
        x.v[u][e][1] = v[1];
      } else {
        const i32x4 v = load_codes<ONCE, i32x4>(row);
#pragma unroll
        for (int b = 0; b < 4; ++b) x.v[u][e][b] = v[b];
      }
    }
  }
}

// Running state of one wave: rows = lane & 15, each lane a quarter of a row's
// output (elements (lane / 16) * D/4 ...), and its own part of the row's sum.
template <int D>
struct RowState {
  f32x4 o[D / 16];
  float m, l;
};

// The positions that this lane's row of a row tile sees, [see_lo, see_hi].
struct Rows {
  int see_lo, see_hi;
};

// A row's value from its four lanes (l, l + 16, l + 32, l + 48): a swap of two
// copies leaves both values of a pair in every lane.
template <typename F>
__device__ __forceinline__ float quarters(float v, F f) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
  v = f(__int_as_float(r[0]), __int_as_float(r[1]));
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return f(__int_as_float(h[0]), __int_as_float(h[1]));
}

// S^T of a tile: lane = its row, tokens 16 u + 4 g4 + i.
template <int D, int MT>
__device__ __forceinline__ void scores(const Tile<D>& x, const bf16x8 (&q)[MT][D / 32], f32x4 (&sc)[MT][2]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int k = 0; k < MT; ++k) sc[k][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const i32x2 a = fp8x4_to_bf16(x.k[u][2 * j]), b = fp8x4_to_bf16(x.k[u][2 * j + 1]);
      const bf16x8 kf = __builtin_bit_cast(bf16x8, i32x4{a[0], a[1], b[0], b[1]});
#pragma unroll
      for (int k = 0; k < MT; ++k) sc[k][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[k][j], sc[k][u], 0, 0, 0);
    }
  }
}

// The larger one; NaN if one is NaN.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Weights of a tile: the running maxima and sums move on, the outputs so far
// are scaled to the new maxima; pf gets P^T as the second product wants it.
// whole: every row sees all 32 positions.
// The maximum is rounded to a multiple of 2^-16 (of coarser powers past 64): so
// log2 sv + 14 - M is exact, V's scale being a power of two, and a weight's
// exponent takes one rounding, that of the FMA; and the largest weight is 2^14
// nearly enough to stay that in FP16, which matters to rows with few others.
// A maximum past FAR stays as it is, and the exponents are rounded as it was, so
// that the largest is 14 again: from scores of 2^24 on FP32's spacing is 2 and
// more, and exponents rounded in another way could pass FP16's range, or all
// fall below it.
template <int D, int MT, bool P16>
__device__ __forceinline__ void weigh(const f32x4 (&sc)[MT][2], const Scales& x, const Rows (&r)[MT], bool whole, int t,
                                      int g4, float qk, RowState<D> (&st)[MT], f16x8 (&pf)[MT]) {
  float c[2], lsv[2], inv[2];  // (scales count as 1 where a half takes no part)
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float vs = __int_as_float(x.ok[u] ? x.vs[u] : 0x3f800000);
    // (positive: a masked score is -inf, and stays it)
    c[u] = larger(__int_as_float(x.ok[u] ? x.ks[u] : 0x3f800000) * qk, 1.17549435e-38f);
    lsv[u] = __builtin_amdgcn_logf(vs);
    inv[u] = __builtin_amdgcn_rcpf(vs) * (1.0f / P_GAIN);
  }
#pragma unroll
  for (int k = 0; k < MT; ++k) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = sc[k][i / 4][i % 4];
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = t * 32 + 16 * (i / 4) + 4 * g4 + i % 4;
        y[i] = x.ok[i / 4] && at >= r[k].see_lo && at <= r[k].see_hi ? y[i] : -INFINITY;
      }
    }
    float mx = larger(larger(y[0], y[1]), larger(y[2], y[3])), mx1 = larger(larger(y[4], y[5]), larger(y[6], y[7]));
    if (P16) mx = larger(__builtin_fmaf(mx, c[0], lsv[0]), __builtin_fmaf(mx1, c[1], lsv[1]));
    else mx = __builtin_fmaf(larger(mx, mx1), c[0], lsv[0]);
    mx = quarters(mx, larger);
    if (__any(!(mx <= st[k].m))) {  // (seldom, once the largest scores have been seen)
      const float m_new = larger(st[k].m, fabsf(mx) > FAR ? mx : mx + ON_GRID - ON_GRID);
      const float alpha = __builtin_amdgcn_exp2f(st[k].m - (m_new == -INFINITY ? 0.0f : m_new));
      st[k].m = m_new;
      st[k].l *= alpha;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[k].o[i][e] *= alpha;
    }
    const float m_use = st[k].m == -INFINITY ? 0.0f : st[k].m;  // nothing seen so far
    float x2[8];  // exponents
    if (__any(fabsf(m_use) > FAR)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x2[i] = __builtin_fmaf(y[i], c[i / 4], lsv[i / 4]);
        asm volatile("" : "+v"(x2[i]));  // (rounded here)
        x2[i] = (x2[i] - m_use) + P_GAIN_LOG2;
      }
    } else {
      const float d[2] = {lsv[0] + P_GAIN_LOG2 - m_use, lsv[1] + P_GAIN_LOG2 - m_use};
#pragma unroll
      for (int i = 0; i < 8; ++i) x2[i] = __builtin_fmaf(y[i], c[i / 4], d[i / 4]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = __builtin_amdgcn_exp2f(x2[i]);
      st[k].l = __builtin_fmaf(w, inv[i / 4], st[k].l);
      pf[k][i] = (_Float16)w;
    }
  }
}

// Elements 2b and 2b + 1 of a lane's eight tokens, in FP16.
template <int D>
__device__ __forceinline__ void turn_values(const Tile<D>& x, int b, f16x8& v0, f16x8& v1) {
  f16x2 lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // bytes (token 2j, token 2j + 1) of element 2b, then of element 2b + 1
    const int pair = __builtin_amdgcn_perm(x.v[j / 2][2 * j % 4 + 1][b / 2], x.v[j / 2][2 * j % 4][b / 2],
                                           b % 2 == 0 ? 0x05010400u : 0x07030602u);
    lo[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pair, 1.0f, false);
    hi[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pair, 1.0f, true);
  }
  v0 = f16x8{lo[0][0], lo[0][1], lo[1][0], lo[1][1], lo[2][0], lo[2][1], lo[3][0], lo[3][1]};
  v1 = f16x8{hi[0][0], hi[0][1], hi[1][0], hi[1][1], hi[2][0], hi[2][1], hi[3][0], hi[3][1]};
}

// O^T += V^T P^T.
template <int D, int MT>
__device__ __forceinline__ void add_values(const Tile<D>& x, const f16x8 (&pf)[MT], RowState<D> (&st)[MT]) {
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    f16x8 v0, v1;
    turn_values<D>(x, b, v0, v1);
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      st[k].o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[k], st[k].o[2 * b], 0, 0, 0);
      st[k].o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[k], st[k].o[2 * b + 1], 0, 0, 0);
    }
  }
}

// Clears the values of positions outside [lo, hi] and of absent pages: their
// codes may be NaN, and a weight of 0 would not hide that.
template <int D>
__device__ __forceinline__ void clear_values(const Scales& place, int t, int g4, int lo, int hi, Tile<D>& x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = t * 32 + 16 * (i / 4) + 4 * g4 + i % 4;
    const bool seen = place.ok[i / 4] && at >= lo && at <= hi;
#pragma unroll
    for (int b = 0; b < D / 64; ++b) x.v[i / 4][i % 4][b] = seen ? x.v[i / 4][i % 4][b] : 0;
  }
}

// Rows of a tile that do not see the same positions, and a NaN code among the
// values: it has to reach the rows that see it and no others, though a
// weight of 0 times NaN is NaN.  The NaN codes are cleared, and a product of
// their places with what each row sees says which outputs they make NaN.
template <int D, int MT>
__device__ __forceinline__ void take_out_nans(const Scales& place, const Rows (&r)[MT], int t, int g4, Tile<D>& x,
                                              RowState<D> (&st)[MT]) {
  // code 1 (a positive value) where there is a NaN
  const auto nans = [](int w) { return (int)(((((uint32_t)w & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u); };
  int hit = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int b = 0; b < D / 64; ++b) hit |= nans(x.v[i / 4][i % 4][b]);
  if (!__any(hit != 0)) return;
  f16x8 sees[MT];
#pragma unroll
  for (int k = 0; k < MT; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = t * 32 + 16 * (i / 4) + 4 * g4 + i % 4;
      sees[k][i] = (_Float16)(place.ok[i / 4] && at >= r[k].see_lo && at <= r[k].see_hi ? 1.0f : 0.0f);
    }
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    Tile<64> places;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int& w = x.v[i / 4][i % 4][b / 2];
      const int n = nans(w) & (b % 2 == 0 ? 0x0000ffff : (int)0xffff0000);  // elements 2 b and 2 b + 1
      places.v[i / 4][i % 4][0] = n;
      w &= (int)~((uint32_t)n * 0xffu);
    }
    f16x8 v0, v1;
    turn_values<64>(places, b % 2, v0, v1);
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
      const f32x4 c0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, sees[k], zero, 0, 0, 0);
      const f32x4 c1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, sees[k], zero, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st[k].o[2 * b][e] = c0[e] > 0.0f ? __uint_as_float(0x7fc00000u) : st[k].o[2 * b][e];
        st[k].o[2 * b + 1][e] = c1[e] > 0.0f ? __uint_as_float(0x7fc00000u) : st[k].o[2 * b + 1][e];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// A part's place in the workspace: the rows' D sums, then their maxima and sums.
template <int D>
__device__ __forceinline__ float* part_at(const PagedAttnArgs& p, int64_t slot) {
  return p.workspace + slot * (int64_t)(p.rt * 16 * (D + 2));
}
// Which shares a unit was cut into, {first, last}: behind the parts.
__device__ __forceinline__ int32_t* unit_parts(const PagedAttnArgs& p, int64_t unit) {
  return reinterpret_cast<int32_t*>(p.workspace + 2 * (int64_t)p.shares * (p.rt * 16 * (p.D + 2))) + 2 * unit;
}

template <int D>
__device__ __forceinline__ void store_row(const PagedAttnArgs& p, int s, int h, int row, int c4, f32x4 o, float m, float l) {
  const float inv_l = l != 0.0f ? __fdiv_rn(1.0f / P_GAIN, l) : 0.0f;  // (NaN stays NaN)
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = l != 0.0f ? o[e] * inv_l : 0.0f;
  const int qi = row / p.group, qh = h * p.group + row % p.group;
  *reinterpret_cast<i32x2*>(p.out + s * p.so_s + (int64_t)qi * p.so_n + (int64_t)qh * p.so_h + c4) = to_bf16x4_bits(o);
  if (c4 == 0 && p.lse != nullptr)
    // log2 l = exponent + log2 of the mantissa: M plus the exponent is small
    // and exact, the scales of V cancel in it
    p.lse[s * p.sl_s + (int64_t)qi * p.sl_n + (int64_t)qh * p.sl_h] =
        l != 0.0f ? (m + (float)__builtin_amdgcn_frexp_expf(l) + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(l))) * LN2
                  : -INFINITY;
}

// MT: row tiles of a wave: the codes are converted once for up to 16 MT rows.
// A unit with more rows has them spread over wr waves side by side (the second
// and later ones find the codes in the caches); the ATTN_WAVES / wr streams of
// waves take the tiles in turn.
template <int D, int MT, bool SPLIT, bool ONCE, bool P16>
__global__ __launch_bounds__(ATTN_THREADS, WAVES_PER_SIMD(D, MT)) void paged_attention_kernel(const PagedAttnArgs p) {
  constexpr int KB = D / 4;    // bytes of a key per lane
  constexpr int VB = D / 16;   // bytes of a value per lane, and output tiles
  __shared__ float so[ATTN_WAVES][16][D + 4];  // a row tile's sums of every wave
  __shared__ float sm[MT][ATTN_WAVES][16], sl[MT][ATTN_WAVES][16];
  __shared__ float row_m[ATTN_WAVES][16], row_l[ATTN_WAVES][16];
  __shared__ int red[ATTN_WAVES], found[3];
  // (one argument of every 64-byte line, so that the lines come in together:
  // 0.3 to 0.5 us of a short call)
  asm volatile("" ::"s"(p.q), "s"(p.out), "s"(p.sl_s), "s"(p.skc_p), "s"(p.v_scale), "s"(p.lens), "s"(p.workspace), "s"(p.log_p));
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t k_lane = (uint32_t)(r16 * p.skc_t + g4 * 16);
  const uint32_t v_lane = (uint32_t)(4 * g4 * p.svc_t + r16 * VB);
  const float qk = fabsf(p.scale) * LOG2E;  // (its sign goes into the queries)
  const int streams = uniform(ATTN_WAVES / p.wr), stream = uniform(wave / p.wr), wgroup = wave - stream * p.wr;

  Share line = {0, 1, 0, 1, 0, 0, 0};
  if (SPLIT) {
    if (!line_share(p, red, found, line)) return;
  } else {
    line.s = uniform(blockIdx.x / p.units);
    line.len = uniform_load(p.lens + line.s);
  }

  while (line.at < line.end) {
    const int s = line.s;
    const Span sp = span_of(p, line.len);
    const int nt = sp.end - sp.begin;
    const int places = SPLIT ? padded(nt, line.pad) : nt;
    if (SPLIT && line.at - line.before >= places * p.units) {  // next sequence
      line.before += places * p.units;
      ++line.s;
      line.len = uniform_load(p.lens + line.s);
      continue;
    }
    const int rel = line.at - line.before;
    const int unit = uniform(SPLIT ? rel / places : (int)(blockIdx.x - s * p.units));
    const int t0 = SPLIT ? rel - unit * places : 0;
    const int t1 = SPLIT && line.end - line.at < nt - t0 ? t0 + line.end - line.at : nt;
    const int h = uniform(unit / p.groups), row0 = (unit - h * p.groups) * p.wr * MT * 16;
    const int len = sp.len;

    // query positions of the wave's rows, and what they see together and each
    const int wrow0 = row0 + wgroup * MT * 16;
    const int qi_first = uniform(wrow0 / p.group);
    const int qi_last = uniform((wrow0 + 16 * MT < p.rows ? wrow0 + 16 * MT - 1 : p.rows - 1) / p.group);
    const int hi_all = len - p.n + qi_first, hi_any = len - p.n + qi_last;
    const int lo_any = p.window > 0 && hi_all >= p.window ? hi_all - p.window + 1 : 0;
    const int lo_all = p.window > 0 && hi_any >= p.window ? hi_any - p.window + 1 : 0;
    Rows r[MT];
    bf16x8 q[MT][D / 32];  // Q^T fragments: step j holds elements 64 (j / 2) + 16 g4 + 8 (j % 2) ...
    RowState<D> st[MT];
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      const int row = wrow0 + 16 * k + r16;
      const bool row_ok = row < p.rows;
      const int qi = row_ok ? row / p.group : 0, qh = h * p.group + (row_ok ? row - qi * p.group : 0);
      const int qpos = len - p.n + qi;
      r[k].see_hi = row_ok ? qpos : -1;
      r[k].see_lo = p.window > 0 && qpos >= p.window ? qpos - p.window + 1 : 0;
      const uint16_t* from = p.q + s * p.sq_s + (int64_t)qi * p.sq_n + (int64_t)qh * p.sq_h + g4 * 16;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        i32x4 v = {0, 0, 0, 0};
        if (row_ok) v = *reinterpret_cast<const i32x4*>(from + 64 * (j / 2) + 8 * (j % 2));
        q[k][j] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int i = 0; i < VB; ++i) st[k].o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      st[k].m = -INFINITY;
      st[k].l = 0.0f;
    }

    // the piece's tiles that some row of the wave sees, one stream each in turn
    int ta = sp.begin + t0, tb = sp.begin + t1;
    const int t_last = hi_any < 0 ? -1 : hi_any / 32;
    if (ta < lo_any / 32) ta = lo_any / 32;
    if (tb > t_last + 1) tb = t_last + 1;  // (none where the queries see nothing: there may be no page to read)
    if (wrow0 >= p.rows) tb = ta;
    const Heads hd = {p.table + s * p.s_table, p.k_cache + h * p.skc_h, p.v_cache + h * p.svc_h,
                      p.k_scale + h * p.sks_h, p.v_scale + h * p.svs_h, len};
    int t = uniform(ta + stream);
    tb = uniform(tb);
    // Pages are looked up two tiles ahead, keys loaded one tile ahead -- into
    // the registers that the present tile's have just left -- and values
    // while the scores are formed.
    Pages now, next, ahead;
    Tile<D> x;
    if (t < tb) {
      find_pages<P16>(p, hd, t, true, now);
      find_pages<P16>(p, hd, t + streams, t + streams < tb, next);
      load_k<D, ONCE, P16>(p, hd, t, now, k_lane, x);
    }
    if (p.scale < 0.0f) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          q[k][j] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(i32x4, q[k][j]) ^ (int)0x80008000);
    }
    while (t < tb) {
      Scales scl;
      load_scales<P16>(p, hd, now, t, lo_any, hi_any, scl);
      find_pages<P16>(p, hd, t + 2 * streams, t + 2 * streams < tb, ahead);
      load_v<D, ONCE, P16>(p, hd, t, now, v_lane, x);
      f32x4 sc[MT][2];
      scores<D, MT>(x, q, sc);
      __builtin_amdgcn_sched_barrier(0);
      if (t + streams < tb) load_k<D, ONCE, P16>(p, hd, t + streams, next, k_lane, x);
      __builtin_amdgcn_sched_barrier(0);
      const bool whole = t * 32 >= lo_all && t * 32 + 31 <= hi_all && scl.ok[0] && scl.ok[1];
      f16x8 pf[MT];
      weigh<D, MT, P16>(sc, scl, r, whole, t, g4, qk, st, pf);
      if (!whole) {
        clear_values<D>(scl, t, g4, lo_any, hi_any, x);
        if (qi_first != qi_last) take_out_nans<D, MT>(scl, r, t, g4, x, st);
      }
      add_values<D, MT>(x, pf, st);
      now = next;
      next = ahead;
      t += streams;
    }

    // (a cut kernel fetches the arguments of this part again: kept over the tiles
    // they would be spilled, 0.5 us of a call)
    const PagedAttnArgs& pe = SPLIT ? arguments() : p;
    // join the waves: each scales its output to the common maximum, then every
    // thread sums four columns of a row
    if (SPLIT) local_barrier();  // the last piece's join has been read
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      st[k].l = quarters(st[k].l, [](float a, float b) { return a + b; });
      if (g4 == 0) {
        sm[k][wave][r16] = st[k].m;
        sl[k][wave][r16] = st[k].l;
      }
    }
    local_barrier();
    const bool piece = t0 > 0 || t1 < nt;
    float* part = piece ? part_at<D>(pe, 2 * (int64_t)blockIdx.x + (t0 == 0)) : nullptr;
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      if (row0 + 16 * k >= pe.rows) break;
      float m = -INFINITY, l = 0.0f;
      for (int w = wgroup; w < ATTN_WAVES; w += pe.wr) m = fmaxf(m, sm[k][w][r16]);
      // (without a maximum the sums are 0, or NaN where every score is NaN)
      for (int w = wgroup; w < ATTN_WAVES; w += pe.wr)
        l += sl[k][w][r16] * (sm[k][w][r16] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(sm[k][w][r16] - m));
      const float f = st[k].m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st[k].m - m);
      if (k > 0) local_barrier();  // the last row tile's sums have been read
      // element (i, e) of the lane is output element g4 * KB + e * VB + i
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < VB; i += 4)
          *reinterpret_cast<f32x4*>(&so[wave][r16][g4 * KB + e * VB + i]) =
              f32x4{st[k].o[i][e] * f, st[k].o[i + 1][e] * f, st[k].o[i + 2][e] * f, st[k].o[i + 3][e] * f};
      if (stream == 0 && g4 == 0) {
        row_m[wgroup][r16] = m;
        row_l[wgroup][r16] = l;
      }
      local_barrier();
      constexpr int TAKE = D / 64;  // of the row tile's D / 4 x 16 quadruples
      f32x4 sum[TAKE];
      for (int g = 0; g < pe.wr; ++g) {
#pragma unroll
        for (int i = 0; i < TAKE; ++i) {
          const int j = threadIdx.x + i * ATTN_THREADS, c = j % (D / 4) * 4, rw = j / (D / 4);
          sum[i] = *reinterpret_cast<const f32x4*>(&so[g][rw][c]);
        }
        for (int w = g + pe.wr; w < ATTN_WAVES; w += pe.wr)
#pragma unroll
          for (int i = 0; i < TAKE; ++i) {
            const int j = threadIdx.x + i * ATTN_THREADS, c = j % (D / 4) * 4, rw = j / (D / 4);
            const f32x4 v = *reinterpret_cast<const f32x4*>(&so[w][rw][c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[i][e] += v[e];
          }
#pragma unroll
        for (int i = 0; i < TAKE; ++i) {
          const int j = threadIdx.x + i * ATTN_THREADS, c = j % (D / 4) * 4, rw = j / (D / 4), rr = (g * MT + k) * 16 + rw;
          if (row0 + rr >= pe.rows) continue;
          if (SPLIT && piece) {
            *reinterpret_cast<f32x4*>(part + rr * D + c) = sum[i];
            if (c == 0) {
              part[pe.rt * 16 * D + rr] = row_m[g][rw];
              part[pe.rt * 16 * (D + 1) + rr] = row_l[g][rw];
            }
          } else {
            store_row<D>(pe, s, h, row0 + rr, c, sum[i], row_m[g][rw], row_l[g][rw]);
          }
        }
      }
    }
    if (!SPLIT) return;
    if (t0 == 0 && threadIdx.x == 0) {
      int32_t* parts = unit_parts(pe, (int64_t)s * pe.units + unit);
      parts[0] = blockIdx.x;
      parts[1] = (line.at + nt - 1) / line.size;
    }
    if (line.pad > 1) return;
    line.at += t1 - t0;
  }
}

// Join of the units that were cut: a workgroup takes `rps` rows (a power of
// two) of a unit; its threads are D / 4 column quadruples x rps rows x groups
// that walk the parts in turn, each with a running maximum, and are joined in
// order, so that the result does not depend on anything but the lengths.
template <int D>
__global__ __launch_bounds__(ATTN_THREADS) void paged_attention_join_kernel(const PagedAttnArgs p) {
  constexpr int C = D / 4;
  __shared__ f32x4 so[ATTN_THREADS];
  __shared__ float sm[ATTN_THREADS / C], sl[ATTN_THREADS / C];
  const int unit_rows = p.rt * 16, slices = unit_rows / p.rps;
  const int64_t u = blockIdx.x / slices;
  const int32_t* parts = unit_parts(p, u);
  const int w0 = uniform_load(parts), w1 = uniform_load(parts + 1);
  if (w0 == w1) return;
  const int r0 = blockIdx.x % slices * p.rps;
  const int s = (int)(u / p.units), unit = (int)(u % p.units);
  const int h = unit / p.groups, row0 = (unit - h * p.groups) * unit_rows + r0;
  if (row0 >= p.rows) return;
  const int n = w1 - w0 + 1;
  const int64_t part_size = unit_rows * (D + 2);
  const float* base = part_at<D>(p, 2 * (int64_t)w0);  // part i at 2 i, the first one at 1

  const int c = threadIdx.x % C, r = threadIdx.x / C % p.rps, g = threadIdx.x / C / p.rps;
  const int groups = ATTN_THREADS / C / p.rps;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  // (a part without a maximum has sums of 0, or of NaN where every score is NaN)
  auto add = [&](f32x4 v, float pm, float pl) {
    const float top = fmaxf(m, pm);
    const float f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - top);
    const float e = pm == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(pm - top);
    m = top;
    l = __builtin_fmaf(pl, e, l * f);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[i], e, o[i] * f);
  };
#pragma unroll 4
  for (int i = g; i < n; i += groups) {
    const float* part = base + (i == 0 ? 1 : 2 * (int64_t)i) * part_size;
    const float pm = part[unit_rows * D + r0 + r], pl = part[unit_rows * (D + 1) + r0 + r];
    add(*reinterpret_cast<const f32x4*>(part + (r0 + r) * D + 4 * c), pm, pl);
  }
  if (groups > 1) {
    so[threadIdx.x] = o;
    if (c == 0) {
      sm[g * p.rps + r] = m;
      sl[g * p.rps + r] = l;
    }
    __syncthreads();
    if (g > 0) return;
    for (int k = 1; k < groups; ++k)
      add(so[threadIdx.x + k * C * p.rps], sm[k * p.rps + r], sl[k * p.rps + r]);
  }
  if (row0 + r < p.rows) store_row<D>(p, s, h, row0 + r, 4 * c, o, m, l);
}

// What is launched: a pure function of the sizes.
struct AttnPlan {
  int mt, wr, rt;       // row tiles of a wave, waves side by side, row tiles of a unit
  int units;            // units (KV head, group of row tiles) per sequence
  bool split;
  int64_t shares;       // workgroups of the first kernel when split
  bool whole;           // a share is of one unit
  int min_share;        // tiles of a share: a multiple of this power of two
  int rps;              // rows per workgroup of the join
};

AttnPlan attn_plan(int64_t S, int64_t Hkv, int64_t row_tiles, int64_t D, int64_t cap) {
  AttnPlan a;
  // two row tiles a wave where its registers (output and queries: D MT 3 / 8
  // a lane) leave room for two waves a SIMD
  a.mt = row_tiles >= 2 && D <= 128 ? 2 : 1;
  const int64_t groups = (row_tiles + a.mt - 1) / a.mt;
  a.wr = groups >= 3 ? 4 : groups == 2 ? 2 : 1;
  a.rt = a.mt * a.wr;
  a.units = (int)(Hkv * ((row_tiles + a.rt - 1) / a.rt));
  const int64_t cap_tiles = (cap + 31) / 32, units = S * a.units;
  // Short caches are not cut: the cut costs the shares' search, the parts and the
  // join's launch, 3 to 10 us.  How short depends on what a unit's streams of
  // waves do in that time, and the more units there are to fill the machine, the
  // longer.  Not cut / cut, in us (units, cache capacity; lengths from half of it up):
  //   D = 128, four streams: 8 units, 1024 tokens 9.8 / 10.6, 2048 15.2 / 10.7;
  //     128 units, 2048 18.9 / 18.9, 4096 32.1 / 25.7; 512 units, 2048 41 / 48,
  //     4096 76 / 79, 8192 148 / 142; 1024 units of 1 to 8192 tokens 279 / 203
  //   D = 128, two streams (64 rows): 16 units, 256 tokens 11.6 / 14.5, 512 15.4 /
  //     15.1, 1024 22.5 / 16.8; 128 units, 1024 24.1 / 28.7, 2048 38.1 / 30.8
  //   D = 256, two streams (32 rows): 16 units, 512 tokens 16.3 / 14.0, 1024 24.6 /
  //     16.0; 64 units, 512 16.9 / 17.0, 1024 26.0 / 19.8; 256 units, 2048 57.6 / 69
  //   D = 256, four streams: 16 units, 512 tokens 9.8 / 12.4, 1024 14.1 / 11.7; 128
  //     units, 1024 16.0 / 20.8, 2048 25.4 / 28.2 (here the rule cuts a little early)
  const int64_t streams = ATTN_WAVES / a.wr;
  const int64_t direct = streams * (D > 128 ? 4 : 8) + units / 4;
  a.split = cap_tiles > (direct < 128 ? direct : 128);
  a.min_share = (int)streams;  // a tile for each
  // Shares: two workgroups a compute unit, resident at once, so that all end
  // together (its registers would hold a third at D <= 128).  256 / 512 / 768 /
  // 1024 shares, in us, at D = 128: 128 sequences up to 8192 long, 8 heads 226 /
  // 207 / 211 / 225; 4 sequences up to 131071 long, 4 heads 83 / 79 / 80 / 87;
  // few tiles (2 sequences up to 16384 long, 4 heads, 64 rows) 24 / 25.5 / 25.4 / 32.
  int64_t most = 2 * CUS;
  // (and the parts of one call within 40 MiB)
  const int64_t fit = (int64_t(10) << 20) / (2 * a.rt * 16 * (D + 2));
  if (most > fit) most = fit;
  const int64_t want = (units * cap_tiles + a.min_share - 1) / a.min_share;
  a.shares = want < most ? want : most;
  // Few units have each its own count of shares, the last one what is left: the
  // tiles are divided by (shares - units), and the roundings up need no more
  // than the rest.  Else shares that begin in one unit and end in another take
  // half as long again as the others, most of it waiting for a second first tile.
  a.whole = 4 * units <= a.shares && units * cap_tiles < (int64_t(1) << 30);
  // few units: a row to a workgroup; many: as many rows as its threads hold
  a.rps = (int)(ATTN_THREADS / (D / 4));
  if (a.rps > 16) a.rps = 16;
  while (a.rps > 1 && units * (16 * a.rt / a.rps) < 1024) a.rps /= 2;
  return a;
}

// Workgroups of the join.
int64_t join_grid(const AttnPlan& a, int64_t S) { return S * a.units * (a.rt * 16 / a.rps); }

template <int D, int MT, bool ONCE, bool P16>
hipError_t launch(const PagedAttnArgs& p, const AttnPlan& a, hipStream_t stream) {
  if (!a.split) {
    paged_attention_kernel<D, MT, false, ONCE, P16>
        <<<dim3((unsigned)((int64_t)p.S * p.units)), dim3(ATTN_THREADS), 0, stream>>>(p);
    return hipGetLastError();
  }
  paged_attention_kernel<D, MT, true, ONCE, P16><<<dim3((unsigned)p.shares), dim3(ATTN_THREADS), 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  paged_attention_join_kernel<D><<<dim3((unsigned)join_grid(a, p.S)), dim3(ATTN_THREADS), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

int64_t paged_attention_workspace(int64_t S, int64_t n, int64_t Hq, int64_t Hkv, int64_t D, int64_t cap) {
  const AttnPlan a = attn_plan(S, Hkv, (n * (Hq / Hkv) + 15) / 16, D, cap);
  return a.split ? (2 * a.shares * (a.rt * 16 * (D + 2)) + 2 * S * a.units) * 4 : 0;
}

int64_t paged_attention_grid(int64_t S, int64_t Hkv, int64_t row_tiles, int64_t D, int64_t cap) {
  const AttnPlan a = attn_plan(S, Hkv, row_tiles, D, cap);
  return a.split ? join_grid(a, S) : S * a.units;
}

hipError_t launch_paged_attention(PagedAttnArgs p, hipStream_t stream) {
  // what a sequence can hold or, of a window, its queries can see (its first
  // tile may begin up to 31 positions before that); the plan for it needs no
  // more workspace than the whole capacity's
  int64_t seen = (int64_t)p.max_pages * p.P;
  if (p.window > 0 && seen > (int64_t)p.window + p.n + 31) seen = (int64_t)p.window + p.n + 31;
  const AttnPlan a = attn_plan(p.S, p.Hkv, p.row_tiles, p.D, seen);
  p.rt = a.rt;
  p.wr = a.wr;
  p.units = a.units;
  p.groups = a.units / p.Hkv;
  p.shares = (int32_t)a.shares;
  p.min_share = a.min_share;
  p.whole = a.whole;
  const int64_t ends = a.whole ? (int64_t)p.S * a.units : 0;
  p.cuts = (int32_t)(a.shares - ends);
  p.cuts_one = (int32_t)((a.shares < CUS ? a.shares : CUS) - ends);
  p.rps = a.rps;
  p.log_p = __builtin_ctz(p.P);
  // Past the caches where no waves share codes and what the sequences can hold
  // or see is more than the 256 MiB that the last-level cache keeps from call
  // to call.  With / without, at D = 128: 128 sequences up
  // to 8192 long (2 GiB at most) 198 / 218 us, 4 up to 131071 long 71 / 81 us, 64
  // of 1024 to 2048 39.7 / 43.4 us, of 512 to 1024 (128 MiB) 22.7 / 20.8 us; with
  // codes shared by two waves 44 / 33 us.
  const bool once = a.rt == a.mt && p.groups == 1 && 2 * (int64_t)p.S * p.Hkv * seen * p.D >= (int64_t(256) << 20);
#define ATTN_CASE(D_, MT)                              \
  if (p.D == D_ && a.mt == MT)                         \
    return once ? p.P == 16 ? launch<D_, MT, true, true>(p, a, stream) : launch<D_, MT, true, false>(p, a, stream) \
                : p.P == 16 ? launch<D_, MT, false, true>(p, a, stream) : launch<D_, MT, false, false>(p, a, stream);
  ATTN_CASE(64, 1) ATTN_CASE(64, 2)
  ATTN_CASE(128, 1) ATTN_CASE(128, 2)
  ATTN_CASE(256, 1)
#undef ATTN_CASE
  return hipErrorInvalidValue;
}

}  // namespace dgmi
