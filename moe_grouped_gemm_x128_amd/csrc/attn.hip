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
//   - the head's elements are free in the first product: a lane reads D / 4
//     consecutive bytes of a token's key.
// E4M3 is exact in BF16 and in FP16.  Keys meet the BF16 queries in BF16.
// The weights P are rounded to FP16 (11 bits; rounding them to BF16 would add
// as much error again as the BF16 output has); to keep them in FP16's range
// the scale of V is taken into the exponent: with y_t = x_t log2 e + log2 sv,
//   o = sum_t 2^(y_t - M) code_t / sum_t 2^(y_t - M) / sv,  M = max y,
// shifted by 2^14, so that weights down to 2^-28 of the largest are normal.
// Sums, maxima and the output stay in FP32.
//
// Work is cut along the cache by device-side lengths: the 32-token tiles of
// all (sequence, KV head, row tile) units form one line, and each workgroup
// takes an equal share of it, a few units' ends or a piece of one.  A unit that
// lies in one share is finished there; pieces are written to the workspace
// (FP32 sums, maximum, output) and joined by a second kernel in the order of
// the cache, whichever workgroup ran first.

#include "common.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int ATTN_WAVES = 4;
constexpr int ATTN_THREADS = 64 * ATTN_WAVES;
constexpr float P_SHIFT = 14.0f;  // weights are held times 2^14
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

// Tiles of sequence s on the line of all units' tiles.
__device__ __forceinline__ int64_t line_tiles(const PagedAttnArgs& p, int s) {
  if (s >= p.S) return 0;
  const Span sp = span_of(p, p.lens[s]);
  return (int64_t)(sp.end - sp.begin) * p.units;
}

// Inclusive prefix sum of v over the workgroup; *all gets the total.
__device__ __forceinline__ int64_t line_scan(int64_t v, int64_t* red, int64_t* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t up = __shfl_up(v, off, 64);
    if (lane >= off) v += up;
  }
  __syncthreads();  // the last scan's sums have been read
  if (lane == 63) red[wave] = v;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < ATTN_WAVES; ++w) {
    v += w < wave ? red[w] : 0;
    total += red[w];
  }
  *all = total;
  return v;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v & 0xffffffff)) | ((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32));
}

// This workgroup's share [*at, *end) of the line (false: nothing), the
// sequence in which it begins and the tiles before that one.
__device__ __forceinline__ bool line_share(const PagedAttnArgs& p, int64_t* red, int64_t* found, int64_t* share,
                                           int64_t* at, int64_t* end, int* s_out, int64_t* before_out) {
  int64_t mine = line_tiles(p, threadIdx.x), total;
  int64_t upto = line_scan(mine, red, &total);
  for (int base = ATTN_THREADS; base < p.S; base += ATTN_THREADS) {  // (more sequences than threads)
    int64_t all;
    line_scan(line_tiles(p, base + threadIdx.x), red, &all);
    total += all;
  }
  total = uniform64(total);
  int64_t n = (total + p.shares - 1) / p.shares;
  if (n < p.min_share) n = p.min_share;
  *share = n;
  *at = blockIdx.x * n;
  *end = *at + n < total ? *at + n : total;
  if (*at >= *end) return false;
  int64_t before = 0;
  for (int base = 0;; base += ATTN_THREADS) {
    if (base > 0) {
      int64_t all;
      mine = line_tiles(p, base + threadIdx.x);
      upto = before + line_scan(mine, red, &all);
      before += all;
    } else if (p.S > ATTN_THREADS) {
      int64_t all;
      upto = line_scan(mine, red, &all);
      before = all;
    }
    if (*at >= upto - mine && *at < upto) {
      found[0] = base + (int)threadIdx.x;
      found[1] = upto - mine;
    }
    if (p.S <= ATTN_THREADS || *at < before) break;
  }
  __syncthreads();
  *s_out = uniform((int)found[0]);
  *before_out = uniform64(found[1]);
  return true;
}

// A head's place in the caches, for one sequence.
struct Heads {
  const int32_t* table;
  const uint8_t *k, *v;      // of page 0, token 0
  const float *ks, *vs;
  int len;
};

// Where a tile's two 16-token halves lie, and their scales: one page each.
struct TileRef {
  int page[2];  // 0 where the half takes no part
  float ks[2], vs[2];
  bool ok[2];
};

__device__ __forceinline__ void find_tile(const PagedAttnArgs& p, const Heads& hd, int t, bool wanted, TileRef& x) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int at = t * 32 + 16 * u;
    int page = -1;
    if (wanted && at < hd.len) page = uniform_load(hd.table + (at >> p.log_p));
    x.ok[u] = page >= 0 && page < p.pages;
    x.ks[u] = x.vs[u] = 1.0f;
    x.page[u] = 0;
    if (x.ok[u]) {
      x.page[u] = page;
      x.ks[u] = uniform_load(hd.ks + page * p.sks_p);
      x.vs[u] = uniform_load(hd.vs + page * p.svs_p);
    }
  }
}

// A tile's codes in registers.
template <int D>
struct Tile {
  int k[2][D / 16];     // D / 4 bytes of a token in each half
  int v[2][4][D / 64];  // D / 16 bytes of four tokens in each half
};

template <int D>
__device__ __forceinline__ void load_v(const PagedAttnArgs& p, const Heads& hd, int t, const TileRef& ref,
                                       uint32_t v_lane, Tile<D>& x) {
  constexpr int VB = D / 16;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int slot = (t * 32 + 16 * u) & (p.P - 1);
    const uint8_t* vp = hd.v + ref.page[u] * p.svc_p + slot * p.svc_t;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* row = vp + e * p.svc_t + v_lane;
      if constexpr (VB == 4) {
        x.v[u][e][0] = *reinterpret_cast<const int*>(row);
      } else if constexpr (VB == 8) {
        const i32x2 v = *reinterpret_cast<const i32x2*>(row);
        x.v[u][e][0] = v[0];
        x.v[u][e][1] = v[1];
      } else {
        const i32x4 v = *reinterpret_cast<const i32x4*>(row);
#pragma unroll
        for (int b = 0; b < 4; ++b) x.v[u][e][b] = v[b];
      }
    }
  }
}

template <int D>
__device__ __forceinline__ void load_tile(const PagedAttnArgs& p, const Heads& hd, int t, const TileRef& ref,
                                          uint32_t k_lane, uint32_t v_lane, Tile<D>& x) {
  constexpr int KB = D / 4;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int slot = (t * 32 + 16 * u) & (p.P - 1);
    const uint8_t* kp = hd.k + ref.page[u] * p.skc_p + slot * p.skc_t;
#pragma unroll
    for (int j = 0; j < KB / 16; ++j) {
      const i32x4 v = *reinterpret_cast<const i32x4*>(kp + k_lane + 16 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) x.k[u][4 * j + e] = v[e];
    }
  }
  load_v<D>(p, hd, t, ref, v_lane, x);
}

// Running state of one wave: rows = lane & 15, each lane a quarter of a row's
// output (elements (lane / 16) * D/4 ...), and its own part of the row's sum.
template <int D>
struct RowState {
  f32x4 o[D / 16];
  float m, l;
};

// What the 16 rows of a unit look at.
struct Rows {
  int qi, see_lo, see_hi;            // this lane's row
  int qi_first, qi_last;             // query positions of the tile
  int lo_all, hi_all;                // positions that every row sees
};

// Scores and weights of a tile: the running maximum and sum move on, the
// output so far is scaled to the new maximum; returns P^T as the second
// product wants it.  whole: every row sees all 32 positions.
template <int D>
__device__ __forceinline__ f16x8 weigh(const Tile<D>& x, const TileRef& ref, const bf16x8 (&q)[D / 32], const Rows& r,
                                       bool whole, int t, int g4, float qk, RowState<D>& st) {
  // S^T: lane = its row, tokens 16 u + 4 g4 + i
  f32x4 sc[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const i32x2 a = fp8x4_to_bf16(x.k[u][2 * j]), b = fp8x4_to_bf16(x.k[u][2 * j + 1]);
      const bf16x8 kf = __builtin_bit_cast(bf16x8, i32x4{a[0], a[1], b[0], b[1]});
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[j], acc, 0, 0, 0);
    }
    sc[u] = acc;
  }
  float y[8], inv[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float lsv = __builtin_amdgcn_logf(ref.vs[u]);
    inv[u] = __builtin_amdgcn_rcpf(ref.vs[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[4 * u + i] = __builtin_fmaf(sc[u][i], ref.ks[u] * qk, lsv);
  }
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = t * 32 + 16 * (i / 4) + 4 * g4 + i % 4;
      y[i] = ref.ok[i / 4] && at >= r.see_lo && at <= r.see_hi ? y[i] : -INFINITY;
    }
  }
  float mx = y[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, y[i]);
  mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  const float m_new = fmaxf(st.m, mx);
  const float m_use = m_new == -INFINITY ? 0.0f : m_new - P_SHIFT;  // nothing seen so far
  if (__any(m_new != st.m)) {  // (seldom, once the largest scores have been seen)
    const float alpha = __builtin_amdgcn_exp2f(st.m - P_SHIFT - m_use);
    st.m = m_new;
    st.l *= alpha;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[i][e] *= alpha;
  }
  f16x8 pf;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = __builtin_amdgcn_exp2f(y[i] - m_use);
    st.l = __builtin_fmaf(w, inv[i / 4], st.l);
    pf[i] = (_Float16)w;
  }
  return pf;
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
template <int D>
__device__ __forceinline__ void add_values(const Tile<D>& x, f16x8 pf, RowState<D>& st) {
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    f16x8 v0, v1;
    turn_values<D>(x, b, v0, v1);
    st.o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf, st.o[2 * b], 0, 0, 0);
    st.o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf, st.o[2 * b + 1], 0, 0, 0);
  }
}

// Clears the values of positions outside [lo, hi] and of absent pages: their
// codes may be NaN, and a weight of 0 would not hide that.
template <int D>
__device__ __forceinline__ void clear_values(const TileRef& ref, int t, int g4, int lo, int hi, Tile<D>& x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = t * 32 + 16 * (i / 4) + 4 * g4 + i % 4;
    const bool seen = ref.ok[i / 4] && at >= lo && at <= hi;
#pragma unroll
    for (int b = 0; b < D / 64; ++b) x.v[i / 4][i % 4][b] = seen ? x.v[i / 4][i % 4][b] : 0;
  }
}

// Rows of a tile that do not see the same positions, and a NaN code among the
// values: it has to reach the rows that see it and no others, though a
// weight of 0 times NaN is NaN.  The NaN codes are cleared, and a product of
// their places with what each row sees says which outputs they make NaN.
template <int D>
__device__ __forceinline__ void take_out_nans(const TileRef& ref, const Rows& r, int t, int g4, Tile<D>& x,
                                              RowState<D>& st) {
  Tile<D> places;  // code 1 (a positive value) where there is a NaN
  int hit = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      int& w = x.v[i / 4][i % 4][b];
      const int n = (int)(((((uint32_t)w & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u);
      places.v[i / 4][i % 4][b] = n;
      hit |= n;
      w &= (int)~((uint32_t)n * 0xffu);
    }
  if (!__any(hit != 0)) return;
  f16x8 sees;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = t * 32 + 16 * (i / 4) + 4 * g4 + i % 4;
    sees[i] = (_Float16)(ref.ok[i / 4] && at >= r.see_lo && at <= r.see_hi ? 1.0f : 0.0f);
  }
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    f16x8 v0, v1;
    turn_values<D>(places, b, v0, v1);
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const f32x4 c0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, sees, zero, 0, 0, 0);
    const f32x4 c1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, sees, zero, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      st.o[2 * b][e] = c0[e] > 0.0f ? __uint_as_float(0x7fc00000u) : st.o[2 * b][e];
      st.o[2 * b + 1][e] = c1[e] > 0.0f ? __uint_as_float(0x7fc00000u) : st.o[2 * b + 1][e];
    }
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
  const float inv_l = l != 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;  // (NaN stays NaN)
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = l != 0.0f ? o[e] * inv_l : 0.0f;
  const int qi = row / p.group, qh = h * p.group + row % p.group;
  *reinterpret_cast<i32x2*>(p.out + s * p.so_s + (int64_t)qi * p.so_n + (int64_t)qh * p.so_h + c4) = to_bf16x4_bits(o);
  if (c4 == 0 && p.lse != nullptr)
    p.lse[s * p.sl_s + (int64_t)qi * p.sl_n + (int64_t)qh * p.sl_h] =
        l != 0.0f ? (m - P_SHIFT + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
}

// A workgroup's waves: rt of them take the unit's row tiles side by side (the
// second and later ones find the codes in the caches), ATTN_WAVES / rt streams
// take the tiles of the line in turn.
template <int D, bool SPLIT>
__global__ __launch_bounds__(ATTN_THREADS, D > 128 ? 2 : 3) void paged_attention_kernel(const PagedAttnArgs p) {
  constexpr int KB = D / 4;    // bytes of a key per lane
  constexpr int VB = D / 16;   // bytes of a value per lane, and output tiles
  constexpr int CW = D < 128 ? D : 128;  // columns that the waves join at a time
  __shared__ float so[ATTN_WAVES][16][CW + 4];
  __shared__ float sm[ATTN_WAVES][16], sl[ATTN_WAVES][16];
  __shared__ int64_t red[ATTN_WAVES], found[2];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t k_lane = (uint32_t)(r16 * p.skc_t + g4 * KB);
  const uint32_t v_lane = (uint32_t)(4 * g4 * p.svc_t + r16 * VB);
  const float qk = p.scale * LOG2E;
  const int streams = uniform(ATTN_WAVES / p.rt), stream = uniform(wave / p.rt);

  int64_t share = 0, at = 0, end = 1, before = 0;
  int s = uniform(blockIdx.x / p.units);
  if (SPLIT && !line_share(p, red, found, &share, &at, &end, &s, &before)) return;

  while (at < end) {
    const Span sp = span_of(p, uniform_load(p.lens + s));
    const int nt = sp.end - sp.begin;
    if (SPLIT && at - before >= (int64_t)nt * p.units) {  // next sequence
      before += (int64_t)nt * p.units;
      ++s;
      continue;
    }
    const int rel = (int)(at - before);
    const int unit = uniform(SPLIT ? rel / nt : (int)(blockIdx.x - s * p.units));
    const int t0 = SPLIT ? rel - unit * nt : 0;
    const int t1 = SPLIT && end - at < nt - t0 ? t0 + (int)(end - at) : nt;
    const int h = uniform(unit / p.groups), row0 = (unit - h * p.groups) * p.rt * 16;
    const int len = sp.len;

    // this lane's row: query position and the range of positions it sees
    const int first_row = row0 + (wave - stream * p.rt) * 16;
    const int row = first_row + r16;
    const bool row_ok = row < p.rows;
    const int qh = h * p.group + (row_ok ? row % p.group : 0);
    const int last_row = first_row + 15 < p.rows ? first_row + 15 : p.rows - 1;
    Rows r;
    r.qi = row_ok ? row / p.group : 0;
    r.qi_first = uniform(first_row / p.group);
    r.qi_last = uniform(last_row / p.group);
    const int qpos = len - p.n + r.qi;
    r.see_hi = row_ok ? qpos : -1;
    r.see_lo = p.window > 0 && qpos - p.window + 1 > 0 ? qpos - p.window + 1 : 0;
    r.hi_all = len - p.n + r.qi_first;
    const int hi_any = len - p.n + r.qi_last;
    const int lo_any = p.window > 0 && r.hi_all - p.window + 1 > 0 ? r.hi_all - p.window + 1 : 0;
    r.lo_all = p.window > 0 && hi_any - p.window + 1 > 0 ? hi_any - p.window + 1 : 0;

    // Q^T fragments: step j holds elements g4 * KB + 8 j ...
    bf16x8 q[D / 32];
    {
      const uint16_t* from = p.q + s * p.sq_s + (int64_t)r.qi * p.sq_n + (int64_t)qh * p.sq_h + g4 * KB;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        i32x4 v = {0, 0, 0, 0};
        if (row_ok) v = *reinterpret_cast<const i32x4*>(from + 8 * j);
        q[j] = __builtin_bit_cast(bf16x8, v);
      }
    }
    RowState<D> st;
#pragma unroll
    for (int i = 0; i < VB; ++i) st.o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    st.m = -INFINITY;
    st.l = 0.0f;

    // the piece's tiles that some row of this row tile sees, one stream each in turn
    int ta = sp.begin + t0, tb = sp.begin + t1;
    const int t_last = hi_any < 0 ? -1 : hi_any / 32;
    if (ta < lo_any / 32) ta = lo_any / 32;
    if (tb > t_last + 1) tb = t_last + 1;  // (none where the queries see nothing: there may be no page to read)
    if (first_row >= p.rows) tb = ta;
    const Heads hd = {p.table + s * p.s_table, p.k_cache + h * p.skc_h, p.v_cache + h * p.svc_h,
                      p.k_scale + h * p.sks_h, p.v_scale + h * p.svs_h, len};
    int t = uniform(ta + stream);
    tb = uniform(tb);
    TileRef next;
    find_tile(p, hd, t, t < tb, next);
    while (t < tb) {
      const TileRef ref = next;
      Tile<D> x;
      load_tile<D>(p, hd, t, ref, k_lane, v_lane, x);
      find_tile(p, hd, t + streams, t + streams < tb, next);  // (its page is known when its turn comes)
      const bool whole = t * 32 >= r.lo_all && t * 32 + 31 <= r.hi_all && ref.ok[0] && ref.ok[1];
      const f16x8 pf = weigh<D>(x, ref, q, r, whole, t, g4, qk, st);
      if (!whole) {
        clear_values<D>(ref, t, g4, lo_any, hi_any, x);
        if (r.qi_first != r.qi_last) take_out_nans<D>(ref, r, t, g4, x, st);
      }
      add_values<D>(x, pf, st);
      t += streams;
    }

    // join the streams: each scales its output to the common maximum, then
    // every thread sums four columns of a row
    st.l += __shfl_xor(st.l, 16, 64);
    st.l += __shfl_xor(st.l, 32, 64);
    if (SPLIT) __syncthreads();  // the last piece's join has been read
    if (g4 == 0) {
      sm[wave][r16] = st.m;
      sl[wave][r16] = st.l;
    }
    __syncthreads();
    float m = -INFINITY;
    for (int w = wave % p.rt; w < ATTN_WAVES; w += p.rt) m = fmaxf(m, sm[w][r16]);
    // (without a maximum the sums are 0, or NaN where every score is NaN)
    const float f = st.m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    const bool piece = t0 > 0 || t1 < nt;
    float* part = piece ? part_at<D>(p, 2 * (int64_t)blockIdx.x + (t0 == 0)) : nullptr;
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += CW) {
      if (c0 > 0) __syncthreads();
      // element (i, e) of the lane is output element g4 * KB + e * VB + i
      if (g4 * KB >= c0 && g4 * KB < c0 + CW) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < VB; i += 4)
            *reinterpret_cast<f32x4*>(&so[wave][r16][g4 * KB - c0 + e * VB + i]) =
                f32x4{st.o[i][e] * f, st.o[i + 1][e] * f, st.o[i + 2][e] * f, st.o[i + 3][e] * f};
      }
      __syncthreads();
      for (int j = threadIdx.x; j < p.rt * 16 * (CW / 4); j += ATTN_THREADS) {
        const int c = j % (CW / 4) * 4, rr = j / (CW / 4), tile = rr / 16, rw = rr % 16;
        if (row0 + rr >= p.rows) continue;
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
        float mm = -INFINITY, ll = 0.0f;
        for (int w = tile; w < ATTN_WAVES; w += p.rt) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(&so[w][rw][c]);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] += v[e];
          mm = fmaxf(mm, sm[w][rw]);
        }
        for (int w = tile; w < ATTN_WAVES; w += p.rt)
          ll += sl[w][rw] * (sm[w][rw] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(sm[w][rw] - mm));
        if (SPLIT && piece) {
          *reinterpret_cast<f32x4*>(part + rr * D + c0 + c) = o;
          if (c0 + c == 0) {
            part[p.rt * 16 * D + rr] = mm;
            part[p.rt * 16 * (D + 1) + rr] = ll;
          }
        } else {
          store_row<D>(p, s, h, row0 + rr, c0 + c, o, mm, ll);
        }
      }
    }
    if (!SPLIT) return;
    if (t0 == 0 && threadIdx.x == 0) {
      int32_t* parts = unit_parts(p, (int64_t)s * p.units + unit);
      parts[0] = blockIdx.x;
      parts[1] = (int32_t)((at + nt - 1) / share);
    }
    at += t1 - t0;
  }
}

// Join of the units that were cut: a workgroup takes `rps` rows (a power of
// two) of a unit; its threads are D / 4 column quadruples x rps rows x GROUPS
// that walk the parts in turn and are summed in order, so that the result does
// not depend on anything but the lengths.
template <int D>
__global__ __launch_bounds__(ATTN_THREADS) void paged_attention_join_kernel(const PagedAttnArgs p) {
  constexpr int C = D / 4;
  __shared__ f32x4 acc[ATTN_THREADS];
  __shared__ float red[ATTN_WAVES][16];
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
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  // maxima of the rows: lane r of every rps lanes takes row r
  const int rr = threadIdx.x % p.rps;
  float m = -INFINITY;
  for (int i = threadIdx.x / p.rps; i < n; i += ATTN_THREADS / p.rps)
    m = fmaxf(m, base[(i == 0 ? 1 : 2 * (int64_t)i) * part_size + unit_rows * D + r0 + rr]);
  for (int off = p.rps; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if (lane < p.rps) red[wave][lane] = m;
  __syncthreads();

  const int c = threadIdx.x % C, r = threadIdx.x / C % p.rps, g = threadIdx.x / C / p.rps;
  const int n_groups = ATTN_THREADS / C / p.rps;
  m = red[0][r];
#pragma unroll
  for (int w = 1; w < ATTN_WAVES; ++w) m = fmaxf(m, red[w][r]);
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
#pragma unroll 4
  for (int i = g; i < n; i += n_groups) {
    const float* part = base + (i == 0 ? 1 : 2 * (int64_t)i) * part_size;
    const float pm = part[unit_rows * D + r0 + r];
    const float pl = part[unit_rows * (D + 1) + r0 + r];
    const f32x4 v = *reinterpret_cast<const f32x4*>(part + (r0 + r) * D + 4 * c);
    const float f = pm == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(pm - m);
    l = __builtin_fmaf(pl, f, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(v[e], f, o[e]);
  }
  if (n_groups > 1) {
    __syncthreads();  // the maxima have been read
    acc[threadIdx.x] = o;
    if (c == 0) (&red[0][0])[g * p.rps + r] = l;
    __syncthreads();
    if (g > 0) return;
    for (int k = 1; k < n_groups; ++k) {
      const f32x4 v = acc[threadIdx.x + k * C * p.rps];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += v[e];
      l += (&red[0][0])[k * p.rps + r];
    }
  }
  if (row0 + r < p.rows) store_row<D>(p, s, h, row0 + r, 4 * c, o, m, l);
}

// What is launched: a pure function of the sizes.
struct AttnPlan {
  int rt, units;        // row tiles a workgroup takes together; (KV head, group of row tiles) per sequence
  bool split;
  int64_t shares;       // workgroups of the first kernel when split
  int min_share;        // tiles of a share at least
  int rps;              // rows per workgroup of the join
};

// Caches of at most this many tiles (1024 tokens) are not cut: the cut costs
// two scans of the lengths and the join's launch, together about 7 us, and a
// workgroup goes through 1024 tokens of a head of 128 in 12.6 us.
constexpr int64_t DIRECT_TILES = 32;
// Parts of one call: at most 40 MiB.
constexpr int64_t WORKSPACE_FLOATS = 10 << 20;

// Shares: as many as are resident at once on 256 compute units (registers:
// four workgroups a unit at D = 64, three at 128, two at 256), so that all
// end together.  At D = 128 512 / 768 / 1024 shares took 223 / 219 / 227 us
// (128 sequences up to 8192 long, 8 heads) and 80 / 82 / 85 us (4 sequences
// up to 131071 long, 4 heads); at D = 256 512 / 635 took 34 / 45 us.
int64_t most_shares(int64_t D) { return D == 64 ? 1024 : D == 128 ? 768 : 512; }

AttnPlan attn_plan(int64_t S, int64_t Hkv, int64_t row_tiles, int64_t D, int64_t cap) {
  AttnPlan a;
  a.rt = row_tiles >= 3 ? 4 : (int)row_tiles;
  a.units = (int)(Hkv * ((row_tiles + a.rt - 1) / a.rt));
  const int64_t cap_tiles = (cap + 31) / 32, units = S * a.units;
  a.split = cap_tiles > DIRECT_TILES;
  a.min_share = ATTN_WAVES / a.rt;  // a tile for each stream
  const int64_t part = a.rt * 16 * (D + 2);
  int64_t most = WORKSPACE_FLOATS / (2 * part);
  if (most > most_shares(D)) most = most_shares(D);
  const int64_t want = (units * cap_tiles + a.min_share - 1) / a.min_share;
  a.shares = want < most ? want : most;
  // few units: a row to a workgroup; many: as many rows as its threads hold
  a.rps = (int)(ATTN_THREADS / (D / 4));
  if (a.rps > 16) a.rps = 16;
  while (a.rps > 1 && units * (16 * a.rt / a.rps) < 1024) a.rps /= 2;
  return a;
}

// Workgroups of the join.
int64_t join_grid(const AttnPlan& a, int64_t S) { return S * a.units * (a.rt * 16 / a.rps); }

template <int D>
hipError_t launch(const PagedAttnArgs& p, const AttnPlan& a, hipStream_t stream) {
  if (!a.split) {
    paged_attention_kernel<D, false><<<dim3((unsigned)((int64_t)p.S * p.units)), dim3(ATTN_THREADS), 0, stream>>>(p);
    return hipGetLastError();
  }
  paged_attention_kernel<D, true><<<dim3((unsigned)p.shares), dim3(ATTN_THREADS), 0, stream>>>(p);
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
  const AttnPlan a = attn_plan(p.S, p.Hkv, p.row_tiles, p.D, (int64_t)p.max_pages * p.P);
  p.rt = a.rt;
  p.units = a.units;
  p.groups = a.units / p.Hkv;
  p.shares = (int32_t)a.shares;
  p.min_share = a.min_share;
  p.rps = a.rps;
  p.log_p = __builtin_ctz(p.P);
  if (p.D == 64) return launch<64>(p, a, stream);
  if (p.D == 128) return launch<128>(p, a, stream);
  return launch<256>(p, a, stream);
}

}  // namespace dgmi
