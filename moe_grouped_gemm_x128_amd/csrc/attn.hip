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

__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t up = __shfl_up(v, off, 64);
    if (lane >= off) v += up;
  }
  return v;
}

__device__ __forceinline__ int64_t line_total(const PagedAttnArgs& p, int64_t* red) {
  int64_t v = 0;
  for (int s = threadIdx.x; s < p.S; s += ATTN_THREADS) {
    const Span sp = span_of(p, p.lens[s]);
    v += (int64_t)(sp.end - sp.begin) * p.units;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < ATTN_WAVES; ++w) total += red[w];
  __syncthreads();
  return total;
}

// The sequence holding tile `at` of the line (at < total), and the tiles before it.
__device__ __forceinline__ void line_find(const PagedAttnArgs& p, int64_t at, int64_t* red, int64_t* found,
                                          int* s_out, int64_t* before_out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t before = 0;
  for (int base = 0; base < p.S; base += ATTN_THREADS) {
    const int s = base + threadIdx.x;
    int64_t mine = 0;
    if (s < p.S) {
      const Span sp = span_of(p, p.lens[s]);
      mine = (int64_t)(sp.end - sp.begin) * p.units;
    }
    const int64_t incl = wave_scan(mine, lane);
    if (lane == 63) red[wave] = incl;
    __syncthreads();
    int64_t start = before, all = 0;
#pragma unroll
    for (int w = 0; w < ATTN_WAVES; ++w) {
      start += w < wave ? red[w] : 0;
      all += red[w];
    }
    const int64_t lo = start + incl - mine;
    if (s < p.S && at >= lo && at < lo + mine) {
      found[0] = s;
      found[1] = lo;
    }
    __syncthreads();
    before += all;
    if (at < before) break;
  }
  *s_out = uniform((int)found[0]);
  *before_out = (int64_t)((uint64_t)(uint32_t)uniform((int)(found[1] & 0xffffffff)) |
                          ((uint64_t)(uint32_t)uniform((int)(found[1] >> 32)) << 32));
}

// One tile's codes and scales in registers.
template <int D>
struct Tile {
  int k[2][D / 16];        // D / 4 bytes of a token in each of two 16-token halves
  int v[2][4][D / 64];     // D / 16 bytes of four tokens in each half
  float ks[2], vs[2];
  bool ok[2];
};

template <int D>
__device__ __forceinline__ void load_tile(const PagedAttnArgs& p, int s, int h, int len, int t, uint32_t k_lane,
                                          uint32_t v_lane, Tile<D>& x) {
  constexpr int KB = D / 4, VB = D / 16;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int at = t * 32 + 16 * u;
    int page = -1;
    if (at < len) page = uniform_load(p.table + s * p.s_table + (at >> p.log_p));
    x.ok[u] = page >= 0 && page < p.pages;
    x.ks[u] = x.vs[u] = 1.0f;
    if (x.ok[u]) {
      x.ks[u] = uniform_load(p.k_scale + page * p.sks_p + h * p.sks_h);
      x.vs[u] = uniform_load(p.v_scale + page * p.svs_p + h * p.svs_h);
    } else {
      page = 0;
    }
    const int slot = at & (p.P - 1);
    const uint8_t* kp = p.k_cache + page * p.skc_p + h * p.skc_h + slot * p.skc_t;
    const uint8_t* vp = p.v_cache + page * p.svc_p + h * p.svc_h + slot * p.svc_t;
#pragma unroll
    for (int j = 0; j < KB / 16; ++j) {
      const i32x4 v = *reinterpret_cast<const i32x4*>(kp + k_lane + 16 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) x.k[u][4 * j + e] = v[e];
    }
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

template <int D>
__device__ __forceinline__ void attend(const PagedAttnArgs& p, const Tile<D>& x, const bf16x8 (&q)[D / 32],
                                       const Rows& r, int len, int t, int g4, float qk, RowState<D>& st) {
  constexpr int VB = D / 16;
  const int pos0 = t * 32;
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
  const bool whole = pos0 >= r.lo_all && pos0 + 31 <= r.hi_all && x.ok[0] && x.ok[1];
  float y[8], inv[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float lsv = __builtin_amdgcn_logf(x.vs[u]);
    inv[u] = __builtin_amdgcn_rcpf(x.vs[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = pos0 + 16 * u + 4 * g4 + i;
      const float v = __builtin_fmaf(sc[u][i], x.ks[u] * qk, lsv);
      y[4 * u + i] = whole || (x.ok[u] && at >= r.see_lo && at <= r.see_hi) ? v : -INFINITY;
    }
  }
  float mx = y[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, y[i]);
  mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  const float m_new = fmaxf(st.m, mx);
  const float m_use = m_new == -INFINITY ? 0.0f : m_new - P_SHIFT;  // nothing seen so far
  const float alpha = __builtin_amdgcn_exp2f(st.m == -INFINITY ? -INFINITY : st.m - P_SHIFT - m_use);
  st.m = m_new;
  st.l *= alpha;
  f16x8 pf;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = __builtin_amdgcn_exp2f(y[i] - m_use);
    st.l = __builtin_fmaf(w, inv[i / 4], st.l);
    pf[i] = (_Float16)w;
  }
#pragma unroll
  for (int i = 0; i < VB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) st.o[i][e] *= alpha;

  // O^T += V^T P^T.  Where the rows differ in what they see, or slots past
  // the end are among the 32, each query position takes the tile by itself
  // with the values that it does not see cleared (their codes may be NaN),
  // and only the lanes of its rows keep the result.
  const int first = whole ? 0 : r.qi_first, last = whole ? 0 : r.qi_last;
  for (int a = first; a <= last; ++a) {
    int cw[8][VB / 4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool seen = true;
      if (!whole) {
        const int at = pos0 + 16 * (i / 4) + 4 * g4 + i % 4;
        const int ap = len - p.n + a;
        seen = x.ok[i / 4] && at <= ap && (p.window <= 0 || at > ap - p.window);
      }
#pragma unroll
      for (int b = 0; b < VB / 4; ++b) cw[i][b] = seen ? x.v[i / 4][i % 4][b] : 0;
    }
    const bool take = whole || a == r.qi;
#pragma unroll
    for (int b = 0; b < VB / 2; ++b) {  // bytes 2b, 2b + 1 of the eight tokens
      f16x2 lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // bytes (token 2j, token 2j + 1) of element 2b, then of element 2b + 1
        const int pair = __builtin_amdgcn_perm(cw[2 * j + 1][b / 2], cw[2 * j][b / 2],
                                               b % 2 == 0 ? 0x05010400u : 0x07030602u);
        lo[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pair, 1.0f, false);
        hi[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pair, 1.0f, true);
      }
      const f16x8 v0 = {lo[0][0], lo[0][1], lo[1][0], lo[1][1], lo[2][0], lo[2][1], lo[3][0], lo[3][1]};
      const f16x8 v1 = {hi[0][0], hi[0][1], hi[1][0], hi[1][1], hi[2][0], hi[2][1], hi[3][0], hi[3][1]};
      const f32x4 o0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf, st.o[2 * b], 0, 0, 0);
      const f32x4 o1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf, st.o[2 * b + 1], 0, 0, 0);
      st.o[2 * b] = take ? o0 : st.o[2 * b];
      st.o[2 * b + 1] = take ? o1 : st.o[2 * b + 1];
    }
  }
}

// A part's place in the workspace: 16 rows of D sums, then 16 maxima, 16 sums.
template <int D>
__device__ __forceinline__ float* part_at(const PagedAttnArgs& p, int64_t slot) {
  return p.workspace + slot * (16 * D + 32);
}
// Which parts a unit was cut into: {first workgroup, last workgroup}, behind the parts.
__device__ __forceinline__ int32_t* unit_parts(const PagedAttnArgs& p, int64_t unit) {
  return reinterpret_cast<int32_t*>(p.workspace + 2 * (int64_t)p.shares * (16 * p.D + 32)) + 2 * unit;
}

template <int D>
__global__ __launch_bounds__(ATTN_THREADS) void paged_attention_kernel(const PagedAttnArgs p) {
  constexpr int KB = D / 4;    // bytes of a key per lane
  constexpr int VB = D / 16;   // bytes of a value per lane, and output tiles
  __shared__ float so[ATTN_WAVES - 1][16][D + 4];
  __shared__ float sm[ATTN_WAVES][16], sl[ATTN_WAVES][16];
  __shared__ int64_t red[ATTN_WAVES], found[2];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t k_lane = (uint32_t)(r16 * p.skc_t + g4 * KB);
  const uint32_t v_lane = (uint32_t)(4 * g4 * p.svc_t + r16 * VB);
  const float qk = p.scale * LOG2E;

  const int64_t total = line_total(p, red);
  int64_t share = (total + p.shares - 1) / p.shares;
  if (share < p.min_share) share = p.min_share;
  int64_t at = blockIdx.x * share;
  int64_t end = at + share < total ? at + share : total;
  if (at >= end) return;
  int s;
  int64_t before;
  line_find(p, at, red, found, &s, &before);

  for (; at < end; ) {
    Span sp = span_of(p, uniform_load(p.lens + s));
    const int nt = sp.end - sp.begin;
    if (at - before >= (int64_t)nt * p.units) {  // next sequence
      before += (int64_t)nt * p.units;
      ++s;
      continue;
    }
    const int rel = (int)(at - before);
    const int unit = rel / nt, t0 = rel - unit * nt;
    const int t1 = end - at < nt - t0 ? t0 + (int)(end - at) : nt;
    const int mt = unit % p.row_tiles, h = unit / p.row_tiles;
    const int len = sp.len;

    // this lane's row: query position and the range of positions it sees
    const int row = mt * 16 + r16;
    const bool row_ok = row < p.rows;
    const int qh = h * p.group + (row_ok ? row % p.group : 0);
    const int last_row = mt * 16 + 15 < p.rows ? mt * 16 + 15 : p.rows - 1;
    Rows r;
    r.qi = row_ok ? row / p.group : 0;
    r.qi_first = mt * 16 / p.group;
    r.qi_last = last_row / p.group;
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

    // the piece's tiles that some row of this row tile sees, one wave each in turn
    int ta = sp.begin + t0, tb = sp.begin + t1;
    const int t_last = hi_any < 0 ? -1 : hi_any / 32;
    if (ta < lo_any / 32) ta = lo_any / 32;
    if (tb > t_last + 1) tb = t_last + 1;  // (none where the queries see nothing: there may be no page to read)
    for (int t = ta + wave; t < tb; t += ATTN_WAVES) {
      Tile<D> x;
      load_tile<D>(p, s, h, len, t, k_lane, v_lane, x);
      attend<D>(p, x, q, r, len, t, g4, qk, st);
    }

    // join the waves: sums of the four quarters of each row, then the waves
    st.l += __shfl_xor(st.l, 16, 64);
    st.l += __shfl_xor(st.l, 32, 64);
    __syncthreads();  // the last piece's join has been read
    if (g4 == 0) {
      sm[wave][r16] = st.m;
      sl[wave][r16] = st.l;
    }
    __syncthreads();
    float m = sm[0][r16];
#pragma unroll
    for (int w = 1; w < ATTN_WAVES; ++w) m = fmaxf(m, sm[w][r16]);
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < ATTN_WAVES; ++w)
      l += sl[w][r16] * (sm[w][r16] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(sm[w][r16] - m));
    // (without a maximum the sums are 0, or NaN where every score is NaN)
    const float f = st.m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    // element (i, e) of the lane is output element g4 * KB + e * VB + i
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < VB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) so[wave - 1][r16][g4 * KB + e * VB + i] = st.o[i][e] * f;
    }
    __syncthreads();
    const bool piece = t0 > 0 || t1 < nt;
    const int64_t this_unit = (int64_t)s * p.units + unit;
    if (p.workspace != nullptr && t0 == 0 && threadIdx.x == 0) {
      int32_t* parts = unit_parts(p, this_unit);
      parts[0] = blockIdx.x;
      parts[1] = (int32_t)((at + nt - 1) / share);
    }
    if (wave == 0 && row_ok) {
      const float inv_l = l != 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;  // (NaN stays NaN)
      uint16_t* out = p.out + s * p.so_s + (int64_t)r.qi * p.so_n + (int64_t)qh * p.so_h + g4 * KB;
      float* part = piece ? part_at<D>(p, 2 * (int64_t)blockIdx.x + (t0 == 0)) : nullptr;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < VB; i += 4) {
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float a = st.o[i + j][e] * f;
#pragma unroll
            for (int w = 0; w < ATTN_WAVES - 1; ++w) a += so[w][r16][g4 * KB + e * VB + i + j];
            v[j] = a;
          }
          if (piece) {
            *reinterpret_cast<f32x4*>(part + r16 * D + g4 * KB + e * VB + i) = v;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = l != 0.0f ? v[j] * inv_l : 0.0f;
            *reinterpret_cast<i32x2*>(out + e * VB + i) = to_bf16x4_bits(v);
          }
        }
      if (g4 == 0) {
        if (piece) {
          part[16 * D + r16] = m;
          part[16 * D + 16 + r16] = l;
        } else if (p.lse != nullptr) {
          p.lse[s * p.sl_s + (int64_t)r.qi * p.sl_n + (int64_t)qh * p.sl_h] =
              l != 0.0f ? (m - P_SHIFT + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
        }
      }
    }
    at += t1 - t0;
  }
}

// Join of the units that were cut: workgroup (unit, slice) takes every
// slices-th row.  The D / 4 column quadruples of a row times 256 / (D / 4)
// groups of parts, joined through shared memory; each group walks its parts in
// order, so the sums have one order.
template <int D>
__global__ __launch_bounds__(ATTN_THREADS) void paged_attention_join_kernel(const PagedAttnArgs p) {
  constexpr int C = D / 4, GROUPS = ATTN_THREADS / C;
  __shared__ f32x4 acc[GROUPS][C];
  const int slice = blockIdx.x % p.slices;
  const int64_t u = blockIdx.x / p.slices;
  const int32_t* parts = unit_parts(p, u);
  const int w0 = parts[0], w1 = parts[1];
  if (w0 == w1) return;
  const int s = (int)(u / p.units), unit = (int)(u % p.units);
  const int mt = unit % p.row_tiles, h = unit / p.row_tiles;
  const int c = threadIdx.x % C, grp = threadIdx.x / C;
  const int rows = p.rows - mt * 16 < 16 ? p.rows - mt * 16 : 16;
  for (int r = slice; r < rows; r += p.slices) {
    float m = -INFINITY;
    for (int w = w0; w <= w1; ++w) m = fmaxf(m, part_at<D>(p, 2 * (int64_t)w + (w == w0))[16 * D + r]);
    float l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = w0; w <= w1; ++w) {
      const float* part = part_at<D>(p, 2 * (int64_t)w + (w == w0));
      const float pm = part[16 * D + r];
      const float f = pm == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(pm - m);
      l = __builtin_fmaf(part[16 * D + 16 + r], f, l);
      if ((w - w0) % GROUPS != grp) continue;
      const f32x4 v = *reinterpret_cast<const f32x4*>(part + r * D + 4 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(v[e], f, o[e]);
    }
    acc[grp][c] = o;
    __syncthreads();
    if (grp == 0) {
      for (int g = 1; g < GROUPS; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += acc[g][c][e];
      const float inv_l = l != 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = l != 0.0f ? o[e] * inv_l : 0.0f;
      const int row = mt * 16 + r, qi = row / p.group, qh = h * p.group + row % p.group;
      *reinterpret_cast<i32x2*>(p.out + s * p.so_s + (int64_t)qi * p.so_n + (int64_t)qh * p.so_h + 4 * c) =
          to_bf16x4_bits(o);
      if (c == 0 && p.lse != nullptr)
        p.lse[s * p.sl_s + (int64_t)qi * p.sl_n + (int64_t)qh * p.sl_h] =
            l != 0.0f ? (m - P_SHIFT + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
    }
    __syncthreads();
  }
}

template <int D>
hipError_t launch(const PagedAttnArgs& p, hipStream_t stream) {
  paged_attention_kernel<D><<<dim3((unsigned)p.shares), dim3(ATTN_THREADS), 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.workspace == nullptr) return e;
  paged_attention_join_kernel<D><<<dim3((unsigned)((int64_t)p.S * p.units * p.slices)), dim3(ATTN_THREADS), 0, stream>>>(p);
  return hipGetLastError();
}

constexpr int MIN_SHARE = 4;  // tiles: one for each wave

// Workgroups of the first kernel: a pure function of the sizes.
int64_t share_count(int64_t units, int64_t cap_tiles, int64_t D) {
  const int64_t most = D > 128 ? 1024 : 2048;
  const int64_t want = (units * cap_tiles + MIN_SHARE - 1) / MIN_SHARE;
  return want < most ? want : most;
}

}  // namespace

int64_t paged_attention_workspace(int64_t S, int64_t n, int64_t Hq, int64_t Hkv, int64_t D, int64_t cap) {
  const int64_t group = Hq / Hkv, units = S * Hkv * ((n * group + 15) / 16);
  const int64_t shares = share_count(units, (cap + 31) / 32, D);
  return (2 * shares * (16 * D + 32) + 2 * units) * 4;
}

hipError_t launch_paged_attention(PagedAttnArgs p, hipStream_t stream) {
  p.units = p.Hkv * p.row_tiles;
  const int64_t units = (int64_t)p.S * p.units;
  const int64_t cap_tiles = ((int64_t)p.max_pages * p.P + 31) / 32;
  p.shares = (int32_t)share_count(units, cap_tiles > 0 ? cap_tiles : 1, p.D);
  p.min_share = MIN_SHARE;
  p.log_p = __builtin_ctz(p.P);
  p.slices = units >= 1024 ? 1 : units >= 64 ? (int32_t)(1024 / units) : 16;
  if (p.D == 64) return launch<64>(p, stream);
  if (p.D == 128) return launch<128>(p, stream);
  return launch<256>(p, stream);
}

}  // namespace dgmi
