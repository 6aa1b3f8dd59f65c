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

// Running state of one wave: rows = lane & 15, each lane a quarter of a row's
// output (elements (lane / 16) * D/4 ...), and its own part of the row's sum.
template <int D>
struct RowState {
  f32x4 o[D / 16];
  float m, l;
};

template <int D>
__global__ __launch_bounds__(ATTN_THREADS) void paged_attention_kernel(const PagedAttnArgs p) {
  constexpr int KB = D / 4;    // bytes of a key per lane
  constexpr int VB = D / 16;   // bytes of a value per lane, and output tiles
  __shared__ float so[ATTN_WAVES - 1][16][D + 4];
  __shared__ float sm[ATTN_WAVES][16], sl[ATTN_WAVES][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g4 = lane >> 4;

  const int mt = blockIdx.x % p.row_tiles;
  const int h = blockIdx.x / p.row_tiles % p.Hkv;
  const int s = blockIdx.x / p.row_tiles / p.Hkv;
  const int64_t cap = (int64_t)p.max_pages * p.P;
  int64_t len64 = p.lens[s];
  if (len64 > cap) len64 = cap;
  const int len = len64 < 0 || p.pages == 0 ? 0 : (int)len64;

  // this lane's row: query position and the range of positions it sees
  const int row = mt * 16 + r16;
  const bool row_ok = row < p.rows;
  const int qi = row_ok ? row / p.group : 0;
  const int qh = h * p.group + (row_ok ? row % p.group : 0);
  const int qpos = len - p.n + qi;
  const int see_hi = row_ok ? qpos : -1;  // last position seen
  const int see_lo = p.window > 0 && qpos - p.window + 1 > 0 ? qpos - p.window + 1 : 0;
  // the same over all rows of the tile
  const int qi_first = mt * 16 / p.group;
  const int last_row = mt * 16 + 15 < p.rows ? mt * 16 + 15 : p.rows - 1;
  const int qi_last = last_row / p.group;
  const int hi_all = len - p.n + qi_first, hi_any = len - p.n + qi_last;
  const int lo_any = p.window > 0 && hi_all - p.window + 1 > 0 ? hi_all - p.window + 1 : 0;
  const int lo_all = p.window > 0 && hi_any - p.window + 1 > 0 ? hi_any - p.window + 1 : 0;

  // Q^T fragments: step j holds elements g4 * KB + 8 j ...
  bf16x8 q[D / 32];
  {
    const uint16_t* at = p.q + s * p.sq_s + (int64_t)qi * p.sq_n + (int64_t)qh * p.sq_h + g4 * KB;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      i32x4 v = {0, 0, 0, 0};
      if (row_ok) v = *reinterpret_cast<const i32x4*>(at + 8 * j);
      q[j] = __builtin_bit_cast(bf16x8, v);
    }
  }

  RowState<D> st;
#pragma unroll
  for (int i = 0; i < VB; ++i) st.o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  st.m = -INFINITY;
  st.l = 0.0f;

  const uint32_t k_lane = (uint32_t)(r16 * p.skc_t + g4 * KB);
  const uint32_t v_lane = (uint32_t)(4 * g4 * p.svc_t + r16 * VB);
  const float qk = p.scale * LOG2E;

  // tiles of 32 positions, one wave each in turn
  const int t_begin = lo_any / 32, t_end = hi_any < 0 ? 0 : hi_any / 32 + 1;
  for (int t = t_begin + wave; t < t_end; t += ATTN_WAVES) {
    const int pos0 = t * 32;
    const uint8_t* kp[2];
    const uint8_t* vp[2];
    float ks[2], vs[2];
    bool page_ok[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = pos0 + 16 * u;
      int page = at < len ? p.table[s * p.s_table + at / p.P] : -1;
      page_ok[u] = page >= 0 && page < p.pages;
      page = page_ok[u] ? page : 0;
      const int slot = at % p.P;
      kp[u] = p.k_cache + page * p.skc_p + h * p.skc_h + slot * p.skc_t;
      vp[u] = p.v_cache + page * p.svc_p + h * p.svc_h + slot * p.svc_t;
      ks[u] = page_ok[u] ? p.k_scale[page * p.sks_p + h * p.sks_h] : 1.0f;
      vs[u] = page_ok[u] ? p.v_scale[page * p.svs_p + h * p.svs_h] : 1.0f;
    }
    int kw[2][KB / 4], vw[2][4][VB / 4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < KB / 16; ++j) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(kp[u] + k_lane + 16 * j);
#pragma unroll
        for (int e = 0; e < 4; ++e) kw[u][4 * j + e] = v[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t* at = vp[u] + v_lane + e * p.svc_t;
        if constexpr (VB == 4) {
          vw[u][e][0] = *reinterpret_cast<const int*>(at);
        } else if constexpr (VB == 8) {
          const i32x2 v = *reinterpret_cast<const i32x2*>(at);
          vw[u][e][0] = v[0];
          vw[u][e][1] = v[1];
        } else {
          const i32x4 v = *reinterpret_cast<const i32x4*>(at);
#pragma unroll
          for (int b = 0; b < 4; ++b) vw[u][e][b] = v[b];
        }
      }
    }
    // S^T: lane = row r16, tokens 16 u + 4 g4 + i
    f32x4 sc[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const i32x2 a = fp8x4_to_bf16(kw[u][2 * j]), b = fp8x4_to_bf16(kw[u][2 * j + 1]);
        const bf16x8 kf = __builtin_bit_cast(bf16x8, i32x4{a[0], a[1], b[0], b[1]});
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[j], acc, 0, 0, 0);
      }
      sc[u] = acc;
    }
    const bool whole = pos0 >= lo_all && pos0 + 31 <= hi_all && page_ok[0] && page_ok[1];
    float y[8];
    float inv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float lsv = __builtin_amdgcn_logf(vs[u]);
      inv[u] = __builtin_amdgcn_rcpf(vs[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = pos0 + 16 * u + 4 * g4 + i;
        const float v = __builtin_fmaf(sc[u][i], ks[u] * qk, lsv);
        y[4 * u + i] = whole || (page_ok[u] && at >= see_lo && at <= see_hi) ? v : -INFINITY;
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
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = __builtin_amdgcn_exp2f(y[i] - m_use);
      st.l = __builtin_fmaf(w[i], inv[i / 4], st.l);
    }
#pragma unroll
    for (int i = 0; i < VB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[i][e] *= alpha;

    // O^T += V^T P^T.  Where the rows differ in what they see, or slots past
    // the end are among the 32, each query position takes the tile by itself
    // with the values that it does not see cleared (their codes may be NaN),
    // and only the lanes of its rows keep the result.
    const int first = whole ? 0 : qi_first, last = whole ? 0 : qi_last;
    for (int a = first; a <= last; ++a) {
      int cw[8][VB / 4];
      f16x8 pf;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pf[i] = (_Float16)w[i];
        bool seen = true;
        if (!whole) {
          const int at = pos0 + 16 * (i / 4) + 4 * g4 + i % 4;
          const int ap = len - p.n + a;
          seen = page_ok[i / 4] && at <= ap && (p.window <= 0 || at > ap - p.window);
        }
#pragma unroll
        for (int b = 0; b < VB / 4; ++b) cw[i][b] = seen ? vw[i / 4][i % 4][b] : 0;
      }
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
        const bool take = whole || a == qi;
        st.o[2 * b] = take ? o0 : st.o[2 * b];
        st.o[2 * b + 1] = take ? o1 : st.o[2 * b + 1];
      }
    }
  }

  // join the waves: sums of the four quarters of each row, then the waves
  st.l += __shfl_xor(st.l, 16, 64);
  st.l += __shfl_xor(st.l, 32, 64);
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
  if (wave > 0 || !row_ok) return;
  const float inv_l = l != 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;  // (NaN stays NaN)
  uint16_t* out = p.out + s * p.so_s + (int64_t)qi * p.so_n + (int64_t)qh * p.so_h + g4 * KB;
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
        v[j] = l != 0.0f ? a * inv_l : 0.0f;
      }
      *reinterpret_cast<i32x2*>(out + e * VB + i) = to_bf16x4_bits(v);
    }
  if (p.lse != nullptr && g4 == 0)
    p.lse[s * p.sl_s + (int64_t)qi * p.sl_n + (int64_t)qh * p.sl_h] =
        l != 0.0f ? (m - P_SHIFT + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
}

}  // namespace

int64_t paged_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_paged_attention(const PagedAttnArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.S * p.Hkv * p.row_tiles)), block(ATTN_THREADS);
  if (p.D == 64) paged_attention_kernel<64><<<grid, block, 0, stream>>>(p);
  else if (p.D == 128) paged_attention_kernel<128><<<grid, block, 0, stream>>>(p);
  else paged_attention_kernel<256><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace dgmi
