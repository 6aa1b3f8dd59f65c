// BF16 products grouped by expert with ragged sizes, gfx950: the forward product
// of rows sorted by expert, without padding, and its two gradients.  Group g owns
// rows offsets[g] .. offsets[g + 1] - 1 (device memory) of the tokens' tensors.
//
//   NT  d[m] = c[m] + a[m] . b[g]^T      a [M, K], b [G, N, K], d [M, N]
//   NN  d[m] = c[m] + a[m] . b[g]        a [M, K], b [G, K, N], d [M, N]
//   TN  d[g] = c[g] + a_g^T . b_g        a [M, N], b [M, K], d [G, N, K], the
//       contraction over the group's own rows
//
// One kernel body: a tile of BM x BN outputs a workgroup, WM x WN waves, slices of
// 64 in the contraction staged in LDS by buffer loads that write it directly, FP32
// accumulation in v_mfma_f32_16x16x32_bf16.  An operand whose contraction runs
// along its rows (K-major: a of NT and NN, b of NT) is staged as rows of 128 bytes,
// one whose contraction runs across them (MN-major: b of NN, both of TN) as 64 rows
// of the tile's width, whose fragments are read by transposing LDS loads.
//
// NT and NN: the grid holds the most tiles that offsets can ask for,
// floor(M / BM) + min(G, M) times the column tiles; every wave finds its tile by a
// scan of the offsets, and workgroups past the last tile exit at once.

#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

constexpr int SLICE = 64;  // contraction elements of a stage
constexpr int XCDS = 8;

typedef __attribute__((address_space(3))) void lds_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// K-major stage: 16-byte chunk c of tile row r lies at slot c ^ h(r), h linear over
// GF(2) in the bits of r: the 16 rows of a fragment, consecutive or in PERM's order
// (bits 0, 1, 4 and 5), read at one chunk hit distinct banks.
__device__ __host__ constexpr int row_swz(int r) {
  return ((r ^ (r >> 3) ^ (r >> 5)) & 1) | (r & 2) | ((((r >> 2) ^ (r >> 4)) & 1) << 2);
}
// MN-major stage: chunk c of contraction row k lies at slot c ^ hk(k): the four
// rows of each of two lane groups that read together hit distinct banks.
__device__ __host__ constexpr int col_swz(int k) { return 2 * ((k & 3) | ((((k >> 3) ^ (k >> 4)) & 1) << 2)); }

template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
};

// s_waitcnt operand: all LDS traffic done, and all but the last n loads.
constexpr int vmcnt_lgkm0(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

__device__ __forceinline__ bf16x8 lo_bf16(const i32x8& v) { return __builtin_bit_cast(bf16x8, i32x4{v[0], v[1], v[2], v[3]}); }
__device__ __forceinline__ bf16x8 hi_bf16(const i32x8& v) { return __builtin_bit_cast(bf16x8, i32x4{v[4], v[5], v[6], v[7]}); }

// First row and end of group g, inside [0, M].
__device__ __forceinline__ void group_rows(const int32_t* offsets, int g, int M, int& first, int& end) {
  first = min(max(offsets[g], 0), M);
  end = min(max(offsets[g + 1], 0), M);
}

// Row tiles of all groups, and tile `want` of them: its group, first row and the
// group's end.  64 groups a step, a lane each; every lane gets the result.
template <int BM>
__device__ __forceinline__ int count_tiles(const int32_t* offsets, int G, int M) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int base = 0; base < G; base += 64) {
    int first = 0, end = 0;
    if (base + lane < G) group_rows(offsets, base + lane, M, first, end);
    int n = max(0, end - first + BM - 1) / BM;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, 64);
    total += n;
  }
  return total;
}
template <int BM>
__device__ __forceinline__ void find_tile(const int32_t* offsets, int G, int M, int want, int& g, int& m0, int& end_) {
  const int lane = threadIdx.x & 63;
  g = m0 = end_ = 0;
  for (int base = 0; base < G; base += 64) {
    int first = 0, end = 0;
    if (base + lane < G) group_rows(offsets, base + lane, M, first, end);
    const int n = max(0, end - first + BM - 1) / BM;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int up = __shfl_up(incl, off, 64);
      if (lane >= off) incl += up;
    }
    const uint64_t past = __ballot(incl > want);  // the first of them holds the tile
    if (past != 0) {
      const int at = __ffsll((unsigned long long)past) - 1;
      g = base + at;
      m0 = __shfl(first, at, 64) + (want - (__shfl(incl, at, 64) - __shfl(n, at, 64))) * BM;
      end_ = __shfl(end, at, 64);
      return;
    }
    want -= __shfl(incl, 63, 64);
  }
}

// The hardware deals workgroups to the XCDs in turn: XCD x gets a run of tiles.
__device__ __forceinline__ int tile_of(int b, int total) {
  const int q = total / XCDS, r = total % XCDS, x = b % XCDS;
  return x * q + min(x, r) + b / XCDS;
}
// Tile t of tm x tn tiles, in bands of 8 rows taken column by column.
__device__ __forceinline__ void banded(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = t / (8 * tiles_n), first = band * 8, rows = min(8, tiles_m - first);
  const int in = t - band * 8 * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

template <class T, int LAY, bool F32>
__global__ __launch_bounds__(T::NT) void ragged_kernel(const RaggedArgs p) {
  constexpr bool A_MN = LAY == RAGGED_TN, B_MN = LAY != RAGGED_NT;
  constexpr int A_STAGE = T::BM * SLICE * 2, B_STAGE = T::BN * SLICE * 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds_a0[A_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t lds_a1[A_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t lds_b0[B_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t lds_b1[B_STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;

  // the tile: group g, rows m0 .. and columns n0 .. of the output, and its limits
  int g, m0, n0, m_end, n_end, len;
  const uint16_t *A, *B;  // first row of the tile's operands
  if constexpr (LAY == RAGGED_TN) {
    const int per = p.tiles_n * p.tiles_k;
    const int t = tile_of(blockIdx.x, p.G * per);
    g = t / per;
    int tm, tn, first, end;
    banded(t - g * per, p.tiles_n, p.tiles_k, tm, tn);
    group_rows(p.offsets, g, p.M, first, end);
    first = __builtin_amdgcn_readfirstlane(first);
    len = __builtin_amdgcn_readfirstlane(max(0, end - first));
    m0 = tm * T::BM;
    n0 = tn * T::BN;
    m_end = p.N;
    n_end = p.K;
    A = p.a + (int64_t)first * p.lda + m0;
    B = p.b + (int64_t)first * p.ldb + n0;
  } else {
    const int tiles_m = __builtin_amdgcn_readfirstlane(count_tiles<T::BM>(p.offsets, p.G, p.M));
    const int total = tiles_m * p.tiles_n;
    if ((int)blockIdx.x >= total) return;
    int tm, tn;
    banded(tile_of(blockIdx.x, total), tiles_m, p.tiles_n, tm, tn);
    find_tile<T::BM>(p.offsets, p.G, p.M, tm, g, m0, m_end);
    g = __builtin_amdgcn_readfirstlane(g);
    m0 = __builtin_amdgcn_readfirstlane(m0);
    m_end = __builtin_amdgcn_readfirstlane(m_end);
    n0 = tn * T::BN;
    n_end = p.N;
    len = p.K;
    A = p.a + (int64_t)m0 * p.lda;
    B = p.b + (int64_t)g * p.b_gs + (B_MN ? (int64_t)n0 : (int64_t)n0 * p.ldb);
  }
  const int KB = (len + SLICE - 1) / SLICE;

  // One load of a slice into a stage, 1024 bytes a wave.  K-major: load j fills 8 tile rows of 128 bytes; its
  // resource ends after the last row that exists, what lies past it reads as zero.  A slice past the last one has an
  // empty resource: zeros, no memory access.
  constexpr int A_LD = A_STAGE / (1024 * T::NW), B_LD = B_STAGE / (1024 * T::NW);  // loads of a slice, per wave
  const int lrow = lane >> 3;
  const uint32_t vchunk = (uint32_t)((lane & 7) ^ lrow);  // (row_swz of 8 j + lrow is row_swz(8 j) ^ lrow)
  auto rows_vrow = [&](int64_t ld) { return (uint32_t)((wave * 8 + lrow) * ld * 2); };
  auto rows_size = [&](int64_t ld, int rows, int j) {
    return __builtin_amdgcn_readfirstlane((int)(max(0, min(rows - j * T::NW * 8, T::NW * 8)) * ld * 2));
  };
  auto load_rows_one = [&](uint8_t* stage, const uint16_t* base, int64_t ld, uint32_t vrow, int size, int kb, int j) {
    const uint32_t hu = (uint32_t)row_swz((j * T::NW + wave) * 8);
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + (int64_t)j * T::NW * 8 * ld), (short)0, kb < KB ? size : 0, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_t*)(stage + (j * T::NW + wave) * 1024), 16,
                                             vrow + ((vchunk ^ hu) << 4), kb * SLICE * 2, 0, 0);
  };
  // MN-major: load j fills PER contraction rows of W columns.  Rows past `len` read as zero (the resource starts at
  // the slice and ends with the 16-byte chunk of the last column of the last row), columns past the operand's feed
  // outputs that are never stored.
  struct Cols {
    const uint8_t* at;  // the next slice to load
    int64_t left;       // bytes from there to the operand's end
    int64_t step;
  };
  auto cols_of = [&](const uint16_t* base, int64_t ld, int cols) {
    return Cols{reinterpret_cast<const uint8_t*>(base), len > 0 ? ((len - 1) * ld + (cols + 7) / 8 * 8) * 2 : 0, SLICE * ld * 2};
  };
  auto load_cols_one = [&](uint8_t* stage, const Cols& c, const uint32_t* voff, int j) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)c.at, (short)0, (int)min(max(c.left, (int64_t)0), (int64_t)0x7fffffff), 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_t*)(stage + (j * T::NW + wave) * 1024), 16, voff[j], 0, 0, 0);
  };
  auto cols_voff = [&](int64_t ld, int j, auto width) {
    constexpr int W = decltype(width)::value, SLOTS = W / 8, PER = 64 / SLOTS;
    const int k = (j * T::NW + wave) * PER + lane / SLOTS;
    return (uint32_t)(k * ld * 2) + (uint32_t)(((lane % SLOTS) ^ col_swz(k)) << 4);
  };
  int a_size[A_LD], b_size[B_LD];
  uint32_t a_voff[A_LD], b_voff[B_LD];
  Cols a_cols = {}, b_cols = {};
#pragma unroll
  for (int j = 0; j < A_LD; ++j) {
    if constexpr (A_MN) a_voff[j] = cols_voff(p.lda, j, std::integral_constant<int, T::BM>{});
    else a_size[j] = rows_size(p.lda, m_end - m0, j);
  }
#pragma unroll
  for (int j = 0; j < B_LD; ++j) {
    if constexpr (B_MN) b_voff[j] = cols_voff(p.ldb, j, std::integral_constant<int, T::BN>{});
    else b_size[j] = rows_size(p.ldb, n_end - n0, j);
  }
  if constexpr (A_MN) a_cols = cols_of(A, p.lda, m_end - m0);
  if constexpr (B_MN) b_cols = cols_of(B, p.ldb, n_end - n0);
  const uint32_t a_vrow = rows_vrow(p.lda), b_vrow = rows_vrow(p.ldb);
  auto load_a_one = [&](uint8_t* stage, int kb, int j) {
    if constexpr (A_MN) {
      load_cols_one(stage, a_cols, a_voff, j);
      if (j + 1 == A_LD) a_cols.at += a_cols.step, a_cols.left -= a_cols.step;
    } else {
      load_rows_one(stage, A, p.lda, a_vrow, a_size[j], kb, j);
    }
  };
  auto load_b_one = [&](uint8_t* stage, int kb, int j) {
    if constexpr (B_MN) {
      load_cols_one(stage, b_cols, b_voff, j);
      if (j + 1 == B_LD) b_cols.at += b_cols.step, b_cols.left -= b_cols.step;
    } else {
      load_rows_one(stage, B, p.ldb, b_vrow, b_size[j], kb, j);
    }
  };
  auto load_a = [&](uint8_t* stage, int kb) {
#pragma unroll
    for (int j = 0; j < A_LD; ++j) load_a_one(stage, kb, j);
  };
  auto load_b = [&](uint8_t* stage, int kb) {
#pragma unroll
    for (int j = 0; j < B_LD; ++j) load_b_one(stage, kb, j);
  };

  // Fragments of a slice: 16 tile rows (columns) from r0, contraction 32 half + 8 (lane / 16) .. +7 in lane (row
  // lane % 16), half 0 in the first four registers.  With PERM the rows of B's fragment f are permuted so that a lane
  // ends up with 16 consecutive columns of the output.
  const int fr = lane & 15, q = lane >> 4;
  auto frag_rows = [&](const uint8_t* stage, int r) {
    const int off = r * 128 + ((q ^ row_swz(r)) << 4);
    const i32x4 l = *reinterpret_cast<const i32x4*>(stage + off), h = *reinterpret_cast<const i32x4*>(stage + (off ^ 64));
    return i32x8{l[0], l[1], l[2], l[3], h[0], h[1], h[2], h[3]};
  };
  // lane s of a group of 16 reads 4 columns of contraction row 8 q + 4 t + s / 4; transposed, the group hands lane
  // s the four rows of column s
  auto frag_cols = [&](const uint8_t* stage, int r0, auto width) {
    constexpr int W = decltype(width)::value;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    i32x8 v;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int k = (t >> 1) * 32 + 8 * q + 4 * (t & 1) + (fr >> 2);
      const int chunk = r0 / 8 + ((fr >> 1) & 1);
      const i32x2 x = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(stage + k * W * 2 + ((chunk ^ col_swz(k)) << 4) + 8 * (fr & 1))));
      v[2 * t] = x[0];
      v[2 * t + 1] = x[1];
    }
    return v;
  };
  constexpr bool PERM = !B_MN && T::TN == 64;
  auto a_frag = [&](const uint8_t* stage, int i) {
    if constexpr (A_MN) return frag_cols(stage, wm * T::TM + 16 * i, std::integral_constant<int, T::BM>{});
    else return frag_rows(stage, wm * T::TM + 16 * i + fr);
  };
  auto b_frag = [&](const uint8_t* stage, int f) {
    if constexpr (B_MN) return frag_cols(stage, wn * T::TN + 16 * f, std::integral_constant<int, T::BN>{});
    else return frag_rows(stage, wn * T::TN + (PERM ? (fr >> 2) * 16 + f * 4 + (fr & 3) : 16 * f + fr));
  };
  f32x4 acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int f = 0; f < T::FN; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bool live = m0 + wm * T::TM < m_end && n0 + wn * T::TN < n_end;  // else nothing of the wave is stored

  // One software pipeline over the fragment rows of all slices, two barriers a slice.  Early, before the second
  // fragment row: every wave has the slice's B fragments in registers, so the B part of its stage takes slice kb + 2.
  // Late, before the last one: the next slice has landed and every wave is done with this one's A part, which takes
  // slice kb + 2; the next slice's first fragments are read while the last MFMAs run.  The loads of a point go out one
  // after each MFMA that follows it.  Waiting loads in issue order: B of kb + 2 may stay in flight at the late point.
  auto meet = [&](auto loads) {  // all but the wave's last `loads` loads have landed, in every wave
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0(decltype(loads)::value));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");  // (no access moves past it)
    __builtin_amdgcn_sched_barrier(0);
  };
  auto early = [&]() { meet(std::integral_constant<int, 63>{}); };
  auto late = [&]() { meet(std::integral_constant<int, B_LD>{}); };
  if (KB > 0) {
    load_a(lds_a0, 0);
    load_b(lds_b0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_b(lds_b1, 1);
    load_a(lds_a1, 1);
    __builtin_amdgcn_sched_barrier(0);
    meet(std::integral_constant<int, A_LD + B_LD>{});
    if (live) {
      i32x8 bf[T::FN], af;
#pragma unroll
      for (int f = 0; f < T::FN; ++f) bf[f] = b_frag(lds_b0, f);
      af = a_frag(lds_a0, 0);
      auto slice = [&](uint8_t* cur_a, uint8_t* cur_b, const uint8_t* nxt_a, const uint8_t* nxt_b, int kb) {
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          if (i == 1) early();
          if (i + 1 == T::FM) late();
          const i32x8 next = i + 1 < T::FM ? a_frag(cur_a, i + 1) : a_frag(nxt_a, 0);
#pragma unroll
          for (int f = 0; f < T::FN; ++f) {
            __builtin_amdgcn_sched_barrier(0);
            acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo_bf16(bf[f]), lo_bf16(af), acc[i][f], 0, 0, 0);
#pragma unroll
            for (int j = f; j < (i == 1 ? B_LD : i + 1 == T::FM ? A_LD : 0); j += T::FN) {
              if (i == 1) load_b_one(cur_b, kb + 2, j);
              else load_a_one(cur_a, kb + 2, j);
            }
          }
#pragma unroll
          for (int f = 0; f < T::FN; ++f) {
            __builtin_amdgcn_sched_barrier(0);
            acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi_bf16(bf[f]), hi_bf16(af), acc[i][f], 0, 0, 0);
          }
          if (i + 1 == T::FM) {
#pragma unroll
            for (int f = 0; f < T::FN; ++f) bf[f] = b_frag(nxt_b, f);
          }
          af = next;
        }
      };
      int kb = 0;
      for (; kb + 2 <= KB; kb += 2) {
        slice(lds_a0, lds_b0, lds_a1, lds_b1, kb);
        slice(lds_a1, lds_b1, lds_a0, lds_b0, kb + 1);
      }
      if (kb < KB) slice(lds_a0, lds_b0, lds_a1, lds_b1, kb);
    } else {
      for (int kb = 0; kb < KB; ++kb) {  // (loads and barriers only)
        early();
        load_b(kb & 1 ? lds_b1 : lds_b0, kb + 2);
        late();
        load_a(kb & 1 ? lds_a1 : lds_a0, kb + 2);
      }
    }
    __builtin_amdgcn_s_waitcnt(0);  // (no load may write LDS after the workgroup's end)
  }
  if (!live) return;

  // lane: output row lane % 16 of each fragment row and, PERM, 16 consecutive columns, else 4 of each fragment
  const int64_t d_at = LAY == RAGGED_TN ? (int64_t)g * p.d_gs : 0, c_at = LAY == RAGGED_TN ? (int64_t)g * p.c_gs : 0;
  constexpr int RUN = PERM ? 16 : 4;  // consecutive columns of a lane
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int row = m0 + wm * T::TM + 16 * i + fr;
    if (row >= m_end) continue;
#pragma unroll
    for (int f0 = 0; f0 < T::FN; f0 += RUN / 4) {
      const int col = n0 + wn * T::TN + (PERM ? 16 * q : 16 * f0 + 4 * q);
      const int n = min(RUN, n_end - col);
      if (p.c != nullptr) {
        const int64_t at = c_at + (int64_t)row * p.ldc + col;
#pragma unroll
        for (int e = 0; e < RUN; ++e)
          if (e < n) acc[i][f0 + e / 4][e & 3] += p.c_f32 ? static_cast<const float*>(p.c)[at + e]
                                                          : bf16_to_f32(static_cast<const uint16_t*>(p.c)[at + e]);
      }
      const int64_t at = d_at + (int64_t)row * p.ldd + col;
      if constexpr (F32) {
        float* to = static_cast<float*>(p.d) + at;
        if (n == RUN && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
#pragma unroll
          for (int e = 0; e < RUN; e += 4) *reinterpret_cast<f32x4*>(to + e) = acc[i][f0 + e / 4];
        } else {
#pragma unroll
          for (int e = 0; e < RUN; ++e)
            if (e < n) to[e] = acc[i][f0 + e / 4][e & 3];
        }
      } else {
        uint16_t* to = static_cast<uint16_t*>(p.d) + at;
        i32x2 w[RUN / 4];
#pragma unroll
        for (int e = 0; e < RUN / 4; ++e) w[e] = to_bf16x4_bits(acc[i][f0 + e]);
        if (n == RUN && (reinterpret_cast<uintptr_t>(to) & (PERM ? 15 : 7)) == 0) {
          if constexpr (PERM) {
#pragma unroll
            for (int e = 0; e < RUN / 4; e += 2)
              *reinterpret_cast<i32x4*>(to + 4 * e) = i32x4{w[e][0], w[e][1], w[e + 1][0], w[e + 1][1]};
          } else {
            *reinterpret_cast<i32x2*>(to) = w[0];
          }
        } else {
#pragma unroll
          for (int e = 0; e < RUN; ++e)
            if (e < n) to[e] = (uint16_t)((uint32_t)w[e / 4][(e & 3) / 2] >> (16 * (e & 1)));
        }
      }
    }
  }
}

using Big = Shape<256, 256, 2, 4>;

int64_t tiles(int64_t n, int64_t by) { return (n + by - 1) / by; }

template <class T>
hipError_t launch_shape(RaggedArgs p, int layout, int64_t grid, hipStream_t stream) {
  p.tiles_n = (int32_t)tiles(p.N, layout == RAGGED_TN ? T::BM : T::BN);
  p.tiles_k = (int32_t)tiles(p.K, T::BN);
  const dim3 gr((unsigned)grid), b(T::NT);
#define DGMI_RAGGED(L_)                                                       \
  do {                                                                        \
    if (p.d_f32) ragged_kernel<T, L_, true><<<gr, b, 0, stream>>>(p);         \
    else ragged_kernel<T, L_, false><<<gr, b, 0, stream>>>(p);                \
  } while (0)
  if (layout == RAGGED_NT) DGMI_RAGGED(RAGGED_NT);
  else if (layout == RAGGED_NN) DGMI_RAGGED(RAGGED_NN);
  else DGMI_RAGGED(RAGGED_TN);
#undef DGMI_RAGGED
  return hipGetLastError();
}

}  // namespace

// Workgroups of a call, the most that any offsets ask for.
int64_t ragged_grid(int layout, int64_t G, int64_t M, int64_t N, int64_t K) {
  if (layout == RAGGED_TN) return G * tiles(N, Big::BM) * tiles(K, Big::BN);
  return (M / Big::BM + (G < M ? G : M)) * tiles(N, Big::BN);
}

hipError_t launch_ragged(RaggedArgs p, int layout, hipStream_t stream) {
  return launch_shape<Big>(p, layout, ragged_grid(layout, p.G, p.M, p.N, p.K), stream);
}

}  // namespace dgmi
