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
// accumulation in v_mfma_f32_16x16x32_bf16 (its 32 x 32 form, with half the operand
// reads, measured 3% slower).  An operand whose contraction runs along its rows
// (K-major: a of NT and NN, b of NT) is staged as rows of 128 bytes, one whose
// contraction runs across them (MN-major: b of NN, both of TN) as 64 rows of the
// tile's width, whose fragments are read by transposing LDS loads.
//
// The workgroups are as many as fit the machine and take the tiles in turn; the
// pipeline does not stop between them: while a tile ends, the next one's first
// slices are loaded.  (One workgroup a tile: 4 to 7% slower on tiles of 16 to 112
// slices.)  NT and NN find their tile from the running sums of the groups' tiles,
// kept in LDS; a group's last tile, where it is at most half full, is shared out
// among all waves (2 to 3% over groups of 256 to 1760 rows).
//
// What bounds it: 32 groups of 1024 rows, 4096 x 7168, run at 1400 to 1430 TFLOP/s
// (the gradient of a at 1340 to 1360), at which the card's power limit holds the clock
// near 1.75 GHz; with groups of 267 to 1760 rows 1150 to 1270, 12.5% of the tiles' rows
// being empty.  A weight gradient of 2048 x 7168 over 1024 rows a group runs at 940 to
// 960: its tiles are 16 slices long, and their stores (256 KB in FP32), which the loads
// behind them wait for, take a quarter of the time (without them 720 us for 1000).  Few
// rows are bound by the weights' stream: 8 rows in six groups of 4096 x 7168 read them at
// 5.8 TB/s; one group's few rows by the time of a slice (256 rows of 4096 x 4096 21 us).

#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace dgmi {

namespace {

constexpr int SLICE = 64;  // contraction elements of a stage
constexpr int XCDS = 8, CUS = 256;
constexpr int GROUPS_IN_LDS = 2048;  // groups whose first tiles are kept at hand

typedef __attribute__((address_space(3))) void lds_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// K-major stage: 16-byte chunk c of tile row r lies at slot c ^ h(r): the 16 rows of
// a fragment read at one chunk hit distinct banks.  Those of A (and of B without
// PERM) are consecutive, those of B in PERM's order differ in bits 0, 1, 4 and 5.
__device__ __host__ constexpr int row_swz(int r, bool perm) {
  return perm ? ((r ^ (r >> 5)) & 1) | (r & 2) | (((r >> 4) & 1) << 2) : ((r ^ (r >> 3)) & 1) | (r & 6);
}
// MN-major stage: chunk c of contraction row k lies at slot c ^ hk(k): the four
// rows of each of two lane groups that read together hit distinct banks.
__device__ __host__ constexpr int col_swz(int k) { return 2 * ((k & 3) | ((((k >> 4) ^ (k >> 5)) & 1) << 2)); }

template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int PER_CU_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int PER_CU = PER_CU_;  // workgroups that fit a compute unit
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
};

// s_waitcnt operand: all LDS traffic done, and all but the last n loads.
constexpr int vmcnt_lgkm0(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// First row and end of group g, inside [0, M].
__device__ __forceinline__ void group_rows(const int32_t* offsets, int g, int M, int& first, int& end) {
  first = min(max(offsets[g], 0), M);
  end = min(max(offsets[g + 1], 0), M);
}

// NT and NN: the row tiles of groups base .. base+63, a lane each, and their
// running sum over the lanes.
template <int BM>
__device__ __forceinline__ void group_tiles(const int32_t* offsets, int G, int M, int base, int& first, int& end,
                                            int& n, int& sum) {
  const int lane = threadIdx.x & 63;
  first = end = 0;
  if (base + lane < G) group_rows(offsets, base + lane, M, first, end);
  n = sum = max(0, end - first + BM - 1) / BM;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(sum, off, 64);
    if (lane >= off) sum += up;
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

// A tile: group g, rows m0 .. m_end - 1 and columns n0 .. n_end - 1 of the output
// that may be stored, length of the contraction and (TN) its first row.
struct Tile {
  int g, m0, n0, m_end, n_end, len, first;
};

template <class T, int LAY, bool F32>
__global__ __launch_bounds__(T::NT, 2) void ragged_kernel(const RaggedArgs p) {
  constexpr bool A_MN = LAY == RAGGED_TN, B_MN = LAY != RAGGED_NT;
  constexpr int S = T::STAGES;
  static_assert(S == 2 || S == 3, "two or three stages");
  static_assert((!A_MN || T::BM >= 128) && (!B_MN || T::BN >= 128), "the swizzle flips bits of 16 chunks");
  constexpr int A_STAGE = T::BM * SLICE * 2, B_STAGE = T::BN * SLICE * 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds_a0[A_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t lds_a1[A_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t lds_a2[S > 2 ? A_STAGE : 16];
  __shared__ __attribute__((aligned(16))) uint8_t lds_b0[B_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t lds_b1[B_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t lds_b2[S > 2 ? B_STAGE : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;

  // Tiles of all groups, one after the other; NT and NN: those of group g start at column tiles * starts[g].
  __shared__ int starts[LAY == RAGGED_TN ? 1 : GROUPS_IN_LDS];
  int total;
  if constexpr (LAY == RAGGED_TN) {
    total = p.G * p.tiles_n * p.tiles_k;
  } else {
    int sum_before = 0;
    for (int base = 0; base < p.G; base += 64) {
      int first, end, n, sum;
      group_tiles<T::BM>(p.offsets, p.G, p.M, base, first, end, n, sum);
      if (wave == 0 && base + lane < GROUPS_IN_LDS) starts[base + lane] = sum_before + sum - n;
      sum_before += __shfl(sum, 63, 64);
    }
    total = __builtin_amdgcn_readfirstlane(sum_before) * p.tiles_n;
    __syncthreads();
  }
  auto find = [&](int t) __attribute__((always_inline)) {
    Tile x;
    if constexpr (LAY == RAGGED_TN) {
      const int per = p.tiles_n * p.tiles_k;
      int tm, tn, end;
      x.g = t / per;
      banded(t - x.g * per, p.tiles_n, p.tiles_k, tm, tn);
      group_rows(p.offsets, x.g, p.M, x.first, end);
      x.len = max(0, end - x.first);
      x.m0 = tm * T::BM;
      x.n0 = tn * T::BN;
      x.m_end = p.N;
      x.n_end = p.K;
    } else {
      // the last group that starts at or before the tile, and is not empty
      const int want = t / p.tiles_n;
      int g = 0, before = 0;
      if (p.G <= GROUPS_IN_LDS) {
        for (int base = 0; base < p.G; base += 64) {
          const int s = base + lane < p.G ? starts[base + lane] : INT32_MAX;
          const uint64_t m = __ballot(s <= want);
          if (m == 0) break;
          g = base + 63 - __clzll((long long)m);
          before = __shfl(s, 63 - __clzll((long long)m), 64);
        }
      } else {
        int sum_before = 0;
        for (int base = 0; base < p.G; base += 64) {
          int first, end, n, sum;
          group_tiles<T::BM>(p.offsets, p.G, p.M, base, first, end, n, sum);
          const uint64_t m = __ballot(sum_before + sum > want);
          if (m != 0) {
            const int at = __ffsll((unsigned long long)m) - 1;
            g = base + at;
            before = sum_before + __shfl(sum - n, at, 64);
            break;
          }
          sum_before += __shfl(sum, 63, 64);
        }
      }
      x.g = __builtin_amdgcn_readfirstlane(g);
      before = __builtin_amdgcn_readfirstlane(before);
      int end;
      group_rows(p.offsets, x.g, p.M, x.first, end);
      const int tiles_m = max(1, (end - x.first + T::BM - 1) / T::BM);
      int tm, tn;
      banded(t - before * p.tiles_n, tiles_m, p.tiles_n, tm, tn);
      x.m0 = x.first + tm * T::BM;
      x.n0 = tn * T::BN;
      x.m_end = end;
      x.n_end = p.N;
      x.len = p.K;
    }
    // (in scalar registers: the resources of the loads hang on them)
    for (int* v : {&x.g, &x.m0, &x.n0, &x.m_end, &x.n_end, &x.len, &x.first}) *v = __builtin_amdgcn_readfirstlane(*v);
    return x;
  };
  // the workgroup's tile of each round, as many workgroups as tiles in the last one
  auto tile_in = [&](int done) __attribute__((always_inline)) {
    const int left = total - done, grid = (int)gridDim.x;
    return left >= grid ? done + tile_of(blockIdx.x, grid) : (int)blockIdx.x < left ? done + tile_of(blockIdx.x, left) : -1;
  };

  // One load of a slice into a stage, 1024 bytes a wave.  K-major: load j fills 8 tile rows of 128 bytes; the
  // resource ends after the last row that exists, what lies past it reads as zero.  A slice past the last one has an
  // empty resource: zeros, no memory access.
  constexpr int A_LD = A_STAGE / (1024 * T::NW), B_LD = B_STAGE / (1024 * T::NW);  // loads of a slice, per wave
  constexpr bool PERM = !B_MN && T::TN == 64;
  struct Rows {
    const uint16_t* at;  // the tile's first row
    int bytes;           // of its rows
  };
  // the operands of the tile that the loads are at, its slices, and the one that it begins with
  int KB = 0, rot = 0;
  auto rows_voff = [&](int64_t ld, int j, bool perm) __attribute__((always_inline)) {
    const int r = (j * T::NW + wave) * 8 + (lane >> 3);
    return (uint32_t)(r * ld * 2) + (uint32_t)(((lane & 7) ^ row_swz(r, perm)) << 4);
  };
  auto load_rows_one = [&](uint8_t* stage, const Rows& o, uint32_t voff, int kb, int j) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void*)o.at, (short)0, kb < KB ? o.bytes : 0, 0x00020000);
    const int s = kb + rot;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_t*)(stage + (j * T::NW + wave) * 1024), 16, voff,
                                             (s >= KB ? s - KB : s) * SLICE * 2, 0, 0);
  };
  // MN-major: load j fills PER contraction rows of W columns.  Rows past `len` read as zero (the resource starts at
  // the slice and ends with the 16-byte chunk of the last column of the last row), columns past the operand's feed
  // outputs that are never stored.
  struct Cols {
    const uint8_t* at;  // the next slice to load
    int64_t left;       // bytes from there to the operand's end
    int64_t step;
  };
  auto cols_of = [&](const uint16_t* base, int64_t ld, int len, int cols) __attribute__((always_inline)) {
    return Cols{reinterpret_cast<const uint8_t*>(base), len > 0 ? ((int64_t)(len - 1) * ld + (cols + 7) / 8 * 8) * 2 : 0, SLICE * ld * 2};
  };
  auto load_cols_one = [&](uint8_t* stage, const Cols& c, const uint32_t* voff, int j) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)c.at, (short)0, c.left <= 0 ? 0 : c.left >> 31 ? 0x7fffffff : (int)c.left, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_t*)(stage + (j * T::NW + wave) * 1024), 16, voff[j], 0, 0, 0);
  };
  auto cols_voff = [&](int64_t ld, int j, auto width) __attribute__((always_inline)) {
    constexpr int W = decltype(width)::value, SLOTS = W / 8, PER = 64 / SLOTS;
    const int k = (j * T::NW + wave) * PER + lane / SLOTS;
    return (uint32_t)(k * ld * 2) + (uint32_t)(((lane % SLOTS) ^ col_swz(k)) << 4);
  };
  uint32_t a_voff[A_LD], b_voff[B_LD];
#pragma unroll
  for (int j = 0; j < A_LD; ++j) {
    if constexpr (A_MN) a_voff[j] = cols_voff(p.lda, j, std::integral_constant<int, T::BM>{});
    else a_voff[j] = rows_voff(p.lda, j, false);
  }
#pragma unroll
  for (int j = 0; j < B_LD; ++j) {
    if constexpr (B_MN) b_voff[j] = cols_voff(p.ldb, j, std::integral_constant<int, T::BN>{});
    else b_voff[j] = rows_voff(p.ldb, j, PERM);
  }
  Rows a_rows = {}, b_rows = {};
  Cols a_cols = {}, b_cols = {};
  auto load_from = [&](const Tile& x) __attribute__((always_inline)) {
    KB = (x.len + SLICE - 1) / SLICE;
    // Where weight rows are a multiple of 4 KB apart, the XCDs begin with different slices: all at one, they would be at
    // the same few channels of the memory.  An XCD's share of a round is 32 tiles of 256 columns in turn; which slice
    // comes first hangs on the group and the columns alone, not on the XCD itself, so that a row's sum is of one order in
    // every batch (runs of 16: 32 groups of 192 rows, 7168 x 2048 219 us for 224, of one row, 4096 x 4096 182 for 176).
    // (6144 rows of 7168 x 2048: 247 us for 255; without such rows 1% slower.)
    if constexpr (LAY == RAGGED_NT) {
      const int run = (x.g * ((p.N + 255) >> 8) + (x.n0 >> 8)) >> 5;
      rot = p.ldb * 2 % 4096 == 0 ? run % XCDS * KB / XCDS : 0;
    }
    const uint16_t* A = p.a + (A_MN ? (int64_t)x.first * p.lda + x.m0 : (int64_t)x.m0 * p.lda);
    const uint16_t* B = p.b + (LAY == RAGGED_TN ? (int64_t)x.first * p.ldb + x.n0
                                                : (int64_t)x.g * p.b_gs + (B_MN ? (int64_t)x.n0 : (int64_t)x.n0 * p.ldb));
    const int m = x.m_end - x.m0, n = x.n_end - x.n0;
    if constexpr (A_MN) a_cols = cols_of(A, p.lda, x.len, m);
    else a_rows = Rows{A, __builtin_amdgcn_readfirstlane(min(max(m, 0), T::BM) * (int)p.lda * 2)};
    if constexpr (B_MN) b_cols = cols_of(B, p.ldb, x.len, n);
    else b_rows = Rows{B, __builtin_amdgcn_readfirstlane(min(max(n, 0), T::BN) * (int)p.ldb * 2)};
  };
  auto load_a_one = [&](uint8_t* stage, int kb, int j) __attribute__((always_inline)) {
    if constexpr (A_MN) {
      load_cols_one(stage, a_cols, a_voff, j);
      if (j + 1 == A_LD) a_cols.at += a_cols.step, a_cols.left -= a_cols.step;
    } else {
      load_rows_one(stage, a_rows, a_voff[j], kb, j);
    }
  };
  auto load_b_one = [&](uint8_t* stage, int kb, int j) __attribute__((always_inline)) {
    if constexpr (B_MN) {
      load_cols_one(stage, b_cols, b_voff, j);
      if (j + 1 == B_LD) b_cols.at += b_cols.step, b_cols.left -= b_cols.step;
    } else {
      load_rows_one(stage, b_rows, b_voff[j], kb, j);
    }
  };
  auto load_a = [&](uint8_t* stage, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < A_LD; ++j) load_a_one(stage, kb, j);
  };
  auto load_b = [&](uint8_t* stage, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < B_LD; ++j) load_b_one(stage, kb, j);
  };

  // Fragments of a slice: 16 tile rows (columns), contraction 16 (lane / 16) + 8 half .. +7 in lane (row lane % 16),
  // half 0 in the first four registers.  With PERM the rows of B's fragment f are permuted so that a lane ends up with
  // 16 consecutive columns of the output.  The swizzles are linear: a fragment's offset is a base of the lane's with
  // some bits flipped, plus a constant.
  const int fr = lane & 15, q = lane >> 4;
  auto half_rows = [&](const uint8_t* stage, int base, int r, int h) __attribute__((always_inline)) {
    return *reinterpret_cast<const bf16x8*>(stage + (base ^ (h << 4)) + r * 128);
  };
  // lane s of a group of 16 reads 4 columns of contraction row 16 q + 8 h + 4 t + s / 4; transposed, the group hands
  // lane s the four rows of column s
  auto half_cols = [&](const uint8_t* stage, int base, int i, int h, auto width) __attribute__((always_inline)) {
    constexpr int W = decltype(width)::value;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    union { s16x4 x[2]; bf16x8 v; } u;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      u.x[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(stage + (base ^ (i << 5)) + (8 * h + 4 * t) * W * 2));
    return u.v;
  };
  auto rows_base = [&](int r, bool perm) __attribute__((always_inline)) { return r * 128 + (((2 * q) ^ row_swz(r, perm)) << 4); };
  auto cols_base = [&](int r0, int width) __attribute__((always_inline)) {
    const int k = 16 * q + (fr >> 2);
    return k * width * 2 + (((r0 / 8 + ((fr >> 1) & 1)) ^ col_swz(k)) << 4) + 8 * (fr & 1);
  };
  struct Frag {
    bf16x8 h[2];
  };
  int a_base = 0;  // of the tile's rows of the wave (K-major: they vary)
  if constexpr (A_MN) a_base = cols_base(wm * T::TM, T::BM);
  int b_base = B_MN ? cols_base(wn * T::TN, T::BN) : rows_base(wn * T::TN + (PERM ? (fr >> 2) * 16 + (fr & 3) : fr), PERM);
  auto a_frag = [&](const uint8_t* stage, int i) __attribute__((always_inline)) {
    if constexpr (A_MN)
      return Frag{half_cols(stage, a_base, i, 0, std::integral_constant<int, T::BM>{}),
                  half_cols(stage, a_base, i, 1, std::integral_constant<int, T::BM>{})};
    else return Frag{half_rows(stage, a_base, 16 * i, 0), half_rows(stage, a_base, 16 * i, 1)};
  };
  auto b_half = [&](const uint8_t* stage, int f, int h) __attribute__((always_inline)) {
    if constexpr (B_MN) return half_cols(stage, b_base, f, h, std::integral_constant<int, T::BN>{});
    else return half_rows(stage, b_base, PERM ? 4 * f : 16 * f, h);
  };
  f32x4 acc[T::FM][T::FN];

  // One software pipeline over the fragment rows of all slices of all tiles, two barriers a slice; a tile takes a
  // multiple of S slices (the last may be zeros), so that it begins in the first stage.  Early, before the second
  // fragment row: every wave has the slice's B fragments in registers, so the B part of its stage takes slice kb + S.
  // Late, before the last two: the next slice has landed and every wave is done with this one's A part, which takes
  // slice kb + S; the next slice's first fragments are read while the last matrix instructions run.  The loads of a
  // point go out between those that follow it.  Loads land in the order of their issue: at the late point all that
  // were issued behind those of slice kb + 1 may stay in flight.
  auto meet = [&](auto loads) __attribute__((always_inline)) {  // all but the wave's last `loads` loads have landed, in every wave
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0(decltype(loads)::value));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");  // (no access moves past it)
    __builtin_amdgcn_sched_barrier(0);
  };
  auto early = [&]() __attribute__((always_inline)) { meet(std::integral_constant<int, 63>{}); };
  auto late = [&]() __attribute__((always_inline)) { meet(std::integral_constant<int, (S - 1) * B_LD + (S - 2) * A_LD>{}); };
  auto idle = [&](uint8_t* cur_a, uint8_t* cur_b, int kb) __attribute__((always_inline)) {  // a slice of a wave without rows or columns
    early();
    load_b(cur_b, kb);
    late();
    load_a(cur_a, kb);
  };
  // c's values at `at` .. added to RUN accumulators, the first n of them
  constexpr int RUN = PERM ? 16 : 4;  // consecutive columns of a lane
  auto add_c = [&](f32x4* v, int64_t at, int n) __attribute__((always_inline)) {
    if (p.c_f32) {
      const float* c = static_cast<const float*>(p.c) + at;
      if (n == RUN && (reinterpret_cast<uintptr_t>(c) & 15) == 0) {
#pragma unroll
        for (int e = 0; e < RUN / 4; ++e) v[e] += *reinterpret_cast<const f32x4*>(c + 4 * e);
      } else {
#pragma unroll
        for (int e = 0; e < RUN; ++e)
          if (e < n) v[e / 4][e & 3] += c[e];
      }
    } else {
      const uint16_t* c = static_cast<const uint16_t*>(p.c) + at;
      if (n == RUN && (reinterpret_cast<uintptr_t>(c) & 7) == 0) {
#pragma unroll
        for (int e = 0; e < RUN / 4; ++e) {
          const i32x2 w = *reinterpret_cast<const i32x2*>(c + 4 * e);
          v[e] += f32x4{__uint_as_float((uint32_t)w[0] << 16), __uint_as_float((uint32_t)w[0] & 0xffff0000u),
                        __uint_as_float((uint32_t)w[1] << 16), __uint_as_float((uint32_t)w[1] & 0xffff0000u)};
        }
      } else {
#pragma unroll
        for (int e = 0; e < RUN; ++e)
          if (e < n) v[e / 4][e & 3] += bf16_to_f32(c[e]);
      }
    }
  };
  // c's first n values of four at `at`, as they are stored (TN)
  auto load_c = [&](int64_t at, int n) __attribute__((always_inline)) {
    i32x4 w = {0, 0, 0, 0};
    if (p.c_f32) {
      const float* c = static_cast<const float*>(p.c) + at;
      if (n >= 4 && (reinterpret_cast<uintptr_t>(c) & 15) == 0) {
        w = *reinterpret_cast<const i32x4*>(c);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < n) w[e] = __float_as_int(c[e]);
      }
    } else {
      const uint16_t* c = static_cast<const uint16_t*>(p.c) + at;
      if (n >= 4 && (reinterpret_cast<uintptr_t>(c) & 7) == 0) {
        const i32x2 t = *reinterpret_cast<const i32x2*>(c);
        w[0] = t[0];
        w[1] = t[1];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < n) w[e / 2] |= (int)((uint32_t)c[e] << (16 * (e & 1)));
      }
    }
    return w;
  };
  auto add_loaded = [&](f32x4& v, const i32x4& w) __attribute__((always_inline)) {
    if (p.c_f32)
      v += f32x4{__int_as_float(w[0]), __int_as_float(w[1]), __int_as_float(w[2]), __int_as_float(w[3])};
    else
      v += f32x4{__uint_as_float((uint32_t)w[0] << 16), __uint_as_float((uint32_t)w[0] & 0xffff0000u),
                 __uint_as_float((uint32_t)w[1] << 16), __uint_as_float((uint32_t)w[1] & 0xffff0000u)};
  };
  // TN: a fragment row goes through LDS of the wave's own, so that the lanes of an instruction hold 4 whole rows of the
  // wave's 64 columns and not 64 bytes of 16 rows (32 gradients of 2048 x 7168 in FP32 over 256 to 1760 rows 1081 us for
  // 1143; exchanged between lanes in registers 1095).  Chunk c of row r lies at slot c ^ r.
  constexpr bool WHOLE = LAY == RAGGED_TN;
  static_assert(T::FN == 4, "16 chunks of four columns a fragment row");
  __shared__ __attribute__((aligned(16))) f32x4 turn[WHOLE ? T::NW * 256 : 1];
  auto whole_rows = [&](f32x4* v, int fr, int q) __attribute__((always_inline)) {
    f32x4* own = turn + wave * 256;
#pragma unroll
    for (int f = 0; f < 4; ++f) own[fr * 16 + ((4 * f + q) ^ fr)] = v[f];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // (a wave's LDS accesses are done in their order)
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int f = 0; f < 4; ++f) v[f] = own[(4 * f + q) * 16 + (fr ^ (4 * f + q))];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  // lane: output row lane % 16 of each fragment row and, PERM, 16 consecutive columns, else 4 of each fragment; TN: 4
  // columns of four rows
  auto store = [&](const Tile& x, int fm) __attribute__((always_inline)) {
    int l = lane;
    asm volatile("" : "+v"(l));  // (what follows from it is formed here: kept, it costs registers that there are not)
    const int fr = l & 15, q = l >> 4;
    const int64_t d_at = LAY == RAGGED_TN ? (int64_t)x.g * p.d_gs : 0, c_at = LAY == RAGGED_TN ? (int64_t)x.g * p.c_gs : 0;
    // TN: c is loaded a fragment row ahead, before the stores of the one at hand, so that its loads do not wait in turn
    // with them: tiles may have few slices (64 of 178 x 3840 over 0 to 7 rows 84 us for 130; 32 of 2048 x 7168 over 256
    // to 1760 1271 to 1317 for 1547; NT and NN, whose tiles have more, lose 2 to 10%).  c may be d: a lane loads what it stores.
    auto c_row = [&](int i, i32x4* w) __attribute__((always_inline)) {
      const int col = x.n0 + wn * T::TN + 4 * fr;
#pragma unroll
      for (int f = 0; f < T::FN; ++f) {
        w[f] = i32x4{0, 0, 0, 0};
        const int row = x.m0 + wm * 16 * fm + 16 * i + 4 * f + q;
        if (row < x.m_end && col < x.n_end) w[f] = load_c(c_at + (int64_t)row * p.ldc + col, x.n_end - col);
      }
    };
    i32x4 cw[T::FN];
    if (WHOLE && p.c != nullptr) c_row(0, cw);
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      if (i >= fm) continue;
      if constexpr (WHOLE) {
        whole_rows(acc[i], fr, q);
        if (p.c != nullptr) {
#pragma unroll
          for (int f = 0; f < T::FN; ++f) add_loaded(acc[i][f], cw[f]);
          if (i + 1 < T::FM) c_row(i + 1, cw);
        }
      }
#pragma unroll
      for (int f0 = 0; f0 < T::FN; f0 += RUN / 4) {
        const int row = x.m0 + wm * 16 * fm + 16 * i + (WHOLE ? 4 * f0 + q : fr);
        if (row >= x.m_end) continue;
        const int col = x.n0 + wn * T::TN + (PERM ? 16 * q : WHOLE ? 4 * fr : 16 * f0 + 4 * q);
        const int n = min(RUN, x.n_end - col);
        if (!WHOLE && p.c != nullptr) add_c(&acc[i][f0], c_at + (int64_t)row * p.ldc + col, n);
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
  };

  int done = 0, t = tile_in(0);
  if (t < 0) return;
  Tile x = find(t);
  load_from(x);
  load_a(lds_a0, 0);
  load_b(lds_b0, 0);
  __builtin_amdgcn_sched_barrier(0);
  load_b(lds_b1, 1);
  load_a(lds_a1, 1);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (S > 2) {
    load_b(lds_b2, 2);
    load_a(lds_a2, 2);
    __builtin_amdgcn_sched_barrier(0);
  }
  meet(std::integral_constant<int, (S - 1) * (A_LD + B_LD)>{});
  // Fragment rows that a wave takes of the tile's own: all of them, or, where the group ends in the tile's first half
  // and A is K-major, half, so that every wave has a part of the rows that there are.
  constexpr bool HALVES = !A_MN && T::FM >= 4;
  auto rows_for = [&](const Tile& x) __attribute__((always_inline)) {
    return HALVES && x.m_end - x.m0 <= T::BM / 2 ? T::FM / 2 : T::FM;
  };
  int fm = rows_for(x);
  if constexpr (!A_MN) a_base = rows_base(wm * 16 * fm + fr, false);
  Frag bf[T::FN], af;
  auto first_frags = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < T::FN; ++f) bf[f] = Frag{b_half(lds_b0, f, 0), b_half(lds_b0, f, 1)};
    af = a_frag(lds_a0, 0);
  };
  first_frags();
  for (;;) {
    done += gridDim.x;
    t = tile_in(done);
    Tile next = {};
    if (t >= 0) next = find(t);
    const int slices = max(1, (KB + S - 1) / S) * S, fm_next = rows_for(next);
    const int a_next = A_MN ? a_base : rows_base(wm * 16 * fm_next + fr, false);
    const bool live = x.m0 + wm * 16 * fm < x.m_end && x.n0 + wn * T::TN < x.n_end;  // else nothing of the wave is stored
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
      for (int f = 0; f < T::FN; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto slice = [&](auto rows, uint8_t* cur_a, uint8_t* cur_b, const uint8_t* nxt_a, const uint8_t* nxt_b, int kb,
                     bool ends) __attribute__((always_inline)) {
      constexpr int FM = decltype(rows)::value;
      // (the fragments' offsets are formed anew each slice: kept, they cost more registers than there are)
      if constexpr (A_MN) asm volatile("" : "+v"(a_base));
      if constexpr (B_MN) asm volatile("" : "+v"(b_base));
      // all fragment rows but the last two, one after the other, each A fragment read a row ahead
      Frag last = af;
      if constexpr (FM == 2) last = a_frag(cur_a, 1);
#pragma unroll
      for (int i = 0; i + 2 < FM; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if (i == 1) early();
        const Frag ahead = a_frag(cur_a, i + 1);
        if (i + 3 == FM) last = a_frag(cur_a, FM - 1);
#pragma unroll
        for (int m = 0; m < 2 * T::FN; ++m) {
          const int f = m % T::FN, h = m / T::FN;
          __builtin_amdgcn_sched_barrier(0);
          acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[f].h[h], af.h[h], acc[i][f], 0, 0, 0);
          if (i == 1) {
#pragma unroll
            for (int j = m * B_LD / (2 * T::FN); j < (m + 1) * B_LD / (2 * T::FN); ++j) load_b_one(cur_b, kb, j);
          }
        }
        af = ahead;
      }
      // the last two together, half of the contraction at a time, so that the next slice's B fragments take the
      // registers as they fall free; where they are all that there is, the early point is before them and the late one
      // between the halves
      constexpr int N2 = 2 * T::FN;  // matrix instructions of a half
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (FM == 2) early();
      else late();
      Frag ahead = af;
      if constexpr (FM > 2) {
        if (ends) a_base = a_next;
        ahead = a_frag(nxt_a, 0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (FM == 2 && h == 1) {
          __builtin_amdgcn_sched_barrier(0);
          late();
          if (ends) a_base = a_next;
          ahead = a_frag(nxt_a, 0);
#pragma unroll
          for (int f = 0; f < T::FN; ++f) bf[f].h[0] = b_half(nxt_b, f, 0);
        }
#pragma unroll
        for (int m = 0; m < N2; ++m) {
          const int f = m / 2, i = FM - 2 + (m & 1);
          __builtin_amdgcn_sched_barrier(0);
          acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[f].h[h], (m & 1) ? last.h[h] : af.h[h], acc[i][f], 0, 0, 0);
          if ((m & 1) && (FM > 2 || h == 1)) bf[f].h[h] = b_half(nxt_b, f, h);
          const int n = FM > 2 ? h * N2 + m : m, of = FM > 2 ? 2 * N2 : N2;
          if (FM == 2 && h == 0) {
#pragma unroll
            for (int j = n * B_LD / of; j < (n + 1) * B_LD / of; ++j) load_b_one(cur_b, kb, j);
          } else {
#pragma unroll
            for (int j = n * A_LD / of; j < (n + 1) * A_LD / of; ++j) load_a_one(cur_a, kb, j);
          }
        }
      }
      af = ahead;
    };
    auto run = [&](auto rows) __attribute__((always_inline)) {
      for (int kb = S; kb <= slices; kb += S) {  // (kb: the slice that the loads are at)
        int at = kb;
        const bool ends = kb == slices;
        if (ends) {  // the next tile's first ones
          load_from(next);
          at = 0;
        }
        slice(rows, lds_a0, lds_b0, lds_a1, lds_b1, at, false);
        if constexpr (S == 2) {
          slice(rows, lds_a1, lds_b1, lds_a0, lds_b0, at + 1, ends);
        } else {
          slice(rows, lds_a1, lds_b1, lds_a2, lds_b2, at + 1, false);
          slice(rows, lds_a2, lds_b2, lds_a0, lds_b0, at + 2, ends);
        }
      }
    };
    if (!live) {
      for (int kb = S; kb <= slices; kb += S) {  // (loads and barriers only)
        int at = kb;
        if (kb == slices) {
          load_from(next);
          at = 0;
        }
        idle(lds_a0, lds_b0, at);
        idle(lds_a1, lds_b1, at + 1);
        if constexpr (S > 2) idle(lds_a2, lds_b2, at + 2);
      }
      a_base = a_next;
      first_frags();
    } else if (!HALVES || fm == T::FM) {
      run(std::integral_constant<int, T::FM>{});
    } else {
      if constexpr (HALVES) run(std::integral_constant<int, T::FM / 2>{});
    }
    if (live) store(x, fm);
    if (t < 0) break;
    x = next;
    fm = fm_next;
  }
  __builtin_amdgcn_s_waitcnt(0);  // (no load may write LDS after the workgroup's end)
}

using Big = Shape<256, 256, 2, 4, 2, 1>;   // 512 threads, wave tile 128 x 64, 2 stages of 64 KB
using Mid = Shape<128, 128, 2, 2, 2, 2>;   // 256 threads, wave tile 64 x 64, 2 stages of 32 KB, two to a compute unit
using Few = Shape<64, 128, 2, 2, 3, 2>;    // 256 threads, wave tile 32 x 64, 3 stages of 24 KB, two to a compute unit

int64_t tiles(int64_t n, int64_t by) { return (n + by - 1) / by; }

// What a tile shape costs: rounds of its workgroups over the machine times the
// time of a slice, in those of Big.  Row tiles: of full ones, and half a tile for
// each group but one, which seldom ends with a tile.
template <class T>
double shape_cost(int layout, int64_t G, int64_t M, int64_t N, int64_t K, double slice) {
  double count;
  if (layout == RAGGED_TN) {
    count = (double)G * (double)tiles(N, T::BM) * (double)tiles(K, T::BN);
  } else {
    const double groups = (double)(G < M ? G : M);
    double rows = (double)M / T::BM + 0.5 * (groups - 1.0);
    if (rows < groups) rows = groups;
    count = rows * (double)tiles(N, T::BN);
  }
  const double slots = CUS * T::PER_CU;
  return (double)(int64_t)((count + slots - 1.0) / slots) * slice;
}

template <class T>
hipError_t launch_shape(RaggedArgs p, int layout, hipStream_t stream) {
  p.tiles_n = (int32_t)tiles(p.N, layout == RAGGED_TN ? T::BM : T::BN);
  p.tiles_k = (int32_t)tiles(p.K, T::BN);
  const int64_t count = layout == RAGGED_TN ? (int64_t)p.G * p.tiles_n * p.tiles_k
                                            : (p.M / T::BM + (p.G < p.M ? p.G : p.M)) * (int64_t)p.tiles_n;
  const int64_t slots = CUS * T::PER_CU;
  const dim3 gr((unsigned)(count < slots ? count : slots)), b(T::NT);
#define DGMI_RAGGED(L_)                                                       \
  do {                                                                        \
    if (p.d_f32) ragged_kernel<T, L_, true><<<gr, b, 0, stream>>>(p);         \
    else ragged_kernel<T, L_, false><<<gr, b, 0, stream>>>(p);                \
  } while (0)
  if (layout == RAGGED_NT) {
    DGMI_RAGGED(RAGGED_NT);
  } else if (layout == RAGGED_NN) {
    DGMI_RAGGED(RAGGED_NN);
  } else if constexpr (T::BM >= 128) {
    DGMI_RAGGED(RAGGED_TN);
  } else {
    return hipErrorInvalidValue;  // (no such plan)
  }
#undef DGMI_RAGGED
  return hipGetLastError();
}

}  // namespace

// Tiles that a call may have to count: with offsets that fall each group may hold all rows.
double ragged_tiles(int layout, int64_t G, int64_t M, int64_t N, int64_t K) {
  if (layout == RAGGED_TN) return (double)G * (double)tiles(N, Mid::BM) * (double)tiles(K, Mid::BN);
  return (double)G * (double)(M / Few::BM + 1) * (double)tiles(N, Few::BN);
}

// Slice times in those of Big, from sweeps of 4 to 8192 rows in 1 to 64 groups
// (32 groups of 4096 x 2048: 8192 rows 160 us with Big, 190 with Mid, 239 with
// Few; 8 of 1024 x 1024: 1024 rows 24, 11 and 9.5; 8 weight gradients of 512 x
// 512, 4096 rows: 27 and 13).
hipError_t launch_ragged(RaggedArgs p, int layout, hipStream_t stream) {
  const double big = shape_cost<Big>(layout, p.G, p.M, p.N, p.K, 1.0), mid = shape_cost<Mid>(layout, p.G, p.M, p.N, p.K, 0.72);
  if (layout != RAGGED_TN) {
    const double few = shape_cost<Few>(layout, p.G, p.M, p.N, p.K, 0.55);
    if (few < big && few < mid) return launch_shape<Few>(p, layout, stream);
  }
  return mid < big ? launch_shape<Mid>(p, layout, stream) : launch_shape<Big>(p, layout, stream);
}

}  // namespace dgmi
