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
typedef __bf16 bf16x4v __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// K-major stage: 16-byte chunk c of tile row r lies at slot c ^ h(r); the 16 rows
// of a fragment read at one chunk then hit distinct banks.
__device__ __host__ constexpr int row_swz(int r) { return ((r ^ (r >> 3)) & 1) | (r & 6); }
// MN-major stage: chunk c of contraction row k lies at slot c ^ hk(k): the four
// rows of each of two lane groups that read together hit distinct banks.
__device__ __host__ constexpr int col_swz(int k) { return 2 * ((k & 3) | ((((k >> 3) ^ (k >> 4)) & 1) << 2)); }

template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
};

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

  // loads of slice kb into a stage, 1024 bytes a wave and instruction.  K-major: 8 tile rows of 128 bytes;
  // the resource ends after the last row that exists, and what lies past it reads as zero.
  auto load_rows = [&](uint8_t* stage, const uint16_t* base, int64_t ld, int rows, int kb, auto tile_rows) {
    constexpr int R = decltype(tile_rows)::value;
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)base, (short)0, (int)(min(max(rows, 0), R) * ld * 2), 0x00020000);
#pragma unroll
    for (int j = 0; j < R / (8 * T::NW); ++j) {
      const int r = (j * T::NW + wave) * 8 + (lane >> 3);
      const uint32_t off = (uint32_t)(r * ld * 2) + (uint32_t)(((lane & 7) ^ row_swz(r)) << 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_t*)(stage + (j * T::NW + wave) * 1024), 16, off,
                                               kb * SLICE * 2, 0, 0);
    }
  };
  // MN-major: SLICE contraction rows of W columns; rows past `len` read as zero (the resource is the slice's own and
  // ends with the 16-byte chunk of the last column of the last row), columns past the operand's feed outputs that
  // are never stored.
  auto load_cols = [&](uint8_t* stage, const uint16_t* base, int64_t ld, int cols, int kb, auto width) {
    constexpr int W = decltype(width)::value, SLOTS = W / 8, PER = 64 / SLOTS;
    const int left = len - kb * SLICE;
    const int64_t bytes = left > 0 && cols > 0 ? ((int64_t)(left - 1) * ld + (cols + 7) / 8 * 8) * 2 : 0;
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + (int64_t)kb * SLICE * ld), (short)0, (int)min(bytes, (int64_t)0x7fffffff), 0x00020000);
#pragma unroll
    for (int j = 0; j < SLICE / (PER * T::NW); ++j) {
      const int k = (j * T::NW + wave) * PER + lane / SLOTS;
      const uint32_t off = (uint32_t)(k * ld * 2) + (uint32_t)(((lane % SLOTS) ^ col_swz(k)) << 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_t*)(stage + (j * T::NW + wave) * 1024), 16, off, 0, 0, 0);
    }
  };
  auto load = [&](uint8_t* sa, uint8_t* sb, int kb) {
    if constexpr (A_MN) load_cols(sa, A, p.lda, m_end - m0, kb, std::integral_constant<int, T::BM>{});
    else load_rows(sa, A, p.lda, m_end - m0, kb, std::integral_constant<int, T::BM>{});
    if constexpr (B_MN) load_cols(sb, B, p.ldb, n_end - n0, kb, std::integral_constant<int, T::BN>{});
    else load_rows(sb, B, p.ldb, n_end - n0, kb, std::integral_constant<int, T::BN>{});
  };

  // fragments: 16 tile rows (columns) at r0, contraction 32 half + 8 (lane / 16) .. +7 in lane (row lane % 16)
  const int fr = lane & 15, q = lane >> 4;
  auto frag_rows = [&](const uint8_t* stage, int r0, int half) {
    const int r = r0 + fr;
    return *reinterpret_cast<const bf16x8*>(stage + r * 128 + (((half * 4 + q) ^ row_swz(r)) << 4));
  };
  // lane s of a group of 16 reads 4 columns of contraction row 8 q + 4 t + s / 4; transposed, the group hands lane
  // s the four rows of column s
  auto frag_cols = [&](const uint8_t* stage, int r0, int half, auto width) {
    constexpr int W = decltype(width)::value;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    union { bf16x8 v; s16x4 h[2]; } u;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int k = half * 32 + 8 * q + 4 * t + (fr >> 2);
      const int chunk = r0 / 8 + ((fr >> 1) & 1);
      u.h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(stage + k * W * 2 + ((chunk ^ col_swz(k)) << 4) + 8 * (fr & 1)));
    }
    return u.v;
  };
  f32x4 acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int f = 0; f < T::FN; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bool live = m0 + wm * T::TM < m_end && n0 + wn * T::TN < n_end;  // else nothing of the wave is stored
  auto compute = [&](const uint8_t* sa, const uint8_t* sb) {
    if (!live) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      bf16x8 bf[T::FN];
#pragma unroll
      for (int f = 0; f < T::FN; ++f) {
        if constexpr (B_MN) bf[f] = frag_cols(sb, wn * T::TN + 16 * f, half, std::integral_constant<int, T::BN>{});
        else bf[f] = frag_rows(sb, wn * T::TN + 16 * f, half);
      }
#pragma unroll
      for (int i = 0; i < T::FM; ++i) {
        bf16x8 af;
        if constexpr (A_MN) af = frag_cols(sa, wm * T::TM + 16 * i, half, std::integral_constant<int, T::BM>{});
        else af = frag_rows(sa, wm * T::TM + 16 * i, half);
#pragma unroll
        for (int f = 0; f < T::FN; ++f) acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[f], af, acc[i][f], 0, 0, 0);
      }
    }
  };
  // every wave's loads have landed and its reads of the other stage are done
  auto ready = [&]() {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
  };
  if (KB > 0) load(lds_a0, lds_b0, 0);
  for (int kb = 0; kb < KB; kb += 2) {
    ready();
    if (kb + 1 < KB) load(lds_a1, lds_b1, kb + 1);
    compute(lds_a0, lds_b0);
    if (kb + 1 < KB) {
      ready();
      if (kb + 2 < KB) load(lds_a0, lds_b0, kb + 2);
      compute(lds_a1, lds_b1);
    }
  }
  if (!live) return;

  // lane: output row lane % 16 and columns 4 (lane / 16) .. +3 of each fragment
  const int64_t d_at = LAY == RAGGED_TN ? (int64_t)g * p.d_gs : 0, c_at = LAY == RAGGED_TN ? (int64_t)g * p.c_gs : 0;
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int row = m0 + wm * T::TM + 16 * i + fr;
    if (row >= m_end) continue;
#pragma unroll
    for (int f = 0; f < T::FN; ++f) {
      const int col = n0 + wn * T::TN + 16 * f + 4 * q;
      f32x4 v = acc[i][f];
      const int n = min(4, n_end - col);
      if (p.c != nullptr) {
        const int64_t at = c_at + (int64_t)row * p.ldc + col;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < n) v[e] += p.c_f32 ? static_cast<const float*>(p.c)[at + e]
                                     : bf16_to_f32(static_cast<const uint16_t*>(p.c)[at + e]);
      }
      const int64_t at = d_at + (int64_t)row * p.ldd + col;
      if constexpr (F32) {
        float* to = static_cast<float*>(p.d) + at;
        if (n == 4 && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
          *reinterpret_cast<f32x4*>(to) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < n) to[e] = v[e];
        }
      } else {
        uint16_t* to = static_cast<uint16_t*>(p.d) + at;
        const i32x2 w = to_bf16x4_bits(v);
        if (n == 4 && (reinterpret_cast<uintptr_t>(to) & 7) == 0) {
          *reinterpret_cast<i32x2*>(to) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < n) to[e] = (uint16_t)((uint32_t)w[e / 2] >> (16 * (e & 1)));
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
