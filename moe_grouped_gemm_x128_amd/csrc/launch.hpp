// Kernel launchers of libdgmi, called by the host-side ABI (abi.cpp) after
// it has validated every argument.  Internal interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace dgmi {

// Quantizer arguments.  x is viewed as [G, R, K] (R = rows, or N for the
// per-block cast); strides in elements.  sf is [G, R or ceil(R/128), ceil(K/128)].
struct QuantArgs {
  const void* x;
  int32_t x_bf16;
  int64_t sx_g, sx_r;
  uint8_t* q;
  int64_t sq_g, sq_r;
  float* sf;
  int64_t ssf_g, ssf_r, ssf_k;
  int32_t G, R, K;
  int32_t ue8m0;
};

// Casts of an MN-major x: element (g, r, k) at x[g * sx_g + k * sx_k + r]
// (sx_r unused); vec: 16-byte (f32) / 8-byte (bf16) loads along r are
// aligned; qvec: q rows take 16-byte stores.
struct QuantTArgs : QuantArgs {
  int64_t sx_k;
  int32_t vec, qvec;
};

// Per-token cast of the tokens x [T, K] (G = 1, R = T) into the rows their
// slots name: slot[t * k + j] = e * max_m + row in [0, rows) selects row
// `row` of group e of q and sf (strides sq_g / sq_r, ssf_g / ssf_r); other
// values are skipped.
struct QuantScatterArgs : QuantArgs {
  const int32_t* slot;
  int32_t k, max_m, rows;
  int32_t flat;  // sq_g == max_m * sq_r and ssf_g == max_m * ssf_r
  int32_t qvec;  // q, sq_r and sq_g are multiples of 16 bytes
};

// MoE routing into the masked layout (moe.hip): topk [T, k] contiguous,
// slot [T, k] contiguous, src [G, max_m] contiguous, masked_m [G].
struct MoeRouteArgs {
  const int32_t* topk;
  int32_t T, k, G, max_m;
  int32_t vec;  // topk is 16-byte aligned: 16-byte loads
  int32_t* masked_m;
  int32_t* slot;
  int32_t* src;
  // contiguous layout: counts [G] (written by the count pass, then read),
  // layout [mcap / 128], capacity mcap rows (a multiple of 128)
  int32_t* counts;
  int32_t* layout;
  int64_t mcap;
  int32_t align;  // region granule in rows: 128 or 256
};

// MoE combine (moe.hip): d BF16 [G, max_m, N] (strides in elements), slot and
// w [T, k] contiguous, y BF16 [T, N] (row stride sy).
struct MoeCombineArgs {
  const uint16_t* d;
  int64_t sd_g, sd_r;
  int32_t G, max_m, N;
  const int32_t* slot;
  const float* w;
  int32_t T, k;
  uint16_t* y;
  int64_t sy;
  int32_t vec, y_vec;  // 16-byte loads of d rows, 16-byte stores of y rows
  int32_t col_blocks;  // set by the launcher
};

// Expert routing (route.hip): logits [T, E] (row stride sl, FP32 or BF16),
// bias [E] or NULL, idx and w [T, k] (row strides si, sw).
struct RouteTopkArgs {
  const void* logits;
  int64_t sl;
  int32_t bf16;
  const float* bias;
  int32_t* idx;
  int64_t si;
  float* w;
  int64_t sw;
  int32_t T, E, k;
  int32_t n_group, group_size, topk_group, group_top;
  int32_t softmax, renorm;
  float scale;
  // set by the launcher: log2 of a group's lanes, 16-byte loads
  int32_t log_l, vec, vec_bias;
};

struct RouteTopkBwdArgs {
  const void* logits;
  int64_t sl;
  int32_t bf16;
  const int32_t* idx;
  int64_t si;
  const float* g;
  int64_t sg;
  void* dlogits;
  int64_t so;
  int32_t out_bf16;
  int32_t T, E, k;
  int32_t softmax, renorm;
  float scale;
  int32_t vec, vec_out;  // set by the launcher
};

// Append to the paged FP8 cache (kvcache.hip): k, v [T, Hkv, D], q and q_out
// [T, Hq, D], caches [pages, Hkv, P, D], scales [pages, Hkv], table
// [S, max_pages], cu [S + 1], start [S], cos_sin [positions, rot].
struct KvAppendArgs {
  const void *k, *v, *q;
  int32_t bf16;
  int64_t sk_t, sk_h, sv_t, sv_h, sq_t, sq_h;
  uint16_t* q_out;
  int64_t so_t, so_h;
  const float* cos_sin;
  int64_t s_cs;
  int32_t rot, interleaved;
  int64_t positions;
  uint8_t *k_cache, *v_cache;
  int64_t skc_p, skc_h, skc_t, svc_p, svc_h, svc_t;
  float *k_scale, *v_scale;
  int64_t sks_p, sks_h, svs_p, svs_h;
  const int32_t* table;
  int64_t s_table;
  int32_t max_pages, pages;
  const int32_t *cu, *start;
  int32_t T, S, Hkv, Hq, D, P;
  // set by the launcher: workgroups before those of q, workgroups of a page
  // slot, kinds (a head's K or V) of a workgroup, tokens of q of a workgroup,
  // one slot per token (else per page), log2 P
  int64_t kv_blocks;
  int32_t kind_blocks, kinds, q_tokens, by_token, log_p;
};

struct KvAppendPlan {
  int64_t grid, kv_blocks, kind_blocks, kinds, q_tokens;
  bool by_token;
};

// Attention over the paged FP8 cache (attn.hip): q and out [S, n, Hq, D],
// lse [S, n, Hq] or NULL; rows = n * group, row_tiles = ceil(rows / 16).
struct PagedAttnArgs {
  const uint16_t* q;
  int64_t sq_s, sq_n, sq_h;
  uint16_t* out;
  int64_t so_s, so_n, so_h;
  float* lse;
  int64_t sl_s, sl_n, sl_h;
  const uint8_t *k_cache, *v_cache;
  int64_t skc_h, svc_h;
  uint32_t skc_p, skc_t, svc_p, svc_t;
  const float *k_scale, *v_scale;
  int64_t sks_h, svs_h;
  uint32_t sks_p, svs_p;  // bytes
  const int32_t* table;
  int64_t s_table;
  const int32_t* lens;
  int32_t S, n, Hkv, group, rows, row_tiles, D, P, max_pages, pages, window;
  float scale;
  float* workspace;
  // set by the launcher: row tiles of a unit, waves that take them side by
  // side, units (KV head, group of row tiles) per sequence, groups per head,
  // workgroups of the first kernel, what all tiles are divided by for a share's
  // size (with two workgroups a compute unit, and with one), what the size is a
  // multiple of, rows per workgroup of the join, log2 P; a share is of one unit
  int32_t rt, wr, units, groups, shares, cuts, cuts_one, min_share, rps, log_p;
  bool whole;
};

// Root-mean-square norm (norm.hip) of `rows` rows, row i at index (i / heads,
// i % heads) of each tensor; strides in elements, *_vec: rows start on 16 bytes
// (q: on 8).
struct RmsNormArgs {
  const void *x, *res, *w;
  void *h, *y;
  uint8_t* q;
  float* sf;
  int64_t sx_0, sx_1, sr_0, sr_1, sh_0, sh_1, sy_0, sy_1, sq_0, sq_1, ss_0, ss_1, ss_k;
  int64_t rows, heads;
  int32_t H;
  int32_t x_bf16, r_bf16, w_bf16, y_bf16;  // h has the residual's type
  int32_t x_vec, r_vec, w_vec, h_vec, y_vec, q_vec;
  int32_t ue8m0;
  float eps;
};

struct RmsNormBwdArgs {
  const void *dy, *h, *w, *dh;
  void* dx;
  void* dw;     // or NULL
  float* part;  // rms_norm_bwd_parts rows of H, NULL without dw
  int64_t sg_0, sg_1, sh_0, sh_1, sd_0, sd_1, sx_0, sx_1;
  int64_t rows, heads;
  int32_t H;
  int32_t dy_bf16, h_bf16, w_bf16, dh_bf16, dx_bf16, dw_bf16;
  int32_t dy_vec, h_vec, w_vec, dh_vec, dx_vec;
  float eps;
};

// Gated activation (swiglu.hip): x [G, R, 2I], y, q and dy [G, R, I]; masked [G]
// or NULL, w [G R] or NULL.
struct SwigluArgs {
  const void* x;
  const int32_t* masked;
  const float* w;
  void* y;
  uint8_t* q;
  float* sf;
  int64_t sx_g, sx_r, sy_g, sy_r, sq_g, sq_r, ss_g, ss_r, ss_k, sw;
  int32_t G, R, I;
  int32_t x_bf16, y_bf16, x_vec, u_vec, y_vec, q_vec, ue8m0;
};

struct SwigluBwdArgs {
  const void *x, *dy;
  const int32_t* masked;
  const float* w;
  void* dx;
  float* dw;
  int64_t sx_g, sx_r, sy_g, sy_r, sd_g, sd_r, sw, sdw;
  int32_t G, R, I;
  int32_t x_bf16, dy_bf16, dx_bf16, x_vec, u_vec, dy_vec, dx_vec, du_vec;
};

// BF16 products grouped by ragged offsets (ragged.hip).  Strides in elements,
// gs between groups.  Rows of the operands run along the group's tokens (a of
// nt and nn, both operands of tn) or the group's own matrix (b of nt and nn).
struct RaggedArgs {
  const uint16_t *a, *b;
  void* d;
  const void* c;  // or NULL
  const int32_t* offsets;
  int64_t lda, ldb, b_gs, ldd, d_gs, ldc, c_gs;
  int32_t G, M, N, K;  // nt, nn: d [M, N], contraction K; tn: M tokens, d [G, K, N]
  int32_t c_f32, d_f32;
  int32_t tiles_n, tiles_k;  // set by the launcher
};

enum RaggedLayout : int { RAGGED_NT = 0, RAGGED_NN = 1, RAGGED_TN = 2 };

struct PackArgs {
  const float* x;
  int64_t sx_g, sx_r;
  int32_t* out;
  int64_t so_g, so_r;
  int32_t G, R, n, nw;
  int32_t* invalid;
};

// Tile configuration of a GEMM launch (a pure function of the shapes).
struct TileCfg {
  int bm, bn, threads, lds_bytes;
  int variant;  // index of the kernel instance
};

hipError_t launch_per_token(const QuantArgs& p, hipStream_t stream);
hipError_t launch_per_token_scatter(const QuantScatterArgs& p, hipStream_t stream);
hipError_t launch_cast_mn(const QuantTArgs& p, bool per_block, hipStream_t stream);
hipError_t launch_moe_route(const MoeRouteArgs& p, hipStream_t stream);
hipError_t launch_moe_route_contiguous(const MoeRouteArgs& p, hipStream_t stream);
hipError_t launch_moe_combine(const MoeCombineArgs& p, hipStream_t stream);
hipError_t launch_moe_route_topk(RouteTopkArgs p, hipStream_t stream);
hipError_t launch_moe_route_topk_bwd(RouteTopkBwdArgs p, hipStream_t stream);
KvAppendPlan kv_append_plan(int64_t T, int64_t S, int64_t P, int64_t Hkv, int64_t D, bool q);
hipError_t launch_kv_append(KvAppendArgs p, hipStream_t stream);
int64_t paged_attention_workspace(int64_t S, int64_t n, int64_t Hq, int64_t Hkv, int64_t D, int64_t cap);
// largest grid of the call's kernels
int64_t paged_attention_grid(int64_t S, int64_t Hkv, int64_t row_tiles, int64_t D, int64_t cap);
hipError_t launch_paged_attention(PagedAttnArgs p, hipStream_t stream);
int64_t rms_norm_max_rows(int64_t H);
int64_t rms_norm_bwd_parts(int64_t rows, int64_t H);
hipError_t launch_rms_norm(const RmsNormArgs& p, hipStream_t stream);
hipError_t launch_rms_norm_bwd(const RmsNormBwdArgs& p, hipStream_t stream);
int64_t swiglu_grid(int64_t rows, int64_t I);
int64_t swiglu_bwd_grid(int64_t rows, int64_t I);
hipError_t launch_swiglu(const SwigluArgs& p, hipStream_t stream);
hipError_t launch_swiglu_bwd(const SwigluBwdArgs& p, hipStream_t stream);
// tiles of a call at most (a kernel counts them in 31 bits)
double ragged_tiles(int layout, int64_t G, int64_t M, int64_t N, int64_t K);
hipError_t launch_ragged(RaggedArgs p, int layout, hipStream_t stream);
hipError_t launch_per_block(const QuantArgs& p, hipStream_t stream);
hipError_t launch_pack_ue8m0(const PackArgs& p, hipStream_t stream);

// Launch plan of a GEMM: one launch over all N columns, or two launches on
// the same stream, cfg[0] over columns [0, n_split) and cfg[1] over
// [n_split, N) (n_split a multiple of 256).
struct GemmPlan {
  TileCfg cfg[2];
  int64_t n_split;
  int parts;
};

// Contiguous layouts of more 128-row blocks than this take 128-row tiles: the
// 256-row tiles list their tile starts in LDS (4 bytes a block).
constexpr int64_t RUNS_MAX_BLOCKS = 8192;

// GEMMs: the plan for (mode, G, M, N, K) and the grid of each launch (pure
// functions of the shapes), and the launchers.
GemmPlan fp8_gemm_plan(int mode, int64_t G, int64_t M, int64_t N, int64_t K, int sf_fmt);
GemmPlan bf16_gemm_plan(int mode, int64_t G, int64_t M, int64_t N, int64_t K);
int64_t gemm_grid(const TileCfg& cfg, int mode, int64_t G, int64_t M, int64_t N);
int64_t plan_grid(const GemmPlan& plan, int part, int mode, int64_t G, int64_t M, int64_t N);
// static LDS of one workgroup of launch `part` (0 past the plan's launches)
int plan_lds(const GemmPlan& plan, int part, int mode);
// sf_fmt: SF_F32 or SF_UE8M0, plus SF_ROWB for one B scale per row of B;
// an MN-major A or B (p.a_mn, p.b_mn: dense, block scales, BF16 d) takes the
// plan of fp8_mn_gemm_plan
hipError_t launch_fp8_gemm(GemmParams p, int mode, int sf_fmt, hipStream_t stream);
GemmPlan fp8_mn_gemm_plan();
// Dense FP8 GEMM whose output D is cast per token to FP8 (p.q, p.sfq) in the
// epilogue; sf_fmt SF_F32 or SF_UE8M0, plus SF_ROWB for one B scale per row.
GemmPlan fp8_out_gemm_plan(int64_t M, int64_t N, int sf_fmt);
hipError_t launch_fp8_gemm_fp8_out(GemmParams p, int sf_fmt, hipStream_t stream);
// BF16 GEMMs: same kernel body; byte strides in p, no scales
hipError_t launch_bf16_gemm(GemmParams p, int mode, hipStream_t stream);

}  // namespace dgmi
