/*
 * dgmi.h -- C ABI of the block-scaled FP8 (grouped) GEMM library for MI355X.
 *
 * The library (libdgmi.so) computes DeepGEMM-style FP8 GEMMs with
 * fine-grained scaling on gfx950: E4M3 operands, one FP32 scale per 1x128
 * K-block of each activation row and one per 128x128 block of the weights
 * (or the same scales as power-of-two UE8M0 exponents packed four to an
 * int32), each 128-wide K-block contracted on the matrix cores and promoted
 * into an FP32 accumulator multiplied by both scales, BF16 out.
 *   "DeepInside DeepGEMM: Unpacking DeepSeek's Unified Tensor Core Library
 *    for SM90 and SM100", section 2 (NT layout, FP32 or packed UE8M0 scale
 *    factors) and section 4 (fp8_gemm_nt(a, b, a_sf, b_sf, c, bf16)).
 * Around them: casts, the MoE steps (choice of experts, dispatch, combine),
 * a paged FP8 key/value cache with the attention over it, and what a layer is
 * trained with: norm and activation with their gradients, BF16 products of
 * ragged groups.
 *
 * Conventions shared by every entry point
 *   - Every buffer is device memory allocated and owned by the caller,
 *     outputs included.  The library never allocates, frees, synchronises,
 *     reads device memory on the host, or keeps a pointer after returning
 *     ("DeepGEMM CUDA Graph Compatibility for Masked Grouped GEMMs",
 *     sections "Eliminating Host-Side Allocation" and "Tensor-Based
 *     Metadata Arguments").
 *   - Each call validates shapes/dtypes/strides on the host, then enqueues
 *     its kernels on `stream` (NULL = the null stream) and returns.  The
 *     launch configuration depends only on the shapes, never on device
 *     data, so every entry point except dgmi_init may be captured into a
 *     hipGraph and replayed (same page, section "Stateless Kernel
 *     Architecture").  Device faults surface at the caller's next sync.
 *   - Tensors are described by dg_tensor: shape and strides in ELEMENTS.
 *     The innermost (last) stride of every data operand must be 1.
 *   - On error nothing is launched, the call returns a non-zero status and
 *     dg_last_error() describes it.  Calls are reentrant and thread-safe.
 */
#ifndef DGMI_H
#define DGMI_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
enum {
  DG_F32 = 0,  /* IEEE binary32 */
  DG_BF16 = 1, /* bfloat16 */
  DG_E4M3 = 2, /* OCP FP8 E4M3 ("fn": max 448, no inf), one byte */
  DG_I32 = 3   /* int32: masked_m, grouped_layout, packed UE8M0 scales */
};

/* status codes */
enum {
  DG_OK = 0,
  DG_INVALID_ARG = 1,   /* null / dtype / ndim / shape / stride / alignment / aliasing */
  DG_UNSUPPORTED = 2,   /* legal but not implemented (K % 128 != 0; GEMM operand row strides of 8 MiB or more;
                         * more experts, head sizes or lengths than a kernel takes: see each call) */
  DG_LAUNCH_FAILED = 3  /* the HIP runtime rejected a launch */
};

typedef struct dg_tensor {
  void* data;        /* device pointer, caller-owned */
  int32_t dtype;     /* DG_* element type */
  int32_t ndim;      /* 1..4 */
  int64_t shape[4];
  int64_t stride[4]; /* in elements */
} dg_tensor;

/* Message for the last non-zero status returned on this thread. */
const char* dg_last_error(void);

/* Optional eager set-up (checks that a gfx950 device is current).  Not
 * capture-safe; every other entry point works without calling it. */
int dgmi_init(void);

/*
 * D = A . B^T, block-scaled FP8, BF16 out ("DeepInside DeepGEMM", section 4:
 * the NT GEMM fp8_gemm_nt with D = C + A @ B.T).
 *   a   E4M3 [M, K]          row stride lda (elements = bytes), 16-B aligned
 *   b   E4M3 [N, K]          weights in NT layout (K contiguous)
 *   sfa F32  [M, K/128]      any strides (K-major or M-major), or
 *       I32  [M, ceil(K/512)] packed UE8M0 (byte j of word i: K-block 4i+j)
 *   sfb F32  [ceil(N/128), K/128] or I32 [ceil(N/128), ceil(K/512)]: one
 *       scale per 128x128 block of B; or F32 [N, K/128] or I32
 *       [N, ceil(K/512)]: one scale per row of B (the per-row b_sf of the
 *       section's example), told apart by the row count (for N = 1 the two
 *       forms are the same).  sfa and sfb must use the same format.
 *   c   NULL, or the accumulate input C: BF16 or F32 [M, N], any row stride
 *       (innermost stride 1), element-aligned; it may be d itself (same base,
 *       dtype and strides: an in-place D += A . B^T), any other overlap with d
 *       is rejected.  Each element of C is added to the FP32 accumulator
 *       before the BF16 rounding (same section: D = C + A @ B.T).
 *   d   BF16 [M, N], any row stride (innermost stride 1); or F32 [M, N],
 *       4-B aligned: the FP32 accumulator (C added) stored without rounding
 *       (the section's call takes the output dtype as an argument); with
 *       c = d in F32 this is the in-place D += A . B^T.  Either scale form
 *       of B goes with either output dtype.
 * D[m,n] = C[m,n] + sum_kb (sum_{k in kb} A[m,k] B[n,k]) * sfa[m,kb] * sfb[n/128,kb]
 * (sfb[n,kb] with one scale per row of B).
 * K must be a multiple of 128; M and N are arbitrary.
 * a or b may also be MN-major: the transposed view ([M, K] with strides
 * (1, lda)) of a row-major [K, M] tensor, likewise b of a [K, N] one -- the
 * layouts of fp8_gemm_nn / _tn / _tt below, with their conditions.
 */
int fp8_gemm_nt(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa,
                const dg_tensor* sfb, const dg_tensor* c, const dg_tensor* d,
                hipStream_t stream);

/*
 * The NN, TN and TT layouts of the same GEMM ("DeepInside DeepGEMM", section
 * 2: besides NT, the NN, TN and TT layouts of the FP8 GEMM), for operands
 * already in FP8 and stored MN-major.  The first letter is A's layout, the
 * second B's, read as D = op(A) . op(B):
 *   fp8_gemm_nn  a E4M3 [M, K] (K contiguous),  b E4M3 [K, N] (N contiguous)
 *   fp8_gemm_tn  a E4M3 [K, M] (M contiguous),  b E4M3 [K, N]
 *   fp8_gemm_tt  a E4M3 [K, M],                 b E4M3 [N, K] (K contiguous)
 * so D[m,n] = C[m,n] + sum_kb (sum_{k in kb} A[m,k] B[n,k]) sfa[m,kb] sfb[n/128,kb]
 * (sfb[n,kb] with one scale per row of B) with A[m,k] and B[n,k] read from
 * the stored layouts.  sfa, sfb, c and d as for fp8_gemm_nt (sfa is
 * [M, K/128], sfb [ceil(N/128), K/128] or [N, K/128] whatever the operands'
 * layout).  An MN-major operand is row-major in its stored shape,
 * with a 16-byte aligned base and a K-row stride (bytes) that is a multiple
 * of 16, at least its row count, and small enough that K x stride < 2^31 - 256
 * (the operand is addressed with 32-bit offsets); its row count (M or N) must
 * be a multiple of 16
 * (else DG_UNSUPPORTED).  Either scale form of B (one per 128x128 block or
 * one per row), FP32 or packed UE8M0; BF16 or F32 d.  The fragments of an
 * MN-major operand are read from LDS with transposing loads; results equal
 * fp8_gemm_nt's on the same values bit for bit.
 */
int fp8_gemm_nn(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                const dg_tensor* c, const dg_tensor* d, hipStream_t stream);
int fp8_gemm_tn(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                const dg_tensor* c, const dg_tensor* d, hipStream_t stream);
int fp8_gemm_tt(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                const dg_tensor* c, const dg_tensor* d, hipStream_t stream);

/*
 * fp8_gemm_nt with its output cast to FP8 in the same kernel ("DeepInside
 * DeepGEMM", section 5: FP8 casting done by separate helpers costs HBM
 * bandwidth, and belongs in the kernel that produces the tensor): D is
 * formed and rounded to BF16 as by fp8_gemm_nt (C added first), then cast
 * per token exactly as per_token_cast_to_fp8 casts that BF16 tensor, so q
 * and sfq are bit-identical to fp8_gemm_nt followed by per_token_cast_to_fp8
 * with the same use_ue8m0.  The BF16 D is never written to memory.
 *   a, b, sfa, sfb, c  as fp8_gemm_nt (sfb one scale per 128x128 block of B
 *       or one per row of B)
 *   q   E4M3 [M, N], any row stride that is a multiple of 4 (innermost
 *       stride 1), 4-B aligned base; must not overlap any input
 *   sfq F32 [M, ceil(N/128)], any strides, 4-B aligned: the scale of each
 *       1x128 block of D (amax/448 floored as for per_token_cast_to_fp8;
 *       with use_ue8m0 rounded up to a power of two)
 * K must be a multiple of 128; M and N are arbitrary.
 */
int fp8_gemm_nt_fp8_out(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa,
                        const dg_tensor* sfb, const dg_tensor* c, const dg_tensor* q,
                        const dg_tensor* sfq, int use_ue8m0, hipStream_t stream);

/*
 * Contiguous grouped FP8 GEMM: groups concatenated along M ("DeepGEMM tested
 * by Novita AI", section on the contiguous layout for prefill / training).
 *   a   E4M3 [Msum, K], Msum % 128 == 0
 *   b   E4M3 [G, N, K]
 *   sfa as fp8_gemm_nt with M = Msum;  sfb [G, ceil(N/128), ...] or, one
 *       per row of B, [G, N, ...]
 *   d   BF16 [Msum, N], or F32 [Msum, N] (4-B aligned): the FP32
 *       accumulator stored without rounding
 *   grouped_layout I32 [Msum/128] on the device: group id of each 128-row
 *       block; a negative id marks a block to skip (its rows of d are not
 *       written).  Ids >= G are treated as skipped as well.
 */
int m_grouped_fp8_gemm_nt_contiguous(const dg_tensor* a, const dg_tensor* b,
                                     const dg_tensor* sfa, const dg_tensor* sfb,
                                     const dg_tensor* d, const dg_tensor* grouped_layout,
                                     hipStream_t stream);

/*
 * Masked grouped FP8 GEMM for MoE decode ("DeepGEMM CUDA Graph Compatibility
 * for Masked Grouped GEMMs", section "Tensor-Based Metadata Arguments").
 *   a   E4M3 [G, max_m, K] (or [G*max_m, K])
 *   b   E4M3 [G, N, K]
 *   sfa F32 [G, max_m, K/128] (or [G*max_m, K/128]) or packed I32
 *   sfb F32 [G, ceil(N/128), K/128] or packed I32 (or one per row of B:
 *       [G, N, ...])
 *   d   BF16 [G, max_m, N] (or [G*max_m, N]), or F32 of that shape (4-B
 *       aligned): the FP32 accumulator stored without rounding
 *   masked_m I32 [G] on the device: group g computes its first
 *       clamp(masked_m[g], 0, max_m) rows; every other row of d is left
 *       untouched.  Read only by the kernels, never by the host.
 *   max_m_per_group  rows per group of the padded buffers (fixes the grid).
 */
int m_grouped_fp8_gemm_nt_masked(const dg_tensor* a, const dg_tensor* b,
                                 const dg_tensor* sfa, const dg_tensor* sfb,
                                 const dg_tensor* d, const dg_tensor* masked_m,
                                 int64_t max_m_per_group, hipStream_t stream);

/*
 * The two grouped FP8 GEMMs in the accumulate form D = C + A . B^T of
 * fp8_gemm_nt ("DeepInside DeepGEMM", section 4), the other arguments as
 * above.  c is BF16 or F32 with d's shape ([Msum, N]; [G, max_m, N] or
 * [G*max_m, N]), innermost stride 1, element-aligned; each element of C is
 * added to the FP32 accumulator before d is rounded (BF16) or stored (F32).
 * c may be d itself (same base, dtype and strides: an in-place D += A . B^T);
 * any other overlap with d is rejected.  Rows that are not computed (skipped
 * blocks, rows past masked_m) are neither read from c nor written to d.
 */
int m_grouped_fp8_gemm_nt_contiguous_acc(const dg_tensor* a, const dg_tensor* b,
                                         const dg_tensor* sfa, const dg_tensor* sfb,
                                         const dg_tensor* c, const dg_tensor* d,
                                         const dg_tensor* grouped_layout, hipStream_t stream);
int m_grouped_fp8_gemm_nt_masked_acc(const dg_tensor* a, const dg_tensor* b,
                                     const dg_tensor* sfa, const dg_tensor* sfb,
                                     const dg_tensor* c, const dg_tensor* d,
                                     const dg_tensor* masked_m, int64_t max_m_per_group,
                                     hipStream_t stream);

/*
 * Masked grouped BF16 GEMM, argument order of the pages' capture example
 * (a, b, d, masked_m, max_m_per_group): D[g,m,:] = A[g,m,:] . B[g]^T for
 * m < clamp(masked_m[g], 0, max_m), FP32 accumulation, BF16 out.
 *   a BF16 [G, max_m, K] or [G*max_m, K]; b BF16 [G, N, K]; d like a with N,
 *   BF16, or F32 (4-B aligned: the FP32 accumulator stored without rounding).
 *   Rows past masked_m are not written.  K must be a multiple of 64.
 */
int m_grouped_bf16_gemm_nt_masked(const dg_tensor* a, const dg_tensor* b,
                                  const dg_tensor* d, const dg_tensor* masked_m,
                                  int64_t max_m_per_group, hipStream_t stream);

/*
 * Dense BF16 GEMM D = C + A . B^T: the BF16 GEMM primitive ("DeepGEMM: Why
 * DeepSeek Built Its Own BLAS Kernels", its table of primitives) in the NT
 * layout and accumulate form of fp8_gemm_nt, FP32 accumulation, BF16 out.
 *   a BF16 [M, K], b BF16 [N, K] (row strides multiples of 8 elements,
 *   16-B aligned bases); c NULL or BF16/F32 [M, N] as for fp8_gemm_nt (may be
 *   d itself); d BF16 [M, N] or F32 [M, N] (4-B aligned, the FP32 accumulator
 *   stored as is), any row stride.  K must be a multiple of 64.
 */
int bf16_gemm_nt(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c, const dg_tensor* d,
                 hipStream_t stream);

/*
 * Contiguous grouped BF16 GEMM: the layout of m_grouped_fp8_gemm_nt_contiguous
 * without scales.
 *   a BF16 [Msum, K] (Msum % 128 == 0), b BF16 [G, N, K], d BF16 [Msum, N]
 *   or F32 [Msum, N] (4-B aligned: the FP32 accumulator stored without rounding)
 *   grouped_layout I32 [Msum/128]: group id per 128-row block; negative ids
 *   (and ids >= G) skip the block, its rows of d are not written.
 *   K must be a multiple of 64.
 */
int m_grouped_bf16_gemm_nt_contiguous(const dg_tensor* a, const dg_tensor* b, const dg_tensor* d,
                                      const dg_tensor* grouped_layout, hipStream_t stream);

/*
 * The two grouped BF16 GEMMs in the accumulate form D = C + A . B^T of
 * bf16_gemm_nt (the accumulate form of fp8_gemm_nt, "DeepInside DeepGEMM",
 * section 4), the other arguments as above.  c is BF16 or F32 with d's
 * shape ([Msum, N]; [G, max_m, N] or [G*max_m, N]), innermost stride 1,
 * element-aligned; each element of C is added to the FP32 accumulator before
 * d is rounded (BF16) or stored (F32).  c may be d itself (same base, dtype
 * and strides: an in-place D += A . B^T); any other overlap with d is
 * rejected.  Rows that are not computed (skipped blocks, rows past masked_m)
 * are neither read from c nor written to d.
 */
int m_grouped_bf16_gemm_nt_contiguous_acc(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c,
                                          const dg_tensor* d, const dg_tensor* grouped_layout, hipStream_t stream);
int m_grouped_bf16_gemm_nt_masked_acc(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c,
                                      const dg_tensor* d, const dg_tensor* masked_m, int64_t max_m_per_group,
                                      hipStream_t stream);

/*
 * Per-token FP8 cast: each row of x cut into 1x128 blocks along K; block
 * scale s = amax/448 (amax floored at 1e-4; with use_ue8m0 rounded up to a
 * power of two), q = e4m3(x/s) rounded to nearest even after clamping to
 * +-448 ("DeepInside DeepGEMM", section 5: the FP8 casting helpers).
 *   x  F32 or BF16 [R, K] or [G, R, K]: K-major (innermost stride 1, 16-B
 *      aligned rows), or MN-major (stride 1 along R: the transpose of a
 *      row-major [K, R] tensor, e.g. an activation kept [K, M] for the TN
 *      GEMM), read through a transposing LDS tile ("DeepInside DeepGEMM",
 *      section 5: transposition and casting fused into the producer)
 *   q  E4M3 same shape, K-major: the operand layout of the NT GEMMs
 *   sf F32 [R, ceil(K/128)] (or [G, R, ...]) with any strides
 * The bytes do not depend on the layout of x.
 */
int per_token_cast_to_fp8(const dg_tensor* x, const dg_tensor* q, const dg_tensor* sf,
                          int use_ue8m0, hipStream_t stream);

/*
 * Per-block FP8 cast over 128x128 blocks (weights): as per_token_cast_to_fp8
 * with one scale per block.
 *   x  F32 or BF16 [N, K] or [G, N, K], K-major or MN-major as for
 *      per_token_cast_to_fp8 (a weight kept [K, N] for the NN / TT GEMMs);
 *      q E4M3 same shape, K-major
 *   sf F32 [ceil(N/128), ceil(K/128)] or [G, ...] with any strides
 */
int per_block_cast_to_fp8(const dg_tensor* x, const dg_tensor* q, const dg_tensor* sf,
                          int use_ue8m0, hipStream_t stream);

/*
 * Pack FP32 power-of-two scales into UE8M0 bytes, four per int32 ("[GH-ISSUE
 * #414] pack_ue8m0_to_int is not CUDA Graph capture safe", section "Expected
 * behavior"): byte j of out[..., i] = bits 30..23 of x[..., 4i+j]; missing
 * tail elements give zero bytes.  Shape and dtype checks stay on the host;
 * the value check of the issue's Summary (x >= 0 with a zero mantissa) is
 * done on the device without any host synchronisation: when invalid_count
 * is not NULL, the number of offending elements is ADDED to the int32 it
 * points to (device memory; the caller zeroes it).
 *   x   F32 [..., n] (1 to 3 dims, innermost stride 1)
 *   out I32 [..., ceil(n/4)] same leading shape
 */
int pack_ue8m0_to_int(const dg_tensor* x, const dg_tensor* out, int32_t* invalid_count,
                      hipStream_t stream);

/*
 * MoE dispatch into the masked layout, with the per-token FP8 cast of the
 * routed tokens ("DeepGEMM tested by Novita AI", decode section: each expert
 * owns a padded buffer of max_m rows of which masked_m[e] are valid;
 * "DeepGEMM CUDA Graph Compatibility for Masked Grouped GEMMs", last
 * section: the fused MoE path chains the input casting and the masked GEMM
 * calls; "DeepInside DeepGEMM", section 5: the cast done where the tensor
 * is produced).  Two kernels on `stream`, no allocation, no host sync.
 *   x        F32 or BF16 [T, K] tokens (16-B aligned base and row stride)
 *   topk_idx I32 [T, k] contiguous: the expert of each (token, choice); ids
 *            outside [0, G) route nowhere
 *   a        E4M3 [G, max_m, K] out (4-B aligned rows): row r of expert e is
 *            its r-th routed token, cast as per_token_cast_to_fp8 casts it;
 *            rows >= masked_m[e] are left untouched
 *   sfa      F32 [G, max_m, ceil(K/128)] out, any strides: its scales
 *   masked_m I32 [G] out: min(tokens routed to e, max_m)
 *   slot     I32 [T, k] out, contiguous: e * max_m + r where (t, j) landed,
 *            -1 if routed nowhere or dropped
 *   src      I32 [G, max_m] out, contiguous: the token of each row (rows <
 *            masked_m[e] only)
 * Pairs routed to an expert take its rows in row-major (t, j) order; those
 * beyond max_m rows are dropped (slot -1).  The outputs feed
 * m_grouped_fp8_gemm_nt_masked (a, sfa, masked_m, max_m) and moe_combine
 * (slot).  G * max_m and T * k must fit in int32 (else DG_UNSUPPORTED).
 */
int moe_dispatch_masked_fp8(const dg_tensor* x, const dg_tensor* topk_idx, const dg_tensor* a,
                            const dg_tensor* sfa, const dg_tensor* masked_m, const dg_tensor* slot,
                            const dg_tensor* src, int use_ue8m0, hipStream_t stream);

/*
 * MoE dispatch into the contiguous layout of m_grouped_fp8_gemm_nt_contiguous
 * (prefill: "DeepGEMM tested by Novita AI", contiguous layout, groups
 * concatenated along M in 128-row blocks with a group id per block), with
 * the per-token FP8 cast of the routed tokens as in moe_dispatch_masked_fp8.
 * Three kernels on `stream` (count, place, cast), no allocation, no host sync.
 *   x, topk_idx     as moe_dispatch_masked_fp8
 *   a               E4M3 [Mcap, K] out (Mcap % 128 == 0, 4-B aligned rows):
 *                   expert e's routed tokens fill a region of
 *                   ceil(count_e / align) * align rows, regions in expert
 *                   order, tokens in row-major (t, j) order; the rows of a
 *                   region past count_e are padding and left untouched
 *   sfa             F32 [Mcap, ceil(K/128)] out, any strides: their scales
 *   grouped_layout  I32 [Mcap/128] out: e for the blocks of e's region, -1
 *                   for the blocks past the last region
 *   counts          I32 [G] out: pairs routed to each expert
 *   slot            I32 [T, k] out, contiguous: the row of a where (t, j)
 *                   landed, -1 if routed nowhere or past the capacity Mcap
 *   align           128 (whole blocks), or 256 (whole 256-row tiles of the
 *                   contiguous GEMM: no region then ends in a one-block
 *                   tile, at the cost of more padding rows)
 * Mcap >= T * k + (align - 1) * G holds every routing.  The outputs feed
 * m_grouped_fp8_gemm_nt_contiguous (a, sfa, grouped_layout) and moe_combine
 * (slot, with the GEMM's [Mcap, N] output viewed as [1, Mcap, N]).
 */
int moe_dispatch_contiguous_fp8(const dg_tensor* x, const dg_tensor* topk_idx, const dg_tensor* a,
                                const dg_tensor* sfa, const dg_tensor* grouped_layout,
                                const dg_tensor* counts, const dg_tensor* slot, int32_t align,
                                int use_ue8m0, hipStream_t stream);

/*
 * MoE combine: y[t] = sum over j of topk_weights[t, j] * d[slot[t, j]], the
 * rows of the masked GEMM's output picked by moe_dispatch_masked_fp8's slot
 * table; slots outside [0, G * max_m) (not routed, dropped) add nothing.
 * FP32 sum in increasing j, one FMA per term, rounded to BF16.
 *   d            BF16 [G, max_m, N], any row/group strides (innermost 1)
 *   slot         I32 [T, k] contiguous
 *   topk_weights F32 [T, k] contiguous
 *   y            BF16 [T, N] out, any row stride; must not overlap d
 */
int moe_combine(const dg_tensor* d, const dg_tensor* slot, const dg_tensor* topk_weights,
                const dg_tensor* y, hipStream_t stream);

/* score functions of the routing */
enum {
  DG_SCORE_SOFTMAX = 0,
  DG_SCORE_SIGMOID = 1
};

/*
 * Expert routing: from the router's logits to the tables that
 * moe_dispatch_*_fp8 (topk_idx) and moe_combine (topk_weights) read.
 *   logits       F32 or BF16 [T, E], any row stride; E <= 1024
 *   bias         NULL, or F32 [E]: added to the scores for the choice only
 *                (a balance term), never to the weights
 *   topk_idx     I32 [T, k] out, k <= 64, by falling choice; -1 where fewer
 *                than k experts can be chosen.  (moe_dispatch_*_fp8 wants it
 *                contiguous; any row stride is written here.)
 *   topk_weights F32 [T, k] out, 0 where topk_idx is -1
 *   score        scores s: DG_SCORE_SOFTMAX or DG_SCORE_SIGMOID of the logits
 *   n_group, topk_group, group_top
 *                the experts are n_group equal ranges (at most 64); a group's
 *                score is the sum of its group_top (1 or 2) best choices s +
 *                bias, and only the experts of the topk_group best groups can
 *                be chosen.  n_group = 1: no groups
 *   renormalize  weights are divided by their sum (sigmoid: s_j / (sum +
 *                1e-20); softmax: the softmax over the chosen logits)
 *   scale        factor of every weight
 * Without a bias the choices are ordered by the logits themselves, with one
 * by the FP32 sums of score and bias; equal ones go to the lowest index.  An
 * expert whose logit or bias is -inf cannot be chosen (a token whose logits are
 * all -inf is routed nowhere); NaN ranks below every number.  A +inf softmax
 * logit makes the row's weights NaN, and so does a NaN one (with
 * renormalisation: a NaN among the chosen).  Scores are FP32, each operation
 * rounded once.
 */
int moe_route_topk(const dg_tensor* logits, const dg_tensor* bias, const dg_tensor* topk_idx,
                   const dg_tensor* topk_weights, int32_t score, int32_t n_group, int32_t topk_group,
                   int32_t group_top, int renormalize, float scale, hipStream_t stream);

/*
 * Gradient of moe_route_topk's weights with respect to the logits, the choice
 * taken as given.
 *   logits, topk_idx, score, renormalize, scale  as moe_route_topk; entries
 *                of topk_idx outside [0, E) give nothing, an expert named
 *                twice in a row gets both parts
 *   grad_weights F32 [T, k], any row stride
 *   grad_logits  F32 or BF16 [T, E] out, written whole
 */
int moe_route_topk_bwd(const dg_tensor* logits, const dg_tensor* topk_idx, const dg_tensor* grad_weights,
                       const dg_tensor* grad_logits, int32_t score, int renormalize, float scale,
                       hipStream_t stream);

/*
 * Append new tokens to a paged FP8 key/value cache, rotating keys (and
 * queries) by their position on the way.  One kernel.
 *   k, v         F32 or BF16 [T, Hkv, D], the sequences' new tokens one after
 *                another; D = 64, 128 or 256
 *   k_cache, v_cache  E4M3 [pages, Hkv, P, D], P = 16, 32, 64 or 128; any
 *                strides that are multiples of 16 (innermost 1; tokens less
 *                than 2^24 bytes apart, pages less than 2^32): pages may be
 *                laid out head by head or token by token, and the two caches
 *                may be parts of one pool, interleaved in any way that shares
 *                no memory (with unlike page strides: one after the other)
 *   k_scale, v_scale  F32 [pages, Hkv], any strides (pages less than 2^30
 *                elements apart): the scale of each page and head, a power of
 *                two
 *   block_table  I32 [S, max_pages]: the pages of each sequence, in order
 *   cu_tokens    I32 [S + 1]: sequence s brings tokens cu[s] .. cu[s+1]-1
 *   start        I32 [S]: how many tokens of it are in the cache already, so
 *                that token t has position start[s] + t - cu[s]
 *   cos_sin      NULL, or F32 [positions, rot], 16-byte aligned rows: the
 *                cosines of the rot/2 angles of a position, then the sines.
 *                rot is a multiple of 16, at most D; the other elements of a
 *                head are not rotated.  The pair (x, y) becomes (x cos - y
 *                sin, y cos + x sin), in FP32
 *   interleaved  pairs are elements (2j, 2j+1); else (j, j + rot/2)
 *   q, q_out     both NULL, or q of k's type [T, Hq, D] and q_out BF16 of the
 *                same shape: q rotated, for paged_attention_fp8
 * A page that gets its first tokens takes the scale 2^ceil(log2(a / 448)), a
 * the largest absolute value of what it gets (floored at 1e-4); a page that
 * holds tokens already takes the larger of that and its present scale, and
 * its older codes are re-encoded when the scale grows.  Values that are not
 * finite become NaN codes and do not count for a.  Tokens whose position
 * lies outside the block table or the rows of cos_sin, or whose page is
 * outside [0, pages), are dropped (their rows of q_out stay as they are where
 * the position has no row of cos_sin).  No page may be named for appending by
 * two sequences.
 */
int kv_append_fp8(const dg_tensor* k, const dg_tensor* v, const dg_tensor* k_cache, const dg_tensor* v_cache,
                  const dg_tensor* k_scale, const dg_tensor* v_scale, const dg_tensor* block_table,
                  const dg_tensor* cu_tokens, const dg_tensor* start, const dg_tensor* cos_sin,
                  const dg_tensor* q, const dg_tensor* q_out, int interleaved, hipStream_t stream);

/*
 * Attention of the n newest tokens of each sequence over its paged FP8 cache.
 *   q         BF16 [S, n, Hq, D]; out BF16, the same shape.  Strides multiples
 *             of 8 elements, 16-byte aligned bases
 *   caches, scales, block_table  as kv_append_fp8; Hq a multiple of Hkv (query
 *             heads h * Hq / Hkv .. share KV head h).  Scales of pages that
 *             a query sees are positive, finite and not subnormal, V's within
 *             a factor of 2^120 of each other
 *   seq_lens  I32 [S]: tokens in the cache, the n queries' own included (cut
 *             to what the block table holds).  Query i stands at position
 *             seq_lens[s] - n + i
 *   lse       NULL, or F32 [S, n, Hq] out, any strides: the natural logarithm
 *             of the sum of exp(scores)
 *   workspace F32, at least paged_attention_fp8_workspace bytes (NULL if that
 *             is 0), 16-byte aligned; its contents mean nothing between calls,
 *             but two calls that may run at once need one each
 *   scale     factor of the scores
 *   window    a query sees the window positions up to its own; 0: all of them
 * Positions past a query's own or before its window, and pages outside
 * [0, pages), take no part, whatever their memory holds (NaN codes too, and
 * the scales of pages that no query sees).  A query that sees nothing gives 0,
 * with lse -inf.  Weights are rounded to FP16 (11 bits) on their way into the
 * second product -- those below 2^-38 of the row's largest, V's scales counted
 * in, are lost there -- while scores, sums and output accumulate in FP32; a
 * finite score gives a finite row, however large it is.  The result does not
 * depend on the order in which workgroups run.
 */
int paged_attention_fp8(const dg_tensor* q, const dg_tensor* k_cache, const dg_tensor* v_cache,
                        const dg_tensor* k_scale, const dg_tensor* v_scale, const dg_tensor* block_table,
                        const dg_tensor* seq_lens, const dg_tensor* out, const dg_tensor* lse,
                        const dg_tensor* workspace, float scale, int32_t window, hipStream_t stream);

/* Bytes of workspace that paged_attention_fp8 needs for these sizes
 * (max_tokens = max_pages * P); a pure function of its arguments.  0 for sizes
 * that no call takes. */
int64_t paged_attention_fp8_workspace(int64_t S, int64_t n, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_tokens);

/*
 * Root-mean-square norm with the residual's addition, and its result cast to
 * FP8 in the same kernel (the operand of the FP8 GEMMs):
 *   h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight
 *   x         F32 or BF16 [T, H], or [T, heads, H] (each head of a projection's
 *             output), any strides of the outer dims (innermost 1); H <= 16384,
 *             at most 2^22 - 1 rows (2^24 - 4 up to H = 2048, 2^26 - 16 up to
 *             1024, 2^28 - 64 up to 128)
 *   weight    F32 or BF16 [H]
 *   residual  NULL, or F32 or BF16 of x's shape
 *   h         NULL, or of the residual's type and x's shape, out: the sum,
 *             rounded once.  The norm is of the rounded sum, stored or not
 *   y         NULL, or F32 or BF16 of x's shape, out
 *   q, sf     both NULL, or E4M3 of x's shape and F32 [.., ceil(H/128)] (any
 *             strides), out: y, unrounded, cast as per_token_cast_to_fp8 casts
 *             (one scale per 128 elements of a row, amax floored at 1e-4; with
 *             use_ue8m0 rounded up to a power of two).  Values that are not
 *             finite become NaN codes and do not count for the scale
 *   eps       positive and finite
 * One of y and q is wanted.  h and y may take the place of x or the residual
 * (same base, type and strides); any other overlap is rejected.  Rows whose
 * squares leave FP32's range, at either end, are computed as others are.
 */
int rms_norm(const dg_tensor* x, const dg_tensor* weight, const dg_tensor* y, const dg_tensor* q, const dg_tensor* sf,
             const dg_tensor* residual, const dg_tensor* h, float eps, int use_ue8m0, hipStream_t stream);

/*
 * Gradients of rms_norm's y with respect to the sum h (so to x and to the
 * residual alike) and to the weight; a cast of y counts as the identity.
 *   grad_y       F32 or BF16 [T, H] or [T, heads, H]
 *   h            the sum that rms_norm stored (x, where it had no residual)
 *   grad_x       F32 or BF16 of that shape, out; it may take the place of
 *                grad_y, h or grad_h (same base, type and strides)
 *   grad_weight  NULL, or F32 or BF16 [H], out
 *   workspace    F32, rms_norm_bwd_workspace(rows, H) bytes (rows = T heads), 16-byte
 *                aligned; NULL without grad_weight.  Its contents mean nothing
 *                between calls, but two calls that may run at once need one each
 *   grad_h       NULL, or F32 or BF16 of that shape: a gradient that reaches h
 *                from elsewhere (the residual stream), added to grad_x
 * FP32 sums in an order that depends on the sizes only.  Rows and gradients may be
 * of any size whose products grad_y weight and whose results FP32 holds.
 */
int rms_norm_bwd(const dg_tensor* grad_y, const dg_tensor* h, const dg_tensor* weight, const dg_tensor* grad_x,
                 const dg_tensor* grad_weight, const dg_tensor* workspace, const dg_tensor* grad_h, float eps,
                 hipStream_t stream);

/* Bytes of workspace that rms_norm_bwd needs for a weight's gradient; a pure
 * function of its arguments.  0 for sizes that no call takes. */
int64_t rms_norm_bwd_workspace(int64_t rows, int64_t H);

/*
 * The gated activation between an expert's two products, with its cast to FP8:
 *   y = row_weight * silu(gate) * up,  silu(g) = g / (1 + exp(-g))
 *   x            F32 or BF16 [R, 2 I] or [G, R, 2 I]: the gate's I columns, then
 *                the up projection's
 *   y            NULL, or F32 or BF16 [.., I], out
 *   q, sf        both NULL, or E4M3 [.., I] and F32 [.., ceil(I/128)], out: y,
 *                unrounded, cast as by rms_norm
 *   masked_m     NULL, or I32 [G] ([1] for a 2-D x) on the device: only the
 *                first masked_m[g] rows of group g are read and written (the
 *                masked GEMM's layout; with a 2-D x the rows in use of a buffer)
 *   row_weights  NULL, or F32 [G R]: a factor of each row (the router's weights)
 */
int swiglu(const dg_tensor* x, const dg_tensor* y, const dg_tensor* q, const dg_tensor* sf, const dg_tensor* masked_m,
           const dg_tensor* row_weights, int use_ue8m0, hipStream_t stream);

/*
 * Gradients of swiglu's y; a cast of y counts as the identity.
 *   grad_y            F32 or BF16 [.., I]
 *   grad_x            F32 or BF16 of x's shape, out; it may be x itself
 *   grad_row_weights  NULL, or F32 [G R], out: the sum over each row of grad_y
 *                     silu(gate) up (for moe_route_topk_bwd)
 * masked_m and row_weights as for swiglu; rows past masked_m are left alone.
 */
int swiglu_bwd(const dg_tensor* x, const dg_tensor* grad_y, const dg_tensor* grad_x, const dg_tensor* masked_m,
               const dg_tensor* row_weights, const dg_tensor* grad_row_weights, hipStream_t stream);

/*
 * BF16 products grouped by expert with ragged sizes: rows sorted by expert, no
 * padding between the groups.  Group g holds rows offsets[g] .. offsets[g+1]-1
 * of the tokens' tensors (device memory, never read by the host; values are cut
 * to [0, M], a group whose end is not past its start is empty).  offsets is
 * expected not to fall: where it does, which rows of d are computed is not
 * specified.  FP32 accumulation, in an order that depends on the group's index
 * and b's sizes and strides (tn: on the group's rows) and on nothing else of the
 * call: a row keeps its bits whatever the other groups hold.
 *   nt  d[m] = c[m] + a[m] . b[g]^T   a [M, K], b [G, N, K], d [M, N]: the
 *       forward product of m_grouped_bf16_gemm_nt_contiguous without its blocks
 *   nn  d[m] = c[m] + a[m] . b[g]     a [M, K], b [G, K, N], d [M, N]: the
 *       gradient of nt's a, from nt's b as it is stored
 *   tn  d[g] = c[g] + a_g^T . b_g     a [M, N], b [M, K], d [G, N, K]: the
 *       gradient of nt's b, the contraction over the group's rows; an empty
 *       group gives c[g], or zeros
 *   a, b     BF16, row and group strides multiples of 8 elements, rows that do
 *            not overlap, 16-byte aligned bases; any M, N and (tn) K, K of nt and
 *            nn a multiple of 64
 *   c        NULL, or BF16 or F32 of d's shape; it may be d itself (same base,
 *            type and strides), any other overlap is rejected
 *   d        BF16 or F32, any row stride (innermost 1).  Rows of nt and nn
 *            outside every group are neither read from a and c nor written
 *   offsets  I32 [G + 1]
 */
int m_grouped_bf16_gemm_nt_ragged(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c, const dg_tensor* d,
                                  const dg_tensor* offsets, hipStream_t stream);
int m_grouped_bf16_gemm_nn_ragged(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c, const dg_tensor* d,
                                  const dg_tensor* offsets, hipStream_t stream);
int k_grouped_bf16_gemm_tn(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c, const dg_tensor* d,
                           const dg_tensor* offsets, hipStream_t stream);

/* Launch configuration chosen for a GEMM (a pure function of the shapes).
 * A GEMM is one launch over all N columns, or two launches in stream order:
 * the first over columns [0, n_split), the second (block_n2 > 0) over
 * [n_split, N) with a narrower tile, when that fills the last round of
 * workgroups over the compute units better (block sizes that are not powers
 * of two: "DeepGEMM tested by Novita AI", section "Technological Innovations
 * of DeepGEMM", item "Support for Arbitrary Matrix Sizes"). */
typedef struct dg_config {
  int32_t block_m, block_n;   /* output tile of one workgroup (first launch) */
  int32_t threads;            /* workgroup size */
  int64_t grid;               /* workgroups of the first launch */
  int32_t lds_bytes;          /* static LDS per workgroup of the first launch */
  int64_t n_split;            /* columns of the first launch (N when there is one launch) */
  int32_t block_n2;           /* tile width of the second launch, 0 if none (block_m, threads as above) */
  int64_t grid2;              /* workgroups of the second launch, 0 if none */
  int32_t lds_bytes2;         /* static LDS per workgroup of the second launch */
} dg_config;

enum {
  DG_KIND_DENSE = 0, DG_KIND_CONTIGUOUS = 1, DG_KIND_MASKED = 2,            /* FP8 GEMMs */
  DG_KIND_BF16_MASKED = 3, DG_KIND_BF16_DENSE = 4, DG_KIND_BF16_CONTIGUOUS = 5, /* BF16 GEMMs */
  DG_KIND_DENSE_ROWB = 6, DG_KIND_CONTIGUOUS_ROWB = 7, DG_KIND_MASKED_ROWB = 8, /* FP8, one B scale per row */
  DG_KIND_DENSE_FP8_OUT = 9,                                                      /* fp8_gemm_nt_fp8_out */
  DG_KIND_DENSE_MN = 10,                        /* fp8_gemm_nn / _tn / _tt (an MN-major operand) */
  DG_KIND_DENSE_FP8_OUT_ROWB = 11               /* fp8_gemm_nt_fp8_out, one B scale per row */
};

/* Fill *out with the configuration `kind` would launch for these sizes
 * (M = rows: M, Msum or max_m; G = groups, 1 for dense). */
int dg_query_config(int32_t kind, int64_t G, int64_t M, int64_t N, int64_t K, dg_config* out);

#ifdef __cplusplus
}
#endif
#endif /* DGMI_H */
