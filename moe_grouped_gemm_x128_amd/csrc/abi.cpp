// Host side of libdgmi: the extern "C" entry points declared in dgmi.h.
//
// Every entry point validates its descriptors on the host (dtype, rank,
// shape consistency, unit innermost stride, alignment, aliasing of the
// output), then enqueues the kernels on the caller's stream and returns.
// Nothing here allocates, synchronises or reads device memory, so each call
// can be captured into a hipGraph ("DeepGEMM CUDA Graph Compatibility for
// Masked Grouped GEMMs", sections "Eliminating Host-Side Allocation" and
// "Tensor-Based Metadata Arguments"; "[GH-ISSUE #414] pack_ue8m0_to_int is
// not CUDA Graph capture safe", section "Expected behavior": shape and dtype
// checks stay on the host, value checks never synchronise).

#include <stdarg.h>
#include <stdio.h>

#include <string>

#include "dgmi.h"
#include "launch.hpp"

namespace {

thread_local std::string g_err;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

int ok() {
  g_err.clear();
  return DG_OK;
}

int elem_size(int32_t dtype) {
  switch (dtype) {
    case DG_F32: return 4;
    case DG_BF16: return 2;
    case DG_E4M3: return 1;
    case DG_I32: return 4;
    default: return 0;
  }
}

const char* dtype_name(int32_t dtype) {
  switch (dtype) {
    case DG_F32: return "F32";
    case DG_BF16: return "BF16";
    case DG_E4M3: return "E4M3";
    case DG_I32: return "I32";
    default: return "?";
  }
}

// Basic well-formedness: non-null, known dtype, 1..4 dims, non-negative
// shape, non-negative strides, innermost stride 1 when `unit_inner` (for a
// tensor with elements).
int check_basic(const dg_tensor* t, const char* name, bool unit_inner) {
  if (t == nullptr) return fail(DG_INVALID_ARG, "%s: descriptor is NULL", name);
  if (elem_size(t->dtype) == 0) return fail(DG_INVALID_ARG, "%s: unknown dtype %d", name, t->dtype);
  if (t->ndim < 1 || t->ndim > 4) return fail(DG_INVALID_ARG, "%s: ndim %d not in 1..4", name, t->ndim);
  int64_t numel = 1;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] < 0) return fail(DG_INVALID_ARG, "%s: negative extent in dim %d", name, i);
    if (t->stride[i] < 0) return fail(DG_INVALID_ARG, "%s: negative stride in dim %d", name, i);
    if (t->shape[i] > INT32_MAX) return fail(DG_INVALID_ARG, "%s: extent of dim %d exceeds 2^31-1", name, i);
    numel *= t->shape[i];
  }
  if (numel > 0 && t->data == nullptr) return fail(DG_INVALID_ARG, "%s: data pointer is NULL", name);
  if (unit_inner && numel > 0 && t->shape[t->ndim - 1] > 1 && t->stride[t->ndim - 1] != 1)
    return fail(DG_INVALID_ARG, "%s: innermost stride must be 1 (got %lld)", name, (long long)t->stride[t->ndim - 1]);
  return DG_OK;
}

int check_dtype(const dg_tensor* t, const char* name, int32_t want) {
  if (t->dtype != want)
    return fail(DG_INVALID_ARG, "%s: dtype %s, expected %s", name, dtype_name(t->dtype), dtype_name(want));
  return DG_OK;
}

// Byte span [lo, hi) touched by a strided tensor (empty => lo == hi).
void span(const dg_tensor* t, uintptr_t* lo, uintptr_t* hi) {
  int64_t last = 0;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] == 0) {
      *lo = *hi = reinterpret_cast<uintptr_t>(t->data);
      return;
    }
    last += (t->shape[i] - 1) * t->stride[i];
  }
  *lo = reinterpret_cast<uintptr_t>(t->data);
  *hi = *lo + (uintptr_t)((last + 1) * elem_size(t->dtype));
}

int check_no_alias(const dg_tensor* out, const char* oname, const dg_tensor* in, const char* iname) {
  if (in == nullptr) return DG_OK;
  uintptr_t a0, a1, b0, b1;
  span(out, &a0, &a1);
  span(in, &b0, &b1);
  if (a0 < a1 && b0 < b1 && a0 < b1 && b0 < a1)
    return fail(DG_INVALID_ARG, "%s overlaps %s in memory", oname, iname);
  return DG_OK;
}

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }

#define DG_TRY(expr)             \
  do {                           \
    int rc_ = (expr);            \
    if (rc_ != DG_OK) return rc_; \
  } while (0)

// A matrix-like operand viewed as [G, R, C]: either 3-D, or 2-D with R = G*rows
// split by `rows_per_group` (rows_per_group <= 0: 2-D means a single group).
struct View3 {
  int64_t G, R, C;
  int64_t sg, sr;
};

int view3(const dg_tensor* t, const char* name, int64_t G_expect, int64_t rows_per_group, View3* v) {
  if (t->ndim == 3) {
    v->G = t->shape[0];
    v->R = t->shape[1];
    v->C = t->shape[2];
    v->sg = t->stride[0];
    v->sr = t->stride[1];
  } else if (t->ndim == 2) {
    if (rows_per_group > 0) {
      if (t->shape[0] != G_expect * rows_per_group)
        return fail(DG_INVALID_ARG, "%s: 2-D leading extent %lld != groups*rows %lld", name,
                    (long long)t->shape[0], (long long)(G_expect * rows_per_group));
      v->G = G_expect;
      v->R = rows_per_group;
      v->sg = rows_per_group * t->stride[0];
    } else {
      v->G = 1;
      v->R = t->shape[0];
      v->sg = 0;
    }
    v->C = t->shape[1];
    v->sr = t->stride[0];
  } else {
    return fail(DG_INVALID_ARG, "%s: expected 2 or 3 dims, got %d", name, t->ndim);
  }
  if (G_expect >= 0 && v->G != G_expect)
    return fail(DG_INVALID_ARG, "%s: %lld groups, expected %lld", name, (long long)v->G, (long long)G_expect);
  return DG_OK;
}

// Scale-factor operand of the FP8 GEMMs: F32 [.., rows, nkb] or packed I32
// [.., rows, ceil(nkb/4)]; any strides.
int check_scales(const dg_tensor* t, const char* name, int sf_fmt, int64_t G_expect, int64_t rows_per_group,
                 int64_t rows, int64_t nkb, View3* v) {
  DG_TRY(check_basic(t, name, false));
  DG_TRY(check_dtype(t, name, sf_fmt == dgmi::SF_F32 ? DG_F32 : DG_I32));
  DG_TRY(view3(t, name, G_expect, rows_per_group, v));
  const int64_t cols = sf_fmt == dgmi::SF_F32 ? nkb : (nkb + 3) / 4;
  if (v->R != rows || v->C != cols)
    return fail(DG_INVALID_ARG, "%s: shape [..,%lld,%lld], expected [..,%lld,%lld]", name, (long long)v->R,
                (long long)v->C, (long long)rows, (long long)cols);
  return DG_OK;
}

// The kernels address a tile of up to 256 rows of A or B with 32-bit buffer
// offsets (row * row stride + K offset): row strides (bytes) must stay below
// 2^31 / 256, i.e. 8 MiB.
int check_row_strides(int64_t lda_bytes, int64_t ldb_bytes, const char* fname) {
  constexpr int64_t kMax = INT32_MAX / 256;
  if (lda_bytes > kMax || ldb_bytes > kMax)
    return fail(DG_UNSUPPORTED, "%s: row strides of a and b must be below %lld bytes (got %lld, %lld)", fname,
                (long long)kMax, (long long)lda_bytes, (long long)ldb_bytes);
  return DG_OK;
}

int check_launch(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(DG_LAUNCH_FAILED, "%s: launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

// Common FP8 GEMM validation.  mode: dense / contig / masked.  With q != NULL
// (dense only) the output is D cast per token to FP8: q E4M3 [M, N] and sfq
// F32 [M, ceil(N/128)] take the place of d (NULL).
int fp8_gemm_common(int mode, const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                    const dg_tensor* c, const dg_tensor* d, const dg_tensor* meta, int64_t max_m, hipStream_t stream,
                    const char* fname, const dg_tensor* q = nullptr, const dg_tensor* sfq = nullptr,
                    int q_ue8m0 = 0) {
  const bool fp8_out = q != nullptr;
  if (fp8_out) d = q;  // the output operand, for the shape and alias checks
  const char* dname = fp8_out ? "q" : "d";
  // An MN-major operand (dense only) is the transposed view of a row-major
  // [K, M] or [K, N] tensor: a 2-D descriptor with unit stride along its rows
  // and its K-row stride in stride[1].
  auto mn_major = [](const dg_tensor* t) {
    return t != nullptr && t->ndim == 2 && t->shape[1] > 1 && t->stride[1] != 1 &&
           (t->shape[0] <= 1 || t->stride[0] == 1);
  };
  const bool a_mn = mode == dgmi::MODE_DENSE && mn_major(a), b_mn = mode == dgmi::MODE_DENSE && mn_major(b);
  DG_TRY(check_basic(a, "a", !a_mn));
  DG_TRY(check_basic(b, "b", !b_mn));
  DG_TRY(check_basic(d, dname, true));
  DG_TRY(check_dtype(a, "a", DG_E4M3));
  DG_TRY(check_dtype(b, "b", DG_E4M3));
  // d: BF16, or F32 for the dense GEMM (the FP32 accumulator stored as is)
  const bool d_f32 = !fp8_out && d->dtype == DG_F32;
  DG_TRY(check_dtype(d, dname, fp8_out ? DG_E4M3 : (d_f32 ? DG_F32 : DG_BF16)));
  if (sfa == nullptr || sfb == nullptr) return fail(DG_INVALID_ARG, "%s: scale descriptors must not be NULL", fname);
  if (sfa->dtype != sfb->dtype) return fail(DG_INVALID_ARG, "%s: sfa and sfb must have the same dtype", fname);
  const int sf_fmt = sfa->dtype == DG_I32 ? dgmi::SF_UE8M0 : dgmi::SF_F32;

  View3 va, vb, vd, vsa, vsb;
  int64_t G = 1, rows_pg = 0;
  if (mode == dgmi::MODE_DENSE) {
    if (a->ndim != 2 || b->ndim != 2 || d->ndim != 2)
      return fail(DG_INVALID_ARG, "%s: a, b, %s must be 2-D", fname, dname);
    DG_TRY(view3(b, "b", 1, 0, &vb));
  } else {
    if (b->ndim != 3) return fail(DG_INVALID_ARG, "%s: b must be [G, N, K]", fname);
    G = b->shape[0];
    DG_TRY(view3(b, "b", G, 0, &vb));
  }
  if (mode == dgmi::MODE_MASKED) {
    if (max_m < 0) return fail(DG_INVALID_ARG, "%s: max_m_per_group must be >= 0", fname);
    rows_pg = max_m;
    DG_TRY(view3(a, "a", G, rows_pg, &va));
    DG_TRY(view3(d, "d", G, rows_pg, &vd));
  } else {
    if (a->ndim != 2 || d->ndim != 2) return fail(DG_INVALID_ARG, "%s: a and %s must be 2-D", fname, dname);
    DG_TRY(view3(a, "a", 1, 0, &va));
    DG_TRY(view3(d, dname, 1, 0, &vd));
  }
  const int64_t M = va.R, K = va.C, N = vb.R;
  if (vb.C != K) return fail(DG_INVALID_ARG, "%s: K mismatch: a has %lld, b has %lld", fname, (long long)K, (long long)vb.C);
  if (vd.R != M || vd.C != N)
    return fail(DG_INVALID_ARG, "%s: %s is [..,%lld,%lld], expected [..,%lld,%lld]", fname, dname, (long long)vd.R,
                (long long)vd.C, (long long)M, (long long)N);
  if (mode == dgmi::MODE_MASKED && M != max_m)
    return fail(DG_INVALID_ARG, "%s: a has %lld rows per group, max_m_per_group is %lld", fname, (long long)M,
                (long long)max_m);
  if (K % 128 != 0) return fail(DG_UNSUPPORTED, "%s: K = %lld is not a multiple of 128", fname, (long long)K);
  const int64_t nkb = K / 128, nnb = (N + 127) / 128;
  DG_TRY(check_scales(sfa, "sfa", sf_fmt, mode == dgmi::MODE_MASKED ? G : 1, rows_pg, M, nkb, &vsa));
  // sfb: one scale per 128x128 block of B, or one per row of B (N rows; for
  // N = 1 the two forms are the same)
  const bool rowb = sfb->ndim >= 2 && sfb->shape[sfb->ndim - 2] == N && N != nnb;
  DG_TRY(check_scales(sfb, "sfb", sf_fmt, mode == dgmi::MODE_DENSE ? 1 : G, 0, rowb ? N : nnb, nkb, &vsb));
  if (mode == dgmi::MODE_DENSE && (sfb->ndim != 2 || sfa->ndim != 2))
    return fail(DG_INVALID_ARG, "%s: sfa and sfb must be 2-D", fname);
  if (mode == dgmi::MODE_CONTIG && sfb->ndim != 3) return fail(DG_INVALID_ARG, "%s: sfb must be [G, ceil(N/128), ..]", fname);

  // MN-major operands: K-rows of M (N) bytes, 16-byte aligned, ld bytes apart
  const int64_t lda = a_mn ? a->stride[1] : va.sr, ldb = b_mn ? b->stride[1] : vb.sr;
  if (a_mn || b_mn) {
    if (fp8_out) return fail(DG_UNSUPPORTED, "%s: MN-major operands take a BF16 or F32 d", fname);
    if ((a_mn && M % 16) || (b_mn && N % 16))
      return fail(DG_UNSUPPORTED, "%s: an MN-major operand needs its row count (M or N) to be a multiple of 16",
                  fname);
    if ((a_mn && lda < M) || (b_mn && ldb < N))
      return fail(DG_UNSUPPORTED, "%s: the K-row stride of an MN-major operand must be at least its row count", fname);
    // the kernels address an MN-major operand with 32-bit offsets from its first K-row
    const int64_t lim = (int64_t(1) << 31) - 256;
    if ((a_mn && K * lda > lim) || (b_mn && K * ldb > lim))
      return fail(DG_UNSUPPORTED, "%s: an MN-major operand must span less than 2^31 bytes (K x K-row stride)", fname);
  }
  // alignment: 16-B operand rows (the kernels load 16-B chunks), 16-B output rows
  if (!aligned(a->data, 16) || !aligned(b->data, 16) || lda % 16 || ldb % 16 || va.sg % 16 || vb.sg % 16)
    return fail(DG_INVALID_ARG, "%s: a and b need 16-byte aligned bases and row/group strides", fname);
  DG_TRY(check_row_strides(a_mn ? 0 : lda, b_mn ? 0 : ldb, fname));
  if (fp8_out) {
    // q rows are written in 4-byte words (16-byte stores when 16-byte aligned)
    if (!aligned(d->data, 4) || (M > 1 && N > 0 && vd.sr % 4))
      return fail(DG_INVALID_ARG, "%s: q needs a 4-byte aligned base and row stride", fname);
    DG_TRY(check_basic(sfq, "sfq", false));
    DG_TRY(check_dtype(sfq, "sfq", DG_F32));
    if (sfq->ndim != 2 || sfq->shape[0] != M || sfq->shape[1] != nnb)
      return fail(DG_INVALID_ARG, "%s: sfq must be F32 [M, ceil(N/128)] = [%lld, %lld]", fname, (long long)M,
                  (long long)nnb);
    if (!aligned(sfq->data, 4)) return fail(DG_INVALID_ARG, "%s: sfq must be 4-byte aligned", fname);
  } else if (!aligned(d->data, d_f32 ? 4 : 2)) {
    return fail(DG_INVALID_ARG, "%s: d must be element-aligned", fname);
  }
  if (!aligned(sfa->data, 4) || !aligned(sfb->data, 4)) return fail(DG_INVALID_ARG, "%s: scales must be 4-byte aligned", fname);

  if (mode == dgmi::MODE_CONTIG) {
    if (M % 128 != 0) return fail(DG_INVALID_ARG, "%s: Msum = %lld is not a multiple of 128", fname, (long long)M);
    DG_TRY(check_basic(meta, "grouped_layout", true));
    DG_TRY(check_dtype(meta, "grouped_layout", DG_I32));
    if (meta->ndim != 1 || meta->shape[0] != M / 128)
      return fail(DG_INVALID_ARG, "%s: grouped_layout must be I32 [Msum/128 = %lld]", fname, (long long)(M / 128));
  } else if (mode == dgmi::MODE_MASKED) {
    DG_TRY(check_basic(meta, "masked_m", true));
    DG_TRY(check_dtype(meta, "masked_m", DG_I32));
    if (meta->ndim != 1 || meta->shape[0] != G)
      return fail(DG_INVALID_ARG, "%s: masked_m must be I32 [G = %lld]", fname, (long long)G);
  }
  DG_TRY(check_no_alias(d, dname, a, "a"));
  DG_TRY(check_no_alias(d, dname, b, "b"));
  DG_TRY(check_no_alias(d, dname, sfa, "sfa"));
  DG_TRY(check_no_alias(d, dname, sfb, "sfb"));
  if (meta != nullptr) DG_TRY(check_no_alias(d, dname, meta, "metadata"));
  if (fp8_out) {
    DG_TRY(check_no_alias(sfq, "sfq", a, "a"));
    DG_TRY(check_no_alias(sfq, "sfq", b, "b"));
    DG_TRY(check_no_alias(sfq, "sfq", sfa, "sfa"));
    DG_TRY(check_no_alias(sfq, "sfq", sfb, "sfb"));
    DG_TRY(check_no_alias(sfq, "sfq", q, "q"));
    DG_TRY(check_no_alias(sfq, "sfq", c, "c"));
  }
  // accumulate input: D = C + A . B^T, C BF16 or F32 with d's shape ([M, N],
  // [Msum, N], or [G, max_m, N] / [G * max_m, N]); c may be d itself (same
  // base and strides), any other overlap is rejected
  bool c_f32 = false;
  int64_t ldc = 0, c_gs = 0;
  if (c != nullptr) {
    DG_TRY(check_basic(c, "c", true));
    if (c->dtype != DG_BF16 && c->dtype != DG_F32) return fail(DG_INVALID_ARG, "%s: c must be BF16 or F32", fname);
    View3 vc;
    if (mode == dgmi::MODE_MASKED) {
      DG_TRY(view3(c, "c", G, rows_pg, &vc));
    } else {
      if (c->ndim != 2) return fail(DG_INVALID_ARG, "%s: c must be 2-D", fname);
      DG_TRY(view3(c, "c", 1, 0, &vc));
    }
    if ((mode == dgmi::MODE_MASKED && vc.G != G) || vc.R != M || vc.C != N)
      return fail(DG_INVALID_ARG, "%s: c must have the shape of %s ([..,%lld,%lld])", fname, dname, (long long)M,
                  (long long)N);
    c_f32 = c->dtype == DG_F32;
    if (!aligned(c->data, c_f32 ? 4 : 2)) return fail(DG_INVALID_ARG, "%s: c must be element-aligned", fname);
    ldc = vc.sr;
    c_gs = vc.sg;
    // (with FP8 output, c and q differ in dtype and must not overlap)
    const bool same_as_d = c->data == d->data && c->dtype == d->dtype && ldc == vd.sr && (G <= 1 || c_gs == vd.sg);
    if (!same_as_d) DG_TRY(check_no_alias(d, dname, c, "c"));
  }

  dgmi::GemmParams p = {};
  p.a = static_cast<const uint8_t*>(a->data);
  p.b = static_cast<const uint8_t*>(b->data);
  p.sfa = sfa->data;
  p.sfb = sfb->data;
  p.d = fp8_out ? nullptr : static_cast<uint16_t*>(d->data);
  p.d_f32 = d_f32 ? 1 : 0;
  if (fp8_out) {
    p.q = static_cast<uint8_t*>(q->data);
    p.ldq = vd.sr;
    p.sfq = static_cast<float*>(sfq->data);
    p.sfq_sm = sfq->stride[0];
    p.sfq_sn = sfq->stride[1];
    p.q_ue8m0 = q_ue8m0 ? 1 : 0;
  }
  p.c = c != nullptr ? c->data : nullptr;
  p.ldc = ldc;
  p.c_gs = c_gs;
  p.c_f32 = c_f32 ? 1 : 0;
  p.meta = meta ? static_cast<const int32_t*>(meta->data) : nullptr;
  p.lda = lda;
  p.a_gs = va.sg;
  p.ldb = ldb;
  p.b_gs = vb.sg;
  p.a_mn = a_mn ? 1 : 0;
  p.b_mn = b_mn ? 1 : 0;
  p.sfa_sm = vsa.sr;
  p.sfa_sk = sfa->stride[sfa->ndim - 1];
  p.sfa_gs = vsa.sg;
  p.sfb_sn = vsb.sr;
  p.sfb_sk = sfb->stride[sfb->ndim - 1];
  p.sfb_gs = vsb.sg;
  p.ldd = vd.sr;
  p.d_gs = d_f32 ? 2 * vd.sg : vd.sg;  // (the kernels step d in BF16-sized units)
  p.M = (int32_t)M;
  p.N = (int32_t)N;
  p.k_bytes = (int32_t)K;
  p.G = (int32_t)G;
  if (M == 0 || N == 0 || G == 0) return ok();
  if (K == 0) return fail(DG_UNSUPPORTED, "%s: K = 0 is not supported", fname);
  if (fp8_out)
    return check_launch(dgmi::launch_fp8_gemm_fp8_out(p, sf_fmt | (rowb ? dgmi::SF_ROWB : 0), stream), fname);
  return check_launch(dgmi::launch_fp8_gemm(p, mode, sf_fmt | (rowb ? dgmi::SF_ROWB : 0), stream), fname);
}

// Quantizer validation: x [R, K] or [G, R, K]; q same shape; sf [.., R', KB].
// x is K-major (innermost stride 1) or MN-major (stride 1 along the rows:
// the transpose of a row-major [K, R] tensor), q is K-major.
int quant_common(const dg_tensor* x, const dg_tensor* q, const dg_tensor* sf, int use_ue8m0, hipStream_t stream,
                 bool per_block, const char* fname) {
  const bool mn_major = x != nullptr && x->ndim >= 2 && x->shape[x->ndim - 1] > 1 && x->stride[x->ndim - 1] != 1 &&
                        (x->shape[x->ndim - 2] <= 1 || x->stride[x->ndim - 2] == 1);
  DG_TRY(check_basic(x, "x", !mn_major));
  DG_TRY(check_basic(q, "q", true));
  DG_TRY(check_basic(sf, "sf", false));
  if (x->dtype != DG_F32 && x->dtype != DG_BF16) return fail(DG_INVALID_ARG, "%s: x must be F32 or BF16", fname);
  DG_TRY(check_dtype(q, "q", DG_E4M3));
  DG_TRY(check_dtype(sf, "sf", DG_F32));
  if (x->ndim != q->ndim || x->ndim != sf->ndim || (x->ndim != 2 && x->ndim != 3))
    return fail(DG_INVALID_ARG, "%s: x, q and sf must all be 2-D or all 3-D", fname);
  for (int i = 0; i < x->ndim; ++i)
    if (x->shape[i] != q->shape[i]) return fail(DG_INVALID_ARG, "%s: q must have the shape of x", fname);
  View3 vx, vq, vs;
  DG_TRY(view3(x, "x", -1, 0, &vx));
  DG_TRY(view3(q, "q", vx.G, 0, &vq));
  DG_TRY(view3(sf, "sf", vx.G, 0, &vs));
  const int64_t R = vx.R, K = vx.C;
  const int64_t srows = per_block ? (R + 127) / 128 : R;
  if (vs.R != srows || vs.C != (K + 127) / 128)
    return fail(DG_INVALID_ARG, "%s: sf is [..,%lld,%lld], expected [..,%lld,%lld]", fname, (long long)vs.R,
                (long long)vs.C, (long long)srows, (long long)((K + 127) / 128));
  const int xe = elem_size(x->dtype);
  if (!mn_major && (!aligned(x->data, 16) || (vx.sr * xe) % 16 || (vx.sg * xe) % 16))
    return fail(DG_INVALID_ARG, "%s: x needs a 16-byte aligned base and row/group strides", fname);
  if (mn_major && !aligned(x->data, xe)) return fail(DG_INVALID_ARG, "%s: x must be element-aligned", fname);
  if (!aligned(q->data, 4) || vq.sr % 4 || vq.sg % 4)
    return fail(DG_INVALID_ARG, "%s: q needs a 4-byte aligned base and row/group strides", fname);
  if (!aligned(sf->data, 4)) return fail(DG_INVALID_ARG, "%s: sf must be 4-byte aligned", fname);
  DG_TRY(check_no_alias(q, "q", x, "x"));
  DG_TRY(check_no_alias(sf, "sf", x, "x"));
  DG_TRY(check_no_alias(sf, "sf", q, "q"));
  dgmi::QuantArgs p = {};
  p.x = x->data;
  p.x_bf16 = x->dtype == DG_BF16;
  p.sx_g = vx.sg;
  p.sx_r = vx.sr;
  p.q = static_cast<uint8_t*>(q->data);
  p.sq_g = vq.sg;
  p.sq_r = vq.sr;
  p.sf = static_cast<float*>(sf->data);
  p.ssf_g = vs.sg;
  p.ssf_r = vs.sr;
  p.ssf_k = sf->stride[sf->ndim - 1];
  p.G = (int32_t)vx.G;
  p.R = (int32_t)R;
  p.K = (int32_t)K;
  p.ue8m0 = use_ue8m0 ? 1 : 0;
  if (vx.G == 0 || R == 0 || K == 0) return ok();
  if (mn_major) {
    // read through a transposing LDS tile
    dgmi::QuantTArgs t = {};
    static_cast<dgmi::QuantArgs&>(t) = p;
    t.sx_k = x->stride[x->ndim - 1];
    const int64_t lb = x->dtype == DG_F32 ? 16 : 8;  // bytes of four elements
    t.vec = (aligned(x->data, (int)lb) && (t.sx_k * xe) % lb == 0 && (vx.sg * xe) % lb == 0) ? 1 : 0;
    t.qvec = (aligned(q->data, 16) && (R <= 1 || vq.sr % 16 == 0) && (vx.G <= 1 || vq.sg % 16 == 0)) ? 1 : 0;
    return check_launch(dgmi::launch_cast_mn(t, per_block, stream), fname);
  }
  return check_launch(per_block ? dgmi::launch_per_block(p, stream) : dgmi::launch_per_token(p, stream), fname);
}

// The BF16 GEMMs (dense with optional C, contiguous, masked): the same
// kernel body as the FP8 GEMM with BF16 operands and no scales.
int bf16_gemm_common(int mode, const dg_tensor* a, const dg_tensor* b, const dg_tensor* c, const dg_tensor* d,
                     const dg_tensor* meta, int64_t max_m, hipStream_t stream, const char* fname) {
  DG_TRY(check_basic(a, "a", true));
  DG_TRY(check_basic(b, "b", true));
  DG_TRY(check_basic(d, "d", true));
  DG_TRY(check_dtype(a, "a", DG_BF16));
  DG_TRY(check_dtype(b, "b", DG_BF16));
  // d: BF16, or F32 (the FP32 accumulator stored as is)
  const bool d_f32 = d->dtype == DG_F32;
  DG_TRY(check_dtype(d, "d", d_f32 ? DG_F32 : DG_BF16));
  View3 va, vb, vd;
  int64_t G = 1;
  if (mode == dgmi::MODE_DENSE) {
    if (a->ndim != 2 || b->ndim != 2 || d->ndim != 2) return fail(DG_INVALID_ARG, "%s: a, b, d must be 2-D", fname);
    DG_TRY(view3(b, "b", 1, 0, &vb));
  } else {
    if (b->ndim != 3) return fail(DG_INVALID_ARG, "%s: b must be [G, N, K]", fname);
    G = b->shape[0];
    DG_TRY(view3(b, "b", G, 0, &vb));
  }
  if (mode == dgmi::MODE_MASKED) {
    if (max_m < 0) return fail(DG_INVALID_ARG, "%s: max_m_per_group must be >= 0", fname);
    DG_TRY(view3(a, "a", G, max_m, &va));
    DG_TRY(view3(d, "d", G, max_m, &vd));
  } else {
    if (a->ndim != 2 || d->ndim != 2) return fail(DG_INVALID_ARG, "%s: a and d must be 2-D", fname);
    DG_TRY(view3(a, "a", 1, 0, &va));
    DG_TRY(view3(d, "d", 1, 0, &vd));
  }
  const int64_t M = va.R, K = va.C, N = vb.R;
  if (mode == dgmi::MODE_MASKED && M != max_m)
    return fail(DG_INVALID_ARG, "%s: a has %lld rows per group, max_m_per_group is %lld", fname, (long long)M, (long long)max_m);
  if (vb.C != K) return fail(DG_INVALID_ARG, "%s: K mismatch", fname);
  if (vd.R != M || vd.C != N) return fail(DG_INVALID_ARG, "%s: d must be [.., %lld, %lld]", fname, (long long)M, (long long)N);
  if (K % 64 != 0) return fail(DG_UNSUPPORTED, "%s: K = %lld is not a multiple of 64", fname, (long long)K);
  if (!aligned(a->data, 16) || !aligned(b->data, 16) || va.sr % 8 || vb.sr % 8 || va.sg % 8 || vb.sg % 8)
    return fail(DG_INVALID_ARG, "%s: a and b need 16-byte aligned bases and row/group strides", fname);
  DG_TRY(check_row_strides(2 * va.sr, 2 * vb.sr, fname));
  if (!aligned(d->data, d_f32 ? 4 : 2)) return fail(DG_INVALID_ARG, "%s: d must be element-aligned", fname);
  if (mode == dgmi::MODE_CONTIG) {
    if (M % 128 != 0) return fail(DG_INVALID_ARG, "%s: Msum = %lld is not a multiple of 128", fname, (long long)M);
    DG_TRY(check_basic(meta, "grouped_layout", true));
    DG_TRY(check_dtype(meta, "grouped_layout", DG_I32));
    if (meta->ndim != 1 || meta->shape[0] != M / 128)
      return fail(DG_INVALID_ARG, "%s: grouped_layout must be I32 [Msum/128 = %lld]", fname, (long long)(M / 128));
  } else if (mode == dgmi::MODE_MASKED) {
    DG_TRY(check_basic(meta, "masked_m", true));
    DG_TRY(check_dtype(meta, "masked_m", DG_I32));
    if (meta->ndim != 1 || meta->shape[0] != G) return fail(DG_INVALID_ARG, "%s: masked_m must be I32 [G]", fname);
  }
  DG_TRY(check_no_alias(d, "d", a, "a"));
  DG_TRY(check_no_alias(d, "d", b, "b"));
  if (meta != nullptr) DG_TRY(check_no_alias(d, "d", meta, "metadata"));
  bool c_f32 = false;
  int64_t ldc = 0, c_gs = 0;
  if (c != nullptr) {
    // C shaped like d: [M, N] (dense), [Msum, N] (contiguous), [G, max_m, N]
    // or [G*max_m, N] (masked, its own group stride)
    DG_TRY(check_basic(c, "c", true));
    if (c->dtype != DG_BF16 && c->dtype != DG_F32) return fail(DG_INVALID_ARG, "%s: c must be BF16 or F32", fname);
    View3 vc;
    if (mode == dgmi::MODE_MASKED) {
      DG_TRY(view3(c, "c", G, max_m, &vc));
    } else {
      if (c->ndim != 2) return fail(DG_INVALID_ARG, "%s: c must be 2-D", fname);
      DG_TRY(view3(c, "c", 1, 0, &vc));
    }
    if ((mode == dgmi::MODE_MASKED && vc.G != G) || vc.R != M || vc.C != N)
      return fail(DG_INVALID_ARG, "%s: c must have the shape of d ([..,%lld,%lld])", fname, (long long)M,
                  (long long)N);
    c_f32 = c->dtype == DG_F32;
    if (!aligned(c->data, c_f32 ? 4 : 2)) return fail(DG_INVALID_ARG, "%s: c must be element-aligned", fname);
    ldc = vc.sr;
    c_gs = vc.sg;
    const bool same_as_d = c->data == d->data && c->dtype == d->dtype && ldc == vd.sr && (G <= 1 || c_gs == vd.sg);
    if (!same_as_d) DG_TRY(check_no_alias(d, "d", c, "c"));
  }
  // the kernel addresses A and B in bytes
  dgmi::GemmParams p = {};
  p.a = static_cast<const uint8_t*>(a->data);
  p.b = static_cast<const uint8_t*>(b->data);
  p.d = static_cast<uint16_t*>(d->data);
  p.d_f32 = d_f32 ? 1 : 0;
  p.c = c != nullptr ? c->data : nullptr;
  p.ldc = ldc;
  p.c_gs = c_gs;
  p.c_f32 = c_f32 ? 1 : 0;
  p.meta = meta ? static_cast<const int32_t*>(meta->data) : nullptr;
  p.lda = 2 * va.sr;
  p.a_gs = 2 * va.sg;
  p.ldb = 2 * vb.sr;
  p.b_gs = 2 * vb.sg;
  p.ldd = vd.sr;
  p.d_gs = d_f32 ? 2 * vd.sg : vd.sg;  // (the kernels step d in BF16-sized units)
  p.M = (int32_t)M;
  p.N = (int32_t)N;
  p.k_bytes = (int32_t)(2 * K);
  p.G = (int32_t)G;
  if (G == 0 || M == 0 || N == 0) return ok();
  if (K == 0) return fail(DG_UNSUPPORTED, "%s: K = 0 is not supported", fname);
  return check_launch(dgmi::launch_bf16_gemm(p, mode, stream), fname);
}

}  // namespace

extern "C" {

const char* dg_last_error(void) { return g_err.c_str(); }

int dgmi_init(void) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(DG_LAUNCH_FAILED, "dgmi_init: no HIP device: %s", hipGetErrorString(e));
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return fail(DG_LAUNCH_FAILED, "dgmi_init: %s", hipGetErrorString(e));
  if (std::string(prop.gcnArchName).rfind("gfx950", 0) != 0)
    return fail(DG_UNSUPPORTED, "dgmi_init: device %d is %s, this library is built for gfx950", dev, prop.gcnArchName);
  return ok();
}

int fp8_gemm_nt(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                const dg_tensor* c, const dg_tensor* d, hipStream_t stream) {
  return fp8_gemm_common(dgmi::MODE_DENSE, a, b, sfa, sfb, c, d, nullptr, 0, stream, "fp8_gemm_nt");
}

// The other three layouts: a descriptor given in its stored shape ([K, M]
// for A, [K, N] for B, row-major) is viewed as its transpose and handed to
// the common path, which takes the view as MN-major.
namespace {
int transposed(const dg_tensor* t, const char* name, const char* fname, dg_tensor* out) {
  if (t == nullptr) return fail(DG_INVALID_ARG, "%s: %s descriptor is NULL", fname, name);
  if (t->ndim != 2) return fail(DG_INVALID_ARG, "%s: %s must be 2-D", fname, name);
  *out = *t;
  out->shape[0] = t->shape[1];
  out->shape[1] = t->shape[0];
  out->stride[0] = t->stride[1];
  out->stride[1] = t->stride[0];
  if (t->shape[1] > 1 && t->stride[1] != 1)
    return fail(DG_INVALID_ARG, "%s: %s must be row-major (innermost stride 1)", fname, name);
  return DG_OK;
}
}  // namespace

int fp8_gemm_nn(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                const dg_tensor* c, const dg_tensor* d, hipStream_t stream) {
  dg_tensor bt;
  DG_TRY(transposed(b, "b", "fp8_gemm_nn", &bt));
  return fp8_gemm_common(dgmi::MODE_DENSE, a, &bt, sfa, sfb, c, d, nullptr, 0, stream, "fp8_gemm_nn");
}

int fp8_gemm_tn(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                const dg_tensor* c, const dg_tensor* d, hipStream_t stream) {
  dg_tensor at, bt;
  DG_TRY(transposed(a, "a", "fp8_gemm_tn", &at));
  DG_TRY(transposed(b, "b", "fp8_gemm_tn", &bt));
  return fp8_gemm_common(dgmi::MODE_DENSE, &at, &bt, sfa, sfb, c, d, nullptr, 0, stream, "fp8_gemm_tn");
}

int fp8_gemm_tt(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                const dg_tensor* c, const dg_tensor* d, hipStream_t stream) {
  dg_tensor at;
  DG_TRY(transposed(a, "a", "fp8_gemm_tt", &at));
  return fp8_gemm_common(dgmi::MODE_DENSE, &at, b, sfa, sfb, c, d, nullptr, 0, stream, "fp8_gemm_tt");
}

int fp8_gemm_nt_fp8_out(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                        const dg_tensor* c, const dg_tensor* q, const dg_tensor* sfq, int use_ue8m0,
                        hipStream_t stream) {
  if (q == nullptr || sfq == nullptr) return fail(DG_INVALID_ARG, "fp8_gemm_nt_fp8_out: q and sfq must not be NULL");
  return fp8_gemm_common(dgmi::MODE_DENSE, a, b, sfa, sfb, c, nullptr, nullptr, 0, stream, "fp8_gemm_nt_fp8_out", q,
                         sfq, use_ue8m0);
}

int m_grouped_fp8_gemm_nt_contiguous(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa,
                                     const dg_tensor* sfb, const dg_tensor* d, const dg_tensor* grouped_layout,
                                     hipStream_t stream) {
  if (grouped_layout == nullptr) return fail(DG_INVALID_ARG, "m_grouped_fp8_gemm_nt_contiguous: grouped_layout is NULL");
  return fp8_gemm_common(dgmi::MODE_CONTIG, a, b, sfa, sfb, nullptr, d, grouped_layout, 0, stream,
                         "m_grouped_fp8_gemm_nt_contiguous");
}

int m_grouped_fp8_gemm_nt_masked(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa, const dg_tensor* sfb,
                                 const dg_tensor* d, const dg_tensor* masked_m, int64_t max_m_per_group,
                                 hipStream_t stream) {
  if (masked_m == nullptr) return fail(DG_INVALID_ARG, "m_grouped_fp8_gemm_nt_masked: masked_m is NULL");
  return fp8_gemm_common(dgmi::MODE_MASKED, a, b, sfa, sfb, nullptr, d, masked_m, max_m_per_group, stream,
                         "m_grouped_fp8_gemm_nt_masked");
}

int m_grouped_fp8_gemm_nt_contiguous_acc(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa,
                                         const dg_tensor* sfb, const dg_tensor* c, const dg_tensor* d,
                                         const dg_tensor* grouped_layout, hipStream_t stream) {
  if (grouped_layout == nullptr)
    return fail(DG_INVALID_ARG, "m_grouped_fp8_gemm_nt_contiguous_acc: grouped_layout is NULL");
  return fp8_gemm_common(dgmi::MODE_CONTIG, a, b, sfa, sfb, c, d, grouped_layout, 0, stream,
                         "m_grouped_fp8_gemm_nt_contiguous_acc");
}

int m_grouped_fp8_gemm_nt_masked_acc(const dg_tensor* a, const dg_tensor* b, const dg_tensor* sfa,
                                     const dg_tensor* sfb, const dg_tensor* c, const dg_tensor* d,
                                     const dg_tensor* masked_m, int64_t max_m_per_group, hipStream_t stream) {
  if (masked_m == nullptr) return fail(DG_INVALID_ARG, "m_grouped_fp8_gemm_nt_masked_acc: masked_m is NULL");
  return fp8_gemm_common(dgmi::MODE_MASKED, a, b, sfa, sfb, c, d, masked_m, max_m_per_group, stream,
                         "m_grouped_fp8_gemm_nt_masked_acc");
}

int bf16_gemm_nt(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c, const dg_tensor* d, hipStream_t stream) {
  return bf16_gemm_common(dgmi::MODE_DENSE, a, b, c, d, nullptr, 0, stream, "bf16_gemm_nt");
}

int m_grouped_bf16_gemm_nt_contiguous(const dg_tensor* a, const dg_tensor* b, const dg_tensor* d,
                                      const dg_tensor* grouped_layout, hipStream_t stream) {
  if (grouped_layout == nullptr) return fail(DG_INVALID_ARG, "m_grouped_bf16_gemm_nt_contiguous: grouped_layout is NULL");
  return bf16_gemm_common(dgmi::MODE_CONTIG, a, b, nullptr, d, grouped_layout, 0, stream,
                          "m_grouped_bf16_gemm_nt_contiguous");
}

int m_grouped_bf16_gemm_nt_masked(const dg_tensor* a, const dg_tensor* b, const dg_tensor* d,
                                  const dg_tensor* masked_m, int64_t max_m_per_group, hipStream_t stream) {
  if (masked_m == nullptr) return fail(DG_INVALID_ARG, "m_grouped_bf16_gemm_nt_masked: masked_m is NULL");
  return bf16_gemm_common(dgmi::MODE_MASKED, a, b, nullptr, d, masked_m, max_m_per_group, stream,
                          "m_grouped_bf16_gemm_nt_masked");
}

int m_grouped_bf16_gemm_nt_contiguous_acc(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c,
                                          const dg_tensor* d, const dg_tensor* grouped_layout, hipStream_t stream) {
  if (grouped_layout == nullptr)
    return fail(DG_INVALID_ARG, "m_grouped_bf16_gemm_nt_contiguous_acc: grouped_layout is NULL");
  return bf16_gemm_common(dgmi::MODE_CONTIG, a, b, c, d, grouped_layout, 0, stream,
                          "m_grouped_bf16_gemm_nt_contiguous_acc");
}

int m_grouped_bf16_gemm_nt_masked_acc(const dg_tensor* a, const dg_tensor* b, const dg_tensor* c, const dg_tensor* d,
                                      const dg_tensor* masked_m, int64_t max_m_per_group, hipStream_t stream) {
  if (masked_m == nullptr) return fail(DG_INVALID_ARG, "m_grouped_bf16_gemm_nt_masked_acc: masked_m is NULL");
  return bf16_gemm_common(dgmi::MODE_MASKED, a, b, c, d, masked_m, max_m_per_group, stream,
                          "m_grouped_bf16_gemm_nt_masked_acc");
}

int per_token_cast_to_fp8(const dg_tensor* x, const dg_tensor* q, const dg_tensor* sf, int use_ue8m0,
                          hipStream_t stream) {
  return quant_common(x, q, sf, use_ue8m0, stream, false, "per_token_cast_to_fp8");
}

int per_block_cast_to_fp8(const dg_tensor* x, const dg_tensor* q, const dg_tensor* sf, int use_ue8m0,
                          hipStream_t stream) {
  return quant_common(x, q, sf, use_ue8m0, stream, true, "per_block_cast_to_fp8");
}

int pack_ue8m0_to_int(const dg_tensor* x, const dg_tensor* out, int32_t* invalid_count, hipStream_t stream) {
  const char* fname = "pack_ue8m0_to_int";
  DG_TRY(check_basic(x, "x", true));
  DG_TRY(check_basic(out, "out", true));
  DG_TRY(check_dtype(x, "x", DG_F32));
  DG_TRY(check_dtype(out, "out", DG_I32));
  if (x->ndim != out->ndim || x->ndim > 3) return fail(DG_INVALID_ARG, "%s: x and out must have the same rank (1..3)", fname);
  for (int i = 0; i + 1 < x->ndim; ++i)
    if (x->shape[i] != out->shape[i]) return fail(DG_INVALID_ARG, "%s: leading shapes of x and out differ", fname);
  const int64_t n = x->shape[x->ndim - 1];
  const int64_t nw = (n + 3) / 4;
  if (out->shape[out->ndim - 1] != nw)
    return fail(DG_INVALID_ARG, "%s: out has %lld words per row, expected ceil(%lld/4) = %lld", fname,
                (long long)out->shape[out->ndim - 1], (long long)n, (long long)nw);
  if (!aligned(x->data, 4) || !aligned(out->data, 4)) return fail(DG_INVALID_ARG, "%s: x and out must be 4-byte aligned", fname);
  DG_TRY(check_no_alias(out, "out", x, "x"));
  dgmi::PackArgs p = {};
  p.x = static_cast<const float*>(x->data);
  p.out = static_cast<int32_t*>(out->data);
  p.n = (int32_t)n;
  p.nw = (int32_t)nw;
  p.invalid = invalid_count;
  if (x->ndim == 1) {
    p.G = 1; p.R = 1; p.sx_g = p.sx_r = 0; p.so_g = p.so_r = 0;
  } else if (x->ndim == 2) {
    p.G = 1; p.R = (int32_t)x->shape[0]; p.sx_g = 0; p.sx_r = x->stride[0]; p.so_g = 0; p.so_r = out->stride[0];
  } else {
    p.G = (int32_t)x->shape[0]; p.R = (int32_t)x->shape[1];
    p.sx_g = x->stride[0]; p.sx_r = x->stride[1]; p.so_g = out->stride[0]; p.so_r = out->stride[1];
  }
  if (p.G == 0 || p.R == 0 || nw == 0) return ok();
  return check_launch(dgmi::launch_pack_ue8m0(p, stream), fname);
}

int moe_dispatch_masked_fp8(const dg_tensor* x, const dg_tensor* topk_idx, const dg_tensor* a, const dg_tensor* sfa,
                            const dg_tensor* masked_m, const dg_tensor* slot, const dg_tensor* src, int use_ue8m0,
                            hipStream_t stream) {
  const char* fname = "moe_dispatch_masked_fp8";
  DG_TRY(check_basic(x, "x", true));
  DG_TRY(check_basic(topk_idx, "topk_idx", true));
  DG_TRY(check_basic(a, "a", true));
  DG_TRY(check_basic(sfa, "sfa", false));
  DG_TRY(check_basic(masked_m, "masked_m", true));
  DG_TRY(check_basic(slot, "slot", true));
  DG_TRY(check_basic(src, "src", true));
  if (x->dtype != DG_F32 && x->dtype != DG_BF16) return fail(DG_INVALID_ARG, "%s: x must be F32 or BF16", fname);
  DG_TRY(check_dtype(topk_idx, "topk_idx", DG_I32));
  DG_TRY(check_dtype(a, "a", DG_E4M3));
  DG_TRY(check_dtype(sfa, "sfa", DG_F32));
  DG_TRY(check_dtype(masked_m, "masked_m", DG_I32));
  DG_TRY(check_dtype(slot, "slot", DG_I32));
  DG_TRY(check_dtype(src, "src", DG_I32));
  if (x->ndim != 2 || topk_idx->ndim != 2 || a->ndim != 3 || sfa->ndim != 3 || masked_m->ndim != 1 ||
      slot->ndim != 2 || src->ndim != 2)
    return fail(DG_INVALID_ARG, "%s: x [T, K], topk_idx [T, k], a [G, max_m, K], sfa [G, max_m, K/128], "
                "masked_m [G], slot [T, k], src [G, max_m]", fname);
  const int64_t T = x->shape[0], K = x->shape[1], k = topk_idx->shape[1];
  const int64_t G = a->shape[0], max_m = a->shape[1];
  if (topk_idx->shape[0] != T) return fail(DG_INVALID_ARG, "%s: topk_idx must have T = %lld rows", fname, (long long)T);
  if (a->shape[2] != K) return fail(DG_INVALID_ARG, "%s: a must be [G, max_m, K = %lld]", fname, (long long)K);
  if (sfa->shape[0] != G || sfa->shape[1] != max_m || sfa->shape[2] != (K + 127) / 128)
    return fail(DG_INVALID_ARG, "%s: sfa must be [G, max_m, ceil(K/128)] = [%lld, %lld, %lld]", fname, (long long)G,
                (long long)max_m, (long long)((K + 127) / 128));
  if (masked_m->shape[0] != G) return fail(DG_INVALID_ARG, "%s: masked_m must be [G = %lld]", fname, (long long)G);
  if (slot->shape[0] != T || slot->shape[1] != k)
    return fail(DG_INVALID_ARG, "%s: slot must have the shape of topk_idx", fname);
  if (src->shape[0] != G || src->shape[1] != max_m)
    return fail(DG_INVALID_ARG, "%s: src must be [G, max_m] = [%lld, %lld]", fname, (long long)G, (long long)max_m);
  // the routing tables are read and written as flat arrays
  if ((T > 1 && topk_idx->stride[0] != k) || (T > 1 && slot->stride[0] != k) || (G > 1 && src->stride[0] != max_m))
    return fail(DG_INVALID_ARG, "%s: topk_idx, slot and src must be contiguous", fname);
  if (G * max_m > INT32_MAX || T * k > INT32_MAX)
    return fail(DG_UNSUPPORTED, "%s: G * max_m and T * k must fit in int32", fname);
  const int xe = elem_size(x->dtype);
  if (!aligned(x->data, 16) || (T > 1 && (x->stride[0] * xe) % 16))
    return fail(DG_INVALID_ARG, "%s: x needs a 16-byte aligned base and row stride", fname);
  if (!aligned(a->data, 4) || (max_m > 1 && a->stride[1] % 4) || (G > 1 && a->stride[0] % 4))
    return fail(DG_INVALID_ARG, "%s: a needs a 4-byte aligned base and row/group strides", fname);
  if (!aligned(sfa->data, 4)) return fail(DG_INVALID_ARG, "%s: sfa must be 4-byte aligned", fname);
  const dg_tensor* outs[] = {a, sfa, masked_m, slot, src};
  const char* onames[] = {"a", "sfa", "masked_m", "slot", "src"};
  for (int i = 0; i < 5; ++i) {
    DG_TRY(check_no_alias(outs[i], onames[i], x, "x"));
    DG_TRY(check_no_alias(outs[i], onames[i], topk_idx, "topk_idx"));
    for (int j = i + 1; j < 5; ++j) DG_TRY(check_no_alias(outs[i], onames[i], outs[j], onames[j]));
  }
  if (G == 0) return ok();
  dgmi::MoeRouteArgs r = {};
  r.topk = static_cast<const int32_t*>(topk_idx->data);
  r.T = (int32_t)T;
  r.k = (int32_t)k;
  r.G = (int32_t)G;
  r.max_m = (int32_t)max_m;
  r.vec = aligned(topk_idx->data, 16) ? 1 : 0;
  r.masked_m = static_cast<int32_t*>(masked_m->data);
  r.slot = static_cast<int32_t*>(slot->data);
  r.src = static_cast<int32_t*>(src->data);
  hipError_t e = dgmi::launch_moe_route(r, stream);
  if (e != hipSuccess || max_m == 0 || K == 0 || T == 0 || k == 0) return check_launch(e, fname);
  // the per-token cast of each token, stored into every row its slots name
  dgmi::QuantScatterArgs q = {};
  q.x = x->data;
  q.x_bf16 = x->dtype == DG_BF16;
  q.sx_g = 0;
  q.sx_r = x->stride[0];
  q.q = static_cast<uint8_t*>(a->data);
  q.sq_g = a->stride[0];
  q.sq_r = a->stride[1];
  q.sf = static_cast<float*>(sfa->data);
  q.ssf_g = sfa->stride[0];
  q.ssf_r = sfa->stride[1];
  q.ssf_k = sfa->stride[2];
  q.G = 1;
  q.R = (int32_t)T;
  q.K = (int32_t)K;
  q.ue8m0 = use_ue8m0 ? 1 : 0;
  q.slot = r.slot;
  q.k = (int32_t)k;
  q.max_m = (int32_t)max_m;
  q.rows = (int32_t)(G * max_m);
  q.flat = (q.sq_g == max_m * q.sq_r && q.ssf_g == max_m * q.ssf_r) ? 1 : 0;
  q.qvec = (aligned(a->data, 16) && q.sq_r % 16 == 0 && q.sq_g % 16 == 0) ? 1 : 0;
  return check_launch(dgmi::launch_per_token_scatter(q, stream), fname);
}

int moe_dispatch_contiguous_fp8(const dg_tensor* x, const dg_tensor* topk_idx, const dg_tensor* a,
                                const dg_tensor* sfa, const dg_tensor* grouped_layout, const dg_tensor* counts,
                                const dg_tensor* slot, int32_t align, int use_ue8m0, hipStream_t stream) {
  const char* fname = "moe_dispatch_contiguous_fp8";
  if (align != 128 && align != 256) return fail(DG_INVALID_ARG, "%s: align must be 128 or 256 (got %d)", fname, align);
  DG_TRY(check_basic(x, "x", true));
  DG_TRY(check_basic(topk_idx, "topk_idx", true));
  DG_TRY(check_basic(a, "a", true));
  DG_TRY(check_basic(sfa, "sfa", false));
  DG_TRY(check_basic(grouped_layout, "grouped_layout", true));
  DG_TRY(check_basic(counts, "counts", true));
  DG_TRY(check_basic(slot, "slot", true));
  if (x->dtype != DG_F32 && x->dtype != DG_BF16) return fail(DG_INVALID_ARG, "%s: x must be F32 or BF16", fname);
  DG_TRY(check_dtype(topk_idx, "topk_idx", DG_I32));
  DG_TRY(check_dtype(a, "a", DG_E4M3));
  DG_TRY(check_dtype(sfa, "sfa", DG_F32));
  DG_TRY(check_dtype(grouped_layout, "grouped_layout", DG_I32));
  DG_TRY(check_dtype(counts, "counts", DG_I32));
  DG_TRY(check_dtype(slot, "slot", DG_I32));
  if (x->ndim != 2 || topk_idx->ndim != 2 || a->ndim != 2 || sfa->ndim != 2 || grouped_layout->ndim != 1 ||
      counts->ndim != 1 || slot->ndim != 2)
    return fail(DG_INVALID_ARG, "%s: x [T, K], topk_idx [T, k], a [Mcap, K], sfa [Mcap, K/128], "
                "grouped_layout [Mcap/128], counts [G], slot [T, k]", fname);
  const int64_t T = x->shape[0], K = x->shape[1], k = topk_idx->shape[1];
  const int64_t Mcap = a->shape[0], G = counts->shape[0];
  if (topk_idx->shape[0] != T) return fail(DG_INVALID_ARG, "%s: topk_idx must have T = %lld rows", fname, (long long)T);
  if (a->shape[1] != K) return fail(DG_INVALID_ARG, "%s: a must be [Mcap, K = %lld]", fname, (long long)K);
  if (Mcap % 128 != 0) return fail(DG_INVALID_ARG, "%s: Mcap = %lld is not a multiple of 128", fname, (long long)Mcap);
  if (sfa->shape[0] != Mcap || sfa->shape[1] != (K + 127) / 128)
    return fail(DG_INVALID_ARG, "%s: sfa must be [Mcap, ceil(K/128)] = [%lld, %lld]", fname, (long long)Mcap,
                (long long)((K + 127) / 128));
  if (grouped_layout->shape[0] != Mcap / 128)
    return fail(DG_INVALID_ARG, "%s: grouped_layout must be [Mcap/128 = %lld]", fname, (long long)(Mcap / 128));
  if (slot->shape[0] != T || slot->shape[1] != k)
    return fail(DG_INVALID_ARG, "%s: slot must have the shape of topk_idx", fname);
  if ((T > 1 && topk_idx->stride[0] != k) || (T > 1 && slot->stride[0] != k))
    return fail(DG_INVALID_ARG, "%s: topk_idx and slot must be contiguous", fname);
  if (Mcap > INT32_MAX || T * k > INT32_MAX)
    return fail(DG_UNSUPPORTED, "%s: Mcap and T * k must fit in int32", fname);
  const int xe = elem_size(x->dtype);
  if (!aligned(x->data, 16) || (T > 1 && (x->stride[0] * xe) % 16))
    return fail(DG_INVALID_ARG, "%s: x needs a 16-byte aligned base and row stride", fname);
  if (!aligned(a->data, 4) || (Mcap > 1 && a->stride[0] % 4))
    return fail(DG_INVALID_ARG, "%s: a needs a 4-byte aligned base and row stride", fname);
  if (!aligned(sfa->data, 4)) return fail(DG_INVALID_ARG, "%s: sfa must be 4-byte aligned", fname);
  const dg_tensor* outs[] = {a, sfa, grouped_layout, counts, slot};
  const char* onames[] = {"a", "sfa", "grouped_layout", "counts", "slot"};
  for (int i = 0; i < 5; ++i) {
    DG_TRY(check_no_alias(outs[i], onames[i], x, "x"));
    DG_TRY(check_no_alias(outs[i], onames[i], topk_idx, "topk_idx"));
    for (int j = i + 1; j < 5; ++j) DG_TRY(check_no_alias(outs[i], onames[i], outs[j], onames[j]));
  }
  if (Mcap == 0 && G == 0) return ok();
  dgmi::MoeRouteArgs r = {};
  r.topk = static_cast<const int32_t*>(topk_idx->data);
  r.T = (int32_t)T;
  r.k = (int32_t)k;
  r.G = (int32_t)G;
  r.vec = aligned(topk_idx->data, 16) ? 1 : 0;
  r.slot = static_cast<int32_t*>(slot->data);
  r.counts = static_cast<int32_t*>(counts->data);
  r.layout = static_cast<int32_t*>(grouped_layout->data);
  r.mcap = Mcap;
  r.align = align;
  hipError_t e = dgmi::launch_moe_route_contiguous(r, stream);
  if (e != hipSuccess || Mcap == 0 || K == 0 || T == 0 || k == 0) return check_launch(e, fname);
  // the per-token cast of each token, stored into every row its slots name
  dgmi::QuantScatterArgs q = {};
  q.x = x->data;
  q.x_bf16 = x->dtype == DG_BF16;
  q.sx_g = 0;
  q.sx_r = x->stride[0];
  q.q = static_cast<uint8_t*>(a->data);
  q.sq_g = 0;
  q.sq_r = a->stride[0];
  q.sf = static_cast<float*>(sfa->data);
  q.ssf_g = 0;
  q.ssf_r = sfa->stride[0];
  q.ssf_k = sfa->stride[1];
  q.G = 1;
  q.R = (int32_t)T;
  q.K = (int32_t)K;
  q.ue8m0 = use_ue8m0 ? 1 : 0;
  q.slot = r.slot;
  q.k = (int32_t)k;
  q.max_m = (int32_t)Mcap;
  q.rows = (int32_t)Mcap;
  q.flat = 1;  // a slot is a row of a and sfa
  q.qvec = (aligned(a->data, 16) && q.sq_r % 16 == 0) ? 1 : 0;
  return check_launch(dgmi::launch_per_token_scatter(q, stream), fname);
}

int moe_combine(const dg_tensor* d, const dg_tensor* slot, const dg_tensor* topk_weights, const dg_tensor* y,
                hipStream_t stream) {
  const char* fname = "moe_combine";
  DG_TRY(check_basic(d, "d", true));
  DG_TRY(check_basic(slot, "slot", true));
  DG_TRY(check_basic(topk_weights, "topk_weights", true));
  DG_TRY(check_basic(y, "y", true));
  DG_TRY(check_dtype(d, "d", DG_BF16));
  DG_TRY(check_dtype(slot, "slot", DG_I32));
  DG_TRY(check_dtype(topk_weights, "topk_weights", DG_F32));
  DG_TRY(check_dtype(y, "y", DG_BF16));
  if (d->ndim != 3 || slot->ndim != 2 || topk_weights->ndim != 2 || y->ndim != 2)
    return fail(DG_INVALID_ARG, "%s: d [G, max_m, N], slot [T, k], topk_weights [T, k], y [T, N]", fname);
  const int64_t G = d->shape[0], max_m = d->shape[1], N = d->shape[2], T = slot->shape[0], k = slot->shape[1];
  if (topk_weights->shape[0] != T || topk_weights->shape[1] != k)
    return fail(DG_INVALID_ARG, "%s: topk_weights must have the shape of slot", fname);
  if (y->shape[0] != T || y->shape[1] != N)
    return fail(DG_INVALID_ARG, "%s: y must be [T, N] = [%lld, %lld]", fname, (long long)T, (long long)N);
  if ((T > 1 && slot->stride[0] != k) || (T > 1 && topk_weights->stride[0] != k))
    return fail(DG_INVALID_ARG, "%s: slot and topk_weights must be contiguous", fname);
  if (G * max_m > INT32_MAX) return fail(DG_UNSUPPORTED, "%s: G * max_m must fit in int32", fname);
  if (!aligned(d->data, 2) || !aligned(y->data, 2)) return fail(DG_INVALID_ARG, "%s: d and y must be 2-byte aligned", fname);
  DG_TRY(check_no_alias(y, "y", d, "d"));
  DG_TRY(check_no_alias(y, "y", slot, "slot"));
  DG_TRY(check_no_alias(y, "y", topk_weights, "topk_weights"));
  dgmi::MoeCombineArgs p = {};
  p.d = static_cast<const uint16_t*>(d->data);
  p.sd_g = d->stride[0];
  p.sd_r = d->stride[1];
  p.G = (int32_t)G;
  p.max_m = (int32_t)max_m;
  p.N = (int32_t)N;
  p.slot = static_cast<const int32_t*>(slot->data);
  p.w = static_cast<const float*>(topk_weights->data);
  p.T = (int32_t)T;
  p.k = (int32_t)k;
  p.y = static_cast<uint16_t*>(y->data);
  p.sy = y->stride[0];
  p.vec = (aligned(d->data, 16) && (max_m <= 1 || d->stride[1] % 8 == 0) && (G <= 1 || d->stride[0] % 8 == 0)) ? 1 : 0;
  p.y_vec = (aligned(y->data, 16) && (T <= 1 || y->stride[0] % 8 == 0)) ? 1 : 0;
  if (T == 0 || N == 0) return ok();
  return check_launch(dgmi::launch_moe_combine(p, stream), fname);
}

namespace {

// Row indices and weights of the routing: [T, k], unit innermost stride, any row stride.
int check_routes(const dg_tensor* t, const char* name, int32_t dtype, int64_t T, int64_t k, const char* fname) {
  DG_TRY(check_basic(t, name, true));
  DG_TRY(check_dtype(t, name, dtype));
  if (t->ndim != 2 || t->shape[0] != T || t->shape[1] != k)
    return fail(DG_INVALID_ARG, "%s: %s must be [T, k] = [%lld, %lld]", fname, name, (long long)T, (long long)k);
  if (!aligned(t->data, 4)) return fail(DG_INVALID_ARG, "%s: %s must be 4-byte aligned", fname, name);
  return DG_OK;
}

// An output whose rows overlap each other would be written by two workgroups.
int check_rows_apart(const dg_tensor* t, const char* name) {
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] <= 1) continue;
    int64_t inner = 1;  // elements spanned by the dims of smaller stride
    for (int j = 0; j < t->ndim; ++j) {
      if (t->shape[j] == 0) return DG_OK;
      if (j != i && (t->stride[j] < t->stride[i] || (t->stride[j] == t->stride[i] && j > i)))
        inner += (t->shape[j] - 1) * t->stride[j];
    }
    if (t->stride[i] < inner) return fail(DG_INVALID_ARG, "%s: rows overlap in memory", name);
  }
  return DG_OK;
}

// Two strided tensors whose memory ranges may interleave: is there an element
// of both?  That is a combination of their strides, with coefficients in the
// ranges of their indexes (b's negative, equal strides taken together), that
// equals the distance of their bases.  Sought from the largest stride down, where
// what the smaller ones can reach leaves one or two coefficients for tensors of
// alike strides; a search that grows past `budget` steps counts as an overlap.
struct Stride {
  int64_t by, lo, hi;  // stride, range of its coefficient
};
bool reaches(const Stride* d, int n, int64_t left, int* budget) {
  if (n == 0) return left == 0;
  if (--*budget < 0) return true;
  int64_t lo = 0, hi = 0;  // what the smaller strides reach
  for (int i = 1; i < n; ++i) {
    lo += d[i].lo * d[i].by;
    hi += d[i].hi * d[i].by;
  }
  // the first coefficient that leaves no more than hi, up to the last that leaves no less than lo
  const int64_t most = left - hi, least = left - lo;
  int64_t c = most >= 0 ? (most + d->by - 1) / d->by : -(-most / d->by);
  const int64_t end = least >= 0 ? least / d->by : -((-least + d->by - 1) / d->by);
  if (c < d->lo) c = d->lo;
  for (; c <= end && c <= d->hi; ++c)
    if (reaches(d + 1, n - 1, left - c * d->by, budget)) return true;
  return false;
}
int check_apart(const dg_tensor* a, const char* aname, const dg_tensor* b, const char* bname) {
  uintptr_t a0, a1, b0, b1;
  span(a, &a0, &a1);
  span(b, &b0, &b1);
  if (a0 >= a1 || b0 >= b1 || a0 >= b1 || b0 >= a1) return DG_OK;
  Stride d[8];
  int n = 0;
  const auto add = [&](int64_t by, int64_t lo, int64_t hi) {
    if (lo == hi || by == 0) return;
    int at = 0;
    while (at < n && d[at].by > by) ++at;
    if (at < n && d[at].by == by) {
      d[at].lo += lo;
      d[at].hi += hi;
      return;
    }
    for (int i = n++; i > at; --i) d[i] = d[i - 1];
    d[at] = Stride{by, lo, hi};
  };
  for (int i = 0; i < a->ndim; ++i) add(a->stride[i], 0, a->shape[i] - 1);
  for (int i = 0; i < b->ndim; ++i) add(b->stride[i], 1 - b->shape[i], 0);
  const int64_t es = elem_size(a->dtype);  // (both bases are aligned to it)
  int budget = 256;
  if (reaches(d, n, ((int64_t)b0 - (int64_t)a0) / es, &budget))
    return fail(DG_INVALID_ARG, "%s and %s overlap in memory", aname, bname);
  return DG_OK;
}

// Logits [T, E] in FP32 or BF16.
int check_logits(const dg_tensor* t, const char* name, const char* fname) {
  DG_TRY(check_basic(t, name, true));
  if (t->dtype != DG_F32 && t->dtype != DG_BF16) return fail(DG_INVALID_ARG, "%s: %s must be F32 or BF16", fname, name);
  if (t->ndim != 2) return fail(DG_INVALID_ARG, "%s: %s must be [T, E]", fname, name);
  if (!aligned(t->data, elem_size(t->dtype))) return fail(DG_INVALID_ARG, "%s: %s must be element-aligned", fname, name);
  return DG_OK;
}

// Workgroups of one launch of 256 threads each: the grid's threads are counted in 32 bits.
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;

int check_route_limits(int64_t T, int64_t E, int64_t k, int32_t score, float scale, const char* fname) {
  if (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID)
    return fail(DG_INVALID_ARG, "%s: score must be DG_SCORE_SOFTMAX or DG_SCORE_SIGMOID (got %d)", fname, score);
  if (k > E) return fail(DG_INVALID_ARG, "%s: k = %lld choices out of E = %lld experts", fname, (long long)k, (long long)E);
  if (E > 1024 || k > 64)
    return fail(DG_UNSUPPORTED, "%s: at most 1024 experts and 64 choices (got %lld, %lld)", fname, (long long)E, (long long)k);
  if (T > (int64_t(1) << 25)) return fail(DG_UNSUPPORTED, "%s: at most 2^25 tokens a call (got %lld)", fname, (long long)T);
  if (!(scale - scale == 0.0f)) return fail(DG_INVALID_ARG, "%s: scale must be finite", fname);
  return DG_OK;
}

// A paged cache tensor [pages, Hkv, P, D] (strides of the first three dims
// free, rows of D bytes 16-byte aligned) and its scales [pages, Hkv].
int check_cache(const dg_tensor* c, const char* name, const dg_tensor* sc, const char* sname, const char* fname) {
  DG_TRY(check_basic(c, name, true));
  DG_TRY(check_dtype(c, name, DG_E4M3));
  DG_TRY(check_basic(sc, sname, false));
  DG_TRY(check_dtype(sc, sname, DG_F32));
  if (c->ndim != 4) return fail(DG_INVALID_ARG, "%s: %s must be [pages, Hkv, P, D]", fname, name);
  if (sc->ndim != 2 || sc->shape[0] != c->shape[0] || sc->shape[1] != c->shape[1])
    return fail(DG_INVALID_ARG, "%s: %s must be [pages, Hkv] = [%lld, %lld]", fname, sname, (long long)c->shape[0],
                (long long)c->shape[1]);
  if (!aligned(sc->data, 4)) return fail(DG_INVALID_ARG, "%s: %s must be 4-byte aligned", fname, sname);
  const int64_t P = c->shape[2], D = c->shape[3];
  if (D != 64 && D != 128 && D != 256)
    return fail(DG_UNSUPPORTED, "%s: head size %lld is not 64, 128 or 256", fname, (long long)D);
  if (P != 16 && P != 32 && P != 64 && P != 128)
    return fail(DG_UNSUPPORTED, "%s: page size %lld is not 16, 32, 64 or 128", fname, (long long)P);
  if (!aligned(c->data, 16) || c->stride[0] % 16 || c->stride[1] % 16 || c->stride[2] % 16)
    return fail(DG_INVALID_ARG, "%s: %s needs a 16-byte aligned base and strides", fname, name);
  // (a page's tokens and the page strides are reached with 32-bit offsets)
  if (c->stride[2] >= (int64_t(1) << 24) || (c->shape[0] > 1 && c->stride[0] >= (int64_t(1) << 32)) ||
      (sc->shape[0] > 1 && sc->stride[0] >= (int64_t(1) << 30)))
    return fail(DG_UNSUPPORTED, "%s: the token stride of %s must be below 2^24 bytes, its page stride below 2^32 bytes "
                "and that of %s below 2^30 elements", fname, name, sname);
  return DG_OK;
}

int check_caches(const dg_tensor* kc, const dg_tensor* ks, const dg_tensor* vc, const dg_tensor* vs, const char* fname) {
  DG_TRY(check_cache(kc, "k_cache", ks, "k_scale", fname));
  DG_TRY(check_cache(vc, "v_cache", vs, "v_scale", fname));
  for (int i = 0; i < 4; ++i)
    if (kc->shape[i] != vc->shape[i]) return fail(DG_INVALID_ARG, "%s: k_cache and v_cache differ in shape", fname);
  return DG_OK;
}

int check_table(const dg_tensor* t, int64_t S, int64_t P, const char* fname) {
  DG_TRY(check_basic(t, "block_table", true));
  DG_TRY(check_dtype(t, "block_table", DG_I32));
  if (t->ndim != 2 || t->shape[0] != S)
    return fail(DG_INVALID_ARG, "%s: block_table must be [S = %lld, max_pages]", fname, (long long)S);
  if (t->shape[1] * P > INT32_MAX - 256)
    return fail(DG_UNSUPPORTED, "%s: max_pages * P must be below 2^31 - 256", fname);
  if (!aligned(t->data, 4)) return fail(DG_INVALID_ARG, "%s: block_table must be 4-byte aligned", fname);
  return DG_OK;
}

int check_ints(const dg_tensor* t, const char* name, int64_t n, const char* fname) {
  DG_TRY(check_basic(t, name, true));
  DG_TRY(check_dtype(t, name, DG_I32));
  if (t->ndim != 1 || t->shape[0] != n)
    return fail(DG_INVALID_ARG, "%s: %s must be I32 [%lld]", fname, name, (long long)n);
  if (!aligned(t->data, 4)) return fail(DG_INVALID_ARG, "%s: %s must be 4-byte aligned", fname, name);
  return DG_OK;
}

// Head rows of D elements [.., D] read or written 16 bytes at a time.
int check_heads(const dg_tensor* t, const char* name, const char* fname) {
  const int es = elem_size(t->dtype);
  bool ok = aligned(t->data, 16);
  for (int i = 0; i + 1 < t->ndim; ++i) ok = ok && (t->shape[i] <= 1 || t->stride[i] * es % 16 == 0);
  if (!ok) return fail(DG_INVALID_ARG, "%s: %s needs a 16-byte aligned base and strides", fname, name);
  return DG_OK;
}

}  // namespace

int moe_route_topk(const dg_tensor* logits, const dg_tensor* bias, const dg_tensor* topk_idx,
                   const dg_tensor* topk_weights, int32_t score, int32_t n_group, int32_t topk_group,
                   int32_t group_top, int renormalize, float scale, hipStream_t stream) {
  const char* fname = "moe_route_topk";
  DG_TRY(check_logits(logits, "logits", fname));
  DG_TRY(check_basic(topk_idx, "topk_idx", true));
  if (topk_idx->ndim != 2) return fail(DG_INVALID_ARG, "%s: topk_idx must be [T, k]", fname);
  const int64_t T = logits->shape[0], E = logits->shape[1], k = topk_idx->shape[1];
  DG_TRY(check_routes(topk_idx, "topk_idx", DG_I32, T, k, fname));
  DG_TRY(check_routes(topk_weights, "topk_weights", DG_F32, T, k, fname));
  if (bias != nullptr) {
    DG_TRY(check_basic(bias, "bias", true));
    DG_TRY(check_dtype(bias, "bias", DG_F32));
    if (bias->ndim != 1 || bias->shape[0] != E) return fail(DG_INVALID_ARG, "%s: bias must be F32 [E = %lld]", fname, (long long)E);
    if (!aligned(bias->data, 4)) return fail(DG_INVALID_ARG, "%s: bias must be 4-byte aligned", fname);
  }
  DG_TRY(check_route_limits(T, E, k, score, scale, fname));
  if (n_group < 1 || (E > 0 && E % n_group != 0))
    return fail(DG_INVALID_ARG, "%s: n_group = %d must divide E = %lld", fname, n_group, (long long)E);
  if (n_group > 64) return fail(DG_UNSUPPORTED, "%s: at most 64 groups (got %d)", fname, n_group);
  if (topk_group < 1 || topk_group > n_group)
    return fail(DG_INVALID_ARG, "%s: topk_group must be in 1..n_group (got %d)", fname, topk_group);
  if (group_top != 1 && group_top != 2) return fail(DG_INVALID_ARG, "%s: group_top must be 1 or 2 (got %d)", fname, group_top);
  if (topk_group * (E / n_group) < k)
    return fail(DG_INVALID_ARG, "%s: %d groups of %lld experts hold fewer than k = %lld", fname, topk_group,
                (long long)(E / n_group), (long long)k);
  DG_TRY(check_rows_apart(topk_idx, "topk_idx"));
  DG_TRY(check_rows_apart(topk_weights, "topk_weights"));
  DG_TRY(check_no_alias(topk_idx, "topk_idx", logits, "logits"));
  DG_TRY(check_no_alias(topk_idx, "topk_idx", bias, "bias"));
  DG_TRY(check_no_alias(topk_weights, "topk_weights", logits, "logits"));
  DG_TRY(check_no_alias(topk_weights, "topk_weights", bias, "bias"));
  DG_TRY(check_no_alias(topk_weights, "topk_weights", topk_idx, "topk_idx"));
  if (T == 0 || k == 0) return ok();
  dgmi::RouteTopkArgs p = {};
  p.logits = logits->data;
  p.sl = logits->stride[0];
  p.bf16 = logits->dtype == DG_BF16;
  p.bias = bias ? static_cast<const float*>(bias->data) : nullptr;
  p.idx = static_cast<int32_t*>(topk_idx->data);
  p.si = topk_idx->stride[0];
  p.w = static_cast<float*>(topk_weights->data);
  p.sw = topk_weights->stride[0];
  p.T = (int32_t)T;
  p.E = (int32_t)E;
  p.k = (int32_t)k;
  p.n_group = topk_group == n_group ? 1 : n_group;  // every group stays
  p.group_size = (int32_t)(E / p.n_group);
  p.topk_group = topk_group;
  p.group_top = group_top;
  p.softmax = score == DG_SCORE_SOFTMAX;
  p.renorm = renormalize ? 1 : 0;
  p.scale = scale;
  return check_launch(dgmi::launch_moe_route_topk(p, stream), fname);
}

int moe_route_topk_bwd(const dg_tensor* logits, const dg_tensor* topk_idx, const dg_tensor* grad_weights,
                       const dg_tensor* grad_logits, int32_t score, int renormalize, float scale, hipStream_t stream) {
  const char* fname = "moe_route_topk_bwd";
  DG_TRY(check_logits(logits, "logits", fname));
  DG_TRY(check_logits(grad_logits, "grad_logits", fname));
  DG_TRY(check_basic(topk_idx, "topk_idx", true));
  if (topk_idx->ndim != 2) return fail(DG_INVALID_ARG, "%s: topk_idx must be [T, k]", fname);
  const int64_t T = logits->shape[0], E = logits->shape[1], k = topk_idx->shape[1];
  if (grad_logits->shape[0] != T || grad_logits->shape[1] != E)
    return fail(DG_INVALID_ARG, "%s: grad_logits must have the shape of logits", fname);
  DG_TRY(check_routes(topk_idx, "topk_idx", DG_I32, T, k, fname));
  DG_TRY(check_routes(grad_weights, "grad_weights", DG_F32, T, k, fname));
  DG_TRY(check_route_limits(T, E, k, score, scale, fname));
  DG_TRY(check_rows_apart(grad_logits, "grad_logits"));
  DG_TRY(check_no_alias(grad_logits, "grad_logits", logits, "logits"));
  DG_TRY(check_no_alias(grad_logits, "grad_logits", topk_idx, "topk_idx"));
  DG_TRY(check_no_alias(grad_logits, "grad_logits", grad_weights, "grad_weights"));
  if (T == 0 || E == 0) return ok();
  dgmi::RouteTopkBwdArgs p = {};
  p.logits = logits->data;
  p.sl = logits->stride[0];
  p.bf16 = logits->dtype == DG_BF16;
  p.idx = static_cast<const int32_t*>(topk_idx->data);
  p.si = topk_idx->stride[0];
  p.g = static_cast<const float*>(grad_weights->data);
  p.sg = grad_weights->stride[0];
  p.dlogits = grad_logits->data;
  p.so = grad_logits->stride[0];
  p.out_bf16 = grad_logits->dtype == DG_BF16;
  p.T = (int32_t)T;
  p.E = (int32_t)E;
  p.k = (int32_t)k;
  p.softmax = score == DG_SCORE_SOFTMAX;
  p.renorm = renormalize ? 1 : 0;
  p.scale = scale;
  return check_launch(dgmi::launch_moe_route_topk_bwd(p, stream), fname);
}

int kv_append_fp8(const dg_tensor* k, const dg_tensor* v, const dg_tensor* k_cache, const dg_tensor* v_cache,
                  const dg_tensor* k_scale, const dg_tensor* v_scale, const dg_tensor* block_table,
                  const dg_tensor* cu_tokens, const dg_tensor* start, const dg_tensor* cos_sin, const dg_tensor* q,
                  const dg_tensor* q_out, int interleaved, hipStream_t stream) {
  const char* fname = "kv_append_fp8";
  DG_TRY(check_basic(k, "k", true));
  DG_TRY(check_basic(v, "v", true));
  if (k->dtype != DG_F32 && k->dtype != DG_BF16) return fail(DG_INVALID_ARG, "%s: k must be F32 or BF16", fname);
  DG_TRY(check_dtype(v, "v", k->dtype));
  DG_TRY(check_caches(k_cache, k_scale, v_cache, v_scale, fname));
  const int64_t pages = k_cache->shape[0], Hkv = k_cache->shape[1], P = k_cache->shape[2], D = k_cache->shape[3];
  if (k->ndim != 3 || v->ndim != 3) return fail(DG_INVALID_ARG, "%s: k and v must be [T, Hkv, D]", fname);
  const int64_t T = k->shape[0];
  for (const dg_tensor* t : {k, v})
    if (t->shape[0] != T || t->shape[1] != Hkv || t->shape[2] != D)
      return fail(DG_INVALID_ARG, "%s: k and v must be [T, Hkv, D] = [%lld, %lld, %lld]", fname, (long long)T,
                  (long long)Hkv, (long long)D);
  DG_TRY(check_heads(k, "k", fname));
  DG_TRY(check_heads(v, "v", fname));
  DG_TRY(check_basic(start, "start", true));
  if (start->ndim != 1) return fail(DG_INVALID_ARG, "%s: start must be [S]", fname);
  const int64_t S = start->shape[0];
  DG_TRY(check_ints(start, "start", S, fname));
  DG_TRY(check_ints(cu_tokens, "cu_tokens", S + 1, fname));
  DG_TRY(check_table(block_table, S, P, fname));
  int64_t rot = 0;
  if (cos_sin != nullptr) {
    DG_TRY(check_basic(cos_sin, "cos_sin", true));
    DG_TRY(check_dtype(cos_sin, "cos_sin", DG_F32));
    if (cos_sin->ndim != 2) return fail(DG_INVALID_ARG, "%s: cos_sin must be [positions, rot]", fname);
    rot = cos_sin->shape[1];
    if (rot > D || rot % 16 != 0)
      return fail(DG_INVALID_ARG, "%s: rot = %lld must be a multiple of 16, at most D = %lld", fname, (long long)rot, (long long)D);
    DG_TRY(check_heads(cos_sin, "cos_sin", fname));
  }
  if ((q == nullptr) != (q_out == nullptr)) return fail(DG_INVALID_ARG, "%s: q and q_out go together", fname);
  int64_t Hq = 0;
  if (q != nullptr) {
    DG_TRY(check_basic(q, "q", true));
    DG_TRY(check_basic(q_out, "q_out", true));
    DG_TRY(check_dtype(q, "q", k->dtype));
    DG_TRY(check_dtype(q_out, "q_out", DG_BF16));
    if (q->ndim != 3 || q_out->ndim != 3 || q->shape[0] != T || q->shape[2] != D || q_out->shape[0] != T ||
        q_out->shape[1] != q->shape[1] || q_out->shape[2] != D)
      return fail(DG_INVALID_ARG, "%s: q and q_out must be [T, Hq, D] with T = %lld, D = %lld", fname, (long long)T,
                  (long long)D);
    Hq = q->shape[1];
    DG_TRY(check_heads(q, "q", fname));
    DG_TRY(check_heads(q_out, "q_out", fname));
    DG_TRY(check_rows_apart(q_out, "q_out"));
  }
  const dg_tensor* outs[] = {k_cache, v_cache, k_scale, v_scale, q_out};
  const char* onames[] = {"k_cache", "v_cache", "k_scale", "v_scale", "q_out"};
  const dg_tensor* ins[] = {k, v, q, block_table, cu_tokens, start, cos_sin};
  const char* inames[] = {"k", "v", "q", "block_table", "cu_tokens", "start", "cos_sin"};
  for (int i = 0; i < 5; ++i) {
    if (outs[i] == nullptr) continue;
    for (int j = 0; j < 7; ++j) DG_TRY(check_no_alias(outs[i], onames[i], ins[j], inames[j]));
    for (int j = i + 1; j < 5; ++j) {
      if (i % 2 == 0 && i < 4 && j == i + 1) continue;  // K and V of one pool may be interleaved (below)
      DG_TRY(check_no_alias(outs[i], onames[i], outs[j], onames[j]));
    }
    DG_TRY(check_rows_apart(outs[i], onames[i]));
  }
  // k_cache and v_cache (and their scales) may be parts of one pool, page by
  // page, head by head or token by token, but share no memory
  DG_TRY(check_apart(k_cache, "k_cache", v_cache, "v_cache"));
  DG_TRY(check_apart(k_scale, "k_scale", v_scale, "v_scale"));
  if (T == 0 || S == 0 || pages == 0 || Hkv == 0) {
    if (q == nullptr || T == 0 || S == 0 || Hq == 0) return ok();
  }
  dgmi::KvAppendArgs p = {};
  p.k = k->data;
  p.v = v->data;
  p.q = Hq > 0 ? q->data : nullptr;
  p.bf16 = k->dtype == DG_BF16;
  p.sk_t = k->stride[0];
  p.sk_h = k->stride[1];
  p.sv_t = v->stride[0];
  p.sv_h = v->stride[1];
  if (q != nullptr) {
    p.sq_t = q->stride[0];
    p.sq_h = q->stride[1];
    p.q_out = static_cast<uint16_t*>(q_out->data);
    p.so_t = q_out->stride[0];
    p.so_h = q_out->stride[1];
  }
  if (cos_sin != nullptr) {
    p.cos_sin = static_cast<const float*>(cos_sin->data);
    p.s_cs = cos_sin->stride[0];
    p.positions = cos_sin->shape[0];
  }
  p.rot = (int32_t)rot;
  p.interleaved = interleaved ? 1 : 0;
  p.k_cache = static_cast<uint8_t*>(k_cache->data);
  p.v_cache = static_cast<uint8_t*>(v_cache->data);
  p.skc_p = k_cache->stride[0];
  p.skc_h = k_cache->stride[1];
  p.skc_t = k_cache->stride[2];
  p.svc_p = v_cache->stride[0];
  p.svc_h = v_cache->stride[1];
  p.svc_t = v_cache->stride[2];
  p.k_scale = static_cast<float*>(k_scale->data);
  p.v_scale = static_cast<float*>(v_scale->data);
  p.sks_p = k_scale->stride[0];
  p.sks_h = k_scale->stride[1];
  p.svs_p = v_scale->stride[0];
  p.svs_h = v_scale->stride[1];
  p.table = static_cast<const int32_t*>(block_table->data);
  p.s_table = block_table->stride[0];
  p.max_pages = (int32_t)block_table->shape[1];
  p.pages = (int32_t)pages;
  p.cu = static_cast<const int32_t*>(cu_tokens->data);
  p.start = static_cast<const int32_t*>(start->data);
  p.T = (int32_t)T;
  p.S = (int32_t)S;
  p.Hkv = (int32_t)Hkv;
  p.Hq = (int32_t)Hq;
  p.D = (int32_t)D;
  p.P = (int32_t)P;
  if (dgmi::kv_append_plan(T, S, P, Hkv, D, p.q != nullptr).grid > kMaxGroups)
    return fail(DG_UNSUPPORTED, "%s: too many tokens times heads for one launch", fname);
  return check_launch(dgmi::launch_kv_append(p, stream), fname);
}

int64_t paged_attention_fp8_workspace(int64_t S, int64_t n, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_tokens) {
  // sizes that no call takes need none (and the plan is made for those that one takes)
  for (int64_t v : {S, n, Hq, Hkv, max_tokens})
    if (v <= 0 || v > INT32_MAX) return 0;
  if ((D != 64 && D != 128 && D != 256) || Hq % Hkv != 0) return 0;
  return dgmi::paged_attention_workspace(S, n, Hq, Hkv, D, max_tokens);
}

int paged_attention_fp8(const dg_tensor* q, const dg_tensor* k_cache, const dg_tensor* v_cache,
                        const dg_tensor* k_scale, const dg_tensor* v_scale, const dg_tensor* block_table,
                        const dg_tensor* seq_lens, const dg_tensor* out, const dg_tensor* lse,
                        const dg_tensor* workspace, float scale, int32_t window, hipStream_t stream) {
  const char* fname = "paged_attention_fp8";
  DG_TRY(check_basic(q, "q", true));
  DG_TRY(check_basic(out, "out", true));
  DG_TRY(check_dtype(q, "q", DG_BF16));
  DG_TRY(check_dtype(out, "out", DG_BF16));
  DG_TRY(check_caches(k_cache, k_scale, v_cache, v_scale, fname));
  const int64_t pages = k_cache->shape[0], Hkv = k_cache->shape[1], P = k_cache->shape[2], D = k_cache->shape[3];
  if (q->ndim != 4 || q->shape[3] != D) return fail(DG_INVALID_ARG, "%s: q must be [S, n, Hq, D = %lld]", fname, (long long)D);
  const int64_t S = q->shape[0], n = q->shape[1], Hq = q->shape[2];
  if (out->ndim != 4 || out->shape[0] != S || out->shape[1] != n || out->shape[2] != Hq || out->shape[3] != D)
    return fail(DG_INVALID_ARG, "%s: out must have the shape of q", fname);
  if (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0)
    return fail(DG_INVALID_ARG, "%s: Hq = %lld is not a multiple of Hkv = %lld", fname, (long long)Hq, (long long)Hkv);
  DG_TRY(check_heads(q, "q", fname));
  DG_TRY(check_heads(out, "out", fname));
  DG_TRY(check_rows_apart(out, "out"));
  DG_TRY(check_ints(seq_lens, "seq_lens", S, fname));
  DG_TRY(check_table(block_table, S, P, fname));
  if (window < 0) return fail(DG_INVALID_ARG, "%s: window must be >= 0 (got %d)", fname, window);
  if (!(scale - scale == 0.0f)) return fail(DG_INVALID_ARG, "%s: scale must be finite", fname);
  if (lse != nullptr) {
    DG_TRY(check_basic(lse, "lse", false));
    DG_TRY(check_dtype(lse, "lse", DG_F32));
    if (lse->ndim != 3 || lse->shape[0] != S || lse->shape[1] != n || lse->shape[2] != Hq)
      return fail(DG_INVALID_ARG, "%s: lse must be [S, n, Hq]", fname);
    if (!aligned(lse->data, 4)) return fail(DG_INVALID_ARG, "%s: lse must be 4-byte aligned", fname);
    DG_TRY(check_rows_apart(lse, "lse"));
  }
  const int64_t group = Hkv > 0 ? Hq / Hkv : 0, rows = n * group, row_tiles = (rows + 15) / 16;
  if (rows > INT32_MAX - 16 || Hkv * row_tiles > INT32_MAX ||
      (row_tiles > 0 && dgmi::paged_attention_grid(S, Hkv, row_tiles, D, block_table->shape[1] * P) > kMaxGroups))
    return fail(DG_UNSUPPORTED, "%s: too many queries for one launch", fname);
  // the work is counted in 32-token tiles of every head and 16 query rows, in 31 bits
  if (S * Hkv * row_tiles > INT32_MAX || S * Hkv * row_tiles * (block_table->shape[1] * P / 32 + 1) > INT32_MAX - 65536)
    return fail(DG_UNSUPPORTED, "%s: too many tokens times heads for one call", fname);
  const int64_t need = paged_attention_fp8_workspace(S, n, Hq, Hkv, D, block_table->shape[1] * P);
  if (need > 0) {
    if (workspace == nullptr) return fail(DG_INVALID_ARG, "%s: workspace of %lld bytes needed", fname, (long long)need);
    DG_TRY(check_basic(workspace, "workspace", true));
    DG_TRY(check_dtype(workspace, "workspace", DG_F32));
    if (workspace->ndim != 1 || workspace->shape[0] * 4 < need)
      return fail(DG_INVALID_ARG, "%s: workspace must be F32 [at least %lld]", fname, (long long)((need + 3) / 4));
    if (!aligned(workspace->data, 16)) return fail(DG_INVALID_ARG, "%s: workspace must be 16-byte aligned", fname);
  }
  const dg_tensor* outs[] = {out, lse, need > 0 ? workspace : nullptr};
  const char* onames[] = {"out", "lse", "workspace"};
  const dg_tensor* ins[] = {q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens};
  const char* inames[] = {"q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "seq_lens"};
  for (int i = 0; i < 3; ++i) {
    if (outs[i] == nullptr) continue;
    for (int j = 0; j < 7; ++j) DG_TRY(check_no_alias(outs[i], onames[i], ins[j], inames[j]));
    for (int j = i + 1; j < 3; ++j) DG_TRY(check_no_alias(outs[i], onames[i], outs[j], onames[j]));
  }
  if (S == 0 || rows == 0) return ok();
  dgmi::PagedAttnArgs p = {};
  p.q = static_cast<const uint16_t*>(q->data);
  p.sq_s = q->stride[0];
  p.sq_n = q->stride[1];
  p.sq_h = q->stride[2];
  p.out = static_cast<uint16_t*>(out->data);
  p.so_s = out->stride[0];
  p.so_n = out->stride[1];
  p.so_h = out->stride[2];
  if (lse != nullptr) {
    p.lse = static_cast<float*>(lse->data);
    p.sl_s = lse->stride[0];
    p.sl_n = lse->stride[1];
    p.sl_h = lse->stride[2];
  }
  p.k_cache = static_cast<const uint8_t*>(k_cache->data);
  p.v_cache = static_cast<const uint8_t*>(v_cache->data);
  p.skc_p = (uint32_t)k_cache->stride[0];
  p.skc_h = k_cache->stride[1];
  p.skc_t = (uint32_t)k_cache->stride[2];
  p.svc_p = (uint32_t)v_cache->stride[0];
  p.svc_h = v_cache->stride[1];
  p.svc_t = (uint32_t)v_cache->stride[2];
  p.k_scale = static_cast<const float*>(k_scale->data);
  p.v_scale = static_cast<const float*>(v_scale->data);
  p.sks_p = (uint32_t)(k_scale->stride[0] * 4);
  p.sks_h = k_scale->stride[1];
  p.svs_p = (uint32_t)(v_scale->stride[0] * 4);
  p.svs_h = v_scale->stride[1];
  p.table = static_cast<const int32_t*>(block_table->data);
  p.s_table = block_table->stride[0];
  p.lens = static_cast<const int32_t*>(seq_lens->data);
  p.S = (int32_t)S;
  p.n = (int32_t)n;
  p.Hkv = (int32_t)Hkv;
  p.group = (int32_t)group;
  p.rows = (int32_t)rows;
  p.row_tiles = (int32_t)row_tiles;
  p.D = (int32_t)D;
  p.P = (int32_t)P;
  p.max_pages = (int32_t)block_table->shape[1];
  p.pages = (int32_t)pages;
  p.window = window;
  p.scale = scale;
  p.workspace = need > 0 ? static_cast<float*>(workspace->data) : nullptr;
  return check_launch(dgmi::launch_paged_attention(p, stream), fname);
}

int dg_query_config(int32_t kind, int64_t G, int64_t M, int64_t N, int64_t K, dg_config* out) {
  if (out == nullptr) return fail(DG_INVALID_ARG, "dg_query_config: out is NULL");
  if (G < 0 || M < 0 || N < 0 || K < 0) return fail(DG_INVALID_ARG, "dg_query_config: negative size");
  dgmi::GemmPlan c;
  int mode;
  if (kind == DG_KIND_BF16_MASKED || kind == DG_KIND_BF16_DENSE || kind == DG_KIND_BF16_CONTIGUOUS) {
    mode = kind == DG_KIND_BF16_DENSE ? dgmi::MODE_DENSE
                                      : (kind == DG_KIND_BF16_CONTIGUOUS ? dgmi::MODE_CONTIG : dgmi::MODE_MASKED);
    c = dgmi::bf16_gemm_plan(mode, G, M, N, K);
  } else if (kind >= DG_KIND_DENSE && kind <= DG_KIND_MASKED) {
    mode = kind == DG_KIND_DENSE ? dgmi::MODE_DENSE : (kind == DG_KIND_CONTIGUOUS ? dgmi::MODE_CONTIG : dgmi::MODE_MASKED);
    c = dgmi::fp8_gemm_plan(mode, G, M, N, K, dgmi::SF_F32);
  } else if (kind == DG_KIND_DENSE_FP8_OUT || kind == DG_KIND_DENSE_FP8_OUT_ROWB) {
    mode = dgmi::MODE_DENSE;
    c = dgmi::fp8_out_gemm_plan(M, N, dgmi::SF_F32 | (kind == DG_KIND_DENSE_FP8_OUT_ROWB ? dgmi::SF_ROWB : 0));
  } else if (kind == DG_KIND_DENSE_MN) {
    mode = dgmi::MODE_DENSE;
    c = dgmi::fp8_mn_gemm_plan();
  } else if (kind >= DG_KIND_DENSE_ROWB && kind <= DG_KIND_MASKED_ROWB) {
    mode = kind == DG_KIND_DENSE_ROWB ? dgmi::MODE_DENSE
                                      : (kind == DG_KIND_CONTIGUOUS_ROWB ? dgmi::MODE_CONTIG : dgmi::MODE_MASKED);
    c = dgmi::fp8_gemm_plan(mode, G, M, N, K, dgmi::SF_F32 | dgmi::SF_ROWB);
  } else {
    return fail(DG_INVALID_ARG, "dg_query_config: unknown kind %d", kind);
  }
  out->block_m = c.cfg[0].bm;
  out->block_n = c.cfg[0].bn;
  out->threads = c.cfg[0].threads;
  out->grid = dgmi::plan_grid(c, 0, mode, G, M, N);
  out->lds_bytes = dgmi::plan_lds(c, 0, mode);
  out->n_split = c.parts == 2 ? c.n_split : N;
  out->block_n2 = c.parts == 2 ? c.cfg[1].bn : 0;
  out->grid2 = dgmi::plan_grid(c, 1, mode, G, M, N);
  out->lds_bytes2 = dgmi::plan_lds(c, 1, mode);
  return ok();
}

}  // extern "C"
