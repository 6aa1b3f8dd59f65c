"""ctypes binding of libdgmi (include/dgmi.h).

Argument marshalling only: every function below builds dg_tensor
descriptors from torch tensors (device memory owned by the caller), passes
the current HIP stream, and calls the C entry point of the same name.  All
computation happens in the library's HIP kernels; there is no fallback.  A
missing or unloadable library raises at once.
"""

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdgmi.so")

DG_F32, DG_BF16, DG_E4M3, DG_I32 = 0, 1, 2, 3
DG_OK, DG_INVALID_ARG, DG_UNSUPPORTED, DG_LAUNCH_FAILED = 0, 1, 2, 3
DG_SCORE_SOFTMAX, DG_SCORE_SIGMOID = 0, 1
DG_KIND_DENSE, DG_KIND_CONTIGUOUS, DG_KIND_MASKED = 0, 1, 2
DG_KIND_BF16_MASKED, DG_KIND_BF16_DENSE, DG_KIND_BF16_CONTIGUOUS = 3, 4, 5
DG_KIND_DENSE_ROWB, DG_KIND_CONTIGUOUS_ROWB, DG_KIND_MASKED_ROWB = 6, 7, 8  # FP8, one B scale per row of B
DG_KIND_DENSE_FP8_OUT = 9  # fp8_gemm_nt_fp8_out
DG_KIND_DENSE_MN = 10  # fp8_gemm_nn / _tn / _tt
DG_KIND_DENSE_FP8_OUT_ROWB = 11  # fp8_gemm_nt_fp8_out, one B scale per row

ENTRY_POINTS = (
    "dg_last_error",
    "dgmi_init",
    "fp8_gemm_nt",
    "fp8_gemm_nt_fp8_out",
    "fp8_gemm_nn",
    "fp8_gemm_tn",
    "fp8_gemm_tt",
    "m_grouped_fp8_gemm_nt_contiguous",
    "m_grouped_fp8_gemm_nt_masked",
    "m_grouped_fp8_gemm_nt_contiguous_acc",
    "m_grouped_fp8_gemm_nt_masked_acc",
    "m_grouped_bf16_gemm_nt_masked",
    "bf16_gemm_nt",
    "m_grouped_bf16_gemm_nt_contiguous",
    "m_grouped_bf16_gemm_nt_contiguous_acc",
    "m_grouped_bf16_gemm_nt_masked_acc",
    "per_token_cast_to_fp8",
    "per_block_cast_to_fp8",
    "pack_ue8m0_to_int",
    "moe_dispatch_masked_fp8",
    "moe_dispatch_contiguous_fp8",
    "moe_combine",
    "moe_route_topk",
    "moe_route_topk_bwd",
    "kv_append_fp8",
    "paged_attention_fp8",
    "paged_attention_fp8_workspace",
    "rms_norm",
    "rms_norm_bwd",
    "rms_norm_bwd_workspace",
    "swiglu",
    "swiglu_bwd",
    "m_grouped_bf16_gemm_nt_ragged",
    "m_grouped_bf16_gemm_nn_ragged",
    "k_grouped_bf16_gemm_tn",
    "dg_query_config",
)


class DgTensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("ndim", ctypes.c_int32),
        ("shape", ctypes.c_int64 * 4),
        ("stride", ctypes.c_int64 * 4),
    ]


class DgConfig(ctypes.Structure):
    _fields_ = [
        ("block_m", ctypes.c_int32),
        ("block_n", ctypes.c_int32),
        ("threads", ctypes.c_int32),
        ("grid", ctypes.c_int64),
        ("lds_bytes", ctypes.c_int32),
        ("n_split", ctypes.c_int64),
        ("block_n2", ctypes.c_int32),
        ("grid2", ctypes.c_int64),
        ("lds_bytes2", ctypes.c_int32),
    ]


class DgmiError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"[dgmi status {code}] {message}")
        self.code = code


_LIB = None
_CALLS = None


def load_library(path=None):
    """Open libdgmi.so (built in-tree by moe_grouped_gemm_x128_amd.build)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    lib = _open(path or LIB_PATH, ctypes.POINTER(DgTensor))
    if path is None:
        _LIB = lib
    return lib


def _calls():
    """The library for this module's own calls, whose descriptors are packed bytes."""
    global _CALLS
    if _CALLS is None:
        _CALLS = _open(LIB_PATH, ctypes.c_void_p)
    return _CALLS


def _open(p, T):
    """The library at p, its const dg_tensor* arguments of ctypes type T."""
    if not os.path.exists(p):
        raise RuntimeError(f"libdgmi.so not found at {p}: build it with `python -m moe_grouped_gemm_x128_amd.build`")
    lib = ctypes.CDLL(p)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    sig = {
        "dg_last_error": ([], ctypes.c_char_p),
        "dgmi_init": ([], ctypes.c_int),
        "fp8_gemm_nt": ([T, T, T, T, T, T, vp], ctypes.c_int),
        "fp8_gemm_nt_fp8_out": ([T, T, T, T, T, T, T, ctypes.c_int, vp], ctypes.c_int),
        "fp8_gemm_nn": ([T, T, T, T, T, T, vp], ctypes.c_int),
        "fp8_gemm_tn": ([T, T, T, T, T, T, vp], ctypes.c_int),
        "fp8_gemm_tt": ([T, T, T, T, T, T, vp], ctypes.c_int),
        "m_grouped_fp8_gemm_nt_contiguous": ([T, T, T, T, T, T, vp], ctypes.c_int),
        "m_grouped_fp8_gemm_nt_masked": ([T, T, T, T, T, T, i64, vp], ctypes.c_int),
        "m_grouped_fp8_gemm_nt_contiguous_acc": ([T, T, T, T, T, T, T, vp], ctypes.c_int),
        "m_grouped_fp8_gemm_nt_masked_acc": ([T, T, T, T, T, T, T, i64, vp], ctypes.c_int),
        "m_grouped_bf16_gemm_nt_contiguous_acc": ([T, T, T, T, T, vp], ctypes.c_int),
        "m_grouped_bf16_gemm_nt_masked_acc": ([T, T, T, T, T, i64, vp], ctypes.c_int),
        "m_grouped_bf16_gemm_nt_masked": ([T, T, T, T, i64, vp], ctypes.c_int),
        "bf16_gemm_nt": ([T, T, T, T, vp], ctypes.c_int),
        "m_grouped_bf16_gemm_nt_contiguous": ([T, T, T, T, vp], ctypes.c_int),
        "per_token_cast_to_fp8": ([T, T, T, ctypes.c_int, vp], ctypes.c_int),
        "per_block_cast_to_fp8": ([T, T, T, ctypes.c_int, vp], ctypes.c_int),
        "pack_ue8m0_to_int": ([T, T, vp, vp], ctypes.c_int),
        "moe_dispatch_masked_fp8": ([T, T, T, T, T, T, T, ctypes.c_int, vp], ctypes.c_int),
        "moe_dispatch_contiguous_fp8": ([T, T, T, T, T, T, T, i32, ctypes.c_int, vp], ctypes.c_int),
        "moe_combine": ([T, T, T, T, vp], ctypes.c_int),
        "moe_route_topk": ([T, T, T, T, i32, i32, i32, i32, ctypes.c_int, f32, vp], ctypes.c_int),
        "moe_route_topk_bwd": ([T, T, T, T, i32, ctypes.c_int, f32, vp], ctypes.c_int),
        "kv_append_fp8": ([T] * 12 + [ctypes.c_int, vp], ctypes.c_int),
        "paged_attention_fp8": ([T] * 10 + [f32, i32, vp], ctypes.c_int),
        "paged_attention_fp8_workspace": ([i64] * 6, i64),
        "rms_norm": ([T] * 7 + [f32, ctypes.c_int, vp], ctypes.c_int),
        "rms_norm_bwd": ([T] * 7 + [f32, vp], ctypes.c_int),
        "rms_norm_bwd_workspace": ([i64] * 2, i64),
        "swiglu": ([T] * 6 + [ctypes.c_int, vp], ctypes.c_int),
        "swiglu_bwd": ([T] * 6 + [vp], ctypes.c_int),
        "m_grouped_bf16_gemm_nt_ragged": ([T] * 5 + [vp], ctypes.c_int),
        "m_grouped_bf16_gemm_nn_ragged": ([T] * 5 + [vp], ctypes.c_int),
        "k_grouped_bf16_gemm_tn": ([T] * 5 + [vp], ctypes.c_int),
        "dg_query_config": ([i32, i64, i64, i64, i64, ctypes.POINTER(DgConfig)], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


class _DtypeCodes(dict):
    """dg dtype codes by torch dtype (torch is imported with the first tensor seen)."""

    def __missing__(self, dtype):
        import torch

        if not self:
            self.update({
                torch.float32: DG_F32,
                torch.bfloat16: DG_BF16,
                torch.uint8: DG_E4M3,
                torch.int32: DG_I32,
            })
            f8 = getattr(torch, "float8_e4m3fn", None)
            if f8 is not None:
                self[f8] = DG_E4M3
            if dtype in self:
                return self[dtype]
        raise TypeError(f"unsupported tensor dtype {dtype}")


class _Packers(dict):
    def __missing__(self, ndim):
        raise ValueError("dg_tensor supports 1 to 4 dims")


_DTYPE_CODES = _DtypeCodes()

# a dg_tensor as bytes, by rank: data, dtype, ndim, shape[4], stride[4], what
# the rank leaves over zero
_PACK = _Packers((n, struct.Struct(f"@Qii{n}q{32 - 8 * n}x{n}q{32 - 8 * n}x").pack) for n in range(1, 5))


def _arg(t):
    """The descriptor argument of a call: a torch tensor's dg_tensor as bytes, or
    NULL.  (Packed in one go and without a helper: a call passes up to a dozen
    tensors, and setting the structure's fields takes 4 us each, this 0.45.)"""
    if t is None:
        return None
    shape = t.shape
    n = len(shape)
    return _PACK[n](t.data_ptr(), _DTYPE_CODES[t.dtype], n, *shape, *t.stride())


def describe(t, dtype=None):
    """dg_tensor for a torch tensor (None -> NULL descriptor); dtype replaces its own code."""
    if t is None:
        return None
    n = len(t.shape)
    code = _DTYPE_CODES[t.dtype] if dtype is None else dtype
    return DgTensor.from_buffer_copy(_PACK[n](t.data_ptr(), code, n, *t.shape, *t.stride()))


# torch's current stream as a handle: (device index of this thread, handle of a device's stream)
_CURRENT = None


def _stream(stream):
    global _CURRENT
    if stream is not None:
        return stream.cuda_stream
    if _CURRENT is None:
        import torch

        torch.cuda.init()
        device, raw = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if device is None or raw is None:
            return torch.cuda.current_stream().cuda_stream
        _CURRENT = device, raw  # (0.1 us a call; a Stream object takes 3)
    device, raw = _CURRENT
    return raw(device())


def _check(rc):
    if rc != DG_OK:
        raise DgmiError(rc, _calls().dg_last_error().decode())


def last_error():
    return _calls().dg_last_error().decode()


def dgmi_init():
    _check(_calls().dgmi_init())


def fp8_gemm_nt(a, b, sfa, sfb, c, d, stream=None):
    """d = c + a . b^T with block scales; c is None or a BF16/F32 [M, N] tensor (may be d)."""
    lib = _calls()
    _check(lib.fp8_gemm_nt(_arg(a), _arg(b), _arg(sfa), _arg(sfb),
                           _arg(c), _arg(d), _stream(stream)))
    return d


def _fp8_gemm_layout(name, a, b, sfa, sfb, c, d, stream):
    lib = _calls()
    _check(getattr(lib, name)(_arg(a), _arg(b), _arg(sfa), _arg(sfb),
                              _arg(c), _arg(d), _stream(stream)))
    return d


def fp8_gemm_nn(a, b, sfa, sfb, c, d, stream=None):
    """d = c + a . b with a [M, K] (K contiguous) and b [K, N] (N contiguous), FP8."""
    return _fp8_gemm_layout("fp8_gemm_nn", a, b, sfa, sfb, c, d, stream)


def fp8_gemm_tn(a, b, sfa, sfb, c, d, stream=None):
    """d = c + a^T . b with a [K, M] (M contiguous) and b [K, N], FP8."""
    return _fp8_gemm_layout("fp8_gemm_tn", a, b, sfa, sfb, c, d, stream)


def fp8_gemm_tt(a, b, sfa, sfb, c, d, stream=None):
    """d = c + a^T . b^T with a [K, M] (M contiguous) and b [N, K] (K contiguous), FP8."""
    return _fp8_gemm_layout("fp8_gemm_tt", a, b, sfa, sfb, c, d, stream)


def fp8_gemm_nt_fp8_out(a, b, sfa, sfb, c, q, sfq, use_ue8m0=False, stream=None):
    """(q, sfq) = per-token FP8 cast of the BF16 D = c + a . b^T, in one kernel."""
    lib = _calls()
    _check(lib.fp8_gemm_nt_fp8_out(_arg(a), _arg(b), _arg(sfa), _arg(sfb),
                                   _arg(c), _arg(q), _arg(sfq), int(bool(use_ue8m0)),
                                   _stream(stream)))
    return q, sfq


def m_grouped_fp8_gemm_nt_contiguous(a, b, sfa, sfb, d, grouped_layout, stream=None, c=None):
    """Contiguous grouped GEMM; with c (BF16/F32, d's shape, may be d) the
    accumulate form d = c + a . b^T (m_grouped_fp8_gemm_nt_contiguous_acc)."""
    lib = _calls()
    if c is not None:
        _check(lib.m_grouped_fp8_gemm_nt_contiguous_acc(_arg(a), _arg(b), _arg(sfa),
                                                        _arg(sfb), _arg(c), _arg(d),
                                                        _arg(grouped_layout), _stream(stream)))
        return d
    _check(lib.m_grouped_fp8_gemm_nt_contiguous(_arg(a), _arg(b), _arg(sfa),
                                                _arg(sfb), _arg(d),
                                                _arg(grouped_layout), _stream(stream)))
    return d


def m_grouped_fp8_gemm_nt_masked(a, b, sfa, sfb, d, masked_m, max_m_per_group, stream=None, c=None):
    """Masked grouped GEMM; with c (BF16/F32, d's shape, may be d) the
    accumulate form d = c + a . b^T (m_grouped_fp8_gemm_nt_masked_acc)."""
    lib = _calls()
    if c is not None:
        _check(lib.m_grouped_fp8_gemm_nt_masked_acc(_arg(a), _arg(b), _arg(sfa),
                                                    _arg(sfb), _arg(c), _arg(d),
                                                    _arg(masked_m), int(max_m_per_group), _stream(stream)))
        return d
    _check(lib.m_grouped_fp8_gemm_nt_masked(_arg(a), _arg(b), _arg(sfa),
                                            _arg(sfb), _arg(d), _arg(masked_m),
                                            int(max_m_per_group), _stream(stream)))
    return d


def m_grouped_bf16_gemm_nt_masked(a, b, d, masked_m, max_m_per_group, stream=None, c=None):
    """Masked grouped BF16 GEMM; with c (BF16/F32, d's shape, may be d) the
    accumulate form d = c + a . b^T (m_grouped_bf16_gemm_nt_masked_acc)."""
    lib = _calls()
    if c is not None:
        _check(lib.m_grouped_bf16_gemm_nt_masked_acc(_arg(a), _arg(b), _arg(c),
                                                     _arg(d), _arg(masked_m), int(max_m_per_group),
                                                     _stream(stream)))
        return d
    _check(lib.m_grouped_bf16_gemm_nt_masked(_arg(a), _arg(b), _arg(d),
                                             _arg(masked_m), int(max_m_per_group), _stream(stream)))
    return d


def bf16_gemm_nt(a, b, c, d, stream=None):
    """d = c + a . b^T in BF16 (FP32 accumulation); c is None or a BF16/F32 [M, N] tensor (may be d)."""
    lib = _calls()
    _check(lib.bf16_gemm_nt(_arg(a), _arg(b), _arg(c), _arg(d),
                            _stream(stream)))
    return d


def m_grouped_bf16_gemm_nt_contiguous(a, b, d, grouped_layout, stream=None, c=None):
    """Contiguous grouped BF16 GEMM; with c (BF16/F32, d's shape, may be d)
    the accumulate form d = c + a . b^T (m_grouped_bf16_gemm_nt_contiguous_acc)."""
    lib = _calls()
    if c is not None:
        _check(lib.m_grouped_bf16_gemm_nt_contiguous_acc(_arg(a), _arg(b), _arg(c),
                                                         _arg(d), _arg(grouped_layout),
                                                         _stream(stream)))
        return d
    _check(lib.m_grouped_bf16_gemm_nt_contiguous(_arg(a), _arg(b), _arg(d),
                                                 _arg(grouped_layout), _stream(stream)))
    return d


def per_token_cast_to_fp8(x, q, sf, use_ue8m0=False, stream=None):
    lib = _calls()
    _check(lib.per_token_cast_to_fp8(_arg(x), _arg(q), _arg(sf),
                                     int(bool(use_ue8m0)), _stream(stream)))
    return q, sf


def per_block_cast_to_fp8(x, q, sf, use_ue8m0=False, stream=None):
    lib = _calls()
    _check(lib.per_block_cast_to_fp8(_arg(x), _arg(q), _arg(sf),
                                     int(bool(use_ue8m0)), _stream(stream)))
    return q, sf


def pack_ue8m0_to_int(x, out, invalid_count=None, stream=None):
    """Pack FP32 power-of-two scales into int32 words of four UE8M0 bytes.
    invalid_count: optional int32 device tensor (1 element) that receives the
    number of non-UE8M0 inputs, added on the device."""
    lib = _calls()
    cnt = ctypes.c_void_p(invalid_count.data_ptr()) if invalid_count is not None else None
    _check(lib.pack_ue8m0_to_int(_arg(x), _arg(out), cnt, _stream(stream)))
    return out


def moe_dispatch_masked_fp8(x, topk_idx, a, sfa, masked_m, slot, src, use_ue8m0=False, stream=None):
    """Route (token, choice) pairs into the expert buffers a / sfa (masked
    layout) with the per-token FP8 cast; fills masked_m, slot and src."""
    lib = _calls()
    _check(lib.moe_dispatch_masked_fp8(_arg(x), _arg(topk_idx), _arg(a),
                                       _arg(sfa), _arg(masked_m), _arg(slot),
                                       _arg(src), int(bool(use_ue8m0)), _stream(stream)))
    return a, sfa, masked_m, slot, src


def moe_dispatch_contiguous_fp8(x, topk_idx, a, sfa, grouped_layout, counts, slot, align=128, use_ue8m0=False,
                                stream=None):
    """Route (token, choice) pairs into the contiguous layout (a region of
    whole `align`-row granules per expert, align 128 or 256) with the
    per-token FP8 cast; fills grouped_layout, counts and slot."""
    lib = _calls()
    _check(lib.moe_dispatch_contiguous_fp8(_arg(x), _arg(topk_idx), _arg(a),
                                           _arg(sfa), _arg(grouped_layout), _arg(counts),
                                           _arg(slot), int(align), int(bool(use_ue8m0)), _stream(stream)))
    return a, sfa, grouped_layout, counts, slot


def moe_combine(d, slot, topk_weights, y, stream=None):
    """y[t] = sum_j topk_weights[t, j] * d[slot[t, j]] (BF16 out)."""
    lib = _calls()
    _check(lib.moe_combine(_arg(d), _arg(slot), _arg(topk_weights), _arg(y),
                           _stream(stream)))
    return y


_SCORES = {"softmax": DG_SCORE_SOFTMAX, "sigmoid": DG_SCORE_SIGMOID}


def _score_code(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _SCORES[score]


def moe_route_topk(logits, topk_idx, topk_weights, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1,
                   renormalize=True, scale=1.0, stream=None):
    """Choose topk_idx.shape[1] experts per row of logits, with their weights
    (the tables of moe_dispatch_* and moe_combine).  score "softmax" or
    "sigmoid"; bias counts for the choice only; groups: the topk_group best of
    n_group ranges of experts by the sum of their group_top best choices."""
    lib = _calls()
    _check(lib.moe_route_topk(_arg(logits), _arg(bias), _arg(topk_idx),
                              _arg(topk_weights), _score_code(score), int(n_group), int(topk_group),
                              int(group_top), int(bool(renormalize)), float(scale), _stream(stream)))
    return topk_idx, topk_weights


def moe_route_topk_bwd(logits, topk_idx, grad_weights, grad_logits, score="softmax", renormalize=True, scale=1.0,
                       stream=None):
    """grad_logits from the gradient of moe_route_topk's weights (the choice taken as given)."""
    lib = _calls()
    _check(lib.moe_route_topk_bwd(_arg(logits), _arg(topk_idx), _arg(grad_weights),
                                  _arg(grad_logits), _score_code(score), int(bool(renormalize)),
                                  float(scale), _stream(stream)))
    return grad_logits


def kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_tokens, start, cos_sin=None, q=None,
                  q_out=None, interleaved=False, stream=None):
    """Append the tokens k, v [T, Hkv, D] to the paged FP8 caches
    [pages, Hkv, P, D] (scales [pages, Hkv]), keys rotated by position with
    cos_sin [positions, rot]; q [T, Hq, D] is rotated into q_out on the way."""
    lib = _calls()
    _check(lib.kv_append_fp8(_arg(k), _arg(v), _arg(k_cache), _arg(v_cache),
                             _arg(k_scale), _arg(v_scale), _arg(block_table),
                             _arg(cu_tokens), _arg(start), _arg(cos_sin),
                             _arg(q), _arg(q_out), int(bool(interleaved)), _stream(stream)))
    return k_cache, v_cache, k_scale, v_scale


def paged_attention_fp8_workspace(S, n, Hq, Hkv, D, max_tokens):
    """Bytes of workspace paged_attention_fp8 needs (max_tokens = max_pages * P)."""
    return int(_calls().paged_attention_fp8_workspace(int(S), int(n), int(Hq), int(Hkv), int(D),
                                                            int(max_tokens)))


def paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out, scale, workspace=None,
                        lse=None, window=0, stream=None):
    """Attention of the n newest tokens of each sequence, q [S, n, Hq, D],
    over its pages of the FP8 caches; lse [S, n, Hq] is optional."""
    lib = _calls()
    _check(lib.paged_attention_fp8(_arg(q), _arg(k_cache), _arg(v_cache),
                                   _arg(k_scale), _arg(v_scale), _arg(block_table),
                                   _arg(seq_lens), _arg(out), _arg(lse),
                                   _arg(workspace), float(scale), int(window), _stream(stream)))
    return out


def rms_norm(x, weight, y=None, q=None, sf=None, residual=None, h=None, eps=1e-6, use_ue8m0=False, stream=None):
    """Norm of the rows of x [T, H] or [T, heads, H], or of x + residual (stored
    in h): y, and / or its FP8 cast q with the scales sf [.., ceil(H / 128)]."""
    lib = _calls()
    _check(lib.rms_norm(_arg(x), _arg(weight), _arg(y), _arg(q), _arg(sf), _arg(residual),
                        _arg(h), float(eps), int(bool(use_ue8m0)), _stream(stream)))
    return y if q is None else (q, sf)


def rms_norm_bwd_workspace(rows, H):
    """Bytes of workspace rms_norm_bwd needs for the gradient of the weight (rows = T * heads)."""
    return int(_calls().rms_norm_bwd_workspace(int(rows), int(H)))


def rms_norm_bwd(grad_y, h, weight, grad_x, grad_weight=None, workspace=None, grad_h=None, eps=1e-6, stream=None):
    """grad_x (of x and of the residual alike; grad_h, what reaches the sum from
    elsewhere, is added) and grad_weight from the gradient of rms_norm's y."""
    lib = _calls()
    _check(lib.rms_norm_bwd(_arg(grad_y), _arg(h), _arg(weight), _arg(grad_x), _arg(grad_weight),
                            _arg(workspace), _arg(grad_h), float(eps), _stream(stream)))
    return grad_x


def swiglu(x, y=None, q=None, sf=None, masked_m=None, row_weights=None, use_ue8m0=False, stream=None):
    """row_weights * silu(gate) * up of x [.., 2 I] (the gate's columns first): y,
    and / or its FP8 cast q, sf; of the first masked_m[g] rows of each group only."""
    lib = _calls()
    _check(lib.swiglu(_arg(x), _arg(y), _arg(q), _arg(sf), _arg(masked_m), _arg(row_weights),
                      int(bool(use_ue8m0)), _stream(stream)))
    return y if q is None else (q, sf)


def swiglu_bwd(x, grad_y, grad_x, masked_m=None, row_weights=None, grad_row_weights=None, stream=None):
    """grad_x (it may be x) and grad_row_weights from the gradient of swiglu's y."""
    lib = _calls()
    _check(lib.swiglu_bwd(_arg(x), _arg(grad_y), _arg(grad_x), _arg(masked_m), _arg(row_weights),
                          _arg(grad_row_weights), _stream(stream)))
    return grad_x


def m_grouped_bf16_gemm_nt_ragged(a, b, d, offsets, stream=None, c=None):
    """d[m] = c[m] + a[m] . b[g]^T for rows offsets[g] <= m < offsets[g + 1]."""
    lib = _calls()
    _check(lib.m_grouped_bf16_gemm_nt_ragged(_arg(a), _arg(b), _arg(c), _arg(d), _arg(offsets), _stream(stream)))
    return d


def m_grouped_bf16_gemm_nn_ragged(a, b, d, offsets, stream=None, c=None):
    """d[m] = c[m] + a[m] . b[g] for rows offsets[g] <= m < offsets[g + 1], b [G, K, N]."""
    lib = _calls()
    _check(lib.m_grouped_bf16_gemm_nn_ragged(_arg(a), _arg(b), _arg(c), _arg(d), _arg(offsets), _stream(stream)))
    return d


def k_grouped_bf16_gemm_tn(a, b, d, offsets, stream=None, c=None):
    """d[g] = c[g] + a_g^T . b_g over rows offsets[g] .. offsets[g + 1] - 1 of a [M, N] and b [M, K]."""
    lib = _calls()
    _check(lib.k_grouped_bf16_gemm_tn(_arg(a), _arg(b), _arg(c), _arg(d), _arg(offsets), _stream(stream)))
    return d


def query_config(kind, G, M, N, K):
    cfg = DgConfig()
    _check(_calls().dg_query_config(int(kind), int(G), int(M), int(N), int(K), ctypes.byref(cfg)))
    return dict(block_m=cfg.block_m, block_n=cfg.block_n, threads=cfg.threads, grid=cfg.grid, lds_bytes=cfg.lds_bytes,
                n_split=cfg.n_split, block_n2=cfg.block_n2, grid2=cfg.grid2, lds_bytes2=cfg.lds_bytes2)
