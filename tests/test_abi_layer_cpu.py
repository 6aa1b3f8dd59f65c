"""Refusals of the norm, the activation, their gradients and the ragged products:
every malformed argument is rejected on the host, before any launch (no GPU
needed; on a machine with one they are skipped, because calls that pass every
check would run on these descriptors of host memory)."""

import os

import pytest
import torch

import moe_grouped_gemm_x128_amd as mg
from moe_grouped_gemm_x128_amd import binding

I32, F32, BF16, U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
INVALID, UNSUPPORTED = binding.DG_INVALID_ARG, binding.DG_UNSUPPORTED


@pytest.fixture(autouse=True)
def _built():
    if torch.cuda.is_available():
        pytest.skip("descriptors of host memory: the launches would run")
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libdgmi.so is not built (python -m moe_grouped_gemm_x128_amd.build)")


def _t(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


class _Null:
    cuda_stream = 0


def _refused(call, code, *args, **kw):
    with pytest.raises(mg.DgmiError) as e:
        call(*args, stream=_Null(), **kw)
    assert e.value.code == code, str(e.value)
    return str(e.value)


def _taken(call, *args, **kw):
    """Past every check: without a GPU the launch itself fails."""
    try:
        call(*args, stream=_Null(), **kw)
    except mg.DgmiError as e:
        assert e.code == binding.DG_LAUNCH_FAILED, str(e)


def test_norm_refusals():
    T, H = 4, 256
    x, w, y, q, sf = _t((T, H), BF16), _t(H), _t((T, H), BF16), _t((T, H), U8), _t((T, 2))
    n = mg.rms_norm
    _refused(n, INVALID, x, w)                                                 # nothing wanted
    _refused(n, INVALID, x, w, q=q)                                            # codes without scales
    _refused(n, INVALID, x, w, y=y, sf=sf)
    _refused(n, INVALID, _t((T, H), I32), w, y=y)
    _refused(n, INVALID, _t((1, T, 1, H), BF16), w, y=y)                       # rank
    _refused(n, INVALID, _t((H, T), BF16).t(), w, y=y)                         # innermost stride
    _refused(n, INVALID, x, _t(H + 1), y=y)
    _refused(n, INVALID, x, _t(H, I32), y=y)
    _refused(n, INVALID, x, w, y=_t((T + 1, H), BF16))
    _refused(n, INVALID, x, w, y=_t((T, H), U8))
    _refused(n, INVALID, x, w, q=q, sf=_t((T, 3)))
    _refused(n, INVALID, x, w, q=q, sf=_t((T, 2), I32))
    _refused(n, INVALID, x, w, q=_t((T, H + 128), U8), sf=_t((T, 3)))
    _refused(n, INVALID, x, w, y=y, h=_t((T, H), BF16))                        # a sum of nothing
    _refused(n, INVALID, x, w, y=y, residual=_t((T, H)), h=_t((T, H), BF16))   # not the residual's type
    _refused(n, INVALID, x, w, y=y, residual=_t((T, H + 8), BF16))
    _refused(n, INVALID, x, w, y=y[:1].expand(T, H))                           # rows on top of each other
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        _refused(n, INVALID, x, w, y=y, eps=eps)
    _refused(n, UNSUPPORTED, _t((1, 16392), BF16), _t(16392), y=_t((1, 16392), BF16))
    _refused(n, UNSUPPORTED, _t((1, 1), BF16).expand(2 ** 28, 1), _t(1), y=torch.empty((2 ** 28, 1), dtype=BF16))
    _taken(n, _t((1, 8), BF16).expand(2 ** 22, 8), _t(8), y=torch.empty((2 ** 22, 8), dtype=BF16))
    # in place over x or the residual as they are, and nothing else
    _taken(n, x, w, y=x)
    r = _t((T, H), BF16)
    _taken(n, x, w, y=x, residual=r, h=r)
    _taken(n, x, w, y=r, residual=r, h=x)
    assert "overlaps" in _refused(n, INVALID, x, w, y=y, residual=r, h=y)
    assert "overlaps" in _refused(n, INVALID, x[:2], w, y=x[1:3])
    _refused(n, INVALID, x, w, q=x.view(U8)[:, :H], sf=sf)
    _refused(n, INVALID, x, w[:H], y=y, residual=w.expand(T, H), h=w.expand(T, H))
    big = _t((T, 3, H), BF16)
    _taken(n, big[:, :2], w, q=_t((T, 2, H), U8), sf=_t((2, T, 2)).transpose(0, 1), y=_t((T, 2, H)))
    _taken(n, _t((0, H), BF16), w, y=_t((0, H), BF16))


def test_norm_gradient_refusals():
    T, H = 4, 256
    dy, h, w, dx = _t((T, H), BF16), _t((T, H), BF16), _t(H), _t((T, H), BF16)
    dw, need = _t(H), mg.rms_norm_bwd_workspace(T, H)
    ws = _t(need // 4)
    b = mg.rms_norm_bwd
    assert need > 0
    assert mg.rms_norm_bwd_workspace(0, H) == mg.rms_norm_bwd_workspace(T, 16385) == 0
    assert mg.rms_norm_bwd_workspace(2 ** 40, H) == mg.rms_norm_bwd_workspace(-1, H) == mg.rms_norm_bwd_workspace(T, -1) == 0
    for rows in (1, 7, 1000, 2 ** 22 - 1):
        for H_ in (1, 128, 1000, 7168, 16384):
            assert 0 < mg.rms_norm_bwd_workspace(rows, H_) <= 1024 * H_ * 4
    _refused(b, INVALID, _t((T, H + 8), BF16), h, w, dx)
    _refused(b, INVALID, dy, h, w, _t((T, H), U8))
    _refused(b, INVALID, dy, h, _t(H, I32), dx)
    _refused(b, INVALID, dy, h, w, dx, grad_weight=_t(H + 1), workspace=ws)
    _refused(b, INVALID, dy, h, w, dx, grad_weight=dw)                         # no workspace
    _refused(b, INVALID, dy, h, w, dx, grad_weight=dw, workspace=ws[:-1])
    _refused(b, INVALID, dy, h, w, dx, grad_weight=dw, workspace=_t(need, I32))
    _refused(b, INVALID, dy, h, w, dx, grad_weight=dw, workspace=_t(need // 4 + 1)[1:])
    _refused(b, INVALID, dy, h, w, dx, grad_h=_t((T - 1, H), BF16))
    _refused(b, INVALID, dy, h, w, dx, eps=0.0)
    _refused(b, UNSUPPORTED, *(_t((1, 16392)) for _ in range(2)), _t(16392), _t((1, 16392)))
    _refused(b, INVALID, dy, h, w, dx[:1].expand(T, H))
    _refused(b, INVALID, dy, h, w, dx, grad_weight=w, workspace=ws)            # the weight's own memory
    _refused(b, INVALID, dy, h, w, dx, grad_weight=ws[:H], workspace=ws)
    _taken(b, dy, h, w, dy)
    _taken(b, dy, h, w, h, grad_weight=dw, workspace=ws)
    _taken(b, dy, h, w, dx, grad_weight=dw.to(BF16), workspace=ws, grad_h=dx)
    assert "overlaps" in _refused(b, INVALID, dy[:2], h[:2], w, dy[1:3])


def test_activation_refusals():
    R, I = 6, 200
    x, y, q, sf = _t((R, 2 * I), BF16), _t((R, I), BF16), _t((R, I), U8), _t((R, 2))
    a = mg.swiglu
    _refused(a, INVALID, x)
    _refused(a, INVALID, x, q=q)
    _refused(a, INVALID, _t((R, 2 * I + 1), BF16), y=y)                        # an odd width has no halves
    _refused(a, INVALID, _t(2 * I, BF16), y=y)
    _refused(a, INVALID, x.to(I32), y=y)
    _refused(a, INVALID, x, y=_t((R, I + 1), BF16))
    _refused(a, INVALID, x, y=_t((R, 1, I), BF16))
    _refused(a, INVALID, x, q=q, sf=_t((R, 1)))
    _refused(a, INVALID, x, y=y, masked_m=_t(R, I32))                          # one group
    _refused(a, INVALID, x, y=y, masked_m=_t(1))
    _refused(a, INVALID, x, y=y, row_weights=_t(R + 1))
    _refused(a, INVALID, x, y=y, row_weights=_t(R, BF16))
    _refused(a, INVALID, x, y=y, row_weights=_t((R, 1)))
    assert "overlaps" in _refused(a, INVALID, x, y=x[:, :I])
    _refused(a, INVALID, x, y=y[:1].expand(R, I))
    many = _t((1, 2), BF16).expand(2 ** 28 + 16, 2)
    _refused(a, UNSUPPORTED, many, y=_t((2 ** 28 + 16, 1), BF16))
    _taken(a, _t((2, R, 2 * I)), y=_t((2, R, I)), q=_t((2, R, I), U8), sf=_t((2, R, 2)), masked_m=_t(2, I32),
           row_weights=_t(2 * R))
    _taken(a, x, y=y, masked_m=_t(1, I32))
    g, dx, dw = _t((R, I), BF16), _t((R, 2 * I), BF16), _t(R)
    b = mg.swiglu_bwd
    _refused(b, INVALID, x, _t((R, I + 1), BF16), dx)
    _refused(b, INVALID, x, g, _t((R, 2 * I + 2), BF16))
    _refused(b, INVALID, x, g, dx, grad_row_weights=_t(R + 1))
    _refused(b, INVALID, x, g, dx, grad_row_weights=dw[:1].expand(R))
    _refused(b, INVALID, x, g, dx, row_weights=dw, grad_row_weights=dw)
    _refused(b, INVALID, x, x[:, :I], x)                                       # over the gradient's rows
    _refused(b, INVALID, x, g, dx[1:])
    _taken(b, x, g, x, row_weights=_t(R), grad_row_weights=dw)


def _far(shape):
    """Rows 8 MiB apart (memory that nothing touches)."""
    return torch.empty(shape[0] << 22, dtype=BF16).as_strided(shape, (1 << 22, 1))


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_ragged_refusals(form):
    G, M, N, K = 3, 20, 40, 128
    call = {"nt": mg.m_grouped_bf16_gemm_nt_ragged, "nn": mg.m_grouped_bf16_gemm_nn_ragged,
            "tn": mg.k_grouped_bf16_gemm_tn}[form]
    sa = (M, N) if form == "tn" else (M, K)
    sb = (G, N, K) if form == "nt" else (G, K, N) if form == "nn" else (M, K)
    sd = (G, N, K) if form == "tn" else (M, N)
    a, b, d, off = _t(sa, BF16), _t(sb, BF16), _t(sd, BF16), _t(G + 1, I32)

    def no(code, a=a, b=b, d=d, off=off, c=None):
        return _refused(call, code, a, b, d, off, c=c)

    no(INVALID, a=a.float())
    no(INVALID, b=b.float())
    no(INVALID, d=d.to(I32))
    no(INVALID, a=a[None])
    no(INVALID, b=b[0])
    no(INVALID, a=_t((sa[0], sa[1] + 64), BF16))
    no(INVALID, d=_t(sd[:-1] + (sd[-1] + 1,), BF16))
    no(INVALID, off=_t(G, I32))
    no(INVALID, off=_t(G + 1))
    no(INVALID, off=_t((G + 1, 1), I32))
    no(INVALID, off=_t(2 * G + 2, I32)[::2])
    no(INVALID, a=_t((sa[0], sa[1] + 4), BF16)[:, :sa[1]])                     # rows not 16-byte aligned
    no(INVALID, b=_t(sb[:-1] + (sb[-1] + 4,), BF16)[..., :sb[-1]])
    no(INVALID, a=_t((sa[0], sa[1] + 8), BF16)[:, 1:sa[1] + 1])
    no(INVALID, c=_t(sd[:-1] + (sd[-1] + 1,)))
    no(INVALID, c=_t(sd, I32))
    wide = _t(sd[:-1] + (sd[-1] + 8,), BF16)
    assert "overlaps" in no(INVALID, d=wide[..., :sd[-1]], c=wide[..., 8:])
    no(INVALID, d=d[:1].expand(sd))
    assert "overlap" in no(INVALID, a=a[:1].expand(sa))
    assert "overlap" in no(INVALID, b=b[..., :1, :].expand(sb))
    assert "overlap" in no(INVALID, a=a.view(-1)[:8 * sa[0] + sa[1]].as_strided(sa, (8, 1)))
    no(UNSUPPORTED, a=_far(sa))
    many = 2 ** 31 - 1
    if form == "nt":
        no(UNSUPPORTED, a=_t((1, 0), BF16), b=_t((G, many, 0), BF16), d=torch.empty((1, many), dtype=BF16))
    if form == "nn":
        no(UNSUPPORTED, a=_t((many, 0), BF16), b=_t((G, 0, 1), BF16), d=torch.empty((many, 1), dtype=BF16))
    if form == "tn":
        no(UNSUPPORTED, a=_t((0, many), BF16), b=_t((0, 1), BF16), d=torch.empty((1, many, 1), dtype=BF16), off=_t(2, I32))
    if form != "tn":
        no(UNSUPPORTED, a=_t((M, 96), BF16), b=_t((G, N, 96) if form == "nt" else (G, 96, N), BF16))
    _taken(call, a, b, d, off)
    _taken(call, a, b, d, off, c=d)
    _taken(call, a, b, _t(sd), off, c=d)
