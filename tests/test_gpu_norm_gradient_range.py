"""Gradients of the norm where the rows' values and their gradients lie far from
one, so that products of the two leave FP32's range though the results do not:
against oracle/layer.py, with the bounds of test_gpu_norm_large_rows.  A product
grad_y weight is a FP32 number in all of them."""

import numpy as np
import pytest

from oracle import layer

from helpers import say
from test_gpu_norm import BF, F32, U, _blank, _close, _gen, _np, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402

HS = [64, 100, 200, 512, 1000, 2048, 4096, 7168, 16384]


def _check(h, dy, w, eps, what, dh=None):
    T, H = h.shape
    dx, dw = _blank((T, H), F32), torch.full((H,), float("nan"), device="cuda")
    ws = torch.full((mg.rms_norm_bwd_workspace(T, H) // 4,), float("nan"), device="cuda")
    mg.rms_norm_bwd(dy, h, w, dx, grad_weight=dw, workspace=ws, grad_h=dh, eps=eps)
    eps = float(np.float32(eps))
    rx, rw, size, wsize = layer.rms_norm_bwd(_np(dy), _np(h), _np(w), eps, None if dh is None else _np(dh))
    _close(dx, rx, 114 * U * size + 2.0 ** -140, f"{what}: grad_x")
    _close(dw, rw, 40 * U * wsize + 2.0 ** -140, f"{what}: grad_weight")
    return dx


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("dt", [F32, BF])
def test_products_past_the_largest(H, dt):
    """dy w h past 2^128: of a few values, of the sum, and beside rows of ordinary size."""
    say(f"rms_norm_bwd, dy w h past FP32, H={H} {dt}")
    gen = _gen(H)
    w = _rows(gen, (H,), F32)
    for hs, gs in (((1e15, 1.0, 1e18), (1e25, 1.0, 1e24)), ((1e12, 3.0, 1e30), (1e26, 1e-3, 1e10)),
                   ((1.0, 2.0, 1e3), (1e36, 1.0, 1e35))):
        h = _rows(gen, (3, H), F32) * torch.tensor(hs, device="cuda")[:, None]
        dy = _rows(gen, (3, H), F32) * torch.tensor(gs, device="cuda")[:, None]
        _check(h.to(dt), dy.to(dt), w, 1e-6, f"h {hs} dy {gs}")
    # all of one sign: the sum itself
    h, dy = torch.full((2, H), 1e19, device="cuda", dtype=dt), torch.full((2, H), 1e18, device="cuda", dtype=dt)
    _check(h, dy, torch.rand(H, generator=gen, device="cuda") + 0.5, 1e-6, "one sign")


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("dt", [F32, BF])
def test_products_below_the_smallest(H, dt):
    """dy w h below 2^-126 where an eps there too lets the row count."""
    say(f"rms_norm_bwd, dy w h below FP32, H={H} {dt}")
    gen = _gen(H + 1)
    w = _rows(gen, (H,), F32)
    for hs, gs in (((1e-14, 1.0, 1e-13), (1e-26, 1e-30, 1e-28)), ((1e-12, 1e-3, 1e-14), (1e-30, 1e-33, 1e-31))):
        h = _rows(gen, (3, H), F32) * torch.tensor(hs, device="cuda")[:, None]
        dy = _rows(gen, (3, H), F32) * torch.tensor(gs, device="cuda")[:, None]
        _check(h.to(dt), dy.to(dt), w, 1e-37, f"h {hs} dy {gs}")


@pytest.mark.parametrize("H", [100, 2048, 7168])
def test_rows_without_a_gradient(H):
    """Zeros in, zeros (or grad_h) out, also between rows that have one."""
    say(f"rms_norm_bwd of rows without a gradient, H={H}")
    gen = _gen(H + 2)
    h, dy, dh, w = _rows(gen, (6, H), BF), _rows(gen, (6, H), BF), _rows(gen, (6, H), BF), _rows(gen, (H,), F32)
    dy[1] = dy[4] = 0.0
    h[4] = 0.0
    for eps in (1e-6, 1e-14, 1e-37):
        dx = _check(h, dy, w, eps, f"eps {eps}")
        assert not dx[[1, 4]].any()
        dx = _check(h, dy, w, eps, f"eps {eps}, grad_h", dh)
        assert torch.equal(dx[[1, 4]], dh[[1, 4]].float())
