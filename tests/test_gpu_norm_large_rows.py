"""Rows of the norm whose squares leave FP32's range by far: whole rows up to the
largest values of F32 and BF16, forward and gradients, against oracle/layer.py.
u = 2^-24.

Such a row's squares are summed again of scaled values, a product and an addition
each: at most 1 + 24 roundings a lane, 6 over a wave and 16 over the waves, of
terms of one sign, 47 u of the sum and 24 u of its root; the mean, the root, the
quotient and the two products are one u each: 29 u of |y|.  Gradients: 29 u in r
and in xh for 24, so 110 u of the absolute terms where test_gpu_norm has 100; r of
the largest values is as small as 2^-128, held to 2^-150: 2^-22, 4 u more.  The
weight's gradient adds up four rows at most beside xh's 29 u: 40 u."""

import numpy as np
import pytest

from oracle import layer

from helpers import say
from test_gpu_norm import BF, F32, HALF, U, _blank, _close, _gen, _np, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402

SIZES = (5e36, 1e37, 1e38, 3e38)  # of a row's values


def _large(gen, H, dtype):
    """A row of each size: signs at random, values within a tenth of each other, one row of equal ones."""
    part = 1.0 - 0.1 * torch.rand(len(SIZES), H, generator=gen, device="cuda", dtype=torch.float64)
    part[-1] = 1.0
    sign = torch.randint(0, 2, part.shape, generator=gen, device="cuda") * 2 - 1
    return (part * sign * torch.tensor(SIZES, device="cuda", dtype=torch.float64)[:, None]).to(dtype)


@pytest.mark.parametrize("H", [1, 2, 16, 100, 300, 1024, 4096, 5120, 7168, 16384])
@pytest.mark.parametrize("dt", [F32, BF])
def test_forward(H, dt):
    say(f"rms_norm of rows of 5e36 to 3e38, H={H} {dt}")
    gen = _gen(H)
    x, w, T = _large(gen, H, dt), _rows(gen, (H,), F32), len(SIZES)
    y, q = _blank((T, H), F32), torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(T, -(-H // 128), device="cuda")
    mg.rms_norm(x, w, y=y, q=q, sf=sf)
    want = layer.rms_norm(_np(x), _np(w), 1e-6)
    _close(y, want, 29 * U * np.abs(want), "y")
    q2, sf2 = torch.empty(T, -(-H // 16) * 16, dtype=torch.uint8, device="cuda")[:, :H], torch.empty_like(sf)
    aligned = torch.zeros(T, -(-H // 4) * 4, device="cuda")[:, :H]
    aligned.copy_(y)
    mg.per_token_cast_to_fp8(aligned, q2, sf2)
    assert torch.equal(sf, sf2) and torch.equal(q, q2)
    y16 = _blank((T, H), BF)
    mg.rms_norm(x, w, y=y16)
    assert torch.equal(y16, y.to(BF))
    # as the sum of two halves, and in place
    h = _blank((T, H), dt)
    half = x * 0.5
    mg.rms_norm(half, w, y=y16, residual=half, h=h)
    assert torch.equal(h, x) and torch.equal(y16, y.to(BF))


@pytest.mark.parametrize("H", [1, 2, 16, 100, 300, 1024, 4096, 5120, 7168, 16384])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("past", [False, True])
def test_gradients(H, dt, past):
    say(f"rms_norm_bwd of rows of 5e36 to 3e38, H={H} {dt} grad_h {past}")
    gen = _gen(H + 1)
    h, w, T = _large(gen, H, dt), _rows(gen, (H,), F32), len(SIZES)
    dy = _rows(gen, (T, H), dt, 1e8)
    dh = _rows(gen, (T, H), dt, 1e-30) if past else None
    dx, dw = _blank((T, H), F32), torch.full((H,), float("nan"), device="cuda")
    ws = torch.full((mg.rms_norm_bwd_workspace(T, H) // 4,), float("nan"), device="cuda")
    mg.rms_norm_bwd(dy, h, w, dx, grad_weight=dw, workspace=ws, grad_h=dh)
    rx, rw, size, wsize = layer.rms_norm_bwd(_np(dy), _np(h), _np(w), 1e-6, None if dh is None else _np(dh))
    _close(dx, rx, 114 * U * size + 2.0 ** -140, "grad_x")
    _close(dw, rw, 40 * U * wsize, "grad_weight")
