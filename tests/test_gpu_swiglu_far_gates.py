"""The activation and its gradients for gates so low that their sigmoid is no
normal FP32 number (below -87.3), while what it is multiplied by may be large:
against oracle/layer.py.  u = 2^-24.

Results are products of factors that each are within 12 u, whatever their size: 20 u
of the absolute terms, as for other gates, and what FP32 cannot hold of the
result, 2^-149 of each of 32 parts (a value is handed on divided by 32)."""

import numpy as np
import pytest

from oracle import layer

from helpers import say
from test_gpu_norm import BF, F32, HALF, U, _blank, _close, _gen, _np, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402

SMALL = 2.0 ** -144


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("R,I,weighted", [(1, 8, False), (3, 100, True), (5, 128, False), (4, 520, True), (2, 2048, True)])
def test_parity(R, I, weighted, dt):
    say(f"swiglu of far gates R={R} I={I} {dt} weighted {weighted}")
    gen = _gen(R + I)
    g = -86.0 - 320.0 * torch.rand(R, I, generator=gen, device="cuda") ** 3
    near = torch.rand(R, I, generator=gen, device="cuda") < 0.3  # ordinary gates between them
    g = torch.where(near, torch.randn(R, I, generator=gen, device="cuda") * 4.0, g)
    u = _rows(gen, (R, I), F32) * torch.where(near, 1.0, 1e37)
    x = torch.cat([g, u], dim=1).to(dt)
    w = torch.rand(R, generator=gen, device="cuda") + 0.5 if weighted else None
    xn, wn = _np(x), None if w is None else _np(w)
    y, dx, dw = _blank((R, I), F32), _blank((R, 2 * I), F32), torch.full((R,), float("nan"), device="cuda")
    mg.swiglu(x, y=y, row_weights=w)
    want = layer.swiglu(xn, wn)
    _close(y, want, 20 * U * np.abs(want) + SMALL, "y")
    q, sf = torch.zeros(R, I, dtype=torch.uint8, device="cuda"), torch.zeros(R, -(-I // 128), device="cuda")
    q2, sf2 = torch.empty(R, -(-I // 16) * 16, dtype=torch.uint8, device="cuda")[:, :I], torch.empty_like(sf)
    mg.swiglu(x, q=q, sf=sf, row_weights=w)
    aligned = torch.zeros(R, -(-I // 4) * 4, device="cuda")[:, :I]
    aligned.copy_(y)
    mg.per_token_cast_to_fp8(aligned, q2, sf2)
    assert torch.equal(sf, sf2) and torch.equal(q, q2)
    dy = _rows(gen, (R, I), dt)
    mg.swiglu_bwd(x, dy, dx, row_weights=w, grad_row_weights=dw)
    rx, rw, size, wsize = layer.swiglu_bwd(xn, _np(dy), wn)
    _close(dx, rx, 20 * U * size + SMALL, "grad_x")
    _close(dw, rw, 60 * U * wsize + I * SMALL, "grad_row_weights")
    mg.swiglu_bwd(x, dy, x, row_weights=w)  # in place
    assert torch.equal(x, dx.to(dt))


def test_gate_by_gate():
    """Every half from -80 to -420 with the largest up: down to results that FP32 does not hold."""
    say("swiglu gate by gate")
    g = -80.0 - 0.5 * torch.arange(680, device="cuda")
    x = torch.cat([g, torch.full_like(g, 3e38)])[None]
    y, dx, dw = _blank((1, 680), F32), _blank((1, 1360), F32), _blank((1,), F32)
    mg.swiglu(x, y=y)
    want = layer.swiglu(_np(x))
    _close(y, want, 20 * U * np.abs(want) + SMALL, "y")
    dy = torch.full((1, 680), 0.01, device="cuda")
    mg.swiglu_bwd(x, dy, dx, grad_row_weights=dw)
    rx, rw, size, wsize = layer.swiglu_bwd(_np(x), _np(dy))
    _close(dx, rx, 20 * U * size + SMALL, "grad_x")
    _close(dw, rw, 60 * U * wsize, "grad_row_weights")


def test_what_is_not_finite():
    """The lowest finite gates give zeros; minus infinity and NaN give NaN, each in its own place."""
    say("swiglu of the lowest gates")
    x = torch.zeros(1, 32, device="cuda")
    x[0, :16], x[0, 16:] = 1.0, 2.0
    x[0, 3], x[0, 5], x[0, 7], x[0, 9] = -1e30, -3.4e38, float("-inf"), float("nan")
    x[0, 21] = 3e38
    y, dx = _blank((1, 16), F32), _blank((1, 32), F32)
    mg.swiglu(x, y=y)
    mg.swiglu_bwd(x, torch.ones(1, 16, device="cuda"), dx)
    odd = torch.zeros(1, 16, dtype=torch.bool, device="cuda")
    odd[0, 7] = odd[0, 9] = True
    assert torch.equal(torch.isnan(y), odd) and torch.equal(torch.isnan(dx), torch.cat([odd, odd], dim=1))
    assert not y[0, [3, 5]].any() and not dx[0, [3, 5, 19, 21]].any()
    assert torch.equal(y[0, :3], y[0, 10:13])
