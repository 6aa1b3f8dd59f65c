"""The gradient of the norm's weight over many rows, with a bound from the rows
that a lane adds up.  u = 2^-24.

rms_norm_bwd leaves P partial rows (its workspace over a row's bytes); a workgroup
takes R rows side by side: 16 up to H = 128, 8 up to 256, 4 up to 1024, else 1.  A
lane adds up ceil(rows / (P R)) products, R - 1 sums join those side by side, then
at most ceil(P / 32) and 32 the partial rows; xh is within 24 u."""

import numpy as np
import pytest

from oracle import layer

from helpers import say
from test_gpu_norm import BF, F32, HALF, U, _blank, _close, _gen, _np, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402


def steps(T, H):
    P = mg.rms_norm_bwd_workspace(T, H) // (4 * H)
    R = 16 if H <= 128 else 8 if H <= 256 else 4 if H <= 1024 else 1
    return -(-T // (P * R)) + R + -(-P // 32) + 32


@pytest.mark.parametrize("T,H", [(2 ** 20 + 5, 8), (200001, 128), (70001, 200), (50003, 512), (30001, 1000), (9001, 2048),
                                 (5003, 4096), (3001, 7168), (1501, 16384), (7, 64), (1, 4096)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_bound(T, H, dt):
    say(f"gradient of the norm's weight, T={T} H={H} {dt}")
    gen = _gen(T + H)
    dy, h, w = _rows(gen, (T, H), dt, 0.1), _rows(gen, (T, H), dt, 3.0), _rows(gen, (H,), F32)
    dx, dw = _blank((T, H), dt), torch.full((H,), float("nan"), device="cuda")
    ws = torch.full((mg.rms_norm_bwd_workspace(T, H) // 4,), float("nan"), device="cuda")
    mg.rms_norm_bwd(dy, h, w, dx, grad_weight=dw, workspace=ws, eps=1e-3)
    _, rw, _, wsize = layer.rms_norm_bwd(_np(dy), _np(h), _np(w), 1e-3)
    _close(dw, rw, (steps(T, H) + 26) * U * wsize + 1e-38, "grad_weight")
