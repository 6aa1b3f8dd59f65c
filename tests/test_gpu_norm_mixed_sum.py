"""The norm's sum of an F32 x and a BF16 residual is rounded once, to BF16: equal,
bit for bit, to the exact sum (float64 holds it) rounded to eight bits, half to even."""

import numpy as np
import pytest

from oracle import layer

from helpers import say
from test_gpu_norm import BF, F32, U, _blank, _close, _gen, _np, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402


def _bf16(v):
    """float64 -> the nearest values of eight bits (normal ones, none near the largest)."""
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def _near_ties(gen, T, H):
    """x that lead from residuals on BF16's grid to halfway between two neighbours, or a last bit beside it."""
    res = _rows(gen, (T, H), BF, 3.0)
    m, e = torch.frexp(res.float())
    half = torch.ldexp(torch.ones_like(m), e - 9)
    off = torch.tensor([0.0, 2.0 ** -22, -2.0 ** -22, 2.0 ** -20, -2.0 ** -20, 0.0, 2.0 ** -23, -2.0 ** -21], device="cuda")
    off = off.repeat(T * H // 8 + 1)[:T * H].view(T, H)
    sign = torch.randint(0, 2, (T, H), generator=gen, device="cuda") * 2 - 1
    return half * sign * (1.0 + off), res


@pytest.mark.parametrize("T,H", [(1, 8), (3, 100), (5, 1000), (4, 4096), (3, 7168), (2, 16384)])
def test_rounded_once(T, H):
    say(f"rms_norm of F32 plus BF16, T={T} H={H}")
    gen = _gen(H)
    w = _rows(gen, (H,), F32)
    cases = [_near_ties(gen, T, H), (_rows(gen, (T, H), F32, 0.01), _rows(gen, (T, H), BF, 3.0)),
             (_rows(gen, (T, H), F32, 300.0), _rows(gen, (T, H), BF, 3.0))]
    cases[0][0][0, 0], cases[0][1][0, 0] = 2.0 ** -8 + 2.0 ** -30, 1.0  # above the tie by less than FP32 holds
    for x, res in cases:
        want = _bf16(_np(x) + _np(res))
        h, y, y2 = _blank((T, H), BF), _blank((T, H), F32), _blank((T, H), F32)
        mg.rms_norm(x, w, y=y, residual=res, h=h)
        assert np.array_equal(_np(h), want)
        mg.rms_norm(h, w, y=y2)  # the norm is of what is stored
        assert torch.equal(y, y2)
        mg.rms_norm(x, w, y=y2, residual=res)
        assert torch.equal(y, y2)


def test_sums_at_the_edges():
    """Zeros, cancelled sums, infinities and NaN, what passes BF16's largest value."""
    say("rms_norm of F32 plus BF16 at the edges")
    inf, nan, top = float("inf"), float("nan"), 3.3895313892515355e38
    x = torch.tensor([0.0, -1.0, 1.0, inf, -inf, nan, 1e36, 1e-40, 1e30, -3e38], device="cuda")
    res = torch.tensor([0.0, 1.0, -0.5, 1.0, inf, 1.0, top, 0.0, -1e30, 3e38], device="cuda").to(BF)
    H = 8
    x, res = x[:, None].repeat(1, H).contiguous(), res[:, None].repeat(1, H).contiguous()
    h = _blank(x.shape, BF)
    mg.rms_norm(x, torch.ones(H, device="cuda"), y=_blank(x.shape, F32), residual=res, h=h)
    got = h[:, 0].float().cpu()
    total = (x.double() + res.double())[:, 0].float().cpu()  # (none of these near a tie)
    want = total.to(BF).float()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])
