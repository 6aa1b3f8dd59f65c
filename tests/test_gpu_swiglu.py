"""GPU parity of the gated activation and its gradients (oracle/layer.py).  u = 2^-24.

The sigmoid: the exponential's argument in two parts (its rest off by 2^-25), the
exponential and the reciprocal within an ulp (2 u) each, the sum: 6 u.  y: three
more products, 10 u of |y|; scales and codes are those of per_token_cast_to_fp8
on the same call's F32 y, bit for bit.  Gradients: up to eight roundings beside
the sigmoid's: 20 u of the absolute terms (for the gate's |z u| s (1 + |g|), 1 -
s being off by u of 1).  A row's sum adds at most 8 I / 2048 FMAs a lane, 6 steps
and 4 waves: 60 u of the absolute terms for I up to 8192.  A sigmoid below 2^-126
counts as zero: 88 * 2^-126 of the other factors at most.  BF16: half a step, 2^-8."""

import numpy as np
import pytest

from oracle import layer

from helpers import say
from test_gpu_norm import BF, F32, HALF, U, _blank, _close, _gen, _np, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402

LOST = 88 * 2.0 ** -126


@pytest.mark.parametrize("R,I", [(1, 1), (3, 7), (5, 64), (2, 100), (17, 128), (4, 129), (9, 512), (3, 520), (2, 1000),
                                 (5, 2048), (2, 4096), (1, 8192)])
@pytest.mark.parametrize("xt,gt,weighted", [(BF, BF, False), (F32, F32, True), (BF, F32, True), (F32, BF, False)])
def test_parity(R, I, xt, gt, weighted):
    say(f"swiglu R={R} I={I} {xt} {gt} weighted {weighted}")
    gen = _gen(R * 1009 + I)
    pad = 8 if R % 2 else 2
    x = _rows(gen, (R, 2 * I), xt, 4.0, pad)
    w = torch.rand(R, 2, generator=gen, device="cuda")[:, 1] if weighted else None
    y = _blank((R, I), F32, pad)
    q = torch.full((R, I + pad), 0xEE, dtype=torch.uint8, device="cuda")[:, :I]
    sf = torch.full((-(-I // 128), R), float("nan"), device="cuda").t()
    xn, wn = _np(x), None if w is None else _np(w)
    want = layer.swiglu(xn, wn)
    for ue8m0 in (False, True):
        assert mg.swiglu(x, y=y, q=q, sf=sf, row_weights=w, use_ue8m0=ue8m0)[1] is sf
        _close(y, want, 10 * U * np.abs(want) + LOST * 50, "y")
        q2, sf2 = torch.empty(R, -(-I // 16) * 16, dtype=torch.uint8, device="cuda")[:, :I], torch.empty_like(sf)
        aligned = torch.zeros(R, -(-I // 4) * 4, device="cuda")[:, :I]
        aligned.copy_(y)
        mg.per_token_cast_to_fp8(aligned, q2, sf2, use_ue8m0=ue8m0)
        assert torch.equal(sf, sf2) and torch.equal(q, q2)
    y16 = _blank((R, I), BF, pad)
    assert mg.swiglu(x, y=y16, row_weights=w) is y16
    assert torch.equal(y16, y.to(BF))
    dy, dx = _rows(gen, (R, I), gt, 1.0, pad), _blank((R, 2 * I), xt, pad)
    dw = torch.full((R, 2), float("nan"), device="cuda")
    assert mg.swiglu_bwd(x, dy, dx, row_weights=w, grad_row_weights=dw[:, 0]) is dx
    rx, rw, size, wsize = layer.swiglu_bwd(xn, _np(dy), wn)
    _close(dx, rx, 20 * U * size + HALF[xt] * np.abs(rx) + LOST * 50, "grad_x")
    _close(dw[:, 0], rw, 60 * U * wsize + LOST * 50 * I, "grad_row_weights")
    assert torch.isnan(dw[:, 1]).all()
    again = _blank((R, 2 * I), xt, pad)
    mg.swiglu_bwd(x, dy, again, row_weights=w)
    assert torch.equal(again, dx)
    mg.swiglu_bwd(x, dy, x, row_weights=w)  # in place
    assert torch.equal(x, dx)


def test_large_gates():
    say("swiglu of gates from -1e30 to 1e30")
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 80, -80, 87, -87, 100, -100, 1e4, -1e4, 1e30, -1e30],
                     device="cuda")
    x = torch.cat([g, torch.full_like(g, 0.75)])[None]
    y, dx, dw = _blank((1, 16), F32), _blank((1, 32), F32), _blank((1,), F32)
    mg.swiglu(x, y=y)
    mg.swiglu_bwd(x, torch.ones(1, 16, device="cuda"), dx, grad_row_weights=dw)
    want = layer.swiglu(_np(x))
    _close(y, want, 10 * U * np.abs(want) + LOST, "y")
    rx, rw, size, wsize = layer.swiglu_bwd(_np(x), np.ones((1, 16)))
    _close(dx, rx, 20 * U * size + LOST * 1e2, "grad_x")
    _close(dw, rw, 60 * U * wsize, "grad_row_weights")


@pytest.mark.parametrize("counts,max_m", [([0, 3, 5, 1], 5), ([7, -2, 100, 0], 9), ([0, 0, 0, 0], 4), ([1, 1, 1, 1], 1)])
def test_masked_rows(counts, max_m):
    say(f"swiglu masked {counts} of {max_m}")
    gen = _gen(3)
    G, I = len(counts), 392
    x = _rows(gen, (G, max_m, 2 * I), BF, 2.0)
    rows = [min(max(c, 0), max_m) for c in counts]
    live = torch.arange(max_m, device="cuda")[None] < torch.tensor(rows, device="cuda")[:, None]
    x[~live] = float("nan")  # what is not read may hold anything
    m = torch.tensor(counts, dtype=torch.int32, device="cuda")
    w = torch.rand(G * max_m, generator=gen, device="cuda")
    y = torch.full((G, max_m, I), 7.0, device="cuda", dtype=BF)
    q = torch.full((G, max_m, I), 0x55, dtype=torch.uint8, device="cuda")
    sf = torch.full((G, 4, max_m), 9.0, device="cuda").transpose(1, 2)
    mg.swiglu(x, y=y, q=q, sf=sf, masked_m=m, row_weights=w)
    dy = _rows(gen, (G, max_m, I), BF)
    dx, dw = torch.full((G, max_m, 2 * I), 5.0, device="cuda", dtype=BF), torch.full((G * max_m,), 3.0, device="cuda")
    mg.swiglu_bwd(x, dy, dx, masked_m=m, row_weights=w, grad_row_weights=dw)
    assert (y[~live] == 7).all() and (q[~live] == 0x55).all() and (sf[~live] == 9).all()
    assert (dx[~live] == 5).all() and (dw.view(G, max_m)[~live] == 3).all()
    if live.any():
        a, b, ws = x[live], dy[live], w.view(G, max_m)[live]
        y2, q2 = torch.empty_like(y[live]), torch.empty_like(q[live])
        sf2, dx2, dw2 = torch.empty(len(a), 4, device="cuda"), torch.empty_like(a), torch.empty(len(a), device="cuda")
        mg.swiglu(a, y=y2, q=q2, sf=sf2, row_weights=ws)
        mg.swiglu_bwd(a, b, dx2, row_weights=ws, grad_row_weights=dw2)
        assert torch.equal(y[live], y2) and torch.equal(q[live], q2) and torch.equal(sf[live], sf2)
        assert torch.equal(dx[live], dx2) and torch.equal(dw.view(G, max_m)[live], dw2)
        want = layer.swiglu(_np(a), _np(ws))
        _close(y2, want, (10 * U + 2.0 ** -8) * np.abs(want) + LOST * 50, "y")


def test_what_is_not_finite():
    say("swiglu of NaN and infinities")
    x = torch.zeros(3, 512, device="cuda")
    x[:, :256], x[:, 256:] = 1.0, 2.0
    x[0, 3], x[1, 300], x[2, 255], x[2, 511] = float("nan"), float("inf"), float("-inf"), 0.0
    q, sf, y = torch.zeros(3, 256, dtype=torch.uint8, device="cuda"), torch.zeros(3, 2, device="cuda"), _blank((3, 256), F32)
    mg.swiglu(x, y=y, q=q, sf=sf)
    bad = torch.zeros(3, 256, dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 44] = bad[2, 255] = True
    assert torch.equal((q & 0x7F) == 0x7F, bad) and torch.equal(torch.isfinite(y), ~bad)
    assert torch.equal(sf, sf[0, 0].expand(3, 2)) and float(y[1, 44]) == float("inf")


def test_empty_calls():
    x, dw = torch.zeros(4, 0, device="cuda"), torch.full((4,), 5.0, device="cuda")
    mg.swiglu(x, y=torch.zeros(4, 0, device="cuda"))
    mg.swiglu_bwd(x, torch.zeros(4, 0, device="cuda"), torch.zeros(4, 0, device="cuda"), grad_row_weights=dw)
    assert torch.equal(dw, torch.zeros_like(dw))
    e = torch.zeros(0, 8, device="cuda")
    mg.swiglu(e, y=torch.zeros(0, 4, device="cuda"))


def test_graph_replays_follow_the_counts():
    say("swiglu replayed with other counts")
    gen = _gen(4)
    x, m = _rows(gen, (4, 6, 256), BF), torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    y, eager = torch.zeros(4, 6, 128, dtype=BF, device="cuda"), torch.zeros(4, 6, 128, dtype=BF, device="cuda")
    mg.swiglu(x, y=y, masked_m=m)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg.swiglu(x, y=y, masked_m=m)
    for counts in ([0, 6, 1, 2], [6, 0, 0, 0], [2, 2, 2, 2]):
        m.copy_(torch.tensor(counts, dtype=torch.int32))
        x.copy_(_rows(gen, (4, 6, 256), BF))
        y.zero_()
        eager.zero_()
        graph.replay()
        torch.cuda.synchronize()
        mg.swiglu(x, y=eager, masked_m=m)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
