"""GPU parity of the norm and its gradients (oracle/layer.py).  u = 2^-24.

y: the sum of squares of a row of at most 16384 elements takes at most 16 FMAs a
lane, 6 steps over a wave and 16 over the waves, of terms of one sign: 38 u of
itself, 19 u of its root; the mean, the root, the quotient and the two products
one u each at most: 24 u of |y|; a BF16 y half a step more, 2^-8.
Codes and scales: those of per_token_cast_to_fp8 on the same call's F32 y, bit
for bit; h: the sum's bits.
grad_x: every term (grad_h, r g, r xh mean) carries the errors of r and of xh,
24 u each, of the mean's sum of at most 38 + 2 roundings, and of the last FMAs:
100 u of the sum of the absolute terms.
grad_weight: a workgroup adds up to ceil(rows / workgroups) terms, then up to 16
rows side by side, up to 32 partial rows and 32 sums: with xh's errors
ceil(rows / 512) + 120 u of the absolute terms (rows past 512 workgroups)."""

import numpy as np
import pytest

from oracle import layer

from helpers import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 0.0}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(gen, shape, dtype, sigma=1.0, pad=0):
    """Rows `pad` elements apart from each other."""
    wide = torch.randn(*shape[:-1], shape[-1] + pad, generator=gen, device="cuda") * sigma
    return wide.to(dtype)[..., :shape[-1]]


def _blank(shape, dtype, pad=0):
    wide = torch.full((*shape[:-1], shape[-1] + pad), float("nan"), device="cuda")
    return wide.to(dtype)[..., :shape[-1]]


def _np(t):
    return t.double().cpu().numpy()


def _close(got, want, bound, what):
    got = _np(got)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    err = np.abs(got - want)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    say(f"  {what}: {worst:.3f} of the bound")
    assert worst <= 1.0, f"{what}: {worst} of the bound"


SHAPES = [(1, 1), (3, 7), (5, 64), (2, 100), (33, 128), (1, 129), (7, 256), (9, 257), (4, 512), (5, 1000), (6, 1024),
          (3, 1025), (2, 2048), (3, 2056), (2, 4096), (3, 5120), (17, 7168), (2, 8192), (2, 8193), (1, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("xt,rt,wt", [(BF, BF, BF), (F32, None, F32), (BF, F32, F32), (F32, BF, BF)])
def test_forward(T, H, xt, rt, wt):
    say(f"rms_norm T={T} H={H} {xt} residual {rt} weight {wt}")
    gen = _gen(T * 100003 + H)
    pad = -H % 8 if T % 2 else 3
    x, w = _rows(gen, (T, H), xt, 2.0, pad), _rows(gen, (H,), wt)
    res = None if rt is None else _rows(gen, (T, H), rt, 5.0, pad)
    h = None if rt is None else _blank((T, H), rt, pad)
    y = _blank((T, H), F32, pad)
    q = torch.full((T, H + pad), 0xEE, dtype=torch.uint8, device="cuda")[:, :H]
    sf = torch.full((-(-H // 128), T), float("nan"), device="cuda").t()
    eps = 1e-5
    for ue8m0 in (False, True):
        assert mg.rms_norm(x, w, y=y, q=q, sf=sf, residual=res, h=h, eps=eps, use_ue8m0=ue8m0)[0] is q
        total = x
        if rt is not None:
            total = (x.float() + res.float()).to(rt)
            assert torch.equal(h, total)
        want = layer.rms_norm(_np(total), _np(w), eps)
        _close(y, want, 24 * U * np.abs(want) + 1e-38, "y")
        q2, sf2 = torch.empty(T, -(-H // 16) * 16, dtype=torch.uint8, device="cuda")[:, :H], torch.empty_like(sf)
        aligned = torch.zeros(T, -(-H // 4) * 4, device="cuda")[:, :H]
        aligned.copy_(y)
        mg.per_token_cast_to_fp8(aligned, q2, sf2, use_ue8m0=ue8m0)
        assert torch.equal(sf, sf2) and torch.equal(q, q2)
    y16 = _blank((T, H), BF, pad)
    assert mg.rms_norm(x, w, y=y16, residual=res, eps=eps) is y16
    assert torch.equal(y16, y.to(BF))


def test_heads_are_views():
    say("rms_norm over heads of a projection's rows")
    gen = _gen(5)
    for T, heads, H, extra in ((1, 1, 128, 0), (13, 6, 128, 2), (4, 3, 64, 1), (3, 5, 200, 1), (2, 2, 1024, 3)):
        big = _rows(gen, (T, heads + extra, H), BF)
        before = big.clone()
        x, w, y = big[:, :heads], _rows(gen, (H,), F32), _blank((T, heads, H), BF)
        q = torch.zeros(heads, T, H, dtype=torch.uint8, device="cuda").transpose(0, 1)
        sf = torch.zeros(T, heads, -(-H // 128), device="cuda")
        mg.rms_norm(x, w, y=y, q=q, sf=sf)
        want = layer.rms_norm(_np(x), _np(w), 1e-6)
        _close(y, want, (24 * U + 2.0 ** -8) * np.abs(want), f"y {T}x{heads}x{H}")
        flat = torch.zeros(T * heads, H, dtype=torch.uint8, device="cuda")
        fsf = torch.zeros(T * heads, -(-H // 128), device="cuda")
        mg.rms_norm(x.reshape(T * heads, H).contiguous(), w, q=flat, sf=fsf)
        assert torch.equal(q.reshape(T * heads, H), flat) and torch.equal(sf.view(T * heads, -1), fsf)
        mg.rms_norm(x, w, y=x)  # in place: the other heads stay
        assert torch.equal(x, y) and torch.equal(big[:, heads:], before[:, heads:])
        dy, dx, dw = _rows(gen, (T, heads, H), BF), _blank((T, heads, H), F32), torch.empty(H, device="cuda")
        ws = torch.full((mg.rms_norm_bwd_workspace(T * heads, H) // 4,), float("nan"), device="cuda")
        mg.rms_norm_bwd(dy, before[:, :heads], w, dx, grad_weight=dw, workspace=ws)
        rx, rw, size, wsize = layer.rms_norm_bwd(_np(dy), _np(before[:, :heads]), _np(w), 1e-6)
        _close(dx, rx, 100 * U * size, "grad_x")
        _close(dw, rw, 130 * U * wsize, "grad_weight")


@pytest.mark.parametrize("T,H", SHAPES + [(2000, 64), (1537, 1024), (1100, 2048), (1030, 4096)])
@pytest.mark.parametrize("gt,ht,dt,wt", [(BF, BF, BF, F32), (F32, F32, None, BF), (BF, F32, F32, F32)])
def test_gradients(T, H, gt, ht, dt, wt):
    say(f"rms_norm_bwd T={T} H={H} {gt} {ht} {dt} {wt}")
    gen = _gen(T * 7 + H)
    pad = -H % 8 if T % 2 else 1
    dy, h, w = _rows(gen, (T, H), gt, 0.1, pad), _rows(gen, (T, H), ht, 3.0, pad), _rows(gen, (H,), wt)
    dh = None if dt is None else _rows(gen, (T, H), dt, 0.1, pad)
    dx, dw = _blank((T, H), ht, pad), torch.full((H,), float("nan"), device="cuda").to(wt)
    ws = torch.full((mg.rms_norm_bwd_workspace(T, H) // 4,), float("nan"), device="cuda")
    assert mg.rms_norm_bwd(dy, h, w, dx, grad_weight=dw, workspace=ws, grad_h=dh, eps=1e-3) is dx
    rx, rw, size, wsize = layer.rms_norm_bwd(_np(dy), _np(h), _np(w), 1e-3, None if dh is None else _np(dh))
    _close(dx, rx, 100 * U * size + HALF[ht] * np.abs(rx) + 1e-38, "grad_x")
    _close(dw, rw, (-(-T // 512) + 120) * U * wsize + HALF[wt] * np.abs(rw) + 1e-38, "grad_weight")
    # without the weight's gradient, and in place of each input
    alone = _blank((T, H), ht, pad)
    mg.rms_norm_bwd(dy, h, w, alone, grad_h=dh, eps=1e-3)
    assert torch.equal(alone, dx)
    for t in (dy, h, dh):
        if t is not None and t.dtype == ht:
            d, hh, g = dy.clone(), h.clone(), None if dh is None else dh.clone()
            out = d if t is dy else hh if t is h else g
            mg.rms_norm_bwd(d, hh, w, out, grad_h=g, eps=1e-3)
            assert torch.equal(out, dx)


@pytest.mark.parametrize("T,H", [(40000, 64), (9001, 256), (6001, 512), (5003, 1024), (2500, 2048), (1301, 4096), (600, 7168), (530, 16384)])
@pytest.mark.parametrize("dt", [None, BF])
def test_gradients_of_many_rows(T, H, dt):
    """Several rows a workgroup, in place; a workgroup adds up at most ceil(T / 256) terms of a column."""
    say(f"rms_norm_bwd T={T} H={H} grad_h {dt}")
    gen = _gen(T + H)
    dy, h, w = _rows(gen, (T, H), BF, 0.1), _rows(gen, (T, H), BF, 3.0), _rows(gen, (H,), F32)
    dh = None if dt is None else _rows(gen, (T, H), dt, 0.1)
    rx, rw, size, wsize = layer.rms_norm_bwd(_np(dy), _np(h), _np(w), 1e-3, None if dh is None else _np(dh))
    ws = torch.full((mg.rms_norm_bwd_workspace(T, H) // 4,), float("nan"), device="cuda")
    far = [_blank((T, H), BF, 8), _blank((T, H), BF, 1)]
    dws = [torch.empty(H, device="cuda") for _ in range(3)]
    for dx, dw in zip(far, dws):
        mg.rms_norm_bwd(dy, h, w, dx, grad_weight=dw, workspace=ws, grad_h=dh, eps=1e-3)
    _close(far[0], rx, 100 * U * size + HALF[BF] * np.abs(rx) + 1e-38, "grad_x")
    _close(dws[0], rw, (-(-T // 256) + 120) * U * wsize + 1e-38, "grad_weight")
    assert torch.equal(far[0], far[1]) and torch.equal(dws[0], dws[1])
    # inputs whose rows are not whole 16-byte words, and in place
    odd = torch.empty(T, H + 1, dtype=BF, device="cuda")[:, :H]
    odd.copy_(h)
    mg.rms_norm_bwd(dy, odd, w, odd, grad_weight=dws[2], workspace=ws, grad_h=dh, eps=1e-3)
    assert torch.equal(odd, far[0]) and torch.equal(dws[2], dws[0])
    mg.rms_norm_bwd(dy, h, w, h, grad_weight=dws[2], workspace=ws, grad_h=dh, eps=1e-3)
    assert torch.equal(h, far[0]) and torch.equal(dws[2], dws[0])


def test_rows_at_the_edges_of_fp32():
    say("rms_norm of rows of zeros, of the smallest and of the largest values")
    H = 300
    gen = _gen(9)
    base = torch.randn(6, H, generator=gen, device="cuda", dtype=torch.float64)
    base[0] = 0.0
    for i, f in ((1, 1e-30), (2, 1e18), (3, 1e30), (4, 1e36)):
        base[i] *= f
    base[5, 0] = 3e38  # one value that outweighs the rest
    x, w = base.float(), _rows(gen, (H,), F32)
    y, q, sf = _blank((6, H), F32), torch.zeros(6, H, dtype=torch.uint8, device="cuda"), torch.zeros(6, 3, device="cuda")
    mg.rms_norm(x, w, y=y, q=q, sf=sf)
    want = layer.rms_norm(_np(x), _np(w), 1e-6)
    _close(y, want, 26 * U * np.abs(want) + 1e-37, "y")
    dy, dh = _rows(gen, (6, H), F32), torch.zeros(6, H, device="cuda")
    dx, dw = _blank((6, H), F32), torch.empty(H, device="cuda")
    ws = torch.empty(mg.rms_norm_bwd_workspace(6, H) // 4, device="cuda")
    mg.rms_norm_bwd(dy, x, w, dx, grad_weight=dw, workspace=ws, grad_h=dh)
    rx, rw, size, wsize = layer.rms_norm_bwd(_np(dy), _np(x), _np(w), 1e-6)
    _close(dx, rx, 104 * U * size + 1e-37, "grad_x")
    _close(dw, rw, 130 * U * wsize + 1e-37, "grad_weight")


@pytest.mark.parametrize("H", [100, 300, 4096])
def test_an_eps_below_the_squares_range(H):
    """Squares that FP32 cannot hold count where eps does not cover them."""
    say(f"rms_norm of small rows with a small eps, H={H}")
    gen = _gen(11)
    x = torch.randn(6, H, generator=gen, device="cuda", dtype=torch.float64)
    for i, f in enumerate((1.0, 1e-14, 1e-16, 1e-20, 1e-25, 1e-36)):
        x[i] *= f
    x, w, dy = x.float(), _rows(gen, (H,), F32), _rows(gen, (6, H), F32, 1e-6)
    for eps in (1e-28, 1e-32, 1e-38, float(np.float32(1e-44))):
        y = _blank((6, H), F32)
        mg.rms_norm(x, w, y=y, eps=eps)
        want = layer.rms_norm(_np(x), _np(w), float(np.float32(eps)))
        _close(y, want, 26 * U * np.abs(want) + 1e-37, f"y, eps {eps}")
        dx, dw = _blank((6, H), F32), torch.empty(H, device="cuda")
        ws = torch.empty(mg.rms_norm_bwd_workspace(6, H) // 4, device="cuda")
        mg.rms_norm_bwd(dy, x, w, dx, grad_weight=dw, workspace=ws, eps=eps)
        rx, rw, size, wsize = layer.rms_norm_bwd(_np(dy), _np(x), _np(w), float(np.float32(eps)))
        _close(dx, rx, 104 * U * size + 1e-37, "grad_x")
        _close(dw, rw, 130 * U * wsize + 1e-37, "grad_weight")


def test_many_short_rows():
    say("rms_norm of 2^22 + 5 rows of 8")
    T = 2 ** 22 + 5
    x, w = _rows(_gen(12), (T, 8), BF), _rows(_gen(13), (8,), F32)
    y = _blank((T, 8), BF)
    mg.rms_norm(x, w, y=y)
    at = [0, 2 ** 21, 2 ** 22 - 1, 2 ** 22, T - 1]
    want = layer.rms_norm(_np(x[at]), _np(w), 1e-6)
    _close(y[at], want, (26 * U + 2.0 ** -8) * np.abs(want) + 1e-37, "y")
    assert torch.isfinite(y).all()
    dx, dw = _blank((T, 8), BF), torch.empty(8, device="cuda")
    ws = torch.empty(mg.rms_norm_bwd_workspace(T, 8) // 4, device="cuda")
    mg.rms_norm_bwd(y, x, w, dx, grad_weight=dw, workspace=ws)
    assert torch.isfinite(dx).all()
    rx, _, size, _ = layer.rms_norm_bwd(_np(y[at]), _np(x[at]), _np(w), 1e-6)
    _close(dx[at], rx, 104 * U * size + 2.0 ** -8 * np.abs(rx) + 1e-37, "grad_x")
    _, rw, _, wsize = layer.rms_norm_bwd(_np(y), _np(x), _np(w), 1e-6)
    _close(dw, rw, (-(-T // 512) + 120) * U * wsize, "grad_weight")


def test_what_is_not_finite_stays_in_its_row():
    say("rms_norm of rows with NaN and infinities")
    H = 640
    gen = _gen(10)
    x, w = _rows(gen, (8, H), BF), _rows(gen, (H,), F32)
    clean = [0, 2, 3, 5, 7]
    want_q, want_sf = torch.zeros(8, H, dtype=torch.uint8, device="cuda"), torch.zeros(8, 5, device="cuda")
    mg.rms_norm(x, w, q=want_q, sf=want_sf)
    x[1, 5], x[4, 600], x[6, 0] = float("nan"), float("inf"), float("-inf")
    y, q, sf = _blank((8, H), F32), torch.zeros_like(want_q), torch.zeros_like(want_sf)
    mg.rms_norm(x, w, y=y, q=q, sf=sf)
    assert torch.equal(q[clean], want_q[clean]) and torch.equal(sf[clean], want_sf[clean])
    assert torch.isnan(y[1]).all() and torch.isnan(y[4, 600]) and torch.isnan(y[6, 0])
    assert torch.equal((q & 0x7F) == 0x7F, ~torch.isfinite(y)) and torch.isfinite(sf).all()
    # a weight that is not finite spoils its column only, not the scale of its block
    w2 = w.clone()
    w2[130], w2[131] = float("inf"), float("nan")
    mg.rms_norm(x[clean], w2, q=q[:5], sf=sf[:5])
    codes, ref = q[:5].clone(), want_q[clean]
    assert ((codes[:, 130:132] & 0x7F) == 0x7F).all()
    other = [0, 2, 3, 4]
    assert torch.equal(sf[:5][:, other], want_sf[clean][:, other]) and torch.isfinite(sf[:5]).all()
    assert torch.equal(codes[:, :128], ref[:, :128]) and torch.equal(codes[:, 256:], ref[:, 256:])
    dx = _blank((8, H), F32)
    mg.rms_norm_bwd(_rows(gen, (8, H), BF), x, w, dx)
    assert torch.isfinite(dx[clean]).all()


def test_no_rows():
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), float("nan"), device="cuda")
    e = torch.empty(0, 64, device="cuda")
    mg.rms_norm(e, w, y=e.clone())
    mg.rms_norm_bwd(e, e, w, e.clone(), grad_weight=dw)
    assert torch.equal(dw, torch.zeros_like(dw))


def test_the_same_bits_every_time_and_on_any_stream():
    say("rms_norm: repeated, on another stream, replayed from a graph")
    gen = _gen(11)
    T, H = 700, 1024
    x, res, w = _rows(gen, (T, H), BF), _rows(gen, (T, H), BF), _rows(gen, (H,), BF)
    dy, dh = _rows(gen, (T, H), BF), _rows(gen, (T, H), BF)

    def room():
        return dict(h=_blank((T, H), BF), q=torch.zeros(T, H, dtype=torch.uint8, device="cuda"),
                    sf=torch.zeros(T, 8, device="cuda"), dx=_blank((T, H), BF), dw=torch.zeros(H, device="cuda"),
                    ws=torch.empty(mg.rms_norm_bwd_workspace(T, H) // 4, device="cuda"))

    def step(o, stream=None):
        mg.rms_norm(x, w, q=o["q"], sf=o["sf"], residual=res, h=o["h"], stream=stream)
        mg.rms_norm_bwd(dy, o["h"], w, o["dx"], grad_weight=o["dw"], workspace=o["ws"], grad_h=dh, stream=stream)

    def same(a, b):
        return all(torch.equal(a[n], b[n]) for n in ("h", "q", "sf", "dx", "dw"))

    first, second, third = room(), room(), room()
    step(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(second, stream=side)
    torch.cuda.synchronize()
    assert same(first, second)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(third)
    for turn in range(3):
        x.copy_(_rows(gen, (T, H), BF))
        graph.replay()
        torch.cuda.synchronize()
        step(first)
        torch.cuda.synchronize()
        assert same(first, third), turn
