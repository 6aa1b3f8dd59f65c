"""GPU parity of the expert routing and its gradient (oracle/router.py).

Indices: equal to the oracle's wherever the choices that decide (the k best,
the next one, and the groups' scores) are apart by more than CHOICE_GAP of
their size: a score is off by at most 4 u of itself (u = 2^-24: the
exponential, the sum, the quotient, each within an ulp), plus u |x - max x|
for the rounding of a softmax argument, a biased choice or a group's sum by
one more rounding each of at most their own size plus the score's; 32 u of
|choice| + score covers arguments up to 16.  Rows with a closer pair are
compared by value.

Weights: relative error at most (k + 20 + 2 max|x - max|) u: the score, the
sum of k scores, the quotient and the factor.  Gradients: every term (g z / D
and the like) carries at most that relative error, so |error| <= (k + 40 + 4
max|x - max|) u times the sum of the absolute terms, plus BF16's 2^-8."""

import numpy as np
import pytest

from moe_grouped_gemm_x128_amd import synth
from oracle import bf16_decode, router

from helpers import say, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
CHOICE_GAP = 32 * U


def _mg():
    import moe_grouped_gemm_x128_amd as mg

    return mg


def _logits(x, bf16, pad=0):
    """Device logits [T, E] (rows `pad` elements apart from each other) and their values."""
    T, E = x.shape
    if bf16:
        bits = synth.bf16_bits_from_f32(x)
        d = to_dev(np.pad(bits, ((0, 0), (0, pad))).view(np.int16)).view(torch.bfloat16)[:, :E]
        return d, bf16_decode(bits)
    d = to_dev(np.pad(np.asarray(x, np.float32), ((0, 0), (0, pad))))[:, :E]
    return d, np.asarray(x, np.float32).astype(np.float64)


def _route(d, k, **kw):
    T = d.shape[0]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), dtype=torch.float32, device="cuda")
    _mg().moe_route_topk(d, idx, w, **kw)
    torch.cuda.synchronize()
    return idx, w


def _check(x, k, idx, w, bias, kw, what):
    bias64 = None if bias is None else bias.astype(np.float64)
    opts = {n: kw.get(n, d) for n, d in (("score", "softmax"), ("n_group", 1), ("topk_group", 1), ("group_top", 1))}
    ridx, rw = router.moe_route_topk(x, k, bias=bias64, renormalize=kw.get("renormalize", True),
                                     scale=kw.get("scale", 1.0), **opts)
    idx, w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    c = router.route_choices(x, bias64, opts["score"], 1, 1, 1)
    size = np.abs(np.where(np.isfinite(c), c, 0.0)) + router._scores(x, opts["score"])  # what rounding errors scale with

    def close(v, mag, count):
        """Rows in which two of the `count` best values, or the last of them and the next, nearly tie."""
        order = np.argsort(-v, axis=1, kind="stable")[:, :count + 1]
        a, m = np.take_along_axis(v, order, 1), np.take_along_axis(mag, order, 1)
        with np.errstate(invalid="ignore"):
            gap = a[:, :-1] - a[:, 1:]
        return np.any((gap > 0) & (gap < CHOICE_GAP * np.maximum(m[:, :-1], m[:, 1:])), axis=1)  # (0: a tie, index order)

    near = np.zeros(len(x), dtype=bool)
    if opts["n_group"] > 1:
        per = np.where(np.isfinite(c), c, 0.0).reshape(len(x), opts["n_group"], -1)
        best = -np.sort(-per, axis=2)[:, :, :opts["group_top"]]
        near |= close(best.sum(axis=2), 2 * size.reshape(per.shape).max(axis=2), opts["topk_group"])
        c = router.route_choices(x, bias64, **opts)
    near |= close(c, size, k)
    # (64 choices of 1024 lie about 1/400 apart: a tenth of such rows is expected to hold a near tie)
    assert near.mean() <= 0.25 or len(x) < 10, f"{what}: {near.mean()} of the rows hold near ties"
    assert np.array_equal(idx[~near], ridx[~near]), f"{what}: indices"
    for t in np.flatnonzero(near):
        a, b = idx[t][idx[t] >= 0], ridx[t][ridx[t] >= 0]
        assert len(a) == len(b) == len(set(a.tolist())), f"{what}: row {t}"
    finite = np.where(np.isfinite(x), x, 0.0)
    spread = np.abs(finite - finite.max(axis=1, keepdims=True)).max() if opts["score"] == "softmax" else 0.0
    tol = (k + 20 + 2 * spread) * U
    err = np.abs(w[~near] - rw[~near])
    assert np.all(err <= tol * np.abs(rw[~near]) + 1e-37), f"{what}: weights off by {err.max()}"
    return idx


@pytest.mark.parametrize("T,E,k,score,bias,groups,renorm,scale,bf16", [
    (300, 256, 8, "sigmoid", True, (8, 4, 2), True, 2.5, False),
    (301, 256, 8, "sigmoid", True, (8, 4, 2), True, 2.5, True),
    (1, 256, 8, "sigmoid", True, (8, 4, 2), True, 2.5, False),
    (257, 128, 8, "softmax", False, (1, 1, 1), True, 1.0, True),
    (130, 64, 6, "softmax", False, (8, 3, 1), False, 16.0, True),
    (77, 60, 4, "softmax", True, (1, 1, 1), False, 1.0, False),
    (65, 33, 33, "sigmoid", False, (1, 1, 1), True, 1.0, False),     # every expert chosen
    (40, 1, 1, "softmax", False, (1, 1, 1), True, 1.0, False),
    (50, 1024, 64, "sigmoid", True, (64, 32, 2), True, 1.0, False),  # the limits
    (50, 513, 5, "softmax", False, (27, 13, 2), True, 1.0, True),    # groups of 19
    (33, 248, 7, "sigmoid", False, (8, 5, 2), False, 1.0, False),    # groups of 31
    (33, 96, 3, "sigmoid", True, (8, 5, 1), True, 1.0, True),        # groups of 12
    (20, 16, 2, "softmax", False, (16, 3, 2), True, 1.0, False),     # groups of one
    (9, 384, 8, "sigmoid", True, (3, 2, 2), True, 1.0, False),
])
def test_route_matches_oracle(T, E, k, score, bias, groups, renorm, scale, bf16):
    say(f"moe_route_topk T={T} E={E} k={k} {score} groups={groups} bias={bias} renorm={renorm} bf16={bf16}")
    rng = np.random.default_rng(700 + E)
    x = rng.normal(size=(T, E)).astype(np.float32) * 2
    b = (rng.normal(size=E) * 0.05).astype(np.float32) if bias else None
    d, xv = _logits(x, bf16, pad=3)
    kw = dict(score=score, n_group=groups[0], topk_group=groups[1], group_top=groups[2], renormalize=renorm, scale=scale)
    idx, w = _route(d, k, bias=None if b is None else to_dev(b), **kw)
    _check(xv, k, idx, w, b, kw, f"T={T} E={E}")


@pytest.mark.parametrize("T,E,k,score,bias,groups,renorm,bf16", [
    (2049, 96, 5, "sigmoid", True, (8, 3, 2), True, False),
    (2500, 400, 8, "softmax", False, (1, 1, 1), False, True),
    (3000, 30, 20, "sigmoid", False, (30, 25, 1), True, False),    # groups of one, more choices than 16 lanes
    (2100, 128, 40, "softmax", False, (1, 1, 1), True, False),     # more than 32
    (8193, 64, 6, "softmax", False, (8, 3, 1), False, True),
    (8200, 256, 8, "sigmoid", True, (8, 4, 2), True, False),
    (8205, 93, 3, "sigmoid", False, (3, 2, 2), True, True),        # groups of 31 on four lanes each
    (8300, 20, 18, "softmax", False, (1, 1, 1), True, False),
    (8193, 1, 1, "sigmoid", False, (1, 1, 1), False, False),
])
def test_many_tokens(T, E, k, score, bias, groups, renorm, bf16):
    """Token counts at which a token takes fewer lanes; ties included."""
    say(f"moe_route_topk many tokens T={T} E={E} k={k} {score} groups={groups}")
    rng = np.random.default_rng(900 + E)
    x = rng.normal(size=(T, E)).astype(np.float32) * 2
    x[5:40] = np.round(x[5:40])      # ties
    x[T - 7:T - 2] = -np.inf
    x[T - 1, E // 2:] = -np.inf
    b = (rng.normal(size=E) * 0.05).astype(np.float32) if bias else None
    d, xv = _logits(x, bf16, pad=8)
    kw = dict(score=score, n_group=groups[0], topk_group=groups[1], group_top=groups[2], renormalize=renorm)
    idx, w = _route(d, k, bias=None if b is None else to_dev(b), **kw)
    _check(xv, k, idx, w, b, kw, f"T={T} E={E}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, (1, 1, 1)), (256, (8, 3, 2)), (96, (8, 4, 1))])
def test_ties_go_to_the_lowest_index(score, E, groups):
    say(f"moe_route_topk ties {score} E={E} groups={groups}")
    rng = np.random.default_rng(3)
    x = rng.integers(0, 3, size=(64, E)).astype(np.float32)
    x[0] = 0.0
    x[1, ::2] = -0.0  # equal to +0
    x[1, 1::2] = 0.0
    kw = dict(score=score, n_group=groups[0], topk_group=groups[1], group_top=groups[2])
    d, xv = _logits(x, False)
    idx, w = _route(d, 8, **kw)
    got = _check(xv, 8, idx, w, None, kw, "ties")
    assert got[0].tolist() == list(range(8))


def test_masked_rows_and_values():
    say("moe_route_topk masks: -inf, the type's lowest value, NaN, +inf")
    E, k = 40, 4
    rng = np.random.default_rng(8)
    low = np.finfo(np.float32).min
    x = rng.normal(size=(8, E)).astype(np.float32)
    x[0] = -np.inf                      # a padded token: nowhere
    x[1, 3:] = -np.inf                  # three experts left
    x[2] = low                          # all at the lowest value: still a softmax
    x[3, 5:] = low
    x[4, 7] = np.nan
    x[5, 9] = np.inf
    x[6, 1:] = -np.inf
    for score in ("softmax", "sigmoid"):
        d, xv = _logits(x, False)
        idx, w = _route(d, k, score=score)
        i, v = idx.cpu().numpy(), w.cpu().numpy()
        assert np.all(i[0] == -1) and np.all(v[0] == 0)
        assert sorted(i[1, :3].tolist()) == [0, 1, 2] and i[1, 3] == -1 and v[1, 3] == 0
        assert abs(v[1].sum() - 1) < 1e-6
        assert i[2].tolist() == [0, 1, 2, 3]
        if score == "softmax":
            assert np.allclose(v[2], 0.25)
            assert np.all(np.isnan(v[5]))
        else:
            assert i[5, 0] == 9 and np.all(np.isfinite(v[5]))
        assert set(i[3].tolist()) <= set(range(5))
        assert 7 not in i[4].tolist() and np.all(np.isfinite(v[4]))
        assert i[6].tolist() == [0, -1, -1, -1] and abs(v[6, 0] - 1) < 1e-6
        for row in i:
            real = row[row >= 0]
            assert len(set(real.tolist())) == len(real) and np.all(real < E)
    # a bias of -inf takes an expert out; a whole group of them comes last
    b = np.zeros(E, dtype=np.float32)
    b[:10] = -np.inf
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2)
    d, xv = _logits(x[7:8], False)
    idx, w = _route(d, k, bias=to_dev(b), **kw)
    assert np.all(idx.cpu().numpy() >= 10)
    _check(xv, k, idx, w, b, kw, "bias -inf")


def test_rows_keep_their_places():
    """Strided tables: only the k columns of each row are written."""
    say("moe_route_topk strided outputs")
    x = np.random.default_rng(2).normal(size=(50, 64)).astype(np.float32)
    d, xv = _logits(x, False, pad=1)
    idx = torch.full((50, 9), -7, dtype=torch.int32, device="cuda")
    w = torch.full((50, 11), 5.0, dtype=torch.float32, device="cuda")
    _mg().moe_route_topk(d, idx[:, 2:8], w[:, 1:7], score="sigmoid")
    torch.cuda.synchronize()
    _check(xv, 6, idx[:, 2:8], w[:, 1:7], None, dict(score="sigmoid"), "strided")
    assert torch.all(idx[:, :2] == -7) and torch.all(idx[:, 8:] == -7)
    assert torch.all(w[:, :1] == 5) and torch.all(w[:, 7:] == 5)


@pytest.mark.parametrize("T,E,k,score,renorm,bf16,out_bf16", [
    (200, 256, 8, "sigmoid", True, False, False),
    (131, 64, 6, "softmax", False, True, True),
    (131, 65, 6, "softmax", True, False, False),
    (64, 33, 4, "sigmoid", False, True, False),
    (1, 128, 8, "softmax", False, False, True),
    (17, 1024, 64, "softmax", False, False, False),
    (17, 513, 7, "sigmoid", True, False, True),
    (5, 1, 1, "softmax", True, False, False),
    (33, 40, 20, "sigmoid", True, False, False),
    (20, 60, 40, "softmax", False, True, False),
    (130, 30, 18, "softmax", True, False, True),
    (70, 200, 12, "softmax", False, False, False),
])
def test_gradient_matches_oracle(T, E, k, score, renorm, bf16, out_bf16):
    say(f"moe_route_topk_bwd T={T} E={E} k={k} {score} renorm={renorm} bf16={bf16}/{out_bf16}")
    rng = np.random.default_rng(40 + E)
    x = rng.normal(size=(T, E)).astype(np.float32) * 2
    idx = np.argsort(rng.uniform(size=(T, E)), axis=1)[:, :k].astype(np.int32)
    if k > 1 and T > 2:
        idx[0, 1] = -1
        idx[1] = -1
        idx[2, 0] = E        # not an expert: nothing
        idx[T - 1, 1] = idx[T - 1, 0]  # named twice: both parts
    g = rng.normal(size=(T, k)).astype(np.float32)
    d, xv = _logits(x, bf16, pad=5)
    dt = torch.bfloat16 if out_bf16 else torch.float32
    out = torch.full((T, E + 2), 7.0, dtype=dt, device="cuda")
    _mg().moe_route_topk_bwd(d, to_dev(idx), to_dev(g), out[:, :E], score=score, renormalize=renorm, scale=1.5)
    torch.cuda.synchronize()
    assert torch.all(out[:, E:] == 7)
    got = out[:, :E].float().cpu().numpy().astype(np.float64)
    ref = router.moe_route_topk_bwd(xv, idx, g, score, renorm, 1.5)
    # absolute terms: the part of the choice itself and the part taken off
    ok = (idx >= 0) & (idx < E)
    s = router._scores(xv, score)
    z = np.where(ok, np.take_along_axis(s, np.clip(idx, 0, E - 1).astype(np.int64), 1), 0.0)
    D = np.maximum(z.sum(axis=1, keepdims=True), 1e-300) if renorm else np.ones((T, 1))
    ga = 1.5 * np.abs(g) * ok / D
    off = (ga * z).sum(axis=1, keepdims=True) / (D if renorm else 1.0)
    terms = np.zeros((T, E))
    for j in range(k):
        r = np.flatnonzero(ok[:, j])
        terms[r, idx[r, j]] += ga[r, j] + (off[r, 0] if renorm else 0.0)
    terms *= s
    if score == "softmax" and not renorm:
        terms += s * (ga * z).sum(axis=1, keepdims=True)
    spread = np.abs(xv - xv.max(axis=1, keepdims=True)).max() if score == "softmax" else 0.0
    bound = (k + 40 + 4 * spread) * U * terms + 1e-37 + (2.0 ** -8 * np.abs(ref) if out_bf16 else 0.0)
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"largest error / bound {np.max(err / bound)}"


def test_gradient_against_differences_of_the_forward():
    """Differences of the GPU's own weights: with step h the formula's third
    order gives h^2 scale / 6 and the FP32 weights 30 u scale / h; at h =
    2^-6 together below 2^-13 for scale 1 (k = 4 terms of weight |g| <= 3)."""
    say("moe_route_topk_bwd against differences of moe_route_topk")
    mg = _mg()
    E, k, h = 24, 4, 2.0 ** -6
    rng = np.random.default_rng(4)
    base = rng.permutation(np.arange(E) * 0.125 - 1.5).astype(np.float32)  # 1/8 apart: steps of 1/64 keep the choice
    x = np.repeat(base[None], 2 * E, axis=0)
    x[np.arange(E), np.arange(E)] += h
    x[np.arange(E) + E, np.arange(E)] -= h
    g = rng.uniform(-3, 3, size=(1, k)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d, _ = _logits(np.concatenate([x, base[None]]), False)
            idx, w = _route(d, k, score=score, renormalize=renorm)
            assert torch.all(idx == idx[:1])
            out = torch.empty(1, E, device="cuda")
            mg.moe_route_topk_bwd(d[2 * E:], idx[:1], to_dev(g), out, score=score, renormalize=renorm)
            wv = w.cpu().numpy().astype(np.float64)
            diff = ((wv[:E] - wv[E:2 * E]) * g).sum(axis=1) / (2 * h)
            err = np.abs(out[0].cpu().numpy() - diff).max()
            assert err <= 4 * 3 * (h * h / 6 + 30 * U / h), err


def test_graph_replays_with_new_logits():
    say("moe_route_topk + bwd under graph capture")
    mg = _mg()
    T, E, k = 100, 128, 6
    rng = np.random.default_rng(12)
    x = torch.empty(T, E, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w, g = torch.empty(T, k, device="cuda"), torch.randn(T, k, device="cuda")
    dx = torch.empty(T, E, device="cuda")
    x.copy_(torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg.moe_route_topk(x, idx, w, score="sigmoid")
        mg.moe_route_topk_bwd(x, idx, g, dx, score="sigmoid")
    for _ in range(3):
        x.copy_(torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (idx, w, dx)]
        mg.moe_route_topk(x, idx, w, score="sigmoid")
        mg.moe_route_topk_bwd(x, idx, g, dx, score="sigmoid")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, dx)))


def test_empty_calls():
    mg = _mg()
    x = torch.empty(0, 16, device="cuda")
    mg.moe_route_topk(x, torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda"))
    mg.moe_route_topk_bwd(x, torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda"),
                          torch.empty(0, 16, device="cuda"))
    # no choices: the gradient is zero
    y = torch.full((3, 16), 7.0, device="cuda")
    mg.moe_route_topk_bwd(torch.randn(3, 16, device="cuda"), torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                          torch.empty(3, 0, device="cuda"), y)
    torch.cuda.synchronize()
    assert torch.all(y == 0)
