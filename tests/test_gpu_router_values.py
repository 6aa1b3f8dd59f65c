"""Expert routing where FP32 scores and their differences run out: saturated and
underflowed scores, rows of one confident expert, NaN beside masked experts.

u = 2^-24.  A sigmoid (an exponential, a sum, a quotient) is off by at most
4 u of itself."""

import numpy as np
import pytest

from oracle import router

from helpers import say, to_dev
from test_gpu_router import CHOICE_GAP, _logits, _mg, _route

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


def test_no_expert_no_weight():
    """A NaN among the chosen and fewer eligible experts than choices: the
    weights of the chosen are NaN, those of the places left over are 0."""
    say("moe_route_topk NaN with fewer eligible experts than choices")
    x = np.full((3, 40), -np.inf, dtype=np.float32)
    x[0, 7], x[0, 30] = np.nan, 1.0
    x[1, 3] = np.nan
    x[2, 5], x[2, 6] = 2.0, 1.0
    d, _ = _logits(x, False)
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            idx, w = _route(d, 4, score=score, renormalize=renorm)
            i, v = idx.cpu().numpy(), w.cpu().numpy()
            assert i.tolist() == [[30, 7, -1, -1], [3, -1, -1, -1], [5, 6, -1, -1]], (score, renorm)
            assert np.all(v[i == -1] == 0), (score, renorm, v.tolist())
            assert np.isnan(v[0, 1]) and np.isnan(v[1, 0]) and np.all(np.isfinite(v[2]))


@pytest.mark.parametrize("T", [300, 2100, 8200])  # 64, 32 and 16 lanes a token
def test_scores_over_the_range_of_the_exponential(T):
    """One expert's sigmoid and a softmax of two, the larger logit 0: the
    exponential within an ulp (2 u), its sum with 1 and the quotient u each:
    4 u of the score, whatever the logit."""
    say(f"moe_route_topk scores over the range of the exponential T={T}")
    x = np.linspace(-80, 80, T).astype(np.float32)[:, None]
    d, xv = _logits(x, False)
    _, w = _route(d, 1, score="sigmoid", renormalize=False)
    ref = 1 / (1 + np.exp(-xv))
    err = np.abs(w.cpu().numpy() - ref)
    assert np.all(err <= 4 * U * ref), f"sigmoid: {np.max(err / ref) / U} u at {xv[np.argmax(err / ref)]}"
    d, xv = _logits(np.concatenate([np.zeros_like(x), -np.abs(x)], axis=1), False)
    ref = np.exp(xv) / (1 + np.exp(xv[:, 1:]))
    for renorm in (True, False):
        idx, w = _route(d, 2, score="softmax", renormalize=renorm)
        want = np.take_along_axis(ref, idx.cpu().numpy().astype(np.int64), 1)
        err = np.abs(w.cpu().numpy() - want)
        assert np.all(err <= 4 * U * want), f"softmax: {np.max(err / want) / U} u"


@pytest.mark.parametrize("T,E,k,bf16", [(64, 40, 20, False), (200, 256, 8, False), (33, 64, 6, True)])
def test_gradient_of_confident_sigmoid_experts(T, E, k, bf16):
    """dx = g scale s(x) s(-x): two sigmoids and three products, at most 12 u of
    itself, from logits of -40 to 40, where 1 - s is far below FP32's spacing at 1."""
    say(f"moe_route_topk_bwd confident sigmoid T={T} E={E} k={k}")
    rng = np.random.default_rng(60 + E)
    x = rng.uniform(-40, 40, size=(T, E)).astype(np.float32)
    x[0] = np.linspace(8, 30, E)
    idx = np.argsort(rng.uniform(size=(T, E)), axis=1)[:, :k].astype(np.int32)
    g = rng.normal(size=(T, k)).astype(np.float32)
    d, xv = _logits(x, bf16)
    out = torch.empty(T, E, device="cuda")
    _mg().moe_route_topk_bwd(d, to_dev(idx), to_dev(g), out, score="sigmoid", renormalize=False, scale=1.5)
    ref = np.zeros((T, E))
    z = np.take_along_axis(xv, idx.astype(np.int64), 1)
    np.put_along_axis(ref, idx.astype(np.int64), 1.5 * g.astype(np.float64) / (1 + np.exp(-z)) / (1 + np.exp(z)), 1)
    err = np.abs(out.cpu().numpy() - ref)
    assert np.all(err <= 12 * U * np.abs(ref)), f"largest relative error {np.max(err / np.maximum(np.abs(ref), 1e-300))}"


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("T,E,k", [(300, 64, 6), (100, 256, 8), (40, 33, 1), (50, 60, 20)])
def test_gradient_of_confident_rows(score, renorm, T, E, k):
    """Weights that are a mean's: the gradient of one is
        q_j sum_i q_i (g_j - g_i),
    which is small where one expert has nearly all of the weight, though the
    g_i are not.  Its terms carry the relative error e = (k + 40 + 4 max|x -
    max|) u of their weights, and the mean that is taken off is off by e of the
    largest |g|, once more by e: |error| <= q_j (4 e sum_i q_i |g_j - g_i| +
    4 e^2 max|g|).  (sigmoid, renormalised: q = s / D, times 1 - s_j, and 1e-20
    g_j / D beside the sum; for softmax weights as they are, the sum is over all
    experts, those not chosen with g = 0.)"""
    say(f"moe_route_topk_bwd confident rows T={T} E={E} k={k} {score} renorm={renorm}")
    rng = np.random.default_rng(80 + E + k)
    x = rng.normal(size=(T, E)).astype(np.float32)
    idx = np.argsort(rng.uniform(size=(T, E)), axis=1)[:, :k].astype(np.int32)
    rows = np.arange(T)
    if score == "softmax":
        x[rows, idx[:, 0]] += rng.uniform(0, 30, size=T).astype(np.float32)  # one chosen expert stands out
    else:
        x[:, :] -= rng.uniform(0, 60, size=(T, 1)).astype(np.float32)
        x[rows, idx[:, 0]] += rng.uniform(0, 40, size=T).astype(np.float32)
    if k > 2:
        idx[5, 2] = -1
        idx[6, 1] = idx[6, 0]          # named twice
    g = (rng.normal(size=(T, k)) + 2.0).astype(np.float32)
    d, xv = _logits(x, False, pad=1)
    out = torch.empty(T, E, device="cuda")
    _mg().moe_route_topk_bwd(d, to_dev(idx), to_dev(g), out, score=score, renormalize=renorm, scale=1.0)
    got = out.cpu().numpy().astype(np.float64)
    ok = idx >= 0
    at = np.clip(idx, 0, E - 1).astype(np.int64)
    g64 = np.where(ok, g, 0.0).astype(np.float64)
    spread = (xv.max(axis=1, keepdims=True) - xv.min(axis=1, keepdims=True)) if score == "softmax" else np.zeros((T, 1))
    e = (k + 40 + 4 * spread) * U
    gmax = np.abs(g64).max(axis=1, keepdims=True)
    ref, bound = np.zeros((T, E)), np.full((T, E), 1e-37)
    if score == "softmax" and not renorm:
        p = router._scores(xv, score)
        ds = np.zeros((T, E))
        for j in range(k):
            ds[rows, at[:, j]] += g64[:, j]
        diff = ds[:, :, None] - ds[:, None, :]
        ref = p * (p[:, None, :] * diff).sum(axis=2)
        bound += p * (4 * e * (p[:, None, :] * np.abs(diff)).sum(axis=2) + 4 * e * e * gmax)
    else:
        z = np.take_along_axis(xv, at, 1)
        if score == "softmax":
            q = np.where(ok, np.exp(z - np.where(ok, z, -np.inf).max(axis=1, keepdims=True)), 0.0)
            q /= q.sum(axis=1, keepdims=True)
            rest, slope = np.zeros((T, 1)), 1.0
        else:
            s = np.where(ok, 1 / (1 + np.exp(-z)), 0.0)
            D = s.sum(axis=1, keepdims=True) + 1e-20
            q, rest, slope = s / D, 1e-20 / D, 1 / (1 + np.exp(z))
        diff = g64[:, :, None] - g64[:, None, :]
        r = q * slope * ((q[:, None, :] * diff).sum(axis=2) + rest * g64)
        b = q * slope * (4 * e * ((q[:, None, :] * np.abs(diff)).sum(axis=2) + rest * np.abs(g64)) + 4 * e * e * gmax)
        for j in range(k):
            ref[rows, at[:, j]] += np.where(ok[:, j], r[:, j], 0.0)
            bound[rows, at[:, j]] += np.where(ok[:, j], b[:, j], 0.0)
    assert np.allclose(ref, router.moe_route_topk_bwd(xv, idx, g, score, renorm, 1.0), rtol=1e-6, atol=1e-12)
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"{np.sum(err > bound)} outside, largest error / bound {np.max(err / bound)}"


@pytest.mark.parametrize("T", [37, 2100, 8200])  # 64, 32 and 16 lanes a token
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(128, (1, 1, 1)), (96, (8, 3, 1)), (33, (1, 1, 1))])
def test_choice_without_a_bias_follows_the_logits(T, score, E, groups):
    """Scores rise with their logits: without a bias the best choices are the
    largest logits, also where FP32 scores are equal -- 0 or 1, or a logit's
    last bits apart.  Equal logits go by index."""
    say(f"moe_route_topk order of the logits T={T} E={E} {score} groups={groups}")
    rng = np.random.default_rng(E + T)
    k = 6
    x = rng.normal(size=(T, E)).astype(np.float32)
    x[0::6, 3] = 150.0                                         # all others underflow in a softmax
    x[1::6] = x[1::6] * 5 + 40                                 # all sigmoids round to 1
    x[2::6] = x[2::6] * 5 - 120                                # all sigmoids underflow
    x[3::6] *= 1e-7                                            # close together
    x[4::6] = np.round(x[4::6]) + 200.0                        # ties
    d, xv = _logits(x, False, pad=2)
    idx, w = _route(d, k, score=score, n_group=groups[0], topk_group=groups[1], group_top=1)
    c = xv.copy()
    if groups[0] > 1:
        per = c.reshape(T, groups[0], -1)
        keep = np.argsort(-per.max(axis=2), axis=1, kind="stable")[:, :groups[1]]
        drop = np.ones((T, groups[0]), dtype=bool)
        np.put_along_axis(drop, keep, False, axis=1)
        per[drop] = -np.inf
    want = np.argsort(-c, axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), want), f"{np.sum(np.any(idx.cpu().numpy() != want, axis=1))} rows differ"


def _picks_by_value(x, k, idx, w, bias, kw, what):
    """Every row of a routing against float64, near ties by value.

    The picks are distinct eligible experts; position by position their float64
    choice is the oracle's within CHOICE_GAP of the values it is made of (a near
    tie may go either way and nothing else may); where there are groups, against
    the best of the groups that the picks show to be kept, each of which scores
    within the gap of the last one that the oracle keeps.  The weights are those
    of the kernel's own picks, in every row."""
    bias64 = None if bias is None else bias.astype(np.float64)
    score, n_group, topk_group, top = (kw.get(n, d) for n, d in (("score", "softmax"), ("n_group", 1), ("topk_group", 1),
                                                                ("group_top", 1)))
    idx, w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    c = router.route_choices(x, bias64, score, 1, 1, 1)
    size = np.abs(np.where(np.isfinite(c), c, 0.0)) + router._scores(x, score)
    finite = np.where(np.isfinite(x), x, 0.0)
    spread = np.abs(finite - finite.max(axis=1, keepdims=True)).max() if score == "softmax" else 0.0
    swapped = 0
    for t in range(len(x)):
        got = idx[t][idx[t] >= 0]
        assert np.all(idx[t][len(got):] == -1) and len(set(got.tolist())) == len(got), f"{what}: row {t}"
        ct = c[t].copy()
        if n_group > 1:
            per = ct.reshape(n_group, -1)
            rank = np.array([np.sort(g[g > -np.inf])[::-1][:top].sum() if np.any(g > -np.inf) else -np.inf for g in per])
            gap = CHOICE_GAP * 2 * size[t].reshape(n_group, -1).max(axis=1)
            cut = np.sort(rank)[::-1][topk_group - 1]
            shown = np.unique(got // per.shape[1])
            with np.errstate(invalid="ignore"):
                near = np.abs(rank - cut) <= gap
            sure = (rank > cut) & ~near
            assert len(shown) <= topk_group and np.all((sure | near)[shown]), f"{what}: row {t}, groups"
            # the groups that can be kept: what is sure, what the picks show, and the best near ones
            rest = [g for g in np.argsort(-rank, kind="stable") if near[g] and g not in shown]
            keep = set(np.flatnonzero(sure).tolist()) | set(shown.tolist())
            keep |= set(rest[:max(0, topk_group - len(keep))])
            per[[g for g in range(n_group) if g not in keep]] = -np.inf
        best = np.argsort(-ct, kind="stable")[:k]
        best = best[ct[best] > -np.inf]
        assert len(best) == len(got), f"{what}: row {t}, {len(got)} picks of {len(best)}"
        off = np.abs(c[t][got] - ct[best])
        assert np.all(off <= CHOICE_GAP * np.maximum(size[t][got], size[t][best])), f"{what}: row {t}"
        swapped += not np.array_equal(got, best)
        rw = router.route_weights(x[t], idx[t], score, kw.get("renormalize", True), kw.get("scale", 1.0))
        assert np.all(np.abs(w[t] - rw) <= (k + 20 + 2 * spread) * U * np.abs(rw) + 1e-37), f"{what}: row {t}, weights"
    return swapped


@pytest.mark.parametrize("T,E,k,score,bias,groups,renorm,step", [
    (300, 256, 8, "sigmoid", True, (8, 4, 2), True, 0),
    (200, 64, 6, "softmax", False, (8, 3, 1), False, 0),
    (50, 1024, 64, "sigmoid", True, (64, 32, 2), True, 0),       # the limits: many near ties
    (50, 513, 5, "softmax", False, (27, 13, 2), True, 0),
    (100, 60, 4, "softmax", True, (1, 1, 1), False, 0),
    # logits so close that most neighbours are near ties
    (200, 128, 8, "sigmoid", True, (1, 1, 1), True, 1e-7),
    (200, 128, 8, "sigmoid", True, (8, 3, 2), False, 2e-7),
    (200, 128, 8, "softmax", True, (8, 3, 1), True, 2e-7),
    (2100, 96, 6, "softmax", False, (8, 3, 2), True, 3e-7),
    (8200, 64, 6, "sigmoid", False, (8, 3, 2), True, 3e-7),
])
def test_near_ties_by_value(T, E, k, score, bias, groups, renorm, step):
    say(f"moe_route_topk near ties T={T} E={E} k={k} {score} groups={groups} step={step}")
    rng = np.random.default_rng(500 + E + T)
    if step:
        x = (0.5 + rng.integers(-20, 20, size=(T, E)) * step).astype(np.float32)
    else:
        x = (rng.normal(size=(T, E)) * 2).astype(np.float32)
    x[7, E // 2:], x[8] = -np.inf, -np.inf
    b = (rng.integers(-3, 4, size=E) * max(step, 0.02)).astype(np.float32) if bias else None
    d, xv = _logits(x, False)
    kw = dict(score=score, n_group=groups[0], topk_group=groups[1], group_top=groups[2], renormalize=renorm, scale=1.5)
    idx, w = _route(d, k, bias=None if b is None else to_dev(b), **kw)
    swapped = _picks_by_value(xv, k, idx, w, b, kw, f"T={T} E={E}")
    say(f"  {swapped} rows with a near tie the other way")
