"""Expert routing where FP32 scores and their differences run out: saturated and
underflowed scores, rows of one confident expert, NaN beside masked experts.

u = 2^-24.  A sigmoid (an exponential, a sum, a quotient) is off by at most
4 u of itself."""

import numpy as np
import pytest

from oracle import router

from helpers import say, to_dev
from test_gpu_router import _logits, _mg, _route

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
