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
