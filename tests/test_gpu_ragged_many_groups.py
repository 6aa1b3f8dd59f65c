"""Ragged products of about as many groups as the kernel keeps the first tiles of
at hand (2048), and of more, which it seeks in the offsets: bounds of
test_gpu_ragged."""

import numpy as np
import pytest

from test_gpu_norm import BF, F32
from test_gpu_ragged import _case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _sizes(G, seed):
    """Most groups empty or of a row or two, some of more than a tile; the last partial run of 64 has both."""
    rng = np.random.default_rng(seed)
    s = rng.choice([0, 0, 0, 1, 2, 3], size=G)
    for i in (0, 63, 64, G // 2, G - 70, G - 3, G - 1):
        s[i] = 65
    s[G - 2] = 0
    return [int(v) for v in s]


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("G", [2047, 2048, 2049, 2112, 2200, 4097])
def test_groups_past_the_table(form, G):
    _case(form, _sizes(G, G), 16, 64, BF, None, first=3, behind=5)
    _case(form, _sizes(G, G + 1), 16, 64, F32, F32)


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("at", [0, 2047, 2048, 2100, 2199])
def test_one_group_with_rows(form, at):
    sizes = [0] * 2200
    sizes[at] = 200
    _case(form, sizes, 264, 64, F32, None, first=1, behind=1)


@pytest.mark.parametrize("form", ["nt", "nn"])
def test_all_empty(form):
    _case(form, [0] * 2200, 16, 64, BF, None, first=4)


def test_weight_gradients_of_many_groups():
    _case("tn", _sizes(2200, 9), 8, 16, F32, None, first=2, behind=2)
