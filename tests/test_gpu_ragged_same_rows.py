"""The same row through the same group's matrix gives the same bits whatever the
other groups hold and whichever tile shape the sizes of the call lead to."""

import pytest

from helpers import say
from test_gpu_norm import BF, F32, _gen, _rows
from test_gpu_ragged import _offsets

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("N,K", [(1032, 2048), (520, 4096), (2560, 1984), (300, 2048)])
def test_rows_in_other_batches(form, N, K):
    if form == "nn":
        N = -(-N // 8) * 8
    say(f"{form} the same rows in other batches, N={N} K={K}")
    gen = _gen(N + K)
    G, own = 12, 5  # rows of each group that come again
    b = _rows(gen, (G, N, K) if form == "nt" else (G, K, N), BF, K ** -0.5)
    rows = _rows(gen, (G, own, K), BF)
    call = mg.m_grouped_bf16_gemm_nt_ragged if form == "nt" else mg.m_grouped_bf16_gemm_nn_ragged
    seen = None
    for extra in ([0] * G, [300] * G, [1, 0, 2000, 7, 0, 130, 64, 0, 700, 1, 2, 3], [0] * 6 + [4000] + [0] * 5,
                  [90, 40, 0, 300] * 3, [2500] + [0] * 11, [0] * 11 + [1500]):
        parts, at, first = [], [], 0
        for g in range(G):  # the rows are the group's last
            parts += [_rows(gen, (extra[g], K), BF), rows[g]]
            at.append(first + extra[g])
            first += extra[g] + own
        a = torch.cat(parts)
        d = torch.empty(first, N, device="cuda")
        call(a, b, d, _offsets([n + own for n in extra]))
        got = torch.stack([d[i:i + own] for i in at])
        if seen is None:
            seen = got
        assert torch.equal(got, seen), extra
