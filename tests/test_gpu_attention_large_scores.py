"""paged_attention_fp8 where the scores are very large: a finite score must give a
finite row, however large it is.

Queries are one-hot, so a score is one product of powers of two with a code and
exact in FP32.  One position of a head holds the largest code in the element
the query looks at (448 against at most 240, or -240 against -448): the next
score is at least 7/15 of it away.  Its exponent is off by a few u = 2^-24 of
itself, so from a score of 2^10 on everything else weighs less than 2^-300,
the output is that position's value, which BF16 holds exactly (4 bits), and
lse the score: 2^-8 |v| and 8 u |score| are allowed."""

import numpy as np
import pytest

from moe_grouped_gemm_x128_amd import synth
from oracle import bf16_decode, e4m3_decode, e4m3_encode

from helpers import say, to_dev
from test_gpu_paged_attention import _case, _run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


def _peaked(seed, S, n, Hq, H, D, P, lens, sign, twins):
    """A cache in which, for element j of a head, one position (two neighbours of
    one page with `twins`) is above all; the queries look at elements of their own."""
    c = _case(seed, S, n, Hq, H, D, P, lens)
    rng = np.random.default_rng(seed + 1)
    shape = c["kc"].shape
    low = rng.uniform(-240, 240, size=shape) if sign > 0 else np.full(shape, -448.0)
    kc = e4m3_encode(low)
    peak = {}
    for s, ln in enumerate(lens):
        seen = ln - n + 1                 # what every query sees
        for h in range(H):
            for j in range(D):
                t = int(rng.integers(0, seen))
                if twins:
                    t = min(t // P * P + t % P // 2 * 2, seen - 2)
                    t -= t % 2
                for u in range(2 if twins else 1):
                    kc[c["table"][s, t // P], h, t % P + u, j] = e4m3_encode(np.array([448.0 if sign > 0 else -240.0]))[0]
                peak[s, h, j] = t
    for s, ln in enumerate(lens):
        if ln % P:
            kc[c["table"][s, ln // P], :, ln % P:] = 0x7F
    used = np.unique(np.concatenate([c["table"][s, :-(-ln // P)] for s, ln in enumerate(lens)]))
    c["kc"], c["ks"] = kc, c["ks"].copy()
    c["ks"][used] = 2.0 ** -6
    q = np.zeros((S, n, Hq, D), dtype=np.float32)
    look = rng.integers(0, D, size=(S, n, Hq))
    np.put_along_axis(q, look[..., None], 1.0, axis=3)
    bits = synth.bf16_bits_from_f32(q)
    c["q"] = bf16_decode(bits)
    c["dq"] = to_dev(bits.view(np.int16)).view(torch.bfloat16)
    c["dev"] = [to_dev(c[x]) for x in ("kc", "vc", "ks", "vs")]
    return c, look, peak


@pytest.mark.parametrize("S,n,Hq,H,D,P,lens,sign,twins", [
    (1, 1, 8, 2, 128, 64, [777], 1, False),
    (2, 2, 4, 1, 64, 16, [90, 33], 1, True),
    (2, 3, 16, 2, 128, 32, [200, 70], -1, False),      # 24 rows: two row tiles a wave
    (1, 1, 4, 1, 256, 128, [700], 1, True),
    (1, 2, 4, 2, 64, 16, [5000], 1, False),            # cut along the cache
    (1, 1, 4, 1, 128, 64, [6001], -1, True),
])
def test_large_scores(S, n, Hq, H, D, P, lens, sign, twins):
    c, look, peak = _peaked(D + P + n, S, n, Hq, H, D, P, lens, sign, twins)
    g = Hq // H
    for power in (10, 15, 18, 20, 21, 22, 23, 24, 26, 29, 33, 45, 80, 115):
        for more in (1.0, 1.3, 1.7):
            scale = float(np.float32(2.0 ** power * more))
            say(f"paged_attention_fp8 D={D} P={P} n={n} lens={lens} sign={sign} scale={scale:g}")
            out, lse = _run(c, scale)
            assert np.all(np.isfinite(out)) and np.all(np.isfinite(lse)), "not finite"
            for s in range(S):
                for i in range(n):
                    for a in range(Hq):
                        h, t = a // g, peak[s, a // g, look[s, i, a]]
                        page = c["table"][s, t // P]
                        v = e4m3_decode(c["vc"][page, h, t % P:t % P + 1 + twins]).mean(axis=0) * float(c["vs"][page, h])
                        assert np.all(np.abs(out[s, i, a] - v) <= 2.0 ** -8 * np.abs(v)), f"row {s, i, a}"
                        x = scale * (448.0 if sign > 0 else -240.0) * 2.0 ** -6
                        assert abs(lse[s, i, a] - x - np.log(1 + twins)) <= 8 * U * (abs(x) + 32), f"lse {s, i, a}"
