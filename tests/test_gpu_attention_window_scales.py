"""paged_attention_fp8 with pages of 16 tokens, two of them to a tile of 32
positions: a page that lies wholly before every window takes no part, whatever
its codes and its scales hold."""

import numpy as np
import pytest

from helpers import say, to_dev
from test_gpu_paged_attention import _case, _run, _compare

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("S,n,Hq,H,D,lens,window", [
    (1, 1, 4, 2, 64, [61], 40),              # sees 21 .. 60
    (2, 3, 8, 2, 128, [200, 122], 50),       # two rows' windows begin on either side of a page's end
    (1, 2, 4, 1, 256, [90], 9),
    (1, 1, 8, 1, 128, [5000], 3220),         # cut along the cache; sees from 1780
    (1, 4, 40, 2, 64, [4700], 1989),
])
def test_pages_before_every_window(S, n, Hq, H, D, lens, window):
    P = 16
    say(f"paged_attention_fp8 unseen pages n={n} D={D} lens={lens} window={window}")
    c = _case(D + n, S, n, Hq, H, D, P, lens)
    clean, lse = _run(c, 0.1, window)
    _compare(c, clean, lse, 0.1, window, "clean")
    gone = []
    for s, ln in enumerate(lens):
        first = max(0, ln - n - window + 1)  # the first position that any query sees
        gone += c["table"][s, :first // P].tolist()
    assert gone
    for ks, vs in ((np.nan, 1.0), (1.0, np.nan), (1.0, 0.0), (0.0, 1.0), (np.inf, np.inf), (-1.0, -1.0), (3e38, 1e-38)):
        d = dict(c, **{x: c[x].copy() for x in ("kc", "vc", "ks", "vs")})
        d["kc"][gone], d["vc"][gone], d["ks"][gone], d["vs"][gone] = 0x7F, 0x7F, ks, vs
        d["dev"] = [to_dev(d[x]) for x in ("kc", "vc", "ks", "vs")]
        out, l = _run(d, 0.1, window)
        assert np.array_equal(out, clean) and np.array_equal(l, lse), f"scales {ks}, {vs}"
