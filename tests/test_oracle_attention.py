"""Pins of the paged-cache oracle: the rotation as a complex product, pages
built by hand, and the attention against a softmax over lists of positions."""

import numpy as np

from oracle import attention as at
from oracle import e4m3_decode, e4m3_encode


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(1)
    T, H, D, rot = 5, 2, 12, 8
    x = rng.normal(size=(T, H, D))
    ang = rng.uniform(0, 6, size=(T, rot // 2))
    for inter in (False, True):
        y = at.rotate(x, np.cos(ang), np.sin(ang), inter)
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
        z = (a + 1j * b) * np.exp(1j * ang)[:, None]
        c, d = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
        assert np.allclose(c + 1j * d, z, atol=1e-14)
        assert np.array_equal(y[..., rot:], x[..., rot:])


def test_scale_is_the_next_power_of_two():
    a = np.array([448.0, 449.0, 224.0, 1.0, 0.0, 447.9], dtype=np.float32)
    assert at.pow2_scale(a).tolist() == [1.0, 2.0, 0.5, 2.0 ** -8, 2.0 ** -22, 1.0]


def test_append_page_by_hand():
    D, P = 16, 16
    kc = np.zeros((2, 1, P, D), dtype=np.uint8)
    vc = kc.copy()
    ks = np.ones((2, 1), dtype=np.float32)
    vs = ks.copy()
    k = np.full((3, 1, D), 1.0, dtype=np.float32)
    v = np.full((3, 1, D), 3.0, dtype=np.float32)
    table = np.array([[1, 0]], dtype=np.int32)
    kc, vc, ks, vs, *_ = at.kv_append_fp8(k, v, kc, vc, ks, vs, table, [0, 3], [0])
    assert ks[1, 0] == 2.0 ** -8 and vs[1, 0] == 2.0 ** -7 and ks[0, 0] == 1.0
    assert np.all(e4m3_decode(kc[1, 0, :3]) == 256.0) and np.all(kc[1, 0, 3:] == 0)
    # sixteen times larger: the scale grows by 16, the old codes shrink by it
    k2 = np.full((1, 1, D), 16.0, dtype=np.float32)
    k2[0, 0, 3] = np.inf
    kc, vc, ks, vs, kn, vn = at.kv_append_fp8(k2, v[:1], kc, vc, ks, vs, table, [0, 1], [3])
    assert ks[1, 0] == 2.0 ** -4
    assert np.all(e4m3_decode(kc[1, 0, :3]) == 16.0) and e4m3_decode(kc[1, 0, 3, 0]) == 256.0
    assert kn[1, 0, 3].nonzero()[0].tolist() == [3] and not vn.any()
    # smaller values keep the page's scale; a run over the page's end starts the next page
    kc, vc, ks, vs, *_ = at.kv_append_fp8(np.full((13, 1, D), 0.5, np.float32), np.ones((13, 1, D), np.float32), kc, vc,
                                          ks, vs, table, [0, 13], [4])
    assert ks[1, 0] == 2.0 ** -4 and np.all(e4m3_decode(kc[1, 0, 4:]) == 8.0)
    assert ks[0, 0] == 2.0 ** -9 and np.all(e4m3_decode(kc[0, 0, 0]) == 256.0)


def test_attention_against_lists():
    rng = np.random.default_rng(3)
    S, n, Hq, H, D, P = 3, 2, 4, 2, 16, 16
    kc = e4m3_encode(rng.normal(size=(7, H, P, D)) * 50)
    vc = e4m3_encode(rng.normal(size=(7, H, P, D)) * 50)
    ks = np.exp2(rng.integers(-6, -3, size=(7, H))).astype(np.float32)
    vs = np.exp2(rng.integers(-6, -3, size=(7, H))).astype(np.float32)
    q = rng.normal(size=(S, n, Hq, D))
    table = np.array([[0, 1, 2], [3, 4, 99], [5, 6, 0]], dtype=np.int32)
    lens = np.array([37, 20, 1])
    for window in (0, 9):
        out, lse, _, _ = at.paged_attention_fp8(q, kc, vc, ks, vs, table, lens, 0.25, window)
        for s in range(S):
            for i in range(n):
                pos = lens[s] - n + i
                for h in range(Hq):
                    num, den = np.zeros(D), 0.0
                    for t in range(pos + 1):
                        if window and t <= pos - window:
                            continue
                        pg = table[s, t // P]
                        kk = e4m3_decode(kc[pg, h // 2, t % P]) * ks[pg, h // 2]
                        vv = e4m3_decode(vc[pg, h // 2, t % P]) * vs[pg, h // 2]
                        e = np.exp(0.25 * float(kk @ q[s, i, h]))
                        num, den = num + e * vv, den + e
                    if den == 0:
                        assert np.all(out[s, i, h] == 0) and lse[s, i, h] == -np.inf
                    else:
                        assert np.allclose(out[s, i, h], num / den, atol=1e-12)
                        assert abs(lse[s, i, h] - np.log(den)) < 1e-12
