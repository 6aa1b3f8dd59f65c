"""GPU parity of the append to the paged FP8 cache (oracle/attention.py).

Codes and scales are compared bit for bit: the definition rounds every product
and sum of the rotation to FP32, the scale is a power of two and the quotient
is correctly rounded.  Slots, pages and scales that no token goes to must stay
as they were.  q_out is within BF16's rounding of the FP32 rotation: 2^-8 |y|
+ 2 u (|x cos| + |y sin|) of the float64 one."""

import numpy as np
import pytest

from moe_grouped_gemm_x128_amd import synth
from oracle import attention as at
from oracle import bf16_decode, e4m3_encode

from helpers import say, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


def _mg():
    import moe_grouped_gemm_x128_amd as mg

    return mg


def _table(positions, rot, theta=10000.0):
    ang = np.arange(positions)[:, None] * theta ** (-np.arange(0, rot, 2) / rot)[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def _values(rng, shape, bf16):
    x = (rng.normal(size=shape) * np.exp2(rng.integers(-2, 3, size=shape[:2] + (1,)))).astype(np.float32)
    if not bf16:
        return to_dev(x), x
    bits = synth.bf16_bits_from_f32(x)
    return to_dev(bits.view(np.int16)).view(torch.bfloat16), bf16_decode(bits).astype(np.float32)


class Pool:
    """Caches on host and device; layout "hpd": [pages, H, P, D] as stored,
    "phd": token by token, "kv": K and V halves of one pool."""

    def __init__(self, rng, pages, H, P, D, layout="hpd"):
        self.kc, self.vc = (e4m3_encode(rng.normal(size=(pages, H, P, D)) * 60) for _ in range(2))
        self.ks, self.vs = (np.exp2(rng.integers(-9, -5, size=(pages, H))).astype(np.float32) for _ in range(2))
        if layout == "kv":
            pool = to_dev(np.stack([self.kc, self.vc], axis=1))
            self.dkc, self.dvc = pool[:, 0], pool[:, 1]
            sc = to_dev(np.stack([self.ks, self.vs], axis=2))
            self.dks, self.dvs = sc[:, :, 0], sc[:, :, 1]
        elif layout == "phd":
            self.dkc, self.dvc = (to_dev(c.transpose(0, 2, 1, 3)).transpose(1, 2) for c in (self.kc, self.vc))
            self.dks, self.dvs = (to_dev(c.T).t() for c in (self.ks, self.vs))
        else:
            self.dkc, self.dvc, self.dks, self.dvs = (to_dev(c) for c in (self.kc, self.vc, self.ks, self.vs))

    def append(self, dk, dv, k, v, table, cu, start, cs, inter, q=None, q_out=None):
        want = at.kv_append_fp8(k, v, self.kc, self.vc, self.ks, self.vs, table, cu, start, cs, inter)
        _mg().kv_append_fp8(dk, dv, self.dkc, self.dvc, self.dks, self.dvs, to_dev(table),
                            to_dev(np.array(cu, np.int32)), to_dev(np.array(start, np.int32)),
                            cos_sin=None if cs is None else to_dev(cs), q=q, q_out=q_out, interleaved=inter)
        torch.cuda.synchronize()
        kc, vc, ks, vs, kn, vn = want
        for name, got, ref, nan in (("k", self.dkc, kc, kn), ("v", self.dvc, vc, vn)):
            got = got.cpu().numpy()
            assert np.all((got[nan] & 0x7F) == 0x7F), f"{name}: NaN codes"
            bad = (got != ref) & ~nan & ~(((got & 0x7F) == 0x7F) & ((ref & 0x7F) == 0x7F))
            assert not bad.any(), f"{name}: {bad.sum()} codes differ, first at {np.argwhere(bad)[:3].tolist()}"
        assert np.array_equal(self.dks.cpu().numpy(), ks) and np.array_equal(self.dvs.cpu().numpy(), vs), "scales"
        self.kc, self.vc, self.ks, self.vs = self.dkc.cpu().numpy(), self.dvc.cpu().numpy(), ks, vs


def _pages(rng, starts, news, P, spare=2):
    need = [max(1, -(-(a + n) // P)) for a, n in zip(starts, news)]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(need), max(need)), -1, dtype=np.int32)
    o = 0
    for i, w in enumerate(need):
        table[i, :w] = order[o:o + w]
        o += w
    return table, sum(need) + spare


@pytest.mark.parametrize("D,P,H,Hq,rot,inter,bf16,layout,starts,news", [
    (128, 64, 2, 8, 128, False, True, "hpd", [0, 63, 64, 130], [1, 1, 1, 1]),        # single tokens
    (128, 64, 2, 4, 128, False, True, "phd", [0, 10, 100, 5, 7], [200, 54, 0, 1, 129]),  # ragged prompts
    (64, 16, 1, 3, 32, True, True, "kv", [3, 0, 15, 16], [40, 1, 2, 16]),
    (256, 32, 3, 3, 96, False, False, "hpd", [31, 32, 0], [33, 31, 70]),
    (64, 128, 2, 2, 64, True, False, "phd", [127, 5], [2, 300]),
    (128, 16, 1, 1, 16, False, True, "hpd", [9], [1]),
    (256, 128, 1, 2, 256, True, True, "kv", [1, 120, 0], [3, 20, 129]),
    (128, 32, 4, 5, 64, False, False, "hpd", list(range(0, 300)), [1] * 300),          # more sequences than threads
])
def test_append_matches_oracle(D, P, H, Hq, rot, inter, bf16, layout, starts, news):
    say(f"kv_append_fp8 D={D} P={P} H={H} rot={rot} inter={inter} bf16={bf16} {layout} S={len(starts)} T={sum(news)}")
    rng = np.random.default_rng(D + P + H)
    table, pages = _pages(rng, starts, news, P)
    pool = Pool(rng, pages, H, P, D, layout)
    cu = np.concatenate([[0], np.cumsum(news)])
    T = int(cu[-1])
    dk, k = _values(rng, (T, H, D), bf16)
    dv, v = _values(rng, (T, H, D), bf16)
    dq, q = _values(rng, (T, Hq, D), bf16)
    cs = _table(max(a + n for a, n in zip(starts, news)), rot)
    q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool.append(dk, dv, k, v, table, cu, starts, cs, inter, dq, q_out)
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(starts, news)]).astype(np.int64)
    rows = cs[pos].astype(np.float64)
    ref = at.rotate(q, rows[:, :rot // 2], rows[:, rot // 2:], inter)
    mag = at.rotate(np.abs(q), np.abs(rows[:, :rot // 2]), np.abs(rows[:, rot // 2:]), inter)  # second of each pair
    neg = at.rotate(np.abs(q), np.abs(rows[:, :rot // 2]), -np.abs(rows[:, rot // 2:]), inter)  # first of each pair
    err = np.abs(q_out.float().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2 * U * np.maximum(np.abs(mag), np.abs(neg)) + 1e-38)
    # the same tokens once more one position on: pages in use, scales kept or grown
    starts2 = [a + n for a, n in zip(starts, news)]
    news2 = [1 if (a % P) and a < table.shape[1] * P else 0 for a in starts2]
    if sum(news2):
        cu2 = np.concatenate([[0], np.cumsum(news2)])
        dk2, k2 = _values(rng, (sum(news2), H, D), bf16)
        dv2, v2 = _values(rng, (sum(news2), H, D), bf16)
        pool.append(dk2 * 32, dv2, k2 * 32, v2, table, cu2, starts2, _table(max(starts2) + 1, rot), inter)


def test_token_by_token_equals_the_definition():
    """Forty single appends to one page, values growing and shrinking."""
    say("kv_append_fp8 token by token")
    rng = np.random.default_rng(6)
    D, P, H = 64, 64, 2
    table = np.array([[1, 0]], dtype=np.int32)
    pool = Pool(rng, 3, H, P, D)
    cs = _table(80, D)
    for t in range(40):
        x = (rng.normal(size=(1, H, D)) * 2.0 ** rng.integers(-12, 12)).astype(np.float32)
        v = (rng.normal(size=(1, H, D)) * 2.0 ** (t - 20)).astype(np.float32)
        pool.append(to_dev(x), to_dev(v), x, v, table, [0, 1], [t], cs, False)


def test_values_that_are_not_finite_and_zeros():
    say("kv_append_fp8 NaN, infinities, zeros, subnormals")
    rng = np.random.default_rng(7)
    D, P, H = 128, 16, 1
    table = np.array([[2, 0, 1]], dtype=np.int32)
    pool = Pool(rng, 4, H, P, D)
    k = rng.normal(size=(40, H, D)).astype(np.float32)
    v = rng.normal(size=(40, H, D)).astype(np.float32)
    k[3, 0, 5], v[4, 0, 6], v[5, 0, 7] = np.nan, np.inf, -np.inf
    k[16:32] = 0.0
    v[16:32] = -0.0
    k[33], v[34] = 1e-42, np.nan
    v[0, 0, 0] = 3e38
    pool.append(to_dev(k), to_dev(v), k, v, table, [0, 40], [0], None, False)


def test_dropped_tokens_touch_nothing():
    """Positions past the block table or the rotation's rows, pages outside
    the pool, negative starts, tokens past the last sequence."""
    say("kv_append_fp8 dropped tokens")
    rng = np.random.default_rng(8)
    D, P, H, Hq = 64, 16, 2, 2
    table = np.array([[0, 99], [-1, 1], [2, 3], [4, 5]], dtype=np.int32)
    starts, news = [10, 12, 30, 3], [10, 8, 9, 4]  # seq 2 runs past its 32 positions
    cu = np.concatenate([[0], np.cumsum(news)])
    T = int(cu[-1]) + 3  # three tokens of no sequence
    pool = Pool(rng, 6, H, P, D)
    x = rng.normal(size=(T, H, D)).astype(np.float32)
    q = torch.randn(T, Hq, D, device="cuda")
    q_out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    cs = _table(19, 32)
    pool.append(to_dev(x), to_dev(x), x, x, table, cu, starts, cs, True, q, q_out)
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(starts, news)])
    kept = torch.all((q_out == 3.0).flatten(1), dim=1).cpu().numpy()
    assert np.array_equal(kept[:len(pos)], pos >= 19) and kept[len(pos):].all()
    pool.append(to_dev(x), to_dev(x), x, x, table, cu, [-3, -100, 0, 0], cs, True)


def test_strided_inputs_and_graph():
    """k and v as views of one packed projection; captured and replayed."""
    say("kv_append_fp8 strided inputs, graph replays")
    mg = _mg()
    rng = np.random.default_rng(9)
    D, P, H, Hq, S = 128, 32, 2, 4, 3
    qkv = torch.randn(S, Hq + 2 * H, D, device="cuda", dtype=torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    table = to_dev(np.array([[0, 1], [2, 3], [4, 5]], dtype=np.int32))
    start = torch.tensor([0, 5, 30], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    cs = to_dev(_table(64, D))
    pool = Pool(rng, 6, H, P, D, "kv")
    q_out = torch.empty(S, Hq, D, dtype=torch.bfloat16, device="cuda")

    def call():
        mg.kv_append_fp8(k, v, pool.dkc, pool.dvc, pool.dks, pool.dvs, table, cu, start, cos_sin=cs, q=q, q_out=q_out)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(4):
        qkv.copy_(torch.randn_like(qkv) * (1 + step))
        kf, vf = k.float().cpu().numpy(), v.float().cpu().numpy()
        want = at.kv_append_fp8(kf, vf, pool.kc, pool.vc, pool.ks, pool.vs, table.cpu().numpy(), [0, 1, 2, 3],
                                start.cpu().numpy(), cs.cpu().numpy(), False)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((pool.dkc, pool.dvc, pool.dks, pool.dvs), want):
            assert np.array_equal(got.cpu().numpy(), ref)
        pool.kc, pool.vc, pool.ks, pool.vs = want[:4]
        start += 1


def test_empty_calls():
    mg = _mg()
    pool = Pool(np.random.default_rng(1), 2, 1, 16, 64)
    none = torch.empty(0, 1, 64, device="cuda")
    cu, start = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    mg.kv_append_fp8(none, none, pool.dkc, pool.dvc, pool.dks, pool.dvs, table, cu, start)
    mg.kv_append_fp8(none, none, pool.dkc, pool.dvc, pool.dks, pool.dvs, table[:0], cu[:1], start[:0])
    one = torch.ones(1, 1, 64, device="cuda")
    mg.kv_append_fp8(one, one, pool.dkc, pool.dvc, pool.dks, pool.dvs, table[:, :0], torch.tensor(
        [0, 1], dtype=torch.int32, device="cuda"), start)
    torch.cuda.synchronize()
    assert np.array_equal(pool.dkc.cpu().numpy(), pool.kc) and np.array_equal(pool.dks.cpu().numpy(), pool.ks)
