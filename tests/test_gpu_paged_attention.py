"""GPU parity of the attention over the paged FP8 cache (oracle/attention.py).

Bound, derived from the kernel's roundings (u = 2^-24).  A score is an FP32
sum of D exact products, off by at most (D + 8) u of scale sum |q| |k| =: dot
times; its exponent y = score log2 e + log2 sv and the exponential add a few u
of |y| + 32, |y| at most 1.5 dot + 24: every weight is off by a relative
  ew = 2 (D + 8) u dot + 16 u (1.5 dot + 56),
and by 2^-11 for its rounding to FP16 (2^-38 of the largest weight, below
FP16's normal range).  Both the sum and the quotient are off by that, so
  |o - ref| <= 2^-8 |ref| + (2^-11 + 2 ew + T 2^-38) sum p |v|,
  |lse - ref| <= ew + 4 u (|ref| + 32)."""

import numpy as np
import pytest

from moe_grouped_gemm_x128_amd import synth
from oracle import attention as at
from oracle import bf16_decode, e4m3_encode

from helpers import say, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TINY = 1e-30


def _mg():
    import moe_grouped_gemm_x128_amd as mg

    return mg


def _case(seed, S, n, Hq, H, D, P, lens, layout="hpd", spare=2, sharp=1.0):
    rng = np.random.default_rng(seed)
    need = [max(1, -(-max(0, ln) // P)) for ln in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = rng.integers(-5, pages + 5, size=(S, max(need))).astype(np.int32)  # past the end: anything
    o = 0
    for i, w in enumerate(need):
        table[i, :w] = order[o:o + w]
        o += w
    c = dict(lens=np.array(lens, dtype=np.int32), table=table)
    for x in "kv":
        codes = e4m3_encode(rng.normal(size=(pages, H, P, D)) * 70)
        for i, ln in enumerate(lens):  # slots past the end: NaN codes
            w = max(0, ln)
            if w % P or w == 0:
                codes[table[i, w // P if w else 0], :, w % P:] = 0x7F
        codes[order[o:]] = 0xFF  # pages of no sequence
        c[x + "c"] = codes
        c[x + "s"] = np.exp2(rng.integers(-8, -4, size=(pages, H))).astype(np.float32)
        c[x + "s"][order[o:]] = 0.0
    bits = synth.bf16_bits_from_f32((rng.normal(size=(S, n, Hq, D)) * sharp).astype(np.float32))
    c["q"] = bf16_decode(bits)
    c["dq"] = to_dev(bits.view(np.int16)).view(torch.bfloat16)
    if layout == "kv":
        pool = to_dev(np.stack([c["kc"], c["vc"]], axis=1))
        c["dev"] = [pool[:, 0], pool[:, 1], to_dev(c["ks"].T).t(), to_dev(c["vs"].T).t()]
    elif layout == "phd":
        c["dev"] = [to_dev(c[x].transpose(0, 2, 1, 3)).transpose(1, 2) for x in ("kc", "vc")] + \
            [to_dev(c["ks"]), to_dev(c["vs"])]
    else:
        c["dev"] = [to_dev(c[x]) for x in ("kc", "vc", "ks", "vs")]
    return c


def _workspace(S, n, Hq, H, D, cap):
    need = _mg().paged_attention_fp8_workspace(S, n, Hq, H, D, cap)
    if need == 0:
        return None
    return torch.full(((need + 3) // 4,), float("nan"), dtype=torch.float32, device="cuda")


def _run(c, scale, window=0, lse=True, pad=0):
    S, n, Hq, D = c["q"].shape
    _, H, P, _ = c["kc"].shape
    out = torch.full((S, n, Hq, D + pad), 9.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((S, n, Hq), 9.0, dtype=torch.float32, device="cuda") if lse else None
    ws = _workspace(S, n, Hq, H, D, c["table"].shape[1] * P)
    _mg().paged_attention_fp8(c["dq"], *c["dev"], to_dev(c["table"]), to_dev(c["lens"]), out[..., :D], scale,
                              workspace=ws, lse=l, window=window)
    torch.cuda.synchronize()
    assert torch.all(out[..., D:] == 9.0)
    return out[..., :D].float().cpu().numpy().astype(np.float64), None if l is None else l.cpu().numpy().astype(np.float64)


def _compare(c, out, lse, scale, window, what):
    ref, rl, mass, dot = at.paged_attention_fp8(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["lens"],
                                                scale, window)
    D, T = ref.shape[3], max(1, int(c["lens"].max()))
    ew = 2 * (D + 8) * U * dot + 16 * U * (1.5 * dot + 56)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * ew[..., None] + T * 2.0 ** -38) * mass + TINY
    assert np.all(np.isfinite(out)), f"{what}: non-finite output"
    err = np.abs(out - ref)
    say(f"  {what}: largest error / bound = {np.max(err / bound):.3g}")
    assert np.all(err <= bound), f"{what}: {np.sum(err > bound)} outside, worst {np.max(err / bound)}"
    if lse is not None:
        empty = rl == -np.inf
        assert np.array_equal(lse == -np.inf, empty), f"{what}: empty rows"
        e = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, rl))
        assert np.all(e <= ew + 4 * U * (np.where(empty, 0.0, np.abs(rl)) + 32)), f"{what}: lse off by {e.max()}"


@pytest.mark.parametrize("S,n,Hq,H,D,P,lens,window,layout", [
    (1, 1, 8, 2, 128, 64, [777], 0, "hpd"),
    (5, 1, 8, 1, 128, 16, [0, 1, 15, 16, 17], 0, "phd"),            # lengths of zero and one, ends inside a tile
    (4, 1, 32, 2, 64, 32, [31, 32, 33, 1000], 0, "kv"),             # sixteen rows a head
    (3, 1, 5, 1, 256, 128, [127, 129, 640], 0, "hpd"),
    (2, 1, 3, 3, 128, 64, [300, 65], 0, "phd"),                     # one row a head
    (3, 4, 10, 2, 128, 32, [3, 70, 401], 0, "hpd"),                 # drafted tokens, more of them than the sequence holds
    (2, 3, 4, 2, 64, 16, [200, 2], 7, "kv"),                        # a window smaller than a tile
    (2, 2, 16, 1, 128, 64, [500, 129], 100, "hpd"),
    (1, 9, 14, 2, 256, 64, [530], 130, "phd"),                      # 63 rows a head
    (2, 1, 40, 1, 64, 64, [90, 200], 1, "hpd"),                     # only itself; three row tiles
    (1, 40, 2, 1, 128, 16, [61], 0, "hpd"),                         # as many queries as a short prompt
])
def test_attention_matches_oracle(S, n, Hq, H, D, P, lens, window, layout):
    say(f"paged_attention_fp8 S={S} n={n} Hq={Hq} H={H} D={D} P={P} lens={lens} window={window} {layout}")
    c = _case(D + P + Hq, S, n, Hq, H, D, P, lens, layout)
    out, lse = _run(c, D ** -0.5, window, pad=8)
    _compare(c, out, lse, D ** -0.5, window, "attention")


@pytest.mark.parametrize("D,P,S,H,group,lens", [
    (128, 64, 2, 2, 4, [9000, 4097]),
    (64, 16, 1, 1, 8, [20011]),
    (256, 128, 3, 1, 2, [5000, 3, 6143]),
])
def test_long_caches(D, P, S, H, group, lens):
    """Lengths that are split over many workgroups and joined again."""
    say(f"paged_attention_fp8 long D={D} lens={lens}")
    c = _case(D, S, 1, H * group, H, D, P, lens)
    out, lse = _run(c, D ** -0.5)
    _compare(c, out, lse, D ** -0.5, 0, "long")


@pytest.mark.parametrize("D,P,S,n,H,group,window,lens", [
    (64, 16, 2, 6, 1, 20, 0, [4500, 77]),       # 120 rows: four row tiles a wave, two waves side by side
    (64, 64, 2, 1, 2, 30, 0, [5000, 4999]),     # two row tiles
    (128, 32, 2, 5, 1, 16, 1000, [6000, 1030]), # 80 rows, a window
    (128, 64, 1, 4, 2, 8, 0, [7001]),
    (128, 16, 1, 7, 1, 25, 0, [4300]),          # 175 rows: more than one workgroup's
    (256, 64, 2, 4, 1, 8, 0, [4400, 9]),
    (256, 16, 1, 3, 1, 33, 333, [5123]),        # 99 rows
])
def test_long_caches_with_many_rows(D, P, S, n, H, group, window, lens):
    say(f"paged_attention_fp8 long, many rows D={D} P={P} n={n} group={group} window={window} lens={lens}")
    c = _case(D + n, S, n, H * group, H, D, P, lens)
    out, lse = _run(c, D ** -0.5, window)
    _compare(c, out, lse, D ** -0.5, window, "long, many rows")


@pytest.mark.parametrize("D,P,S,n,H,group,window,lens", [
    (128, 64, 3, 1, 2, 4, 300, [9000, 8192, 299]),   # what a query sees fits the uncut form, the table does not
    (64, 16, 2, 4, 1, 8, 1500, [6001, 40]),          # cut
    (256, 32, 2, 2, 1, 4, 31, [4100, 4097]),         # the window's positions in two tiles
    (128, 16, 1, 1, 1, 8, 1 << 30, [4500]),          # a window longer than any cache
    (128, 64, 2, 9, 1, 4, 2**31 - 1, [4400, 2]),     # the largest window, queries from before the first position
])
def test_windows_in_long_caches(D, P, S, n, H, group, window, lens):
    say(f"paged_attention_fp8 windows D={D} P={P} n={n} group={group} window={window} lens={lens}")
    c = _case(D + n + group, S, n, H * group, H, D, P, lens)
    out, lse = _run(c, D ** -0.5, window)
    _compare(c, out, lse, D ** -0.5, window, "window")


def test_shares_of_whole_units():
    """Eighty sequences (more than a wave has lanes), few enough that every
    share is of one unit; some end in a short last share, some are empty."""
    say("paged_attention_fp8 80 sequences cut into whole shares")
    rng = np.random.default_rng(80)
    lens = [int(x) for x in rng.integers(0, 1800, 80)]
    lens[0], lens[1], lens[40], lens[79] = 0, 1, 2304, 2304
    c = _case(80, 80, 2, 4, 1, 64, 64, lens)
    out, lse = _run(c, 0.125)
    _compare(c, out, lse, 0.125, 0, "whole shares")


def test_more_sequences_than_threads():
    """Six hundred sequences, most of them short or empty, in a table wide
    enough for the work to be cut along the cache; and without a cut."""
    say("paged_attention_fp8 600 sequences")
    rng = np.random.default_rng(77)
    lens = [int(v) for v in rng.integers(0, 40, size=600)]
    lens[3], lens[255], lens[256], lens[511], lens[599] = 2500, 700, 0, 33, 900
    c = _case(81, 600, 1, 2, 1, 64, 16, lens)
    out, lse = _run(c, 0.125)
    _compare(c, out, lse, 0.125, 0, "600 sequences, not cut")
    wide = np.full((600, 300), -1, dtype=np.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide
    out, lse = _run(c, 0.125)
    _compare(c, out, lse, 0.125, 0, "600 sequences, cut")


def test_sharp_scores():
    """Scores of several hundred: one token takes all the weight, the
    running maximum moves along the cache."""
    say("paged_attention_fp8 sharp scores")
    c = _case(3, 2, 2, 8, 2, 128, 64, [700, 333], sharp=12.0)
    out, lse = _run(c, 0.25)
    _compare(c, out, lse, 0.25, 0, "sharp")
    c = _case(3, 2, 1, 8, 2, 128, 64, [700, 333])
    out, lse = _run(c, 0.0)  # every token the same weight
    _compare(c, out, lse, 0.0, 0, "flat")
    out, lse = _run(c, -0.1)
    _compare(c, out, lse, -0.1, 0, "negative scale")


def test_scales_far_apart():
    """V scales from 2^-22 to 2^20 page by page, K scales small enough that
    the pages' weights stay alike: the largest outputs hide nothing."""
    say("paged_attention_fp8 scales far apart")
    c = _case(21, 2, 1, 8, 2, 64, 16, [400, 100])
    rng = np.random.default_rng(2)
    c["ks"] = np.where(c["ks"] > 0, np.float32(2.0 ** -12), c["ks"]).astype(np.float32)
    c["vs"] = np.where(c["vs"] > 0, np.exp2(rng.integers(-22, 21, size=c["vs"].shape)), 0).astype(np.float32)
    c["dev"][2:] = [to_dev(c["ks"]), to_dev(c["vs"])]
    out, lse = _run(c, 0.1)
    _compare(c, out, lse, 0.1, 0, "scales")


@pytest.mark.parametrize("scale,lens,P", [(0.0, [70, 3, 0], 32), (0.0, [4000, 45, 1], 64), (-0.0, [40, 17, 2], 16)])
def test_a_scale_of_zero_weighs_all_alike(scale, lens, P):
    say(f"paged_attention_fp8 scale {scale} lens={lens} P={P}")
    c = _case(41, 3, 3, 4, 2, 64, P, lens)
    out, lse = _run(c, scale, 30)
    _compare(c, out, lse, scale, 30, "zero scale")
    seen = np.array([[min(30, max(0, ln - 3 + i + 1)) for i in range(3)] for ln in lens])[:, :, None]
    with np.errstate(divide="ignore"):
        want = np.broadcast_to(np.log(seen.astype(np.float64)), lse.shape)
    assert np.array_equal(np.isinf(lse), np.isinf(want))
    some = np.isfinite(want)
    assert np.all(np.abs(lse[some] - want[some]) <= 1e-5)


@pytest.mark.parametrize("D,P,lens", [(128, 64, [900, 31]), (256, 16, [200, 17]), (64, 32, [5000, 3000])])
def test_scales_that_are_no_powers_of_two(D, P, lens):
    say(f"paged_attention_fp8 odd scales D={D} P={P} lens={lens}")
    c = _case(51 + D, 2, 2, 8, 2, D, P, lens)
    rng = np.random.default_rng(5)
    for x in ("ks", "vs"):
        c[x] = (c[x] * rng.uniform(1.0, 2.0, size=c[x].shape)).astype(np.float32)
    c["dev"][2:] = [to_dev(c["ks"]), to_dev(c["vs"])]
    out, lse = _run(c, 0.09)
    _compare(c, out, lse, 0.09, 0, "odd scales")


def test_one_weight_above_all():
    """Queries so sharp that a row is one position, or a few: scores of
    hundreds, up and down."""
    say("paged_attention_fp8 sharp rows")
    for scale in (1.0, -1.0):
        c = _case(61, 2, 2, 8, 2, 128, 64, [700, 90], sharp=4.0)
        out, lse = _run(c, scale)
        _compare(c, out, lse, scale, 0, "sharp")


def test_nan_where_nothing_looks():
    """A NaN value at the newest position of a draft spoils only the queries
    that see it; before a window, none."""
    say("paged_attention_fp8 NaN in masked places")
    c = _case(31, 1, 3, 8, 2, 128, 32, [150])
    clean, lse = _run(c, 0.1, 100)
    _compare(c, clean, lse, 0.1, 100, "clean")
    page, slot = c["table"][0, 149 // 32], 149 % 32
    for x, dev in (("kc", 0), ("vc", 1)):
        d = dict(c, dev=list(c["dev"]))
        codes = c[x].copy()
        codes[page, :, slot] = 0x7F          # the last query's own position
        codes[c["table"][0, 40 // 32], :, 40 % 32] = 0x7F   # before every window (47 - ...)
        d["dev"][dev] = to_dev(codes)
        out, l = _run(d, 0.1, 100)
        assert np.array_equal(out[0, :2], clean[0, :2]) and np.array_equal(l[0, :2], lse[0, :2])
        assert np.all(np.isnan(out[0, 2]))
        assert np.all(np.isnan(l[0, 2])) == (x == "kc")


def test_pages_outside_the_pool_take_no_part():
    say("paged_attention_fp8 pages outside the pool, lengths past the table")
    c = _case(41, 3, 1, 4, 2, 64, 16, [100, 60, 64])
    c["table"][0, 2] = -1
    c["table"][0, 5] = 10 ** 6
    c["table"][1, :] = -7
    c["lens"][2] = 10 ** 6   # cut to the table's length: pages past its own are whatever the table says
    c["table"][2, 4:] = -1
    out, lse = _run(c, 0.125)
    ref = dict(c, lens=np.array([100, 60, c["table"].shape[1] * 16], dtype=np.int32))
    _compare(ref, out, lse, 0.125, 0, "absent pages")
    c["lens"][:] = [-5, 0, 1]
    out, lse = _run(c, 0.125)
    assert np.all(out[:2] == 0) and np.all(lse[:2] == -np.inf) and np.all(np.isfinite(lse[2]))


def test_repeats_are_equal_and_graph_replays():
    say("paged_attention_fp8 repeats, other stream, graph replays")
    mg = _mg()
    S, n, Hq, H, D, P = 3, 1, 16, 2, 128, 64
    c = _case(51, S, n, Hq, H, D, P, [5000, 70, 1999])
    table, lens = to_dev(c["table"]), to_dev(c["lens"])
    ws = _workspace(S, n, Hq, H, D, c["table"].shape[1] * P)
    out = torch.empty(S, n, Hq, D, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        mg.paged_attention_fp8(c["dq"], *c["dev"], table, lens, out, 0.1, workspace=ws, stream=stream)

    call()
    torch.cuda.synchronize()
    first = out.clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        call(side)
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([4999, 0, 1998], [1, 64, 1999], [5000, 70, 1999]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
    assert torch.equal(out, first)


def test_strided_queries():
    say("paged_attention_fp8 strided queries")
    S, Hq, H, D, P = 2, 4, 2, 64, 16
    c = _case(61, S, 1, Hq, H, D, P, [33, 70])
    wide = torch.zeros(S, 1, Hq + 3, D + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1:1 + Hq, :D] = c["dq"]
    c["dq"] = wide[:, :, 1:1 + Hq, :D]
    out, lse = _run(c, 0.2)
    _compare(c, out, lse, 0.2, 0, "strided")


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB, its pages used from both ends."""
    say("paged_attention_fp8 with a pool of over 4 GiB")
    mg = _mg()
    D, P, H, Hq = 256, 128, 8, 16
    pages = (1 << 32) // (P * H * D) + 40
    kc = torch.zeros(pages, H, P, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(pages, H, P, D, dtype=torch.uint8, device="cuda")
    sc = torch.full((pages, H), 2.0 ** -6, device="cuda")
    cs = to_dev(np.concatenate([np.ones((600, 8)), np.zeros((600, 8))], axis=1).astype(np.float32))
    table = torch.tensor([[pages - 1, 0, pages - 2, 1]], dtype=torch.int32, device="cuda")
    x = torch.randn(400, H, D, device="cuda")
    cu, start = torch.tensor([0, 400], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ks, vs = sc.clone(), sc.clone()
    mg.kv_append_fp8(x, x, kc, vc, ks, vs, table, cu, start, cos_sin=cs)
    q = torch.randn(1, 1, Hq, D, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = _workspace(1, 1, Hq, H, D, 4 * P)
    mg.paged_attention_fp8(q, kc, vc, ks, vs, table, start + 400, out, 0.0625, workspace=ws)
    torch.cuda.synchronize()
    small = [pages - 1, 0, pages - 2, 1]
    host = dict(q=q.float().cpu().numpy().astype(np.float64), kc=kc[small].cpu().numpy(), vc=vc[small].cpu().numpy(),
                ks=ks[small].cpu().numpy(), vs=vs[small].cpu().numpy(), lens=np.array([400]),
                table=np.arange(4, dtype=np.int32)[None])
    _compare(host, out.float().cpu().numpy().astype(np.float64), None, 0.0625, 0, "4 GiB")


def test_empty_calls():
    mg = _mg()
    c = _case(71, 1, 1, 2, 1, 64, 16, [5])
    dev = c["dev"]
    mg.paged_attention_fp8(c["dq"][:0], *dev, to_dev(c["table"])[:0], to_dev(c["lens"])[:0],
                           torch.empty_like(c["dq"])[:0], 1.0)
    out = torch.full_like(c["dq"], 5.0)
    none = [t[:0] for t in dev]
    ws = _workspace(1, 1, 2, 1, 64, 16)
    mg.paged_attention_fp8(c["dq"], *none, to_dev(c["table"]), to_dev(c["lens"]), out, 1.0, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(out == 0)
    out.fill_(5.0)
    mg.paged_attention_fp8(c["dq"], *dev, to_dev(c["table"])[:, :0], to_dev(c["lens"]), out, 1.0)
    torch.cuda.synchronize()
    assert torch.all(out == 0)
