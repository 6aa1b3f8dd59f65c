"""GPU parity of the BF16 products of ragged groups (oracle/layer.py).

Products of BF16 values are exact in FP32; the matrix core truncates within groups
of 8 to at most 7 u of the largest product and the sums round once an addition:
an output is off by at most (n + 2) u S, n the length of the contraction, S the
sum of the absolute terms (c included) and u = 2^-24; a BF16 output by half a step
more, 2^-8 of itself."""

import numpy as np
import pytest

from oracle import layer

from helpers import say
from test_gpu_norm import BF, F32, HALF, U, _close, _gen, _np, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import moe_grouped_gemm_x128_amd as mg  # noqa: E402

NAN = float("nan")


def _offsets(sizes, first=0):
    return torch.tensor(np.cumsum([first] + list(sizes)), dtype=torch.int32, device="cuda")


def _case(form, sizes, N, K, dt, ct, first=0, behind=0, pad=0, seed=0):
    """One call against the oracle: rows before and behind the groups hold NaN
    and stay as they are, strides are wider than the rows by `pad`."""
    gen = _gen(seed + 17 * N + K)
    G, M = len(sizes), first + sum(sizes) + behind
    off = _offsets(sizes, first)
    rows = slice(first, first + sum(sizes))

    def held(shape):
        width = -(-shape[-1] // 8) * 8 + pad
        wide = torch.full((*shape[:-1], width), NAN, dtype=BF, device="cuda")
        wide[..., :shape[-1]] = _rows(gen, shape, BF)
        return wide[..., :shape[-1]]

    a = held((M, N) if form == "tn" else (M, K))
    b = held((G, N, K) if form == "nt" else (G, K, N) if form == "nn" else (M, K))
    for t in (a, b) if form == "tn" else (a,):
        t[:first] = NAN
        t[first + sum(sizes):] = NAN
    shape = (G, N, K) if form == "tn" else (M, N)
    wide = torch.full((*shape[:-1], shape[-1] + 3), 77.0, dtype=dt, device="cuda")
    d = wide[..., :shape[-1]]
    c = None
    if ct == "in place":
        c = d
        d.copy_(_rows(gen, shape, dt))
    elif ct is not None:
        c = _rows(gen, shape, ct, 1.0, 5)
    cn = None if c is None else _np(c)
    start = wide.clone()
    call = {"nt": mg.m_grouped_bf16_gemm_nt_ragged, "nn": mg.m_grouped_bf16_gemm_nn_ragged,
            "tn": mg.k_grouped_bf16_gemm_tn}[form]
    what = f"{form} groups {sizes if G < 9 else G} N={N} K={K} {dt} c {ct}"
    say(what)
    assert call(a, b, d, off, c=c) is d
    torch.cuda.synchronize()
    an, bn = np.nan_to_num(_np(a)), np.nan_to_num(_np(b))
    ref = {"nt": layer.ragged_nt, "nn": layer.ragged_nn, "tn": layer.ragged_tn}[form]
    o = off.cpu().numpy()
    want, size = ref(an, bn, o, cn), ref(np.abs(an), np.abs(bn), o, None if cn is None else np.abs(cn))
    assert torch.equal(wide[..., shape[-1]:], start[..., shape[-1]:]), "the stride's rest was written"
    if form == "tn":
        n = max(sizes)
    else:
        n, (want, done), (size, _) = K, want, size
        assert torch.equal(d[~torch.from_numpy(done).cuda()], start[..., :N][~torch.from_numpy(done).cuda()])
        d, want, size = d[rows], want[rows], size[rows]
    _close(d, want, (n + 2) * U * size * (1 + 1e-6) + HALF[dt] * np.abs(want) + 1e-37, what)


SIZES = [[1], [0], [5, 0, 1, 300, 0], [256, 256], [257, 255, 1], [0, 0, 64], [33] * 9, [700]]


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N,K", [(8, 64), (257, 192), (40, 320), (520, 128)])
def test_groups(form, sizes, N, K):
    _case(form, sizes, N, K, BF, None, first=3, behind=5)
    _case(form, sizes, N, K, F32, F32, pad=8)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("dt,ct", [(BF, BF), (BF, F32), (F32, BF), (F32, "in place"), (BF, "in place")])
def test_accumulate(form, dt, ct):
    _case(form, [65, 0, 130, 2], 136, 448, dt, ct, first=1, behind=2)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes,N,K", [
    ([0, 1] * 40, 64, 64),                       # more groups than a wave has lanes, half of them empty
    ([3] * 200, 72, 128),
    ([1] + [0] * 300 + [2], 16, 64),
    ([512, 1, 1023, 256], 300, 704),             # several tiles a group, odd slices
    ([2047], 264, 1024),
    ([64, 65, 128], 256, 4096),                  # rows a multiple of 4 KB apart: slices taken in turns
    ([90, 10, 300], 1, 64),                      # one column
    ([100, 29], 64, 2048),
])
def test_shapes(form, sizes, N, K):
    if form == "nn" or form == "tn":
        N = -(-N // 8) * 8
    _case(form, sizes, N, K, BF, None)


def test_weight_gradient_of_odd_sizes():
    for sizes, N, K in (([1, 2, 3], 1, 1), ([63, 64, 65], 31, 33), ([129], 257, 5), ([0], 7, 9), ([500, 3], 255, 129)):
        _case("tn", sizes, N, K, F32, None, first=2, behind=1)


@pytest.mark.parametrize("K", [0, 64, 128, 192, 256, 320])
def test_few_slices(K):
    """Every phase of the pipeline over the contraction, no slice among them."""
    for form in ("nt", "nn"):
        _case(form, [5, 260], 264, K, F32, F32 if K == 0 else None)


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("sizes,N,K", [
    ([1500, 3, 0, 1200, 129, 257, 2000], 4104, 128),   # more tiles than compute units: several a workgroup
    ([4096], 4096, 64),                                # one slice, whole tiles
    ([70] * 50 + [700], 3008, 192),                    # an odd number of slices, last tiles of every fill
])
def test_large_tiles(form, sizes, N, K):
    _case(form, sizes, N, K, BF, None, first=2, behind=3)
    _case(form, sizes, N, K, F32, BF)


@pytest.mark.parametrize("sizes,N,K", [([40, 0, 200, 1, 64, 129], 2048, 2040), ([300, 65, 3, 10], 2056, 2048)])
def test_large_tiles_of_weight_gradients(sizes, N, K):
    _case("tn", sizes, N, K, F32, None, first=1)
    _case("tn", sizes, N, K, BF, F32, behind=2)


@pytest.mark.parametrize("ct", [F32, BF])
@pytest.mark.parametrize("sizes,N,K", [([40, 0, 200, 1, 64, 129], 2048, 2048), ([5, 70, 0, 1], 256, 384)])
def test_weight_gradients_added_up(sizes, N, K, ct):
    """Whole aligned rows: FP32 sums in place, and a BF16 C beside an FP32 D."""
    say(f"tn groups {sizes} N={N} K={K} added to {ct}")
    gen = _gen(N + K)
    off = _offsets(sizes)
    a, b = _rows(gen, (sum(sizes), N), BF), _rows(gen, (sum(sizes), K), BF)
    c = _rows(gen, (len(sizes), N, K), ct, 4.0)
    d = c if ct == F32 else torch.empty(len(sizes), N, K, device="cuda")
    cn = _np(c)
    mg.k_grouped_bf16_gemm_tn(a, b, d, off, c=c)
    o = off.cpu().numpy()
    want, size = layer.ragged_tn(_np(a), _np(b), o, cn), layer.ragged_tn(np.abs(_np(a)), np.abs(_np(b)), o, np.abs(cn))
    _close(d, want, (max(sizes) + 2) * U * size * (1 + 1e-6), "d")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes", [[900, 500, 0, 1100], [130] * 30])
def test_medium_tiles(form, sizes):
    _case(form, sizes, 1032, 576, BF, None, first=1, behind=1)
    _case(form, sizes, 1032, 512, F32, "in place")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_strides_of_a_single_row(form):
    """The stride of a dimension of one is of no account; weights may be shared by all groups."""
    say(f"{form} of one row, and of one matrix for all groups")
    gen = _gen(31)
    G, N, K = 3, 72, 128
    call, ref = {"nt": (mg.m_grouped_bf16_gemm_nt_ragged, layer.ragged_nt), "nn": (mg.m_grouped_bf16_gemm_nn_ragged, layer.ragged_nn),
                 "tn": (mg.k_grouped_bf16_gemm_tn, layer.ragged_tn)}[form]
    off = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda")
    for stride in (0, 8, 1 << 40):
        a = _rows(gen, (N if form == "tn" else K,), BF).as_strided((1, N if form == "tn" else K), (stride, 1))
        if form == "tn":
            b = _rows(gen, (K,), BF).as_strided((1, K), (stride, 1))
            d = torch.empty(G, N, K, device="cuda")
        else:
            b = _rows(gen, (1, N, K) if form == "nt" else (1, K, N), BF).expand(G, -1, -1)
            d = torch.empty(1, N, device="cuda")
        call(a, b, d, off)
        o = off.cpu().numpy()
        want, size = ref(_np(a), _np(b), o, None), ref(np.abs(_np(a)), np.abs(_np(b)), o, None)
        if form != "tn":
            want, size = want[0], size[0]
        _close(d, want, ((1 if form == "tn" else K) + 2) * U * size * (1 + 1e-6) + 1e-37, f"stride {stride}")
    if form == "nt":  # one output column
        b = _rows(gen, (G, 1, K), BF).as_strided((G, 1, K), (K, 8, 1))
        d = torch.empty(1, 1, device="cuda")
        call(a, b, d, off)
        want, size = ref(_np(a), _np(b), o, None)[0], ref(np.abs(_np(a)), np.abs(_np(b)), o, None)[0]
        _close(d, want, (K + 2) * U * size * (1 + 1e-6) + 1e-37, "one column")


def test_offsets_out_of_range():
    say("offsets past the rows, negative, falling")
    gen = _gen(1)
    G, M, N, K = 4, 50, 64, 128
    a, b = _rows(gen, (M, K), BF), _rows(gen, (G, N, K), BF)
    for off in ([-5, 10, 10, 60, 70], [20, 20, 20, 20, 20], [60, 70, 80, 90, 100], [-9, -8, -7, -6, 50]):
        d = torch.full((M, N), 7.0, device="cuda")
        mg.m_grouped_bf16_gemm_nt_ragged(a, b, d, torch.tensor(off, dtype=torch.int32, device="cuda"))
        want, done = layer.ragged_nt(_np(a), _np(b), off)
        assert torch.equal(d[torch.from_numpy(~done).cuda()], torch.full_like(d, 7.0)[torch.from_numpy(~done).cuda()])
        if done.any():
            size, _ = layer.ragged_nt(np.abs(_np(a)), np.abs(_np(b)), off)
            _close(d[torch.from_numpy(done).cuda()], want[done], (K + 2) * U * size[done], str(off))
    # falling: unspecified rows, and nothing outside d
    room = torch.full((M + 600, N), 7.0, device="cuda")
    mg.m_grouped_bf16_gemm_nt_ragged(a, b, room[300:300 + M], torch.tensor([0, 40, 10, 50, 5], dtype=torch.int32, device="cuda"))
    assert (room[:300] == 7).all() and (room[300 + M:] == 7).all()


def test_what_is_not_finite_stays_in_its_group():
    say("NaN and infinities in one group's rows and weights")
    gen = _gen(2)
    sizes, N, K = [10, 70, 33], 96, 128
    off = _offsets(sizes)
    a, b = _rows(gen, (113, K), BF), _rows(gen, (3, N, K), BF)
    t = _rows(gen, (113, 64), BF)
    d, e, w = (torch.zeros(s, device="cuda") for s in ((113, N), (113, N), (3, K, 64)))
    mg.m_grouped_bf16_gemm_nt_ragged(a, b, d, off)
    mg.k_grouped_bf16_gemm_tn(a, t, w, off)
    a2, b2 = a.clone(), b.clone()
    a2[15, 7], b2[1, 3, 4], b2[1, 90, 0] = NAN, float("inf"), NAN
    mg.m_grouped_bf16_gemm_nt_ragged(a2, b2, e, off)
    assert torch.equal(e[:10], d[:10]) and torch.equal(e[80:], d[80:])
    hit = torch.zeros_like(e, dtype=torch.bool)
    hit[15] = True
    hit[10:80, 3] = hit[10:80, 90] = True
    assert torch.equal(e[~hit], d[~hit]) and not torch.isfinite(e[hit]).any()
    w2 = torch.zeros_like(w)
    mg.k_grouped_bf16_gemm_tn(a2, t, w2, off)
    assert torch.equal(w2[[0, 2]], w[[0, 2]]) and torch.isnan(w2[1, 7]).all()
    assert torch.equal(torch.cat([w2[1, :7], w2[1, 8:]]), torch.cat([w[1, :7], w[1, 8:]]))


def test_gradients_are_differences():
    """nn and tn against central differences of nt, which is linear in each operand."""
    say("gradients of the ragged product against differences")
    gen = _gen(3)
    sizes, N, K = [9, 0, 40], 64, 64
    off = _offsets(sizes)
    a, b, dy = _rows(gen, (49, K), BF), _rows(gen, (3, N, K), BF), _rows(gen, (49, N), BF)
    da, db = torch.zeros(49, K, device="cuda"), torch.zeros(3, N, K, device="cuda")
    mg.m_grouped_bf16_gemm_nn_ragged(dy, b, da, off)
    mg.k_grouped_bf16_gemm_tn(dy, a, db, off)

    def loss(a, b):
        d = torch.zeros(49, N, device="cuda")
        mg.m_grouped_bf16_gemm_nt_ragged(a, b, d, off)
        return float((d.double() * dy.double()).sum())

    # steps of one: the values stay BF16 numbers after rounding, and the quotient takes the step as it was made
    scale = float((a.double().abs().max() * b.double().abs().max() * dy.double().abs().max()))
    for m, k in ((0, 0), (8, 63), (20, 5)):
        up, down = a.clone(), a.clone()
        up[m, k] += 1.0
        down[m, k] -= 1.0
        step = float(up[m, k].double() - down[m, k].double())
        assert abs((loss(up, b) - loss(down, b)) / step - float(da[m, k])) <= 49 * N * (K + 2) * U * scale
    for g, n, k in ((0, 0, 0), (2, 63, 1), (1, 5, 5)):
        up, down = b.clone(), b.clone()
        up[g, n, k] += 1.0
        down[g, n, k] -= 1.0
        step = float(up[g, n, k].double() - down[g, n, k].double())
        assert abs((loss(a, up) - loss(a, down)) / step - float(db[g, n, k])) <= 49 * N * (K + 2) * U * scale


def test_graph_replays_follow_the_offsets():
    say("ragged products replayed with other groups")
    gen = _gen(4)
    M, N, K, G = 300, 128, 192, 5
    a, t = _rows(gen, (M, K), BF), _rows(gen, (M, N), BF)
    b, e = _rows(gen, (G, N, K), BF), _rows(gen, (G, N, K), BF)
    off = _offsets([100, 0, 50, 150, 0])

    def room():
        return [torch.zeros(M, N, dtype=BF, device="cuda"), torch.zeros(M, K, device="cuda"),
                torch.zeros(G, N, K, device="cuda")]

    def step(o):
        mg.m_grouped_bf16_gemm_nt_ragged(a, b, o[0], off)
        mg.m_grouped_bf16_gemm_nn_ragged(t, e, o[1], off)
        mg.k_grouped_bf16_gemm_tn(t, a, o[2], off)

    got, want = room(), room()
    step(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got)
    for sizes in ([0, 300, 0, 0, 0], [1, 2, 3, 4, 290], [60] * 5, [10, 0, 0, 0, 0]):
        off.copy_(_offsets(sizes))
        a.copy_(_rows(gen, (M, K), BF))
        for o in got + want:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        step(want)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), sizes


def test_on_another_stream_and_twice_at_once():
    say("two ragged calls on two streams")
    gen = _gen(6)
    sizes, N, K = [400, 100, 250], 512, 512
    off = _offsets(sizes)
    a, b = _rows(gen, (750, K), BF), _rows(gen, (3, N, K), BF)
    one, two, ref = (torch.zeros(750, N, device="cuda") for _ in range(3))
    mg.m_grouped_bf16_gemm_nt_ragged(a, b, ref, off)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in s:
        st.wait_stream(torch.cuda.current_stream())
    mg.m_grouped_bf16_gemm_nt_ragged(a, b, one, off, stream=s[0])
    mg.m_grouped_bf16_gemm_nt_ragged(a, b, two, off, stream=s[1])
    torch.cuda.synchronize()
    assert torch.equal(one, ref) and torch.equal(two, ref)
