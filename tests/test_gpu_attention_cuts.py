"""Parity of paged_attention_fp8 (oracle/attention.py) as larger batches run it:
many (sequence, KV head) units on one line of tiles, cut where a share ends --
inside a unit, between the heads of a sequence, or between sequences -- and
caches large enough for codes to be loaded past the caches of the machine.

The block tables are wide (-1 past each sequence's pages): how a call is cut and
loaded goes by what the table can hold, S Hkv tables of `room` positions, 2 S Hkv
room D bytes (256 MiB or more: past the caches, where one wave takes a unit's
rows), while the lengths stay short enough for the oracle.  The bounds are
those of test_gpu_paged_attention.py."""

import numpy as np
import pytest

from helpers import say, to_dev
from test_gpu_paged_attention import _case, _compare, _mg, _run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _ragged(S, most, long):
    rng = np.random.default_rng(S + most)
    lens = [int(v) for v in rng.integers(0, most, size=S)]
    lens[0], lens[1], lens[2], lens[S // 2], lens[S - 1] = 0, 1, long, 33, long // 3
    return lens


def _widened(c, room, P):
    wide = np.full((c["table"].shape[0], room // P), -1, dtype=np.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    for i, ln in enumerate(c["lens"]):
        wide[i, max(1, -(-int(ln) // P)):] = -1
    c["table"] = wide


GB = 1 << 28  # bytes of both caches from which codes are loaded past the machine's caches


@pytest.mark.parametrize("S,n,H,group,D,P,room,window,cut,past", [
    # one row tile a unit: four waves take a unit's tiles in turn
    (36, 1, 4, 4, 128, 64, 3840, 0, True, False),
    (36, 1, 4, 4, 128, 64, 8192, 0, True, True),
    (40, 2, 4, 3, 128, 16, 8192, 0, True, True),
    (40, 1, 5, 1, 128, 16, 4096, 700, False, False),   # (what a window shows is not cut)
    (70, 1, 3, 8, 64, 128, 10240, 0, True, True),
    (70, 3, 2, 2, 64, 32, 5120, 0, True, False),
    (36, 1, 4, 4, 128, 16, 3840, 0, True, False),
    (70, 1, 3, 8, 64, 16, 10240, 0, True, True),
    (36, 4, 4, 4, 256, 32, 4096, 0, True, True),
    (36, 4, 4, 4, 256, 16, 4096, 0, True, True),
    (45, 1, 3, 5, 256, 128, 2560, 0, True, False),
    (36, 1, 4, 2, 256, 16, 4096, 900, False, False),
    # more sequences than a wave has lanes, and than a workgroup has
    (300, 1, 2, 4, 128, 64, 4160, 0, True, True),
    (300, 1, 2, 4, 128, 64, 8192, 2500, False, True),
    (300, 1, 2, 4, 128, 64, 8192, 6000, True, True),
    # two row tiles a wave
    (36, 5, 4, 4, 128, 64, 3840, 0, True, False),
    (36, 5, 4, 4, 128, 64, 8192, 0, True, True),
    (36, 5, 4, 4, 128, 16, 8192, 0, True, True),
    (70, 2, 3, 12, 64, 64, 12288, 0, True, True),
    (70, 2, 3, 12, 64, 16, 12288, 0, True, True),
    (33, 7, 4, 4, 128, 32, 4096, 2300, True, False),
    # two and four waves side by side, and more row tiles than they take
    (36, 6, 4, 8, 128, 64, 2560, 0, True, False),
    (36, 6, 4, 8, 128, 16, 2560, 0, True, False),
    (33, 13, 4, 8, 128, 64, 2560, 0, True, False),
    (34, 9, 4, 8, 64, 32, 2560, 0, True, False),
    (20, 19, 4, 8, 128, 64, 2560, 0, True, False),
    (36, 3, 4, 8, 256, 64, 2560, 0, True, False),      # 24 rows
    (34, 5, 4, 8, 256, 16, 2560, 0, True, False),      # 40 rows
    (20, 10, 2, 8, 256, 128, 2560, 1000, True, False),
    # not cut, past the caches
    (200, 1, 2, 4, 128, 64, 4096, 0, False, True),
    (200, 1, 2, 4, 128, 16, 4096, 0, False, True),
    (200, 5, 2, 4, 128, 64, 4096, 0, False, True),
    (200, 5, 2, 4, 128, 16, 4096, 0, False, True),
    (300, 1, 2, 2, 64, 32, 4096, 0, False, True),
    (300, 1, 2, 2, 64, 16, 4096, 0, False, True),
    (300, 9, 2, 2, 64, 32, 4096, 0, False, True),
    (300, 9, 2, 2, 64, 16, 4096, 0, False, True),
    (225, 1, 2, 2, 256, 128, 4096, 0, False, True),
    (225, 1, 2, 2, 256, 16, 4096, 0, False, True),
])
def test_units_of_many_sequences(S, n, H, group, D, P, room, window, cut, past):
    say(f"paged_attention_fp8 units S={S} n={n} H={H} group={group} D={D} P={P} room={room} window={window}")
    shown = min(room, window + n + 31) if window else room
    assert ((2 * S * H * shown * D >= GB) and not (n * group > (32 if D <= 128 else 16))) == past
    if not window:  # (the workspace is that of the whole room)
        assert (_mg().paged_attention_fp8_workspace(S, n, H * group, H, D, room) > 0) == cut
    lens = _ragged(S, 150 if S * n > 200 else 300, 2500)
    c = _case(D + n + S, S, n, H * group, H, D, P, lens)
    _widened(c, room, P)
    out, lse = _run(c, D ** -0.5, window)
    _compare(c, out, lse, D ** -0.5, window, "units")
    again, lse2 = _run(c, D ** -0.5, window)
    assert np.array_equal(out, again) and np.array_equal(lse, lse2), "a repeat differs"


@pytest.mark.parametrize("D,P,n,group", [(128, 64, 1, 8), (64, 16, 5, 4), (256, 32, 3, 8)])
def test_many_units_replayed(D, P, n, group):
    """The general cut under graph capture: other lengths, other shares."""
    say(f"paged_attention_fp8 many units replayed D={D} P={P} n={n}")
    S, H = 40, 4
    c = _case(D, S, n, H * group, H, D, P, _ragged(S, 200, 2400))
    _widened(c, 8192, P)
    table, lens = to_dev(c["table"]), to_dev(c["lens"])
    need = _mg().paged_attention_fp8_workspace(S, n, H * group, H, D, 8192)
    ws = torch.full((need // 4 + 1,), float("nan"), device="cuda")
    out = torch.empty(S, n, H * group, D, dtype=torch.bfloat16, device="cuda")

    def call():
        _mg().paged_attention_fp8(c["dq"], *c["dev"], table, lens, out, 0.1, workspace=ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = c["lens"].copy()
    for step in range(4):
        now = full if step == 3 else np.maximum(full - 37 * (step + 1), 0).astype(np.int32)
        lens.copy_(torch.from_numpy(now))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.fill_(5.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, got), f"replay {step}"


@pytest.mark.parametrize("S,n,H,group,D,P,lens,room,window", [
    (2, 300, 2, 4, 128, 64, [300, 777], 832, 0),          # a fresh prompt, and one after a cached prefix
    (2, 257, 1, 8, 64, 16, [257, 100], 4096, 0),          # more queries than tokens; cut
    (1, 500, 2, 3, 128, 32, [1900], 8192, 400),
    (1, 130, 2, 4, 256, 128, [600], 4096, 0),
])
def test_prompts(S, n, H, group, D, P, lens, room, window):
    say(f"paged_attention_fp8 prompts n={n} H={H} group={group} D={D} P={P} lens={lens} window={window}")
    c = _case(D + n, S, n, H * group, H, D, P, lens)
    _widened(c, room, P)
    out, lse = _run(c, D ** -0.5, window)
    _compare(c, out, lse, D ** -0.5, window, "prompt")
