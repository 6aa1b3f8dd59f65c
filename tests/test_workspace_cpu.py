"""paged_attention_fp8_workspace on any arguments: a number, and 0 for sizes that
no call takes (each in a process of its own, which has to end by itself)."""

import subprocess
import sys

import pytest

import moe_grouped_gemm_x128_amd as mg

BIG = 2 ** 62


@pytest.mark.parametrize("args", [
    (1, 1, 1, 1, 1, 100000), (1, 1, 1, 1, 3, 100000), (1, 1, 1, 1, 96, 100000), (1, 1, 1, 1, 4096, 100000),
    (1, 1, 1, 1, BIG, 100000), (BIG, 1, 1, 1, 64, 100000), (1, BIG, 1, 1, 64, 100000), (1, 1, BIG, 1, 64, 100000),
    (1, 1, BIG, BIG, 64, 100000), (1, 1, 1, 1, 64, BIG), (BIG, BIG, BIG, BIG, BIG, BIG), (1, 1, 3, 2, 64, 100000),
    (1, 1, 1, 2, 64, 100000), (-1, 1, 1, 1, 64, 100000), (0, 1, 1, 1, 64, 100000), (1, 1, 1, 1, 64, -BIG),
])
def test_sizes_that_no_call_takes(args):
    r = subprocess.run([sys.executable, "-c", "import moe_grouped_gemm_x128_amd as mg\n"
                        f"print(mg.paged_attention_fp8_workspace(*{args}))"], capture_output=True, text=True)
    assert r.returncode == 0, f"ended with {r.returncode}"
    assert int(r.stdout) == 0


def test_sizes_that_calls_take():
    for D in (64, 128, 256):
        for S, n, Hq, H in ((1, 1, 8, 2), (128, 1, 64, 8), (3, 40, 32, 4), (600, 4, 16, 1)):
            need = [mg.paged_attention_fp8_workspace(S, n, Hq, H, D, cap) for cap in (16, 1000, 20000, 131072)]
            assert need[0] == 0 and need[3] > 0 and need == sorted(need) and max(need) < 64 << 20, (D, S, n, need)
