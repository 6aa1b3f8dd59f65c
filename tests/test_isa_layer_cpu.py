"""The machine code of the norm, the activation and the ragged products (read from
the in-tree build; skipped where it or the LLVM tools are missing): no kernel may
spill to scratch or hold a packed FP32 instruction, and between the matrix
instructions of a ragged product there is neither a loop over differing lanes (a
load whose resource lost its place in scalar registers) nor a wait for every load
in flight."""

import os
import re
import subprocess

import pytest

from test_isa_cpu import BUILD, LLVM, _extract


def _text(co):
    return subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", co], check=True, capture_output=True,
                          text=True).stdout


@pytest.mark.parametrize("src,kernels", [("norm.hip", 17), ("swiglu.hip", 8), ("ragged.hip", 16)])
def test_no_spills_and_no_packed_fp32(src, kernels, tmp_path):
    co = _extract(os.path.join(BUILD, src + ".o"), tmp_path)
    notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", co], check=True, capture_output=True,
                           text=True).stdout
    sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", notes)
    assert len(sizes) >= kernels
    assert set(sizes) == {"0"}, sizes
    assert not re.search(r"v_pk_(add|mul|fma)_f32", _text(co))


def test_ragged_pipelines_run_through(tmp_path):
    co = _extract(os.path.join(BUILD, "ragged.hip.o"), tmp_path)
    seen = 0
    for body in re.split(r"\n[0-9a-f]+ <", _text(co))[1:]:
        name, _, code = body.partition(">:")
        if "ragged_kernel" not in name:
            continue
        lines = [line.split("//")[0].strip() for line in code.splitlines()]
        at = [i for i, line in enumerate(lines) if line.startswith("v_mfma")]
        assert len(at) >= 16, name
        loop = lines[at[0]:at[-1]]
        assert not any("saveexec" in line for line in loop), name
        assert "s_waitcnt vmcnt(0)" not in loop, name
        seen += 1
    assert seen == 16
