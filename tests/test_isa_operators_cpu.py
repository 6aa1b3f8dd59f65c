"""No kernel of the routing, the cache append or the attention may spill to
scratch, and none may hold a packed FP32 instruction (read from the in-tree
build; skipped where it or the LLVM tools are missing)."""

import os
import re
import subprocess

import pytest

from test_isa_cpu import BUILD, LLVM, _extract


@pytest.mark.parametrize("src,kernels", [("route.hip", 25), ("kvcache.hip", 18), ("attn.hip", 13)])
def test_no_spills_and_no_packed_fp32(src, kernels, tmp_path):
    co = _extract(os.path.join(BUILD, src + ".o"), tmp_path)
    notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", co], check=True, capture_output=True,
                           text=True).stdout
    sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", notes)
    assert len(sizes) >= kernels
    assert set(sizes) == {"0"}, sizes
    text = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", co], check=True, capture_output=True,
                          text=True).stdout
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)
