"""kv_append_fp8 writes two caches and two tables of scales: they may be parts of
one pool in any interleaving, but no byte may belong to both.  Checked on the
host, before any launch (no GPU needed); the expected answers are counted
element by element."""

import ctypes

import numpy as np
import pytest
import torch

import moe_grouped_gemm_x128_amd as mg
from moe_grouped_gemm_x128_amd import binding

from test_abi_operators_cpu import BF16, I32, U8, _built, _refused, _t, _taken  # noqa: F401

INVALID = binding.DG_INVALID_ARG


def _append(kc, vc, ks, vs, ok):
    pages, H, P, D = kc.shape
    args = (_t((5, H, D), BF16), _t((5, H, D), BF16), kc, vc, ks, vs, _t((2, 4), I32), _t((3,), I32), _t((2,), I32))
    if ok:
        _taken(mg.kv_append_fp8, *args)
    else:
        assert "overlap" in _refused(mg.kv_append_fp8, INVALID, *args)


def _elements(t):
    at = np.array([t.storage_offset()])
    for n, s in zip(t.shape, t.stride()):
        at = (at[:, None] + np.arange(n) * s).ravel()
    return set(at.tolist())


def _view(pool, shape, stride, offset):
    return torch.as_strided(pool, shape, stride, offset)


H, P, D = 2, 16, 64


@pytest.mark.parametrize("offset", [16, 64, D * P, D * P * H, 3 * D * P * H - 16])
def test_a_v_cache_that_begins_inside_the_k_cache(offset):
    pool = _t((8 * H * P * D,), U8)
    dense = (H * P * D, P * D, D, 1)
    kc, vc = _view(pool, (3, H, P, D), dense, 0), _view(pool, (3, H, P, D), dense, offset)
    assert _elements(kc) & _elements(vc)
    for a, b in ((kc, vc), (vc, kc)):
        _append(a, b, _t((3, H)), _t((3, H)), False)


@pytest.mark.parametrize("name,ks,vs,off", [
    # strides of (page, head, token) of K and of V, and V's offset
    ("halves of each page", (2 * H * P * D, P * D, D), (2 * H * P * D, P * D, D), H * P * D),
    ("head by head", (2 * H * P * D, 2 * P * D, D), (2 * H * P * D, 2 * P * D, D), P * D),
    ("token by token", (2 * H * P * D, 2 * D, 2 * H * D), (2 * H * P * D, 2 * D, 2 * H * D), D),
    ("tokens of all heads", (2 * H * P * D, D, 2 * H * D), (2 * H * P * D, D, 2 * H * D), H * D),
    ("K by heads, V by tokens", (2 * H * P * D, P * D, D), (2 * H * P * D, D, H * D), H * P * D),
    ("one after the other", (H * P * D, P * D, D), (H * P * D, P * D, D), 3 * H * P * D),
    ("heads first", (P * D, 8 * P * D, D), (P * D, 8 * P * D, D), 4 * P * D),
    # the same, moved into each other
    ("half a half off", (2 * H * P * D, P * D, D), (2 * H * P * D, P * D, D), P * D),
    ("a token early", (2 * H * P * D, P * D, D), (2 * H * P * D, P * D, D), H * P * D - D),
    ("a token late", (2 * H * P * D, P * D, D), (2 * H * P * D, P * D, D), H * P * D + D),
    ("sixteen bytes off", (2 * H * P * D, 2 * D, 2 * H * D), (2 * H * P * D, 2 * D, 2 * H * D), D + 16),
    ("V by tokens, a token early", (2 * H * P * D, P * D, D), (2 * H * P * D, D, H * D), H * P * D - H * D),
    ("V's pages closer", (2 * H * P * D, P * D, D), (H * P * D, P * D, D), H * P * D),
])
def test_caches_in_one_pool(name, ks, vs, off):
    pool = _t((20 * H * P * D,), U8)
    kc, vc = _view(pool, (3, H, P, D), ks + (1,), 0), _view(pool, (3, H, P, D), vs + (1,), off)
    apart = not (_elements(kc) & _elements(vc))
    _append(kc, vc, _t((3, H)), _t((3, H)), apart)
    _append(vc, kc, _t((3, H)), _t((3, H)), apart)


def test_random_layouts_of_one_pool():
    rng = np.random.default_rng(4)
    pool = _t((1 << 16,), U8)
    seen = [0, 0]
    for _ in range(300):
        unit = [D * int(rng.integers(1, 3)), D * P * int(rng.integers(1, 4))]
        page = 2 * D * P * int(rng.integers(2, 5))
        strides = []
        for _ in range(2):
            tok, head = (unit[0], unit[1] * int(rng.integers(1, 3))) if rng.random() < 0.6 else (H * D, D)
            strides.append((page, head, tok, 1))
        kc = _view(pool, (3, H, P, D), strides[0], 0)
        vc = _view(pool, (3, H, P, D), strides[1], 16 * int(rng.integers(0, page // 16)))
        if len(_elements(kc)) < 3 * H * P * D or len(_elements(vc)) < 3 * H * P * D:
            continue  # rows on top of each other: refused for that
        try:
            _taken(mg.kv_append_fp8, _t((5, H, D), BF16), _t((5, H, D), BF16), kc, vc, _t((3, H)), _t((3, H)),
                   _t((2, 4), I32), _t((3,), I32), _t((2,), I32))
            taken = True
        except AssertionError as e:
            if "rows overlap" in str(e):
                continue  # (rows that are apart, but not nested)
            taken = False
        apart = not (_elements(kc) & _elements(vc))
        assert taken == apart, (strides, vc.storage_offset())
        seen[apart] += 1
    assert min(seen) >= 10, seen


def test_scales_in_one_table():
    both = _t((3, 2, H))
    c = [_t((3, H, P, D), U8) for _ in range(2)]
    _append(*c, both[:, 0], both[:, 1], True)
    flat = _t((64,))
    _append(*c, _view(flat, (3, H), (2 * H, 2), 0), _view(flat, (3, H), (2 * H, 2), 1), True)
    _append(*c, _view(flat, (3, H), (1, 3), 0), _view(flat, (3, H), (1, 3), 6), True)
    _append(*c, _view(flat, (3, H), (H, 1), 0), _view(flat, (3, H), (H, 1), 1), False)
    _append(*c, _view(flat, (3, H), (2 * H, 2), 0), _view(flat, (3, H), (2 * H, 2), 2), False)


def test_large_pools_of_unlike_page_strides():
    """A million pages each (descriptors alone, nothing is there): refused, and at once."""
    n = 1 << 20
    lib = binding.load_library()
    k, table, cu, start = (binding.describe(t) for t in (_t((5, H, D), BF16), _t((2, 4), I32), _t((3,), I32), _t((2,), I32)))

    def pool(t, data, page):
        x = binding.describe(t)
        x.data, x.shape[0], x.stride[0] = data, n, page
        return x

    for page_k, page_v, off in ((6144, 4096, 2048), (4096 + 16, 4096 + 32, 16), (12288, 8192, 4096)):
        caches = [pool(_t((3, H, P, D), U8), 1 << 44, page_k), pool(_t((3, H, P, D), U8), (1 << 44) + off, page_v)]
        scales = [pool(_t((3, H)), 1 << 50, H), pool(_t((3, H)), 1 << 51, H)]
        args = [ctypes.byref(x) for x in (k, k, *caches, *scales, table, cu, start)]
        assert lib.kv_append_fp8(*args, None, None, None, 0, None) == INVALID
        assert b"overlap" in lib.dg_last_error()
