"""Refusals of the routing, cache and attention calls: every malformed
argument is rejected on the host, before any launch (no GPU needed)."""

import os

import pytest
import torch

import moe_grouped_gemm_x128_amd as mg
from moe_grouped_gemm_x128_amd import binding

I32, F32, BF16, U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
INVALID, UNSUPPORTED = binding.DG_INVALID_ARG, binding.DG_UNSUPPORTED


@pytest.fixture(autouse=True)
def _built():
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libdgmi.so is not built (python -m moe_grouped_gemm_x128_amd.build)")


def _t(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


class _Null:
    cuda_stream = 0


def _refused(call, code, *args, **kw):
    with pytest.raises(mg.DgmiError) as e:
        call(*args, stream=_Null(), **kw)
    assert e.value.code == code, str(e.value)
    return str(e.value)


def _taken(call, *args, **kw):
    """Past every check: without a GPU the launch itself fails."""
    try:
        call(*args, stream=_Null(), **kw)
    except mg.DgmiError as e:
        assert e.code == binding.DG_LAUNCH_FAILED, str(e)


def test_routing_refusals():
    T, E, k = 4, 32, 4
    x, idx, w, b = _t((T, E)), _t((T, k), I32), _t((T, k)), _t((E,))
    r = mg.moe_route_topk
    _refused(r, INVALID, _t((T, E), I32), idx, w)                              # logits dtype
    _refused(r, INVALID, _t((T, E, 1)), idx, w)                                # rank
    _refused(r, INVALID, x.t().contiguous().t(), idx, w)                       # innermost stride
    _refused(r, INVALID, x, _t((T, k)), w)                                     # idx dtype
    _refused(r, INVALID, x, _t((T + 1, k), I32), w)                            # rows
    _refused(r, INVALID, x, idx, _t((T, k + 1)))                               # weights shape
    _refused(r, INVALID, x, idx, w, bias=_t((E + 1,)))
    _refused(r, INVALID, x, idx, w, bias=b.to(BF16))
    _refused(r, INVALID, x, _t((T, E + 1), I32), _t((T, E + 1)))               # more choices than experts
    _refused(r, INVALID, x, idx, w, n_group=5)                                 # does not divide
    _refused(r, INVALID, x, idx, w, n_group=0)
    _refused(r, INVALID, x, idx, w, n_group=4, topk_group=5)
    _refused(r, INVALID, x, idx, w, n_group=4, topk_group=0)
    _refused(r, INVALID, x, idx, w, n_group=4, group_top=3)
    assert "fewer" in _refused(r, INVALID, x, idx, w, n_group=16, topk_group=1)  # two experts for four choices
    _refused(r, INVALID, x, idx, w, scale=float("nan"))
    _refused(r, UNSUPPORTED, _t((T, 1025)), idx, w)
    _refused(r, UNSUPPORTED, _t((T, 128)), _t((T, 65), I32), _t((T, 65)))
    _refused(r, UNSUPPORTED, _t((T, 130)), idx, w, n_group=65, topk_group=2)
    assert "overlaps" in _refused(r, INVALID, x, idx, x[:, :k])
    _refused(r, INVALID, x, idx, idx.view(F32))
    _refused(r, INVALID, x, idx[:1].expand(T, k), w)                           # rows on top of each other
    far = _t((1, E)).expand(2 ** 25 + 1, E)
    _refused(r, UNSUPPORTED, far, _t((1, 1), I32).expand(2 ** 25 + 1, 1), _t((1, 1)).expand(2 ** 25 + 1, 1))
    with pytest.raises(ValueError):
        r(x, idx, w, score="tanh", stream=_Null())
    _taken(r, x, idx, w, bias=b, score="sigmoid", n_group=8, topk_group=4, group_top=2)
    g = _t((T, k))
    d = mg.moe_route_topk_bwd
    _refused(d, INVALID, x, idx, g, _t((T, E + 1)))
    _refused(d, INVALID, x, idx, g, _t((T, E), I32))
    _refused(d, INVALID, x, idx, g.to(BF16), _t((T, E)))
    _refused(d, INVALID, x, idx, _t((T, k + 1)), _t((T, E)))
    _refused(d, INVALID, x, idx, g, x)                                         # in place
    _refused(d, INVALID, x, idx, g, _t((T, E)), scale=float("inf"))
    _refused(d, UNSUPPORTED, _t((T, 1025)), idx, g, _t((T, 1025)))
    _taken(d, x, idx, g, _t((T, E), BF16))


def _cache(pages=3, H=2, P=16, D=64):
    return [_t((pages, H, P, D), U8), _t((pages, H, P, D), U8), _t((pages, H)), _t((pages, H))]


def test_append_refusals():
    T, H, D, S = 5, 2, 64, 2
    k, v = _t((T, H, D), BF16), _t((T, H, D), BF16)
    c = _cache()
    table, cu, start, cs = _t((S, 4), I32), _t((S + 1,), I32), _t((S,), I32), _t((100, 32))
    a = mg.kv_append_fp8

    def no(code, k=k, v=v, c=c, table=table, cu=cu, start=start, **kw):
        return _refused(a, code, k, v, *c, table, cu, start, **kw)

    no(INVALID, k=k.to(I32))
    no(INVALID, v=v.float())                                                   # k and v differ
    no(INVALID, k=_t((T + 1, H, D), BF16))
    no(INVALID, k=_t((T, H + 1, D), BF16), v=_t((T, H + 1, D), BF16))
    no(INVALID, k=_t((T, H, D + 1), BF16)[..., 1:])                            # rows not 16-byte aligned
    no(INVALID, c=_cache(H=3))
    no(INVALID, c=[c[0], _cache(pages=4)[1], c[2], c[3]])                      # one scale table short
    no(INVALID, c=[c[0].float()] + c[1:])
    no(INVALID, c=c[:2] + [_t((3, 3)), c[3]])
    no(UNSUPPORTED, c=_cache(P=48))
    no(UNSUPPORTED, k=_t((T, H, 96), BF16), v=_t((T, H, 96), BF16), c=_cache(D=96))
    no(INVALID, c=[_t((3, 2, 16, 72), U8)[..., :64]] + c[1:])                  # token stride not a multiple of 16
    no(INVALID, cu=_t((S,), I32))
    no(INVALID, start=_t((S, 1), I32))
    no(INVALID, start=start.float())
    no(INVALID, table=_t((S + 1, 4), I32))
    no(INVALID, cos_sin=_t((100, 24)))                                         # not a multiple of 16
    no(INVALID, cos_sin=_t((100, 80)))                                         # more than the head
    no(INVALID, cos_sin=_t((100, 32), BF16))
    no(INVALID, cos_sin=_t((100, 34))[:, :32])                                 # rows not 16-byte aligned
    q = _t((T, 6, D), BF16)
    no(INVALID, q=q)                                                           # q without q_out
    no(INVALID, q_out=q)
    no(INVALID, q=q, q_out=_t((T, 5, D), BF16))
    no(INVALID, q=q, q_out=_t((T, 6, D)))
    no(INVALID, q=q.float(), q_out=_t((T, 6, D), BF16))                        # not k's type
    assert "overlaps" in no(INVALID, q=q, q_out=q)
    no(INVALID, c=[c[0], c[0], c[2], c[3]])                                    # K and V the same memory
    no(INVALID, c=[c[0], c[1], c[2], c[2]])
    no(INVALID, c=[c[0][:1].expand(3, 2, 16, 64)] + c[1:])                     # pages on top of each other
    pool = _t((3, 2, 2, 16, 64), U8)                                           # K and V halves of one pool: taken
    _taken(a, k, v, pool[:, 0], pool[:, 1], c[2], c[3], table, cu, start, cos_sin=cs, q=q, q_out=_t((T, 6, D), BF16))
    big = _t((1, 1, 64), BF16).expand(2 ** 22, 512, 64)                        # 2^28 workgroups
    no(UNSUPPORTED, k=big, v=big, c=_cache(H=512))


def test_attention_refusals():
    S, n, Hq, H, D = 2, 1, 4, 2, 64
    q, out, lse = _t((S, n, Hq, D), BF16), _t((S, n, Hq, D), BF16), _t((S, n, Hq))
    c = _cache()
    table, lens = _t((S, 4), I32), _t((S,), I32)
    a = mg.paged_attention_fp8

    def no(code, q=q, c=c, table=table, lens=lens, out=out, scale=1.0, **kw):
        return _refused(a, code, q, *c, table, lens, out, scale, **kw)

    no(INVALID, q=q.float())
    no(INVALID, q=q[:, 0])
    no(INVALID, q=_t((S, n, Hq, 128), BF16))
    no(INVALID, out=_t((S, n, Hq + 2, D), BF16))
    no(INVALID, out=out.float())
    no(INVALID, q=_t((S, n, 5, D), BF16), out=_t((S, n, 5, D), BF16))          # not a multiple of Hkv
    no(INVALID, q=_t((S, n, Hq, D + 4), BF16)[..., :D])                        # rows not 16-byte aligned
    no(INVALID, lens=_t((S + 1,), I32))
    no(INVALID, lens=lens.float())
    no(INVALID, table=_t((S + 1, 4), I32))
    no(INVALID, table=_t((S, 4)))
    no(UNSUPPORTED, c=_cache(P=256))
    no(INVALID, scale=float("nan"))
    no(INVALID, window=-1)
    no(INVALID, lse=_t((S, n, Hq + 1)))
    no(INVALID, lse=lse.to(BF16))
    no(INVALID, lse=lse[:1].expand(S, n, Hq))
    assert "overlaps" in no(INVALID, out=q)
    no(INVALID, out=out[:1].expand(S, n, Hq, D))
    no(INVALID, c=[c[0], c[1], c[2], _t((3, 3))])
    # a workspace, where one is needed
    wide = _t((S, 1000), I32)
    need = mg.paged_attention_fp8_workspace(S, n, Hq, H, D, 16000)
    assert need == mg.paged_attention_fp8_workspace(S, n, Hq, H, D, 16000) >= 0
    assert mg.paged_attention_fp8_workspace(0, n, Hq, H, D, 16000) == 0
    if need > 0:
        assert "workspace" in no(INVALID, table=wide)
        no(INVALID, table=wide, workspace=_t((need // 4 - 1,)))
        no(INVALID, table=wide, workspace=_t((need,), I32))
        no(INVALID, table=wide, workspace=_t((need // 4 + 1,))[1:])            # not 16-byte aligned
    _taken(a, q, *c, wide, lens, out, 1.0, lse=lse, window=3, workspace=_t((need // 4 + 4,)))
