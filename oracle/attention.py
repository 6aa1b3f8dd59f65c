"""Paged FP8 key/value cache: appending with the position rotation, and the
attention over it.

kv_append_fp8 follows the definition's own FP32 steps (each product and sum of
the rotation rounded once, the rest exact or correctly rounded), so its codes
and scales are compared bit for bit; rotate gives the rotation in float64.
paged_attention_fp8 is float64 throughout.

Pinned by tests/test_oracle_attention.py: rotations as complex products,
hand-built pages, a brute-force softmax over lists of visible positions.
"""

import numpy as np

from .formats import E4M3_MAX, e4m3_decode, e4m3_encode

AMAX_FLOOR = np.float32(1e-4)


def rotate(x, cos, sin, interleaved, dtype=np.float64):
    """x [T, H, D] with cos, sin [T, rot/2]: pairs (a, b) -> (a c - b s, b c + a s)."""
    x = np.asarray(x, dtype=dtype)
    half = cos.shape[1]
    c, s = np.asarray(cos, dtype=dtype)[:, None], np.asarray(sin, dtype=dtype)[:, None]
    y = x.copy()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    a, b = x[..., first], x[..., second]
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., first] = (a * c).astype(dtype) - (b * s).astype(dtype)
        y[..., second] = (b * c).astype(dtype) + (a * s).astype(dtype)
    return y


def pow2_scale(amax):
    """2^ceil(log2(RN32(max(amax, 1e-4) / 448))) as float32."""
    q = np.maximum(np.asarray(amax, dtype=np.float32), AMAX_FLOOR) / np.float32(E4M3_MAX)
    m, e = np.frexp(q.astype(np.float64))
    return np.ldexp(1.0, e - (m == 0.5)).astype(np.float32)


def _encode(v, scale):
    """E4M3 codes of float32 values over a float32 scale; NaN where not finite."""
    with np.errstate(invalid="ignore", over="ignore"):
        q = v.astype(np.float32) / np.float32(scale)
    fine = np.isfinite(v)
    codes = e4m3_encode(np.where(fine, np.clip(q, -E4M3_MAX, E4M3_MAX), 0.0).astype(np.float64))
    return codes, fine


def kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, table, cu, start, cos_sin=None, interleaved=False):
    """New caches and scales (copies), and one mask per cache of the slots
    whose code stands for a value that was not finite (any NaN code)."""
    pages, H, P, D = k_cache.shape
    T = k.shape[0]
    out = []
    for x, codes, scale, turned in ((k, k_cache, k_scale, True), (v, v_cache, v_scale, False)):
        codes, scale = codes.copy(), scale.copy()
        nan = np.zeros(codes.shape, dtype=bool)
        for s in range(len(start)):
            p, end = int(start[s]), int(start[s]) + int(cu[s + 1]) - int(cu[s])
            if p < 0:
                continue
            if cos_sin is not None:
                end = min(end, cos_sin.shape[0])
            while p < end:
                upto = min(end, (p // P + 1) * P)
                t0 = int(cu[s]) + p - int(start[s])
                lp = p // P
                page = int(table[s, lp]) if lp < table.shape[1] else -1
                if 0 <= page < pages:
                    y = np.asarray(x[t0:t0 + upto - p], dtype=np.float32)
                    if turned and cos_sin is not None:
                        half = cos_sin.shape[1] // 2
                        rows = cos_sin[p:upto]
                        y = rotate(y, rows[:, :half], rows[:, half:], interleaved, np.float32)
                    lo = p % P
                    for h in range(H):
                        a = np.abs(y[:, h][np.isfinite(y[:, h])])
                        sc = pow2_scale(a.max() if a.size else 0.0)
                        if lo and scale[page, h] >= sc:
                            sc = scale[page, h]
                        elif lo:
                            old = e4m3_decode(codes[page, h, :lo]) * (float(scale[page, h]) / float(sc))
                            keep = np.isnan(old)
                            codes[page, h, :lo] = np.where(keep, codes[page, h, :lo],
                                                           e4m3_encode(np.where(keep, 0.0, old)))
                        scale[page, h] = sc
                        c, fine = _encode(y[:, h], sc)
                        codes[page, h, lo:lo + upto - p] = c
                        nan[page, h, lo:lo + upto - p] = ~fine
                p = upto
        out += [codes, scale, nan]
    kc, ks, kn, vc, vs, vn = out
    return kc, vc, ks, vs, kn, vn


def paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale, window=0):
    """(out [S, n, Hq, D], lse [S, n, Hq], mass [S, n, Hq, D], dot [S, n, Hq])
    in float64: mass = sum of weight times |v|, dot = the largest scale *
    sum |q| |k| over the visible tokens (both for error bounds)."""
    S, n, Hq, D = q.shape
    pages, H, P, _ = k_cache.shape
    g = Hq // H
    out = np.zeros((S, n, Hq, D))
    mass = np.zeros((S, n, Hq, D))
    dot = np.zeros((S, n, Hq))
    lse = np.full((S, n, Hq), -np.inf)
    q = np.asarray(q, dtype=np.float64)
    for s in range(S):
        ln = min(max(int(lens[s]), 0), table.shape[1] * P)
        for i in range(n):
            pos = ln - n + i
            lo = max(0, pos - window + 1) if window else 0
            seen = [t for t in range(lo, pos + 1) if 0 <= table[s, t // P] < pages]
            if not seen:
                continue
            pg = np.array([table[s, t // P] for t in seen])
            sl = np.array([t % P for t in seen])
            for h in range(H):
                k = e4m3_decode(k_cache[pg, h, sl]) * k_scale[pg, h].astype(np.float64)[:, None]
                v = e4m3_decode(v_cache[pg, h, sl]) * v_scale[pg, h].astype(np.float64)[:, None]
                for a in range(h * g, (h + 1) * g):
                    x = scale * (k @ q[s, i, a])
                    m = x.max()
                    e = np.exp(x - m)
                    z = e.sum()
                    out[s, i, a] = (e[:, None] * v).sum(axis=0) / z
                    mass[s, i, a] = (e[:, None] * np.abs(v)).sum(axis=0) / z
                    dot[s, i, a] = np.abs(scale) * (np.abs(k) @ np.abs(q[s, i, a])).max()
                    lse[s, i, a] = m + np.log(z)
    return out, lse, mass, dot
