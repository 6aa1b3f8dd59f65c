"""What stands around and between an expert's products, in float64 numpy: the
root-mean-square norm with the residual's addition, the gated activation, their
gradients, and the products of ragged groups.  Pinned by
``tests/test_oracle_layer.py`` (closed forms, differences, brute force)."""

import numpy as np


def rms_norm(h, weight, eps):
    """h [.., H] -> h / sqrt(mean(h^2) + eps) * weight."""
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps) * weight


def rms_norm_bwd(grad_y, h, weight, eps, grad_h=None):
    """(grad of h, grad of weight, and for both the sum of the absolute values of
    the terms that they are sums of)."""
    h, dy = np.asarray(h, np.float64), np.asarray(grad_y, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps)
    hat, g = h * r, dy * weight
    dx = r * (g - hat * (g * hat).mean(axis=-1, keepdims=True))
    size = r * (np.abs(g) + np.abs(hat) * np.abs(g * hat).mean(axis=-1, keepdims=True))
    if grad_h is not None:
        dx = dx + grad_h
        size = size + np.abs(grad_h)
    t = (dy * hat).reshape(-1, h.shape[-1])
    return dx, t.sum(axis=0), size, np.abs(t).sum(axis=0)


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def swiglu(x, row_weights=None):
    """x [R, 2 I] -> row_weights * silu(x[:, :I]) * x[:, I:]."""
    x = np.asarray(x, np.float64)
    n = x.shape[-1] // 2
    y = x[..., :n] * _sigmoid(x[..., :n]) * x[..., n:]
    return y if row_weights is None else y * np.asarray(row_weights, np.float64)[:, None]


def swiglu_bwd(x, grad_y, row_weights=None):
    """(grad of x, grad of row_weights, and what their errors are relative to:
    the absolute terms)."""
    x, dy = np.asarray(x, np.float64), np.asarray(grad_y, np.float64)
    n = x.shape[-1] // 2
    g, u = x[..., :n], x[..., n:]
    w = 1.0 if row_weights is None else np.asarray(row_weights, np.float64)[:, None]
    s, c = _sigmoid(g), _sigmoid(-g)
    dg, du = dy * w * u * s * (1.0 + g * c), dy * w * g * s
    size = np.concatenate([np.abs(dy * w * u) * s * (1.0 + np.abs(g)), np.abs(du)], axis=-1)
    t = dy * g * s * u
    return np.concatenate([dg, du], axis=-1), t.sum(axis=-1), size, np.abs(t).sum(axis=-1)


def ragged_rows(offsets, M):
    """(group, first row, end) of every group, cut to [0, M]."""
    at = np.clip(np.asarray(offsets, np.int64), 0, M)
    return [(g, int(at[g]), int(max(at[g], at[g + 1]))) for g in range(len(at) - 1)]


def ragged_nt(a, b, offsets, c=None):
    """d[m] = c[m] + a[m] . b[g]^T, and the rows that belong to a group."""
    d = np.zeros((a.shape[0], b.shape[1])) if c is None else np.array(c, np.float64)
    done = np.zeros(a.shape[0], bool)
    for g, i, j in ragged_rows(offsets, a.shape[0]):
        d[i:j] += np.asarray(a[i:j], np.float64) @ np.asarray(b[g], np.float64).T
        done[i:j] = True
    return d, done


def ragged_nn(a, b, offsets, c=None):
    """d[m] = c[m] + a[m] . b[g], b [G, K, N]."""
    return ragged_nt(a, np.swapaxes(b, 1, 2), offsets, c)


def ragged_tn(a, b, offsets, c=None):
    """d[g] = c[g] + a_g^T . b_g over the rows of group g."""
    G = len(offsets) - 1
    d = np.zeros((G, a.shape[1], b.shape[1])) if c is None else np.array(c, np.float64)
    for g, i, j in ragged_rows(offsets, a.shape[0]):
        d[g] += np.asarray(a[i:j], np.float64).T @ np.asarray(b[i:j], np.float64)
    return d
