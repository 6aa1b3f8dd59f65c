"""Expert routing of a mixture-of-experts layer and its gradient, float64.

moe_route_topk: scores (sigmoid or softmax of the logits), a choice (score
plus bias) limited to the best groups of experts, the k best choices with
ties to the lowest index, and their weights.  moe_route_topk_bwd: the
gradient of the logits with the choice taken as given.

Pinned by tests/test_oracle_router.py: hand-computed rows, brute force over
the choices, and central differences.
"""

import numpy as np


def _scores(x, score):
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(top > -np.inf, top, 0.0))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total == 0.0, 1.0, total)


def route_choices(x, bias, score, n_group, topk_group, group_top):
    """The choice values [T, E] that are left to pick from (-inf: none)."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    c = _scores(x, score) + b
    c = np.where((x == -np.inf) | (b == -np.inf)[None, :], -np.inf, c)
    if n_group > 1:
        for t in range(T):
            per = c[t].reshape(n_group, -1)
            rank = []
            for g in range(n_group):
                best = np.sort(per[g][per[g] > -np.inf])[::-1][:group_top]
                rank.append(best.sum() if best.size else -np.inf)
            keep = np.argsort(-np.array(rank), kind="stable")[:topk_group]
            drop = np.ones(n_group, dtype=bool)
            drop[keep] = False
            per[drop] = -np.inf
    return c


def moe_route_topk(x, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """(topk_idx int32 [T, k], topk_weights float64 [T, k])."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    c = route_choices(x, bias, score, n_group, topk_group, group_top)
    s = _scores(x, score)
    idx = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        pick = np.argsort(-c[t], kind="stable")[:k]
        pick = pick[c[t, pick] > -np.inf]
        n = len(pick)
        if n == 0:
            continue
        idx[t, :n] = pick
        if not renormalize:
            w[t, :n] = scale * s[t, pick]
        elif score == "sigmoid":
            w[t, :n] = scale * s[t, pick] / (s[t, pick].sum() + 1e-20)
        else:
            e = np.exp(x[t, pick] - x[t, pick].max())
            w[t, :n] = scale * e / e.sum()
    return idx, w


def route_weights(x, idx, score, renormalize, scale):
    """The weights [k] of one row's given choices, as a function of its logits."""
    x = np.asarray(x, dtype=np.float64)
    pick = [i for i in idx if 0 <= i < x.size]
    w = np.zeros(len(idx))
    if not pick:
        return w
    z = _scores(x[None], score)[0][pick]
    if renormalize and score == "softmax":
        z = np.exp(x[pick] - x[pick].max())
        z = z / z.sum()
    elif renormalize:
        z = z / (z.sum() + 1e-20)
    w[[j for j, i in enumerate(idx) if 0 <= i < x.size]] = scale * z
    return w


def moe_route_topk_bwd(x, idx, g, score="softmax", renormalize=True, scale=1.0):
    """Gradient float64 [T, E] of sum(g * weights) for the given choices."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    s = _scores(x, score)
    dx = np.zeros((T, E))
    for t in range(T):
        js = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        if not js:
            continue
        pick = idx[t, js].astype(np.int64)
        gj = scale * np.asarray(g, dtype=np.float64)[t, js]
        if renormalize and score == "softmax":
            q = np.exp(x[t, pick] - x[t, pick].max())
            q /= q.sum()
            np.add.at(dx[t], pick, q * (gj - (gj * q).sum()))
            continue
        z = s[t, pick]
        dz = gj
        if renormalize:
            D = z.sum() + 1e-20
            dz = (gj - (gj * z).sum() / D) / D
        ds = np.zeros(E)
        np.add.at(ds, pick, dz)
        dx[t] = ds * s[t] * (1 - s[t]) if score == "sigmoid" else s[t] * (ds - (ds * s[t]).sum())
    return dx
