"""The operators around the FP8 GEMMs, measured: expert routing with its
gradient, the append to a paged FP8 key/value cache with the position
rotation, and the attention over that cache.

Where `own` is false, `run` computes each operator with elementary torch
operations in 32 bits; where it is true, with the library's calls.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
SCRATCH_F32 = 16 << 20  # scratch a serving program keeps for the attention (64 MiB)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode stream through a large router: latency
        dict(name="route_one", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, bf16=False, pad=0.0, train=False),
        # the decode batch of the framework's MoE workload (768 tokens, 8 choices)
        dict(name="route_decode", op="route", T=768, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, bf16=False, pad=0.0, train=False),
        # a packed prompt batch, BF16 logits, its last tokens padding (masked rows)
        dict(name="route_prompt", op="route", T=16384, E=128, k=8, score="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, renorm=True, scale=1.0, bf16=True, pad=0.03, train=False),
        # a training step's router: forward and gradient of the logits
        dict(name="route_train", op="route", T=4096, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, bf16=False, pad=0.0, train=True),
        # the same with softmax weights kept as they are, an odd token count, BF16
        dict(name="route_train_softmax", op="route", T=8191, E=64, k=6, score="softmax", bias=False, n_group=8,
             topk_group=3, group_top=1, renorm=False, scale=16.0, bf16=True, pad=0.0, train=True),
        # one new token of one sequence: latency; half of each head rotated, pairs interleaved
        dict(name="append_one", op="append", S=1, lo=1, hi=1, start=1500, Hq=8, Hkv=2, D=64, P=16, rot=32,
             interleaved=True, bf16=True),
        # one new token for each sequence of a serving batch
        dict(name="append_decode", op="append", S=256, lo=1, hi=1, start=4096, Hq=64, Hkv=8, D=128, P=64, rot=128,
             interleaved=False, bf16=True),
        # prompts of different lengths written at once
        dict(name="append_prompt", op="append", S=6, lo=37, hi=8192, start=100, Hq=32, Hkv=8, D=128, P=64, rot=128,
             interleaved=False, bf16=True),
        # one sequence, one new token: latency
        dict(name="attn_one", op="attn", S=1, lo=777, hi=777, n=1, Hq=32, Hkv=8, D=128, P=64, window=0),
        # a serving batch of ragged lengths
        dict(name="attn_decode", op="attn", S=128, lo=1, hi=8192, n=1, Hq=64, Hkv=8, D=128, P=64, window=0),
        # a few very long contexts: the work has to be split along the cache
        dict(name="attn_long", op="attn", S=4, lo=60000, hi=131071, n=1, Hq=32, Hkv=4, D=128, P=128, window=0),
        # four drafted tokens checked at once, a sliding window, wide heads, small pages
        dict(name="attn_draft", op="attn", S=32, lo=3, hi=16384, n=4, Hq=16, Hkv=2, D=256, P=32, window=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "append", "attn", "attn"])
    if op == "route":
        n_group = rng.choice([1, 1, 4, 8])
        per = rng.choice([8, 12, 16, 31, 32]) if n_group > 1 else rng.choice([8, 33, 60, 64, 128, 160, 256, 384])
        topk_group = rng.randint((n_group + 1) // 2, n_group)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log(rng, 1, 16384), E=n_group * per, k=rng.randint(1, 8), score=score,
                    bias=score == "sigmoid" and rng.random() < 0.7, n_group=n_group, topk_group=topk_group,
                    group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]),
                    bf16=rng.random() < 0.5, pad=rng.choice([0.0, 0.0, 0.05]), train=rng.random() < 0.5)
    D = rng.choice([64, 128, 128, 256])
    P = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16])
    if op == "append":
        S = _log(rng, 1, 256)
        Hq = min(Hq, 64)
        most = max(1, min(8192, 100_000_000 // (S * (Hq + 2 * Hkv) * D)))
        hi = rng.choice([1, _log(rng, 1, most)])
        return dict(op=op, S=S, lo=rng.randint(1, hi), hi=hi, start=_log(rng, 1, 4096), Hq=Hq, Hkv=Hkv, D=D, P=P,
                    rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.5, bf16=rng.random() < 0.7)
    S = _log(rng, 1, 256)
    n = rng.choice([1, 1, 1, 2, 3, 4])
    most = max(16, min(131072, (400000 * 4 * 128) // (S * Hkv * D)))
    hi = _log(rng, 1, most)
    return dict(op=op, S=S, lo=rng.randint(1, hi), hi=hi, n=n, Hq=Hq, Hkv=Hkv, D=D, P=P,
                window=rng.choice([0, 0, 0, rng.randint(1, hi)]))


def _spread(count, lo, hi):
    """`count` lengths from lo to hi, the first hi: fixed by the case alone."""
    return [hi - int((hi - lo + 0.999) * ((i * 0.6180339887) % 1.0)) for i in range(count)]


def _starts(c):
    return _spread(c["S"], 0, c["start"])


def work(c):
    if c["op"] == "route":
        x = 2 if c["bf16"] else 4
        byt = c["T"] * c["E"] * x + c["T"] * c["k"] * 8 + (4 * c["E"] if c["bias"] else 0)
        flops = 8 * c["T"] * c["E"]
        if c["train"]:
            byt += c["T"] * c["k"] * 4 + c["T"] * c["E"] * x
            flops += 4 * c["T"] * c["E"]
        return dict(bytes=byt, flops=flops)
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "append":
        T, x = sum(_spread(c["S"], c["lo"], c["hi"])), 2 if c["bf16"] else 4
        byt = T * D * (2 * Hkv * (x + 1) + Hq * (x + 2)) + T * c["rot"] * 4
        return dict(bytes=byt, flops=T * D * (6 * Hkv + 3 * Hq))
    tokens = 0
    pairs = 0
    for ln in _spread(c["S"], c["lo"], c["hi"]):
        pos = [p for p in range(ln - c["n"], ln) if p >= 0]
        first = [max(0, p - c["window"] + 1) if c["window"] else 0 for p in pos]
        tokens += ln - min(first)
        pairs += sum(p - f + 1 for p, f in zip(pos, first))
    byt = tokens * Hkv * D * 2 + c["S"] * c["n"] * Hq * (D * 4 + 4)
    return dict(bytes=byt, flops=4 * pairs * Hq * D)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _codes(gen, shape, sigma):
    """E4M3 codes of normal values, made a slab at a time."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_((torch.randn(part.numel(), generator=gen, device=DEV) * sigma).clamp_(-448.0, 448.0))
    return out


def _pool(gen, c, lengths, room):
    """A page pool with sequences of the given lengths in random pages: codes,
    one power-of-two scale per (page, head), and the block table. The slots
    past a sequence's end hold what was left there: NaN codes."""
    P, H, D = c["P"], c["Hkv"], c["D"]
    width = max(1, max(-(-(n + r) // P) for n, r in zip(lengths, room)))
    pages = sum(-(-(n + r) // P) for n, r in zip(lengths, room)) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(len(lengths), width, dtype=torch.int32)
    at = 0
    host = order.cpu()
    for i, (n, r) in enumerate(zip(lengths, room)):
        w = -(-(n + r) // P)
        table[i, :w] = host[at:at + w]
        at += w
    table = table.to(DEV)
    pool = {"block_table": table}
    last = torch.tensor([max(0, n - 1) // P for n in lengths], device=DEV)
    page = table.gather(1, last[:, None])[:, 0].long()
    used = torch.tensor([n - (max(0, n - 1) // P) * P for n in lengths], device=DEV)
    stale = torch.arange(P, device=DEV)[None, :] >= used[:, None]
    for name in ("k", "v"):
        codes = _codes(gen, (pages, H, P, D), 96.0)
        raw = codes.view(torch.uint8)
        edge = raw[page]
        edge[stale[:, None, :, None].expand_as(edge)] = 0x7F
        raw[page] = edge
        pool[name + "_cache"] = codes
        pool[name + "_scale"] = torch.exp2(torch.randint(-8, -5, (pages, H), generator=gen, device=DEV).float())
    return pool


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1_000_003 + seed)
    s = {"case": c}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        x = torch.randn(T, E, generator=gen, device=DEV) * 1.5
        x[:, : max(1, E // 16)] += 1.0  # some experts are liked more
        padded = int(c["pad"] * T)
        if padded:
            x[T - padded:] = -math.inf
        s["logits"] = x.to(torch.bfloat16) if c["bf16"] else x
        s["bias"] = torch.randn(E, generator=gen, device=DEV) * 0.05 if c["bias"] else None
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        if c["train"]:
            s["grad"] = torch.randn(T, k, generator=gen, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    D, Hq, Hkv, P, S = c["D"], c["Hq"], c["Hkv"], c["P"], c["S"]
    if c["op"] == "append":
        new, starts = _spread(S, c["lo"], c["hi"]), _starts(c)
        s.update(_pool(gen, c, starts, new))
        T = sum(new)
        dt = torch.bfloat16 if c["bf16"] else torch.float32
        s["k"] = (torch.randn(T, Hkv, D, generator=gen, device=DEV) * 1.5).to(dt)
        s["v"] = torch.randn(T, Hkv, D, generator=gen, device=DEV).to(dt)
        s["q"] = torch.randn(T, Hq, D, generator=gen, device=DEV).to(dt)
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["start"] = _i32(starts)
        s["cu"] = _i32([0] + [int(v) for v in np.cumsum(new)])
        positions = max(a + b for a, b in zip(starts, new)) + 1
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        ang = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * freq[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        return s
    lens = _spread(S, c["lo"], c["hi"])
    s.update(_pool(gen, c, lens, [0] * S))
    s["seq_lens"] = _i32(lens)
    s["q"] = torch.randn(S, c["n"], Hq, D, generator=gen, device=DEV).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(S, c["n"], Hq, dtype=torch.float32, device=DEV)
    s["workspace"] = torch.empty(SCRATCH_F32, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------

def run(s):
    return {"route": _route, "append": _append, "attn": _attn}[s["case"]["op"]](s)


def _route(s):
    c = s["case"]
    if own:
        import moe_grouped_gemm_x128_amd as mg

        mg.moe_route_topk(s["logits"], s["idx"], s["weights"], bias=s["bias"], score=c["score"], n_group=c["n_group"],
                          topk_group=c["topk_group"], group_top=c["group_top"], renormalize=c["renorm"],
                          scale=c["scale"])
        out = {"idx": s["idx"], "weights": s["weights"]}
        if c["train"]:
            mg.moe_route_topk_bwd(s["logits"], s["idx"], s["grad"], s["dlogits"], score=c["score"],
                                  renormalize=c["renorm"], scale=c["scale"])
            out["dlogits"] = s["dlogits"]
        return out
    x = s["logits"].float()
    T, E = x.shape
    top = x.max(dim=1, keepdim=True).values
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
        choice = p if s["bias"] is None else p + s["bias"]
    else:
        choice = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
        p = choice / choice.sum(dim=1, keepdim=True).clamp_min(1e-30)
    choice = torch.where(x > -math.inf, choice, -math.inf)
    if c["n_group"] > 1:
        per = choice.view(T, c["n_group"], E // c["n_group"])
        best = per.sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(dim=2)
        order = best.sort(dim=1, descending=True, stable=True).indices
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order[:, :c["topk_group"]], True)
        choice = torch.where(kept[:, :, None], per, -math.inf).view(T, E)
    got = choice.sort(dim=1, descending=True, stable=True)
    at = got.indices[:, :c["k"]]
    chosen = got.values[:, :c["k"]] > -math.inf
    z = torch.where(chosen, p.gather(1, at), 0.0)
    if not c["renorm"]:
        w = c["scale"] * z
    elif c["score"] == "sigmoid":
        total = z.sum(dim=1, keepdim=True) + 1e-20
        w = c["scale"] * (z / total)
    else:
        xs = torch.where(chosen, x.gather(1, at), -math.inf)
        m = xs.max(dim=1, keepdim=True).values
        e = torch.where(chosen, torch.exp(xs - torch.where(m > -math.inf, m, 0.0)), 0.0)
        w = c["scale"] * (e / e.sum(dim=1, keepdim=True).clamp_min(1e-30))
    out = {"idx": torch.where(chosen, at, -1).to(torch.int32), "weights": w}
    if c["train"]:
        g = torch.where(chosen, s["grad"], 0.0)
        if c["renorm"] and c["score"] == "softmax":
            dx = torch.zeros_like(x).scatter_(1, at, w * (g - (g * w).sum(dim=1, keepdim=True) / c["scale"]))
        else:
            dz = c["scale"] * g
            if c["renorm"]:
                dz = c["scale"] * (g - (g * z).sum(dim=1, keepdim=True) / total) / total
            ds = torch.zeros_like(x).scatter_(1, at, torch.where(chosen, dz, 0.0))
            if c["score"] == "sigmoid":
                dx = ds * (p * (1.0 - p))
            else:
                dx = p * (ds - (ds * p).sum(dim=1, keepdim=True))
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _rotate(x, table, interleaved):
    rot = table.shape[1]
    cos, sin = table[:, None, :rot // 2], table[:, None, rot // 2:]
    if interleaved:
        a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2)
    else:
        a, b = x[:, :, :rot // 2], x[:, :, rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)
    return torch.cat([y, x[:, :, rot:]], dim=2)


def _append(s):
    c = s["case"]
    result = {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    if own:
        import moe_grouped_gemm_x128_amd as mg

        mg.kv_append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                         s["cu"], s["start"], cos_sin=s["cos_sin"], q=s["q"], q_out=s["q_out"],
                         interleaved=c["interleaved"])
        return {**result, "q_out": s["q_out"]}
    P = c["P"]
    cu, start = s["cu"].long(), s["start"].long()
    t = torch.arange(s["k"].shape[0], device=DEV)
    seq = (t[:, None] >= cu[None, 1:]).sum(dim=1)
    pos = start[seq] + t - cu[seq]
    page, slot = s["block_table"][seq, pos // P].long(), pos % P
    table = s["cos_sin"][pos]
    # the page in which each sequence goes on, and how many older tokens it holds
    grows = (start % P > 0) & (cu[1:] > cu[:-1])
    edge = s["block_table"].gather(1, (start // P).clamp_max(s["block_table"].shape[1] - 1)[:, None])[:, 0].long()
    edge, old = edge[grows], (start % P)[grows]
    older = torch.arange(P, device=DEV)[None, None, :, None] < old[:, None, None, None]
    for name in ("k", "v"):
        y = s[name].float()
        if name == "k":
            y = _rotate(y, table, c["interleaved"])
        codes, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        pages, H = scale.shape
        amax = torch.full((pages, H), -1.0, device=DEV).scatter_reduce_(
            0, page[:, None].expand(-1, H), y.abs().amax(dim=2), "amax")
        need = amax.clamp_min(1e-4) / 448.0
        need = ((need.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32)
        floor = torch.zeros_like(scale)
        floor[edge] = scale[edge]
        now = torch.where(amax >= 0.0, torch.maximum(need, floor), scale)
        was = codes[edge]
        again = was.view(torch.float8_e4m3fn).float() * (scale[edge] / now[edge])[:, :, None, None]
        again = again.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[edge] = torch.where(older, again, was)
        q = (y / now[page][:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[page, :, slot] = q
        scale.copy_(now)
    q = _rotate(s["q"].float(), table, c["interleaved"])
    return {**result, "q_out": q.to(torch.bfloat16)}


def _attn(s):
    c = s["case"]
    S, n, Hq, Hkv, D, P = (c[x] for x in ("S", "n", "Hq", "Hkv", "D", "P"))
    scale = D ** -0.5
    if own:
        import moe_grouped_gemm_x128_amd as mg

        mg.paged_attention_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                               s["seq_lens"], s["out"], scale, workspace=s["workspace"], lse=s["lse"],
                               window=c["window"])
        return {"out": s["out"], "lse": s["lse"]}
    table = s["block_table"].long()
    L = table.shape[1] * P
    lens = s["seq_lens"].long()
    at = torch.arange(L, device=DEV)
    valid = (at[None, :] < lens[:, None])[:, None, :, None]

    def values(name):
        x = s[name + "_cache"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()  # [S, pages, H, P, D]
        x *= s[name + "_scale"][table][:, :, :, None, None]
        return torch.where(valid, x.transpose(1, 2).reshape(S, Hkv, L, D), 0.0)

    q = s["q"].float().view(S, n, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D)
    score = torch.matmul(q, values("k").transpose(2, 3)) * scale
    pos = (lens[:, None] - n + torch.arange(n, device=DEV)[None, :])[:, :, None]
    seen = at[None, None, :] <= pos
    if c["window"]:
        seen = seen & (at[None, None, :] > pos - c["window"])
    seen = seen[:, None, :, None, :].expand(S, 1, n, Hq // Hkv, L).reshape(S, 1, -1, L)
    score = torch.where(seen, score, -math.inf)
    m = score.max(dim=3, keepdim=True).values
    e = torch.exp(score - torch.where(m > -math.inf, m, 0.0))
    total = e.sum(dim=3, keepdim=True)
    o = torch.matmul(e, values("v")) / torch.where(total > 0.0, total, 1.0)
    lse = (m + torch.log(total))[:, :, :, 0]

    def back(x):
        x = x.view(S, Hkv, n, Hq // Hkv, -1).permute(0, 2, 1, 3, 4)
        return x.reshape(S, n, Hq, -1)

    return {"out": back(o).to(torch.bfloat16), "lse": back(lse)[..., 0]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    k, G = c["k"], c["n_group"]
    bias = np.zeros(E) if s["bias"] is None else s["bias"].double().cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        if c["score"] == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-x))
        else:
            m = x.max(axis=1)
            e = np.exp(x - np.where(np.isfinite(m), m, 0.0)[:, None])
            p = e / np.maximum(e.sum(axis=1), 1e-300)[:, None]
    w = np.zeros((T, k))
    idx = np.full((T, k), -1, dtype=np.int64)
    dx = np.zeros((T, E))
    g_in = s["grad"].double().cpu().numpy() if c["train"] else None
    choice = np.where(np.isfinite(x), p + bias, -np.inf)
    for t in range(T):
        ch = choice[t].copy()
        if G > 1:
            best = np.sort(ch.reshape(G, -1), axis=1)[:, ::-1][:, :c["group_top"]].sum(axis=1)
            out_of = np.argsort(-best, kind="stable")[c["topk_group"]:]
            ch.reshape(G, -1)[out_of] = -np.inf
        pick = np.argsort(-ch, kind="stable")[:k]
        pick = pick[ch[pick] > -np.inf]
        r = len(pick)
        if not r:
            continue
        z = p[t, pick]
        total = z.sum()
        idx[t, :r] = pick
        w[t, :r] = c["scale"] * (z / total if c["renorm"] else z)
        if c["train"]:
            g = g_in[t, :r]
            dz = c["scale"] * ((g - (g * z).sum() / total) / total if c["renorm"] else g)
            if c["score"] == "sigmoid":
                dx[t, pick] = dz * z * (1.0 - z)
            else:
                dx[t, pick] = z * dz
                dx[t] -= p[t] * (dz * z).sum()
    out = {"idx": torch.from_numpy(idx), "weights": torch.from_numpy(w)}
    if c["train"]:
        out["dlogits"] = torch.from_numpy(dx)
    return out


def _e4m3(x):
    """The nearest E4M3 values of float64 values up to 448, ties to even."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    unit = torch.exp2(e - 3)
    return torch.sign(x) * torch.round(a / unit) * unit


def _exact_append(s):
    c = s["case"]
    P, rot, H = c["P"], c["rot"], c["Hkv"]
    cu, start, table = s["cu"].tolist(), s["start"].tolist(), s["block_table"].tolist()
    T = s["k"].shape[0]
    at = torch.cat([torch.arange(start[i], start[i] + cu[i + 1] - cu[i]) for i in range(len(start))]).to(DEV)
    cos, sin = s["cos_sin"][at].double().split(rot // 2, dim=1)

    def turned(x):
        z = x.double().clone()
        if c["interleaved"]:
            first, second = slice(0, rot, 2), slice(1, rot, 2)
        else:
            first, second = slice(0, rot // 2), slice(rot // 2, rot)
        a, b = x.double()[..., first], x.double()[..., second]
        z[..., first] = a * cos[:, None] - b * sin[:, None]
        z[..., second] = b * cos[:, None] + a * sin[:, None]
        return z

    out = {"q_out": turned(s["q"])}
    for name, y in (("k", turned(s["k"])), ("v", s["v"].double())):
        codes = s[name + "_cache"].double()
        scale = s[name + "_scale"].double().clone()
        for i in range(len(start)):
            p = start[i]
            end = start[i] + cu[i + 1] - cu[i]
            while p < end:
                upto = min(end, (p // P + 1) * P)
                page, lo = table[i][p // P], p % P
                new = y[cu[i] + p - start[i]: cu[i] + upto - start[i]]  # [tokens, H, D]
                a = new.abs().amax(dim=(0, 2)).clamp_min(float(np.float32(1e-4)))
                man, ex = torch.frexp(a / 448.0)
                sc = torch.exp2((ex - (man == 0.5).to(ex.dtype)).double())
                if lo:
                    sc = torch.maximum(sc, scale[page])
                    codes[page, :, :lo] = _e4m3(codes[page, :, :lo] * (scale[page] / sc)[:, None, None])
                scale[page] = sc
                codes[page, :, lo:lo + upto - p] = _e4m3((new / sc[None, :, None]).clamp(-448, 448)).transpose(0, 1)
                p = upto
        out[name + "_cache"] = codes
        out[name + "_scale"] = scale
    return out


def _exact_attn(s):
    c = s["case"]
    if work(c)["flops"] > 2e11:
        return None
    S, n, Hq, Hkv, D, P = (c[x] for x in ("S", "n", "Hq", "Hkv", "D", "P"))
    out = torch.zeros(S, n, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((S, n, Hq), -math.inf, dtype=torch.float64, device=DEV)
    rep = Hq // Hkv
    for i, ln in enumerate(s["seq_lens"].tolist()):
        pages = s["block_table"][i, :-(-ln // P)].long()
        kv = {}
        for name in ("k", "v"):
            x = s[name + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
            x = x * s[name + "_scale"][pages].double()[:, :, None, None]
            kv[name] = x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :ln]
        for j in range(n):
            p = ln - n + j
            if p < 0:
                continue
            lo = max(0, p - c["window"] + 1) if c["window"] else 0
            qj = s["q"][i, j].double().view(Hkv, rep, D)
            score = torch.einsum("hrd,htd->hrt", qj, kv["k"][:, lo:p + 1]) / math.sqrt(D)
            lse[i, j] = torch.logsumexp(score, dim=2).reshape(Hq)
            out[i, j] = torch.einsum("hrt,htd->hrd", torch.softmax(score, dim=2), kv["v"][:, lo:p + 1]).reshape(Hq, D)
    return {"out": out, "lse": lse}
