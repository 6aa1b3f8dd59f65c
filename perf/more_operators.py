"""The operators of a mixture-of-experts block around and between its matrix
products, measured: the root-mean-square norm with the residual's addition and
FP8 output, the gated activation, both with their gradients, and the BF16
products grouped by expert with ragged sizes (forward, gradient of the inputs,
gradient of the weights).

Where `own` is false, `run` computes each operator with elementary torch
operations in 32 bits; where it is true, with the library's calls.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode stream: latency
        dict(name="norm_one", op="norm", T=1, heads=0, H=7168, f32=False, w_f32=False, residual=True, out="fp8",
             ue8m0=False, train=False),
        # a packed prompt batch in front of an FP8 GEMM, the residual stream carried on
        dict(name="norm_prompt", op="norm", T=16384, heads=0, H=7168, f32=False, w_f32=False, residual=True, out="fp8",
             ue8m0=False, train=False),
        # the norm of each query head, in the projection's output (a view of wider rows)
        dict(name="norm_heads", op="norm", T=4096, heads=32, H=128, f32=False, w_f32=True, residual=False, out="bf16",
             ue8m0=False, train=False),
        # a training step: forward and the gradients of the stream and the weight, an odd token count
        dict(name="norm_train", op="norm", T=8191, heads=0, H=4096, f32=False, w_f32=True, residual=True, out="bf16",
             ue8m0=False, train=True),
        # the experts' activation for one token: 8 of 32 experts hold one row
        dict(name="act_one", op="act", G=32, max_m=8, rows=8, I=2048, f32=False, out="fp8", ue8m0=True, weights=False,
             train=False),
        # ... for the decode batch of the framework's MoE workload (768 tokens, 8 choices, 32 experts)
        dict(name="act_decode", op="act", G=32, max_m=256, rows=6144, I=2048, f32=False, out="fp8", ue8m0=False,
             weights=False, train=False),
        # a training step's activation over the routed rows, weighted by the router, with its gradients
        dict(name="act_train", op="act", G=0, max_m=0, rows=32749, I=2048, f32=False, out="bf16", ue8m0=False,
             weights=True, train=True),
        # one token's 8 rows among 32 experts: whole weights read for a row or two
        dict(name="grouped_one", op="nt", G=32, M=8, N=4096, K=7168, f32=False, acc=False, empty=0.75),
        # the decode batch's down projection: 192 rows an expert on average, uneven
        dict(name="grouped_decode", op="nt", G=32, M=6144, N=7168, K=2048, f32=False, acc=False, empty=0.0),
        # a training step's gate and up projection
        dict(name="grouped_forward", op="nt", G=32, M=32768, N=4096, K=7168, f32=False, acc=False, empty=0.0),
        # its gradient with respect to the routed rows, an odd number of them
        dict(name="grouped_dx", op="nn", G=32, M=32749, N=7168, K=4096, f32=False, acc=False, empty=0.0),
        # the down projection's weight gradient in FP32, two experts without a token
        dict(name="grouped_dw", op="tn", G=32, M=32749, N=2048, K=7168, f32=True, acc=False, empty=0.06),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "act", "act", "nt", "nn", "tn"])
    if op == "norm":
        heads = rng.choice([0, 0, 0, 1, 5, 8, 32])
        H = rng.choice([64, 128, 256]) if heads else rng.choice(
            [_log(rng, 64, 16384), 512, 1024, 2048, 4096, 5120, 7168, 8192, 16384])
        T = _log(rng, 1, max(1, min(16384, 100_000_000 // (H * max(1, heads)))))
        train = rng.random() < 0.4
        out = "bf16" if train else rng.choice(["fp8", "fp8", "bf16"])
        # (a power-of-two scale jumps at its border: few enough blocks that none lies on it)
        return dict(op=op, T=T, heads=heads, H=H, f32=rng.random() < 0.25, w_f32=rng.random() < 0.5,
                    residual=rng.random() < 0.7, out=out,
                    ue8m0=out == "fp8" and T * max(1, heads) * H < 1_000_000 and rng.random() < 0.5, train=train)
    if op == "act":
        I = rng.choice([_log(rng, 64, 8192), 512, 768, 1024, 2048, 4096])
        G = rng.choice([0, 0, 8, 32, 64])
        rows = _log(rng, 1, max(1, min(32768, 70_000_000 // I)))
        train = G == 0 and rng.random() < 0.5
        out = "bf16" if train else rng.choice(["fp8", "fp8", "bf16"])
        return dict(op=op, G=G, max_m=0 if G == 0 else -(-rows * 2 // G) + rng.randint(0, 40), rows=rows, I=I,
                    f32=rng.random() < 0.2, out=out, ue8m0=out == "fp8" and rows * I < 1_000_000 and rng.random() < 0.5,
                    weights=G == 0 and rng.random() < 0.5, train=train)
    G = rng.choice([1, 4, 8, 16, 32, 60, 64, 128])
    N = rng.choice([_log(rng, 32, 7168), 512, 1024, 1536, 2048, 4096, 7168])
    K = 64 * _log(rng, 1, 112)
    if op == "tn":
        K = rng.choice([K, _log(rng, 32, 7168)])
    most = 500_000_000 // (N * K)  # weights of at most 500 million elements
    G = max(1, min(G, most))
    M = _log(rng, 1, max(1, min(32768, 800_000_000_000 // (N * K))))
    return dict(op=op, G=G, M=M, N=N, K=K, f32=rng.random() < (0.7 if op == "tn" else 0.2), acc=rng.random() < 0.3,
                empty=rng.choice([0.0, 0.0, 0.1, 0.5]))


def _sizes(G, rows, empty=0.0, cap=None):
    """Rows of each of G groups, `rows` in all: uneven, a share of the groups
    empty, none above `cap`; fixed by its arguments alone."""
    share = [0.25 + 1.5 * ((i * 0.6180339887 + 0.3) % 1.0) for i in range(G)]
    hollow = min(G - 1, int(empty * G))
    for i in range(hollow):
        share[(i * G) // hollow + (G // hollow) // 2] = 0.0
    total = sum(share)
    out, at = [], 0.0
    for s in share:
        last, at = at, at + s * rows / total
        out.append(int(at + 0.5) - int(last + 0.5))
    out[max(range(G), key=lambda i: share[i])] += rows - sum(out)
    if cap is not None:
        over = 0
        for i in range(G):
            over += max(0, out[i] - cap)
            out[i] = min(out[i], cap)
        for i in range(G):
            more = min(over, cap - out[i])
            out[i] += more
            over -= more
    return out


def work(c):
    if c["op"] == "norm":
        x = 4 if c["f32"] else 2
        rows, H = c["T"] * max(1, c["heads"]), c["H"]
        byt = rows * H * (x * (3 if c["residual"] else 1) + (1 if c["out"] == "fp8" else 2))
        if c["out"] == "fp8":
            byt += rows * -(-H // 128) * 4
        flops = 6 * rows * H
        if c["train"]:
            byt += rows * H * (2 + x + (x if c["residual"] else 0) + x) + 4 * H
            flops += 12 * rows * H
        return dict(bytes=byt + H * (4 if c["w_f32"] else 2), flops=flops)
    if c["op"] == "act":
        x, n = 4 if c["f32"] else 2, c["rows"] * c["I"]
        byt = n * (2 * x + (1 if c["out"] == "fp8" else 2)) + (4 * c["rows"] if c["weights"] else 0)
        if c["out"] == "fp8":
            byt += c["rows"] * -(-c["I"] // 128) * 4
        if c["train"]:
            byt += n * (2 * x + 2 + 2 * x) + (4 * c["rows"] if c["weights"] else 0)
        return dict(bytes=byt, flops=(20 if c["train"] else 8) * n)
    G, M, N, K = c["G"], c["M"], c["N"], c["K"]
    used = sum(1 for s in _sizes(G, M, c["empty"]) if s)
    o = 4 if c["f32"] else 2
    if c["op"] == "tn":
        byt = 2 * M * (N + K) + G * N * K * o * (2 if c["acc"] else 1)
    else:
        byt = 2 * M * K + 2 * used * N * K + M * N * o * (2 if c["acc"] else 1)
    return dict(bytes=byt, flops=2 * M * N * K)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _rows(gen, shape, dtype, sigma=1.0):
    """Normal values in rows that start on 16 bytes (a view of wider rows where the width is odd)."""
    wide = torch.empty(*shape[:-1], -(-shape[-1] // 8) * 8, dtype=dtype, device=DEV)
    flat = wide.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV) * sigma)
    return wide[..., :shape[-1]]


def _room(shape, dtype):
    return torch.zeros(*shape[:-1], -(-shape[-1] // 8) * 8, dtype=dtype, device=DEV)[..., :shape[-1]]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2_000_003 + seed)
    s = {"case": c}
    bf = torch.bfloat16
    dt = torch.float32 if c["f32"] else bf
    if c["op"] == "norm":
        T, H, heads = c["T"], c["H"], c["heads"]
        shape = (T, heads, H) if heads else (T, H)
        if heads:  # the query heads of a projection that holds keys and values too
            s["x"] = _rows(gen, (T, heads + 2, H), dt, 1.5)[:, :heads]
        else:
            s["x"] = _rows(gen, shape, dt, 0.7)
        s["weight"] = 1.0 + torch.randn(H, generator=gen, device=DEV) * 0.2
        if not c["w_f32"]:
            s["weight"] = s["weight"].to(bf)
        # a stream that grew over the layers, a few of its channels far more than the others
        s["residual"] = None
        if c["residual"]:
            s["residual"] = _rows(gen, shape, dt, 3.0)
            s["residual"][..., :: max(1, H // 5)] *= 20.0
        s["h"] = _room(shape, dt) if c["residual"] else None
        s["y"] = s["q"] = s["sf"] = None
        if c["out"] == "fp8":
            s["q"] = _room(shape, torch.uint8).view(torch.float8_e4m3fn)
            s["sf"] = torch.zeros(*shape[:-1], -(-H // 128), device=DEV)
        else:
            s["y"] = _room(shape, bf)
        if c["train"]:
            s["grad_y"] = _rows(gen, shape, bf, 1e-2)
            s["grad_h"] = _rows(gen, shape, dt, 1e-2) if c["residual"] else None
            s["grad_x"] = _room(shape, dt)
            s["grad_weight"] = torch.zeros(H, device=DEV)
            # what the library asks for at most, a row of partial sums for each workgroup
            s["workspace"] = torch.empty(1024 * H, device=DEV)
        return s
    if c["op"] == "act":
        G, I = c["G"], c["I"]
        shape = (G, c["max_m"], 2 * I) if G else (c["rows"], 2 * I)
        s["x"] = _rows(gen, shape, dt, 1.5)
        s["masked_m"] = None
        if G:
            s["masked_m"] = _i32(_sizes(G, c["rows"], 0.1, c["max_m"]))
        s["weights"] = torch.rand(c["rows"], generator=gen, device=DEV) if c["weights"] else None
        s["y"] = s["q"] = s["sf"] = None
        out = shape[:-1] + (I,)
        if c["out"] == "fp8":
            s["q"] = _room(out, torch.uint8).view(torch.float8_e4m3fn)
            s["sf"] = torch.zeros(*out[:-1], -(-I // 128), device=DEV)
        else:
            s["y"] = _room(out, bf)
        if c["train"]:
            s["grad_y"] = _rows(gen, out, bf, 1e-2)
            s["grad_x"] = _room(shape, dt)
            s["grad_weights"] = torch.zeros(c["rows"], device=DEV) if c["weights"] else None
        return s
    G, M, N, K = c["G"], c["M"], c["N"], c["K"]
    sizes = _sizes(G, M, c["empty"])
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    s["offsets"] = _i32(at)
    s["longest"] = max(sizes)
    if c["op"] == "tn":  # tokens' activations and the gradients behind them
        s["a"] = _rows(gen, (M, N), bf)
        s["b"] = _rows(gen, (M, K), bf, 0.1)
        out = (G, N, K)
    else:
        s["a"] = _rows(gen, (M, K), bf)
        s["b"] = _rows(gen, (G, N, K) if c["op"] == "nt" else (G, K, N), bf, K ** -0.5)
        out = (M, N)
    s["c"] = _rows(gen, out, dt) if c["acc"] else None
    s["d"] = _room(out, dt)
    return s


# ---------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------

def run(s):
    return {"norm": _norm, "act": _act}.get(s["case"]["op"], _grouped)(s)


def _cast(y, ue8m0):
    """The FP8 cast of 1x128 blocks: codes and scales."""
    H = y.shape[-1]
    blocks = -(-H // 128)
    z = torch.nn.functional.pad(y, (0, blocks * 128 - H)).unflatten(-1, (blocks, 128))
    sf = z.abs().amax(dim=-1).clamp_min(1e-4) / 448.0
    if ue8m0:
        sf = ((sf.view(torch.int32) + 0x7FFFFF) & 0x7F800000).view(torch.float32)
    q = (z / sf[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.flatten(-2)[..., :H], sf


def _norm(s):
    c = s["case"]
    if own:
        import moe_grouped_gemm_x128_amd as mg

        mg.rms_norm(s["x"], s["weight"], y=s["y"], q=s["q"], sf=s["sf"], residual=s["residual"], h=s["h"], eps=EPS,
                    use_ue8m0=c["ue8m0"])
        out = {n: s[n] for n in ("y", "q", "sf", "h") if s[n] is not None}
        if c["train"]:
            mg.rms_norm_bwd(s["grad_y"], s["h"] if c["residual"] else s["x"], s["weight"], s["grad_x"],
                            grad_weight=s["grad_weight"], workspace=s["workspace"], grad_h=s["grad_h"], eps=EPS)
            out.update(grad_x=s["grad_x"], grad_weight=s["grad_weight"])
        return out
    x = s["x"]
    if c["residual"]:
        x = (x.float() + s["residual"].float()).to(x.dtype)
    h, w = x.float(), s["weight"].float()
    r = 1.0 / torch.sqrt((h * h).mean(dim=-1, keepdim=True) + EPS)
    hat = h * r
    y = hat * w
    out = {}
    if c["out"] == "fp8":
        out["q"], out["sf"] = _cast(y, c["ue8m0"])
    else:
        out["y"] = y.to(torch.bfloat16)
    if c["residual"]:
        out["h"] = x
    if c["train"]:
        dy = s["grad_y"].float()
        g = dy * w
        dx = r * (g - hat * (g * hat).mean(dim=-1, keepdim=True))
        if c["residual"]:
            dx = dx + s["grad_h"].float()
        out["grad_x"] = dx.to(s["grad_x"].dtype)
        out["grad_weight"] = (dy * hat).flatten(0, -2).sum(dim=0)
    return out


def _act(s):
    c = s["case"]
    if own:
        import moe_grouped_gemm_x128_amd as mg

        mg.swiglu(s["x"], y=s["y"], q=s["q"], sf=s["sf"], masked_m=s["masked_m"], row_weights=s["weights"],
                  use_ue8m0=c["ue8m0"])
        out = {n: s[n] for n in ("y", "q", "sf") if s[n] is not None}
        if c["train"]:
            mg.swiglu_bwd(s["x"], s["grad_y"], s["grad_x"], row_weights=s["weights"],
                          grad_row_weights=s["grad_weights"])
            out["grad_x"] = s["grad_x"]
            if c["weights"]:
                out["grad_weights"] = s["grad_weights"]
        return out
    I = c["I"]
    gate, up = s["x"][..., :I].float(), s["x"][..., I:].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    z = gate * sig * up
    w = s["weights"][:, None] if c["weights"] else 1.0
    y = z * w
    out = {}
    if c["out"] == "fp8":
        q, sf = _cast(y, c["ue8m0"])
        if c["G"]:  # rows past a group's own stay as they were
            live = (torch.arange(c["max_m"], device=DEV)[None, :] < s["masked_m"][:, None])[:, :, None]
            q = torch.where(live, q.contiguous().view(torch.uint8), s["q"].contiguous().view(torch.uint8))
            q, sf = q.view(torch.float8_e4m3fn), torch.where(live, sf, s["sf"])
        out["q"], out["sf"] = q, sf
    else:
        y = y.to(torch.bfloat16)
        if c["G"]:
            live = (torch.arange(c["max_m"], device=DEV)[None, :] < s["masked_m"][:, None])[:, :, None]
            y = torch.where(live, y, s["y"])
        out["y"] = y
    if c["train"]:
        dy = s["grad_y"].float()
        dz = dy * w
        dgate = dz * up * sig * (1.0 + gate * (1.0 - sig))
        out["grad_x"] = torch.cat([dgate, dz * gate * sig], dim=-1).to(s["grad_x"].dtype)
        if c["weights"]:
            out["grad_weights"] = (dy * z).sum(dim=-1)
    return out


def _grouped(s):
    c = s["case"]
    if own:
        import moe_grouped_gemm_x128_amd as mg

        call = {"nt": mg.m_grouped_bf16_gemm_nt_ragged, "nn": mg.m_grouped_bf16_gemm_nn_ragged,
                "tn": mg.k_grouped_bf16_gemm_tn}[c["op"]]
        call(s["a"], s["b"], s["d"], s["offsets"], c=s["c"])
        return {"d": s["d"]}
    # the rows of each group side by side, padded with zeros to the longest
    first, last = s["offsets"][:-1].long()[:, None], s["offsets"][1:].long()[:, None]
    row = first + torch.arange(max(1, s["longest"]), device=DEV)[None, :]
    live = row < last
    row = row.clamp_max(c["M"] - 1)

    def padded(x):
        return torch.where(live[:, :, None], x[row].float(), 0.0)

    a = padded(s["a"])
    if c["op"] == "tn":
        d = torch.matmul(a.transpose(1, 2).contiguous(), padded(s["b"]))
        if c["acc"]:
            d = d + s["c"].float()
        return {"d": d.to(s["d"].dtype)}
    b = s["b"].float()
    d = torch.matmul(a, b.transpose(1, 2).contiguous() if c["op"] == "nt" else b)
    # back to their rows; the padding goes to one that is dropped
    back = torch.zeros(c["M"] + 1, c["N"], device=DEV)
    back[torch.where(live, row, c["M"]).flatten()] = d.flatten(0, 1)
    d = back[:c["M"]]
    if c["acc"]:
        d = d + s["c"].float()
    return {"d": d.to(s["d"].dtype)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "act": _exact_act}.get(case["op"], _exact_grouped)(s)


def _exact_cast(y, ue8m0):
    """Scales of 1x128 blocks, and the nearest E4M3 values (ties to even) of y over its scale."""
    H = y.shape[-1]
    sf = torch.stack([p.abs().amax(dim=-1) for p in y.split(128, dim=-1)], dim=-1)
    sf = sf.clamp_min(1e-4) / 448.0
    if ue8m0:
        man, ex = torch.frexp(sf)
        sf = torch.ldexp(torch.ones_like(sf), ex - (man == 0.5).to(ex.dtype))
    v = (y / sf.repeat_interleave(128, dim=-1)[..., :H]).clamp(-448.0, 448.0)
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / unit) * unit, sf


def _exact_norm(s):
    c = s["case"]
    h = s["x"].double()
    out = {}
    if c["residual"]:
        h = (h + s["residual"].double()).to(s["x"].dtype)  # the stream is held in its own type
        out["h"] = h.double()
        h = h.double()
    w = s["weight"].double()
    r = (h.square().mean(dim=-1, keepdim=True) + EPS) ** -0.5
    y = h * r * w
    if c["out"] == "fp8":
        out["q"], out["sf"] = _exact_cast(y, c["ue8m0"])
    else:
        out["y"] = y
    if c["train"]:
        dy = s["grad_y"].double()
        mean = (dy * w * h).mean(dim=-1, keepdim=True)
        dx = r * dy * w - h * r ** 3 * mean
        if c["residual"]:
            dx += s["grad_h"].double()
        out["grad_x"] = dx
        out["grad_weight"] = (dy * h * r).reshape(-1, c["H"]).sum(dim=0)
    return out


def _exact_act(s):
    c = s["case"]
    g, u = s["x"].double().split(c["I"], dim=-1)
    sig = torch.sigmoid(g)
    w = torch.ones(g.shape[:-1], dtype=torch.float64, device=DEV) if s["weights"] is None else s["weights"].double()
    y = w[..., None] * g * sig * u
    dead = None
    if c["G"]:
        dead = torch.arange(c["max_m"], device=DEV) >= s["masked_m"][:, None]
    out = {}
    if c["out"] == "fp8":
        out["q"], out["sf"] = _exact_cast(y, c["ue8m0"])
    else:
        out["y"] = y
    if dead is not None:
        for v in out.values():
            v[dead] = 0.0
    if c["train"]:
        dy = s["grad_y"].double()
        dg = w[:, None] * dy * u * (sig + g * sig * torch.sigmoid(-g))
        du = w[:, None] * dy * g * sig
        out["grad_x"] = torch.cat([dg, du], dim=-1)
        if c["weights"]:
            out["grad_weights"] = torch.einsum("ri,ri->r", dy, g * sig * u)
    return out


def _exact_grouped(s):
    c = s["case"]
    at = s["offsets"].tolist()
    d = torch.zeros(s["d"].shape, dtype=torch.float64, device=DEV)
    for g in range(c["G"]):
        rows = slice(at[g], at[g + 1])
        a = s["a"][rows].double()
        if c["op"] == "tn":
            d[g] = a.t().contiguous() @ s["b"][rows].double()
        elif c["op"] == "nt":
            d[rows] = a @ s["b"][g].double().t().contiguous()
        else:
            d[rows] = a @ s["b"][g].double()
    if c["acc"]:
        d += s["c"].double()
    return {"d": d}
