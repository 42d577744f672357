"""The gated linear recurrence and the 8-bit activation checkpoints: cases, plain forms and exact values.

For gates r and g, input x and a decay parameter lam per channel, in scan order k = 0, 1, ... of a sequence
(its last valid position first, or its first one first):

    log a_k = -8 softplus(lam) sigmoid(r_k)
    h_k     = a_k h_{k-1} + sqrt(1 - a_k^2) sigmoid(g_k) x_k          y_k = h_k

An 8-bit checkpoint of a row holds, for each 64 channels, e4m3 values of x / 2^k and the exponent k, the
smallest (from -126 on) with max|x| <= 448 * 2^k.

Operators ("op" of a case):
    step     one position of each sequence on a running state (serving)
    scan     whole sequences from a state to a state (prefill, a generation block)
    train    the forward that saves the states its gradient needs, and the gradient
    train8   the same, with x, r and g kept between the two in 8 bits instead of 16 or 32
    act8     a hook's hidden state into an 8-bit checkpoint and back
"""
import math

import torch

own = False

TILE = 64        # positions between two saved states
GROUP = 64       # channels that share one scale
DECAY = 8.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one token for each request of a small serving batch: launch latency
        {"name": "step-b8", "op": "step", "B": 8, "L": 1, "E": 4096, "dtype": "bf16", "forward": True, "ragged": False},
        # one token for each of many requests, some of them finished (length 0)
        {"name": "step-b256-ragged", "op": "step", "B": 256, "L": 1, "E": 4096, "dtype": "bf16", "forward": True, "ragged": True},
        # the generation block of cached parallel decoding: 8 requests of 128 positions, right to left
        {"name": "scan-block-b8-l128", "op": "scan", "B": 8, "L": 128, "E": 4096, "dtype": "bf16", "forward": False, "ragged": False},
        # one prompt: few channels, so the position axis has to be split
        {"name": "scan-b1-l2048", "op": "scan", "B": 1, "L": 2048, "E": 4096, "dtype": "bf16", "forward": False, "ragged": False},
        # the prefill of the serving setup
        {"name": "scan-b8-l4096", "op": "scan", "B": 8, "L": 4096, "E": 4096, "dtype": "bf16", "forward": False, "ragged": False},
        # many short requests of all lengths, odd width, true fp32
        {"name": "scan-ragged-fp32", "op": "scan", "B": 61, "L": 512, "E": 1037, "dtype": "fp32", "forward": True, "ragged": True},
        # a training step at the serving setup's width
        {"name": "train-b8-l4096", "op": "train", "B": 8, "L": 4096, "E": 4096, "dtype": "bf16", "forward": False, "ragged": False},
        # a small fp32 training step of ragged sequences and an odd width
        {"name": "train-ragged-fp32", "op": "train", "B": 5, "L": 777, "E": 515, "dtype": "fp32", "forward": True, "ragged": True},
        # the training step with its activations kept in 8 bits
        {"name": "train8-b8-l4096", "op": "train8", "B": 8, "L": 4096, "E": 4096, "dtype": "bf16", "forward": False, "ragged": False},
        # the same on ragged sequences in fp32
        {"name": "train8-ragged-fp32", "op": "train8", "B": 16, "L": 1000, "E": 1024, "dtype": "fp32", "forward": False, "ragged": True},
        # a hook's hidden state at the training setup's size
        {"name": "act8-b8-l4096", "op": "act8", "B": 8, "L": 4096, "E": 2048, "dtype": "bf16", "forward": False, "ragged": False},
        # hidden states of ragged sequences, odd width, fp32
        {"name": "act8-ragged-fp32", "op": "act8", "B": 32, "L": 300, "E": 1037, "dtype": "fp32", "forward": False, "ragged": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))

    op = rng.choice(("step", "scan", "scan", "train", "train8", "act8"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    E = spread(64, 4096)
    if rng.random() < 0.6:
        E = max(64, E // 64 * 64)
    B = spread(1, 256)
    L = 1 if op == "step" else spread(1, 8192)
    most = (1 << 26) if dtype == "fp32" else (1 << 27)
    L = max(1, min(L, most // (B * E)))
    return {"op": op, "B": B, "L": L, "E": E, "dtype": dtype, "forward": rng.random() < 0.5, "ragged": rng.random() < 0.4}


def lengths_of(case):
    """Lengths spread evenly over 0 ... L, the longest first; prepare() shuffles them."""
    B, L = case["B"], case["L"]
    return [L - L * b // max(1, B - 1) for b in range(B)] if case["ragged"] else [L] * B


def make(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, L, E, t = case["B"], case["L"], case["E"], DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device=dev) * std + mean

    s = {"case": case, "x": normal(B * L, E).to(t)}
    lens = torch.tensor(lengths_of(case), dtype=torch.int32, device=dev)
    s["lengths"] = lens[torch.randperm(B, generator=gen, device=dev)].contiguous() if case["ragged"] else None
    if case["op"] == "act8":
        s["out"] = torch.zeros(B * L, E, dtype=t, device=dev)
        return s
    s["r"], s["g"] = normal(B * L, E).to(t), normal(B * L, E).to(t)
    # a^8 uniform in [0.9, 0.999] where the gate is open: memories of 10 to 1000 positions
    sp = -torch.log(0.9 + 0.099 * torch.rand(E, generator=gen, device=dev, dtype=torch.float64)) / DECAY
    s["lam"] = (sp + torch.log(-torch.expm1(-sp))).float()
    s["h0"] = normal(B, E, std=0.5)
    s["y"] = torch.zeros(B * L, E, dtype=t, device=dev)
    s["h_last"] = torch.zeros(B, E, device=dev)
    if case["op"] in ("train", "train8"):
        s["dy"] = normal(B * L, E, std=0.1).to(t)
        s["dh_last"] = normal(B, E, std=0.1)
    return s


def prepare(case, seed):
    return make(case, seed)


# ------------------------------------------------------------------ plain forms

def scan_rows(a, b):
    """h_k = a_k h_{k-1} + b_k along dimension 1 with h_{-1} = 0: pairs are joined, the half is solved, the rest filled in."""
    n = a.shape[1]
    if n == 1:
        return b
    m = n // 2 * 2
    odd = scan_rows(a[:, 1:m:2] * a[:, 0:m:2], a[:, 1:m:2] * b[:, 0:m:2] + b[:, 1:m:2])
    h = torch.empty_like(b)
    h[:, 1:m:2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, : (n - 1) // 2] + b[:, 2::2]
    return h


def scan_order(s):
    """Row index of scan position k of each sequence, [B, L], and which are valid. The same map leads back."""
    c = s["case"]
    k = torch.arange(c["L"], device="cuda").expand(c["B"], c["L"])
    n = torch.full((c["B"], 1), c["L"], device="cuda") if s["lengths"] is None else s["lengths"].long()[:, None]
    i = k if c["forward"] else n - 1 - k
    return (i.clamp(min=0) + torch.arange(c["B"], device="cuda")[:, None] * c["L"]), k < n


def coefficients(x, r, g, lam, valid):
    """a, beta, sigmoid(r), sigmoid(g) and b = beta sigmoid(g) x; a = 1 and b = 0 at positions that are not valid."""
    v = valid[:, :, None]
    sr, sg = torch.sigmoid(r), torch.sigmoid(g)
    rate = -DECAY * torch.log1p(torch.exp(lam))
    l = rate * sr
    beta = torch.sqrt(-torch.expm1(2 * l))
    a = torch.where(v, torch.exp(l), 1.0)
    return a, beta, sr, sg, torch.where(v, beta * sg * x, 0.0), l


def quantised(x):
    """What an 8-bit checkpoint of the rows x (fp32, [..., E]) stands for."""
    E = x.shape[-1]
    p = torch.zeros(*x.shape[:-1], -(-E // GROUP) * GROUP, device=x.device)
    p[..., :E] = x
    p = p.view(*x.shape[:-1], -1, GROUP)
    m, e = torch.frexp(p.abs().amax(-1, keepdim=True))            # max = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    up, down = ((127 + k) << 23).view(torch.float32), ((127 - k) << 23).view(torch.float32)   # 2^k and 2^-k
    return ((p * down).to(torch.float8_e4m3fn).float() * up).flatten(-2)[..., :E]


def plain_scan(s):
    c, t = s["case"], DTYPES[s["case"]["dtype"]]
    at, valid = scan_order(s)
    x, r, g = (s[n][at].float() for n in ("x", "r", "g"))
    a, beta, sr, sg, b, l = coefficients(x, r, g, s["lam"], valid)
    b[:, 0] += a[:, 0] * s["h0"]
    h = scan_rows(a, b)
    row = torch.where(valid[:, :, None], h, 0.0)
    back = row.view(-1, c["E"])[at] if not c["forward"] else row
    y = torch.where(valid[:, :, None], back.view(c["B"], c["L"], -1).to(t), s["y"].view(c["B"], c["L"], -1))
    return y.view(-1, c["E"]), h[:, -1], h


def plain_train(s):
    c, t = s["case"], DTYPES[s["case"]["dtype"]]
    B, L, E = c["B"], c["L"], c["E"]
    y, h_last, h = plain_scan(s)
    at, valid = scan_order(s)
    x, r, g = (s[n].float() for n in ("x", "r", "g"))
    if c["op"] == "train8":
        x, r, g = quantised(x), quantised(r), quantised(g)
    x, r, g = x[at], r[at], g[at]
    a, beta, sr, sg, b, l = coefficients(x, r, g, s["lam"], valid)
    before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)            # state that enters each position
    if c["op"] == "train8":                                         # recomputed from the state saved at each tile's start
        tiles = -(-L // TILE)
        ap, bp = torch.ones(B, tiles * TILE, E, device="cuda"), torch.zeros(B, tiles * TILE, E, device="cuda")
        ap[:, :L], bp[:, :L] = a, b
        bp[:, ::TILE] += ap[:, ::TILE] * before[:, ::TILE]
        inner = scan_rows(ap.view(B * tiles, TILE, E), bp.view(B * tiles, TILE, E)).view(B, -1, E)
        mid = torch.cat([s["h0"][:, None], inner[:, : L - 1]], 1)
        mid[:, ::TILE] = before[:, ::TILE]
        before = mid
    dy = torch.where(valid[:, :, None], s["dy"][at].float(), 0.0)
    dy[:, -1] += s["dh_last"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    G = scan_rows(after.flip(1), dy.flip(1)).flip(1)
    v = valid[:, :, None]
    dx = torch.where(v, G * beta * sg, 0.0)
    dg = torch.where(v, G * beta * x * sg * (1 - sg), 0.0)
    dl = a * G * before - G * sg * x * a * a / beta                 # through a and through beta
    dl = torch.where(v, dl, 0.0)
    dr = dl * l * (1 - sr)
    dlam = (dl * sr).sum((0, 1)) * -DECAY * torch.sigmoid(s["lam"])
    dh0 = a[:, 0] * G[:, 0]
    dx, dr, dg = ((d.view(-1, E)[at] * v if not c["forward"] else d).view(-1, E).to(t) for d in (dx, dr, dg))
    return {"y": y, "h_last": h_last, "dx": dx, "dr": dr, "dg": dg, "dlam": dlam, "dh0": dh0}


def plain_act8(s):
    c = s["case"]
    n = torch.full((c["B"], 1), c["L"], device="cuda") if s["lengths"] is None else s["lengths"].long()[:, None]
    valid = (torch.arange(c["L"], device="cuda")[None] < n).reshape(-1, 1)
    return torch.where(valid, quantised(s["x"].float()).to(s["x"].dtype), s["out"])


def plain(s):
    op = s["case"]["op"]
    if op == "act8":
        return plain_act8(s)
    if op in ("step", "scan"):
        y, h_last, _ = plain_scan(s)
        return {"y": y, "h_last": h_last}
    return plain_train(s)


# ------------------------------------------------------------------ the framework's calls

def kernels(s):
    from reverse_selective_ssm_b200 import binding as bd

    c = s["case"]
    op, B, L, E, t = c["op"], c["B"], c["L"], c["E"], DTYPES[c["dtype"]]
    if op == "act8":
        q, scales = bd.act8_pack(s["x"], B, L, lengths=s["lengths"])
        return bd.act8_unpack(q, scales, B, L, lengths=s["lengths"], out=s["out"])
    flags = (bd.R2L_FLAG_FORWARD_SCAN if c["forward"] else 0) | (bd.R2L_FLAG_ACT8 if op == "train8" else 0)
    dims = bd.gated_dims(E, t, flags)
    if op == "step":
        y = bd.gated_step(s["x"], s["r"], s["g"], s["lam"], dims, s["h0"], new_state=s["h_last"], y=s["y"], lengths=s["lengths"])
        return {"y": y, "h_last": s["h_last"]}
    if op == "scan":
        y, h_last = bd.gated_scan(s["x"], s["r"], s["g"], s["lam"], dims, B, L, h0=s["h0"], y=s["y"], h_last=s["h_last"], lengths=s["lengths"])
        return {"y": y, "h_last": h_last}
    y, h_last, saved = bd.gated_scan_train(s["x"], s["r"], s["g"], s["lam"], dims, B, L, h0=s["h0"], y=s["y"], h_last=s["h_last"], lengths=s["lengths"])
    kept = {} if op == "train8" else {"x": s["x"], "r": s["r"], "g": s["g"]}
    d = bd.gated_scan_backward(s["dy"], s["lam"], dims, B, L, saved, dh_last=s["dh_last"], lengths=s["lengths"], **kept)
    return {"y": y, "h_last": h_last, **d}


def run(state):
    return kernels(state) if own else plain(state)


def work(case):
    n, op, w = sum(lengths_of(case)) * case["E"], case["op"], BYTES[case["dtype"]]
    if op == "act8":
        return {"bytes": n * (2 * w + 1 + 1 / GROUP), "flops": 4 * n}
    ends = case["B"] * case["E"] * 4
    if op in ("step", "scan"):
        return {"bytes": n * 4 * w + 2 * ends + 4 * case["E"], "flops": 20 * n}
    padding = (case["B"] * case["L"] * case["E"] - n) * 3 * w         # rows of zero gradients
    return {"bytes": n * 8 * w + padding + 4 * ends + 8 * case["E"], "flops": 70 * n}


# ------------------------------------------------------------------ exact values

def exact(case, seed):
    """The definition in 64 bits, position by position. A position past the end of its sequence changes nothing."""
    s = make(case, seed)
    B, L, E, op = case["B"], case["L"], case["E"], case["op"]
    f8 = torch.float64
    n = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    live = torch.zeros(B, L, 1, dtype=torch.bool, device="cuda")
    for b in range(B):
        live[b, : n[b]] = True

    def two_to(k):
        return ((k.long() + 1023) << 52).view(f8)

    def eight(v):
        """Nearest e4m3 value of v / 2^k, ties to the even one, times 2^k."""
        out = torch.empty_like(v)
        for at in range(0, E, 64):
            p = v[..., at: at + 64]
            top = p.abs().amax(-1, keepdim=True)
            k = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=-126)
            k = torch.where(top > 448 * two_to(k), k + 1, torch.where(top <= 448 * two_to(k - 1), k - 1, k)).clamp(min=-126)
            u = p / two_to(k)
            grid = two_to(torch.floor(torch.log2(u.abs().clamp(min=1e-300))).clamp(min=-6) - 3)
            out[..., at: at + 64] = torch.round(u / grid) * grid * two_to(k)
        return out

    x = s["x"].to(f8).view(B, L, E)
    if op == "act8":
        return torch.where(live, eight(x), s["out"].to(f8).view(B, L, E)).view(B * L, E)

    def ordered(v):
        """Positions in scan order, and back again."""
        if case["forward"]:
            return v
        w = v.clone()
        for b in range(B):
            w[b, : n[b]] = v[b, : n[b]].flip(0)
        return w

    def gates(r, g):
        up, ug = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-g))
        return -8 * torch.nn.functional.softplus(s["lam"].to(f8)) * up, up, ug

    x, r, g = ordered(x), ordered(s["r"].to(f8).view(B, L, E)), ordered(s["g"].to(f8).view(B, L, E))
    h = s["h0"].to(f8)
    ys, start = torch.zeros(B, L, E, dtype=f8, device="cuda"), []
    for k in range(L):
        if k % 64 == 0:
            start.append(h)
        l, _, ug = gates(r[:, k], g[:, k])
        h = torch.where(live[:, k], torch.exp(l) * h + torch.sqrt(-torch.expm1(2 * l)) * ug * x[:, k], h)
        ys[:, k] = h
    y = torch.where(live, ordered(ys), s["y"].to(f8).view(B, L, E)).view(B * L, E)
    if op in ("step", "scan"):
        return {"y": y, "h_last": h}
    h_last = h
    if op == "train8":
        x, r, g = eight(x), eight(r), eight(g)
    dy = ordered(s["dy"].to(f8).view(B, L, E))
    dx, dr, dg = (torch.zeros(B, L, E, dtype=f8, device="cuda") for _ in range(3))
    rate = -8 * torch.nn.functional.softplus(s["lam"].to(f8))
    drate = torch.zeros(E, dtype=f8, device="cuda")
    D = s["dh_last"].to(f8)                                  # gradient of the state that leaves the position at hand
    for tile in reversed(range(len(start))):
        stop = min(L, tile * 64 + 64)
        h, enters = start[tile], []
        for k in range(tile * 64, stop):
            enters.append(h)
            l, _, ug = gates(r[:, k], g[:, k])
            h = torch.where(live[:, k], torch.exp(l) * h + torch.sqrt(-torch.expm1(2 * l)) * ug * x[:, k], h)
        for k in reversed(range(tile * 64, stop)):
            l, up, ug = gates(r[:, k], g[:, k])
            a, keep = torch.exp(l), torch.sqrt(-torch.expm1(2 * l))
            total = D + dy[:, k]
            dx[:, k] = torch.where(live[:, k], total * keep * ug, 0.0)
            dg[:, k] = torch.where(live[:, k], total * keep * x[:, k] * ug * (1 - ug), 0.0)
            dl = torch.where(live[:, k], total * (a * enters[k - tile * 64] - ug * x[:, k] * a * a / keep), 0.0)
            dr[:, k] = dl * rate * up * (1 - up)
            drate += (dl * up).sum(0)
            D = torch.where(live[:, k], total * a, D)
    dlam = drate * -8 / (1 + torch.exp(-s["lam"].to(f8)))
    dx, dr, dg = (ordered(v).view(B * L, E) for v in (dx, dr, dg))
    return {"y": y, "h_last": h_last, "dx": dx, "dr": dr, "dg": dg, "dlam": dlam, "dh0": D}
