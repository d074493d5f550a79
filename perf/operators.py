"""The recurrent layer's operators as measured cases: short causal convolution,
selective state space scan, rotary positions and the delta rule's single-token
step, each over the sizes it meets in prompts, streams and single tokens.

``run`` computes a case in plain torch operations (``own`` false) or with the
library's calls (``own`` true); ``exact`` computes it in 64 bits from the
definition.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a 480p video block's value channels (2 clips of 21 latent frames, 16 heads of 128), bf16
        {"name": "conv_video", "op": "conv", "B": 2, "T": 32760, "D": 2048, "width": 4, "dtype": "bf16",
         "silu": True, "bias": True, "packed": False, "halves": False},
        # prompts of different lengths in one packed batch, an odd channel count, fp32, three taps
        {"name": "conv_ragged", "op": "conv", "B": 41, "T": 20011, "D": 1001, "width": 3, "dtype": "f32",
         "silu": False, "bias": False, "packed": True, "halves": False},
        # one new token for each of 64 running sequences
        {"name": "conv_step", "op": "conv_step", "B": 64, "slots": 80, "D": 2048, "width": 4, "dtype": "bf16",
         "silu": True, "bias": True},
        # one prompt, x and the gate as the two halves of one projection's rows
        {"name": "ssm_prompt", "op": "ssm", "B": 1, "T": 2048, "D": 4096, "N": 16, "G": 1, "dtype": "bf16",
         "gate": True, "skip": True, "packed": False, "carry": False},
        # a few equal prompts in fp32, odd channel count, a wider state, the state carried in
        {"name": "ssm_batch", "op": "ssm", "B": 4, "T": 777, "D": 1000, "N": 32, "G": 1, "dtype": "f32",
         "gate": False, "skip": True, "packed": False, "carry": True},
        # prompts of different lengths in one packed batch, B and C shared by groups of channels
        {"name": "ssm_ragged", "op": "ssm", "B": 24, "T": 9001, "D": 2048, "N": 16, "G": 2, "dtype": "bf16",
         "gate": True, "skip": True, "packed": True, "carry": True},
        # one long document
        {"name": "ssm_long", "op": "ssm", "B": 1, "T": 32768, "D": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "gate": True, "skip": True, "packed": False, "carry": False},
        # one new token for each of 128 running sequences, states picked out of a pool
        {"name": "ssm_step", "op": "ssm_step", "B": 128, "slots": 150, "D": 4096, "N": 16, "G": 1, "dtype": "bf16",
         "gate": True, "skip": True},
        # half layout over part of the head, far positions with scaled frequencies, q and k slices of fused rows
        {"name": "rotary_part", "op": "rotary", "B": 1, "T": 4096, "Hq": 32, "Hk": 8, "d": 128, "rot": 64,
         "interleaved": False, "axes": 1, "far": 1000000, "dtype": "bf16"},
        # interleaved over the whole head with (frame, row, column) positions of 480p video
        {"name": "rotary_video", "op": "rotary", "B": 2, "T": 32760, "Hq": 16, "Hk": 16, "d": 128, "rot": 128,
         "interleaved": True, "axes": 3, "far": 0, "dtype": "bf16"},
        # one stream's next token (12 heads of 128): the smallest call
        {"name": "delta_step_one", "op": "delta_step", "B": 1, "slots": 1, "H": 12, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # the next token of 128 running sequences, states picked out of a pool
        {"name": "delta_step_many", "op": "delta_step", "B": 128, "slots": 144, "H": 16, "dk": 128, "dv": 128,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "ssm", "ssm", "ssm_step", "rotary", "delta_step"])
    dtype = rng.choice(["bf16", "f32"])
    es = SIZE[dtype]
    if op == "conv":
        D, rows = _log(rng, 64, 8192), _log(rng, 1, 65536)
        rows = max(1, min(rows, 2 ** 28 // (D * es)))
        packed = rng.random() < 0.5
        B = _log(rng, 1, 64) if packed else rng.choice([1, 2, 3, 8])
        return {"op": op, "B": B, "T": rows if packed else max(1, rows // B), "D": D, "width": rng.choice([2, 3, 4]),
                "dtype": dtype, "silu": rng.random() < 0.7, "bias": rng.random() < 0.5, "packed": packed,
                "halves": rng.random() < 0.5}
    if op == "conv_step":
        B = _log(rng, 1, 512)
        return {"op": op, "B": B, "slots": B + rng.randrange(0, 40), "D": _log(rng, 64, 8192),
                "width": rng.choice([2, 3, 4]), "dtype": dtype, "silu": rng.random() < 0.7, "bias": rng.random() < 0.5}
    if op in ("ssm", "ssm_step"):
        N, G = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
        D = _log(rng, 64, 4096)
        if G > 1:
            D = max(1, D // (64 * G)) * 64 * G
        more = {"D": D, "N": N, "G": G, "dtype": dtype, "gate": rng.random() < 0.7, "skip": rng.random() < 0.8}
        if op == "ssm_step":
            B = _log(rng, 1, 128)
            return {"op": op, "B": B, "slots": B + rng.randrange(0, 20), **more}
        rows = max(1, min(_log(rng, 1, 32768), 2 ** 29 // (D * N * (es // 2))))
        packed = rng.random() < 0.5
        B = _log(rng, 1, 32) if packed else rng.choice([1, 2, 3, 8])
        return {"op": op, "B": B, "T": rows if packed else max(1, rows // B), **more, "packed": packed,
                "carry": rng.random() < 0.5}
    if op == "rotary":
        d = rng.choice([64, 96, 128, 192, 256])
        rot = 2 * rng.randrange(4, d // 2 + 1)
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4])
        tokens = max(1, min(_log(rng, 1, 65536), 2 ** 28 // ((Hq + Hk) * d * es)))
        B = rng.choice([1, 2, 5])
        return {"op": op, "B": B, "T": max(1, tokens // B), "Hq": Hq, "Hk": Hk, "d": d, "rot": rot,
                "interleaved": rng.random() < 0.5, "axes": rng.choice([1, 3]), "far": rng.choice([0, 100000, 1000000]),
                "dtype": dtype}
    B = _log(rng, 1, 128)
    return {"op": op, "B": B, "slots": B + rng.randrange(0, 16), "H": _log(rng, 1, 16), "dk": rng.choice([64, 128]),
            "dv": rng.choice([64, 128]), "dtype": dtype}


# ---- inputs -----------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _offsets(case, seed):
    """Row offsets [B + 1] of the sequences: equal ones, or of random lengths with (from three on) one of a single
    token and (from five on) an empty one."""
    B, T = case["B"], case["T"]
    if not case["packed"]:
        return [i * T for i in range(B + 1)]
    r = random.Random(seed * 1009 + 17)
    fixed = [1] * (B >= 3) + [0] * (B >= 5)
    if T < len(fixed):
        fixed = []
    cuts = sorted(r.randrange(0, T - sum(fixed) + 1) for _ in range(B - len(fixed) - 1))
    ends = [0] + cuts + [T - sum(fixed)]
    lens = [b - a for a, b in zip(ends[:-1], ends[1:])] + fixed
    r.shuffle(lens)
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _frequencies(rot, far):
    """Rotary frequencies in 64 bits (base 10000). For far positions the low ones are slowed by 16 and the ones between
    are blended over their wavelengths, with the length scale that goes with it."""
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not far:
        return f, 1.0
    out = []
    for w in f:
        turns = 65536 * w / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
        out.append(w * (keep + (1.0 - keep) / 16.0))
    return out, 0.1 * math.log(16.0) + 1.0


def _sections(pairs, axes):
    return [pairs - (axes - 1) * (pairs // axes)] + [pairs // axes] * (axes - 1)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 13)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, device=dev).normal_(mean, std, generator=g).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.empty(shape, device=dev).uniform_(lo, hi, generator=g)

    def slots_of():
        r = random.Random(seed * 31 + 5)
        return torch.tensor(r.sample(range(case["slots"]), case["B"]), dtype=torch.int32, device=dev)

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("conv", "conv_step"):
        D, W, B = case["D"], case["width"], case["B"]
        s["weight"] = normal(D, W, std=W ** -0.5, dtype=torch.float32)
        s["bias"] = normal(D, std=0.1, dtype=torch.float32) if case["bias"] else None
        if op == "conv_step":
            s["x"], s["index"] = normal(B, D), slots_of()
            s["state"] = normal(case["slots"], W - 1, D)
            return s
        lead = (case["T"],) if case["packed"] else (B, case["T"])
        # the convolved channels are a projection's own rows, or the first half of wider ones
        s["x"] = normal(*lead, 2 * D)[..., :D] if case["halves"] else normal(*lead, D)
        s["state"] = normal(B, W - 1, D)
        s["offsets"] = torch.tensor(_offsets(case, seed), dtype=torch.int32, device=dev)
    elif op in ("ssm", "ssm_step"):
        D, N, G, B = case["D"], case["N"], case["G"], case["B"]
        lead = (B,) if op == "ssm_step" else (case["T"],) if case["packed"] else (B, case["T"])
        xz = normal(*lead, 2 * D)
        s["x"], s["z"] = xz[..., :D], xz[..., D:] if case["gate"] else None
        bc = normal(*lead, 2 * G * N)
        s["B"], s["C"] = bc[..., : G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
        s["dt"] = normal(*lead, D, std=0.5)
        steps = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = steps + torch.log(-torch.expm1(-steps))  # softplus(dt_bias) = steps
        s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(normal(D, N, std=0.1, dtype=torch.float32))
        s["D"] = normal(D, std=0.1, mean=1.0, dtype=torch.float32) if case["skip"] else None
        if op == "ssm_step":
            s["index"], s["state"] = slots_of(), normal(case["slots"], D, N, std=0.3, dtype=torch.float32)
            return s
        s["state"] = normal(B, D, N, std=0.3, dtype=torch.float32) if case["carry"] else None
        s["offsets"] = torch.tensor(_offsets(case, seed), dtype=torch.int32, device=dev)
    elif op == "rotary":
        B, T, d = case["B"], case["T"], case["d"]
        f, s["scale"] = _frequencies(case["rot"], case["far"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
        s["sections"] = _sections(case["rot"] // 2, case["axes"])
        rows = normal(B, T, case["Hq"] + 2 * case["Hk"], d)  # q, k and v of one projection
        s["q"], s["k"] = rows[:, :, : case["Hq"]], rows[:, :, case["Hq"]: case["Hq"] + case["Hk"]]
        t = torch.arange(T, device=dev)
        if case["axes"] == 3:  # (frame, row, column) on a 30 x 52 grid
            pos = torch.stack([t // 1560 + seed % 7, t // 52 % 30, t % 52])[:, None].expand(3, B, T)
        else:
            pos = (t + torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=dev))[None]
        s["pos"] = pos.to(torch.int64).contiguous()
    else:
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        s["q"], s["k"], s["v"] = normal(B, H, dk), normal(B, H, dk), normal(B, H, dv)
        s["log_alpha"] = -torch.nn.functional.softplus(normal(B, H, dtype=torch.float32) - 3.0)
        s["beta"] = torch.sigmoid(normal(B, H, dtype=torch.float32))
        s["index"], s["state"] = slots_of(), normal(case["slots"], H, dv, dk, std=0.1, dtype=torch.float32)
    return s


# ---- one pass ---------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return OWN[op](s)
    return PLAIN[op](s)


def _sequence_of_rows(off, rows):
    """For each packed row its sequence and its place in it."""
    r = torch.arange(rows, device=off.device)
    seq = torch.searchsorted(off, r.to(off.dtype), right=True) - 1
    return seq, r - off[seq]


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def plain_conv(s):
    c = s["case"]
    W, D, B = c["width"], c["D"], c["B"]
    x = s["x"].reshape(-1, D).float()
    rows = x.shape[0]
    ext = torch.cat([s["state"].float().reshape(-1, D), x])  # B * (W - 1) carried rows, then the new ones
    off = s["offsets"]
    seq, place = _sequence_of_rows(off, rows)
    back = torch.arange(W - 1, -1, -1, device=x.device)  # taps, oldest first
    at = place[:, None] - back
    src = torch.where(at >= 0, B * (W - 1) + off[seq].long()[:, None] + at, seq[:, None] * (W - 1) + (W - 1) + at)
    y = s["bias"].expand(rows, D) if s["bias"] is not None else torch.zeros((rows, D), device=x.device)
    y = y.clone()
    for j in range(W):
        y += ext[src[:, j]] * s["weight"][:, j]
    if c["silu"]:
        y = _silu(y)
    # the carried rows: the last W - 1 of (state, x)
    n = (off[1:] - off[:-1]).long()
    at = n[:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
    src = torch.where(at >= 0, B * (W - 1) + off[:-1].long()[:, None] + at,
                      torch.arange(B, device=x.device)[:, None] * (W - 1) + (W - 1) + at)
    dt = s["x"].dtype
    return y.to(dt).view(s["x"].shape), ext[src].to(dt)


def plain_conv_step(s):
    i = s["index"].long()
    win = torch.cat([s["state"][i], s["x"][:, None]], 1)  # [B, W, D]
    y = (win.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["case"]["silu"]:
        y = _silu(y)
    s["state"][i] = win[:, 1:]
    return y.to(s["x"].dtype), s["state"]


def plain_ssm(s):
    c = s["case"]
    D, N, G, B = c["D"], c["N"], c["G"], c["B"]
    x = s["x"].reshape(-1, D).float()
    rows = x.shape[0]
    off = s["offsets"].long()
    dt = _softplus(s["dt"].reshape(-1, D).float() + s["dt_bias"])
    a = torch.exp(dt[..., None] * s["A"])  # [rows, D, N]
    Bm = s["B"].reshape(rows, G, 1, N).float()
    h = ((dt * x).view(rows, G, D // G, 1) * Bm).view(rows, D, N)
    seq, place = _sequence_of_rows(s["offsets"], rows)
    first = (place == 0)[:, None, None]
    if s["state"] is not None:
        h = torch.where(first, torch.addcmul(h, a, s["state"][seq]), h)
    a = torch.where(first, 0.0, a)  # nothing reaches over a sequence's start
    # h_t = a_t h_{t-1} + b_t by doubling: after each step (a, h) span twice as many rows
    d = 1
    while d < rows:
        nh = h.clone()
        nh[d:] += a[d:] * h[:-d]
        h = nh
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    y = (h.view(rows, G, D // G, N) * s["C"].reshape(rows, G, 1, N).float()).sum(-1).reshape(rows, D)
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].reshape(-1, D).float())
    n = off[1:] - off[:-1]
    last = h[(off[1:] - 1).clamp(min=0)]
    start = s["state"] if s["state"] is not None else torch.zeros_like(last)
    return y.to(s["x"].dtype).view(s["x"].shape), torch.where((n > 0)[:, None, None], last, start)


def plain_ssm_step(s):
    c = s["case"]
    D, N, G, B = c["D"], c["N"], c["G"], c["B"]
    i = s["index"].long()
    x = s["x"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    b = ((dt * x).view(B, G, D // G, 1) * s["B"].float()[:, :, None]).view(B, D, N)
    h = torch.exp(dt[..., None] * s["A"]) * s["state"][i] + b
    y = (h.view(B, G, D // G, N) * s["C"].float()[:, :, None]).sum(-1).reshape(B, D)
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][i] = h
    return y.to(s["x"].dtype), s["state"]


def plain_rotary(s):
    c = s["case"]
    pairs = c["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(len(s["sections"])), torch.tensor(s["sections"])).to(s["pos"].device)
    theta = s["pos"][axis].movedim(0, -1).double() * s["freq"]  # [B, T, pairs]
    cos = (torch.cos(theta).float() * s["scale"])[:, :, None]
    sin = (torch.sin(theta).float() * s["scale"])[:, :, None]

    def turn(x):
        head, tail = x[..., : c["rot"]].float(), x[..., c["rot"]:]
        u, v = (head[..., 0::2], head[..., 1::2]) if c["interleaved"] else (head[..., :pairs], head[..., pairs:])
        a, b = u * cos - v * sin, v * cos + u * sin
        y = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([y.to(x.dtype), tail], -1)

    return turn(s["q"]), turn(s["k"])


def plain_delta_step(s):
    i = s["index"].long()

    def unit(x):
        x = x.float()
        return x / torch.clamp((x * x).sum(-1, keepdim=True).sqrt(), min=1e-6)

    q, k, v = unit(s["q"]), unit(s["k"]), s["v"].float()
    S = torch.exp(s["log_alpha"])[..., None, None] * s["state"][i]
    r = (S * k[:, :, None]).sum(-1)
    S = S + (s["beta"][..., None] * (v - r))[..., None] * k[:, :, None]
    s["state"][i] = S
    return (S * q[:, :, None]).sum(-1), s["state"]


PLAIN = {"conv": plain_conv, "conv_step": plain_conv_step, "ssm": plain_ssm, "ssm_step": plain_ssm_step,
         "rotary": plain_rotary, "delta_step": plain_delta_step}


def own_conv(s):
    import gated_delta_rule_scan_amd as gdn

    c = s["case"]
    return gdn.causal_conv(s["x"], s["weight"], s["bias"], state_in=s["state"],
                           activation="silu" if c["silu"] else "none", seq_offsets=s["offsets"] if c["packed"] else None)


def own_conv_step(s):
    import gated_delta_rule_scan_amd as gdn

    y = gdn.causal_conv_step(s["x"], s["weight"], s["bias"], state=s["state"], state_index=s["index"],
                             activation="silu" if s["case"]["silu"] else "none")
    return y, s["state"]


def own_ssm(s):
    import gated_delta_rule_scan_amd as gdn

    return gdn.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                              dt_softplus=True, state_in=s["state"],
                              seq_offsets=s["offsets"] if s["case"]["packed"] else None)


def own_ssm_step(s):
    import gated_delta_rule_scan_amd as gdn

    y = gdn.selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                           dt_softplus=True, state=s["state"], state_index=s["index"])
    return y, s["state"]


def own_rotary(s):
    import gated_delta_rule_scan_amd as gdn

    c = s["case"]
    return gdn.rotary(s["q"], s["k"], s["freq"], s["pos"], interleaved=c["interleaved"], sections=s["sections"],
                      scale=s["scale"])


def own_delta_step(s):
    import gated_delta_rule_scan_amd as gdn

    o = gdn.delta_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], state=s["state"], state_index=s["index"])
    return o, s["state"]


OWN = {"conv": own_conv, "conv_step": own_conv_step, "ssm": own_ssm, "ssm_step": own_ssm_step, "rotary": own_rotary,
       "delta_step": own_delta_step}


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op, es = case["op"], SIZE[case["dtype"]]
    if op in ("conv", "conv_step"):
        B, D, W = case["B"], case["D"], case["width"]
        rows = B if op == "conv_step" else case["T"] if case["packed"] else B * case["T"]
        return {"bytes": 2 * rows * D * es + 2 * B * (W - 1) * D * es + D * W * 4 + (D * 4 if case["bias"] else 0),
                "flops": rows * D * (2 * W + (4 if case["silu"] else 0))}
    if op in ("ssm", "ssm_step"):
        B, D, N, G = case["B"], case["D"], case["N"], case["G"]
        rows = B if op == "ssm_step" else case["T"] if case["packed"] else B * case["T"]
        per_row = (3 + (1 if case["gate"] else 0)) * D * es + 2 * G * N * es
        states = (1 if op == "ssm" and not case["carry"] else 2) * B * D * N * 4
        # per state entry: decay product, exp, input product, update, readout
        return {"bytes": rows * per_row + states + D * N * 4 + 2 * D * 4, "flops": rows * D * (7 * N + 12)}
    if op == "rotary":
        tokens = case["B"] * case["T"]
        vals = tokens * (case["Hq"] + case["Hk"]) * case["d"]
        return {"bytes": 2 * vals * es + 8 * case["axes"] * tokens,
                "flops": 3 * tokens * (case["Hq"] + case["Hk"]) * case["rot"] + 8 * tokens * case["rot"]}
    B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
    return {"bytes": 2 * B * H * dk * dv * 4 + B * H * ((2 * dk + dv) * es + dv * 4 + 8), "flops": 7 * B * H * dk * dv}


# ---- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def _spans(s):
    off = s["offsets"].tolist()
    return list(zip(off[:-1], off[1:]))


def exact_conv(s):
    c = s["case"]
    W, D = c["width"], c["D"]
    x, st, w = s["x"].reshape(-1, D).double(), s["state"].double(), s["weight"].double()
    y, left = torch.zeros_like(x), torch.zeros_like(st)
    for b, (lo, hi) in enumerate(_spans(s)):
        seen = torch.cat([st[b], x[lo:hi]])
        left[b] = seen[hi - lo:]
        y[lo:hi] = sum(w[:, j] * seen[j: j + hi - lo] for j in range(W))
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["silu"]:
        y = y * torch.sigmoid(y)
    return y.view(s["x"].shape), left


def exact_conv_step(s):
    st, w = s["state"].double(), s["weight"].double()
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device=st.device)
    for b, i in enumerate(s["index"].tolist()):
        seen = torch.cat([st[i], s["x"][b: b + 1].double()])
        y[b] = (w * seen.t()).sum(1)
        st[i] = seen[1:]
    if s["bias"] is not None:
        y += s["bias"].double()
    return (y * torch.sigmoid(y) if s["case"]["silu"] else y), st


def _exact_token(h, x, dt, Bm, Cm, s):
    """One token of every sequence: x, dt [S, D], Bm, Cm [S, G, N], h [S, D, N], all in 64 bits."""
    per = s["case"]["D"] // s["case"]["G"]
    dt = torch.logaddexp(dt + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device=dt.device))
    h = torch.exp(dt[..., None] * s["A"].double()) * h + (dt * x)[..., None] * Bm.repeat_interleave(per, 1)
    return h, (h * Cm.repeat_interleave(per, 1)).sum(-1)


def exact_ssm(s):
    c = s["case"]
    D, N, G = c["D"], c["N"], c["G"]
    spans = _spans(s)
    longest = max(hi - lo for lo, hi in spans)
    dev = s["x"].device
    flat = {k: s[k].reshape(-1, *s[k].shape[-(1 if k in ("x", "dt") else 2):]) for k in ("x", "dt", "B", "C")}
    h = torch.zeros((len(spans), D, N), dtype=torch.float64, device=dev) if s["state"] is None else s["state"].double()
    y = torch.zeros((flat["x"].shape[0], D), dtype=torch.float64, device=dev)
    lo = torch.tensor([a for a, _ in spans], device=dev)
    n = torch.tensor([b - a for a, b in spans], device=dev)
    order = sorted(range(len(spans)), key=lambda i: spans[i][0] - spans[i][1])  # longest first
    lens = [spans[i][1] - spans[i][0] for i in order]
    lo, h = lo[order], h[order]
    live = len(order)
    for t in range(longest):
        while live and lens[live - 1] <= t:
            live -= 1
        at = lo[:live] + t
        h[:live], y[at] = _exact_token(h[:live], flat["x"][at].double(), flat["dt"][at].double(),
                                       flat["B"][at].double(), flat["C"][at].double(), s)
    end = torch.empty_like(h)
    end[order] = h
    if s["D"] is not None:
        y += s["D"].double() * flat["x"].double()
    if s["z"] is not None:
        z = s["z"].reshape(-1, D).double()
        y *= z * torch.sigmoid(z)
    return y.view(s["x"].shape), end


def exact_ssm_step(s):
    i = s["index"].long()
    st = s["state"].double()
    h, y = _exact_token(st[i], s["x"].double(), s["dt"].double(), s["B"].double(), s["C"].double(), s)
    st[i] = h
    if s["D"] is not None:
        y = y + s["D"].double() * s["x"].double()
    if s["z"] is not None:
        y = y * s["z"].double() * torch.sigmoid(s["z"].double())
    return y, st


def exact_rotary(s):
    c = s["case"]
    pairs, lo, angles = c["rot"] // 2, 0, []
    for n, p in zip(s["sections"], s["pos"]):
        angles.append(p.double()[..., None] * s["freq"][lo: lo + n])
        lo += n
    turn = torch.polar(torch.full((), float(s["scale"]), dtype=torch.float64, device=s["q"].device), torch.cat(angles, -1))

    def of(x):
        y = x.double()
        if c["interleaved"]:
            z = torch.view_as_complex(y[..., : c["rot"]].unflatten(-1, (pairs, 2)).contiguous()) * turn[:, :, None]
            y[..., : c["rot"]] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :pairs], y[..., pairs: c["rot"]]) * turn[:, :, None]
            y[..., :pairs], y[..., pairs: c["rot"]] = z.real, z.imag
        return y

    return of(s["q"]), of(s["k"])


def exact_delta_step(s):
    st = s["state"].double()
    i = s["index"].long()
    q, k = (x.double() / torch.linalg.vector_norm(x.double(), dim=-1, keepdim=True).clamp(min=1e-6) for x in (s["q"], s["k"]))
    kk = k[..., :, None] * k[..., None, :]
    keep = torch.eye(kk.shape[-1], dtype=torch.float64, device=kk.device) - s["beta"].double()[..., None, None] * kk
    S = torch.exp(s["log_alpha"].double())[..., None, None] * (st[i] @ keep.contiguous())
    S = S + s["beta"].double()[..., None, None] * (s["v"].double()[..., :, None] * k[..., None, :])
    st[i] = S
    return (S @ q[..., None]).squeeze(-1), st


EXACT = {"conv": exact_conv, "conv_step": exact_conv_step, "ssm": exact_ssm, "ssm_step": exact_ssm_step,
         "rotary": exact_rotary, "delta_step": exact_delta_step}
