"""What a hybrid model's layers run beside their recurrent scans, as measured cases: writing keys and values into a
paged cache (as they are or in 8 or 4 bits), reading them back, the attention of one new token over that cache, and
the seam between two blocks (norm, gate, residual, norm) with its gradients, each over the sizes it meets in streams,
batches and training.

``run`` computes a case in plain torch operations (``own`` false) or with the library's calls (``own`` true);
``exact`` computes it in 64 bits from the definition.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
# bytes of one cached row of d channels, scale bytes (one per 32 channels) included
ROW = {"bf16": lambda d: 2 * d, "f32": lambda d: 4 * d, "mxfp8": lambda d: d + d // 32, "mxfp4": lambda d: d // 2 + d // 32}


def listed():
    return [
        # one stream's next token over one latent frame of 480p video, 12 heads of 128: the smallest call
        {"name": "attend_stream", "op": "attend", "B": 1, "L": 1560, "Hq": 12, "Hk": 12, "d": 128, "page": 64,
         "window": 0, "sinks": 0, "format": "bf16", "dtype": "bf16"},
        # the next token of 64 running sequences of all lengths up to 8192, query heads shared by fours
        {"name": "attend_batch", "op": "attend", "B": 64, "L": 8192, "Hq": 32, "Hk": 8, "d": 128, "page": 16,
         "window": 0, "sinks": 0, "format": "bf16", "dtype": "bf16"},
        # one long document, the cache in 8 bits
        {"name": "attend_long", "op": "attend", "B": 1, "L": 131072, "Hq": 32, "Hk": 8, "d": 128, "page": 64,
         "window": 0, "sinks": 0, "format": "mxfp8", "dtype": "bf16"},
        # a rolling window behind a few first tokens, fp32, heads of 64
        {"name": "attend_window", "op": "attend", "B": 24, "L": 9001, "Hq": 16, "Hk": 4, "d": 64, "page": 32,
         "window": 777, "sinks": 16, "format": "f32", "dtype": "f32"},
        # one new token for each of 64 running sequences, k and v slices of a projection's rows
        {"name": "write_step", "op": "write", "B": 64, "T": 1, "L": 4096, "Hk": 8, "d": 128, "page": 16,
         "format": "bf16", "dtype": "bf16", "packed": False},
        # a 480p block's keys and values (2 clips of 21 latent frames, 16 heads of 128) into 8 bits
        {"name": "write_video", "op": "write", "B": 2, "T": 32760, "L": 32760, "Hk": 16, "d": 128, "page": 256,
         "format": "mxfp8", "dtype": "bf16", "packed": False},
        # the rolling window of 8 streams (3 latent frames) out of the cache, as the rows a scan takes
        {"name": "read_window", "op": "read", "B": 8, "T": 4680, "L": 9001, "Hk": 12, "d": 128, "page": 64,
         "format": "bf16", "dtype": "bf16", "packed": False},
        # sequences of different lengths out of a cache in 4 bits, as fp32 rows
        {"name": "read_ragged", "op": "read", "B": 41, "T": 20011, "L": 20011, "Hk": 8, "d": 64, "page": 32,
         "format": "mxfp4", "dtype": "f32", "packed": True},
        # the seam between two blocks for the tokens of a 480p block, a gate per clip, norms on both sides
        {"name": "seam_video", "op": "seam", "B": 2, "T": 32760, "D": 2048, "gate": "sequence", "post": True,
         "packed": False, "dtype": "bf16"},
        # the same for one new token of each of 64 sequences, a learned gate
        {"name": "seam_step", "op": "seam", "B": 64, "T": 1, "D": 4096, "gate": "channel", "post": False,
         "packed": False, "dtype": "bf16"},
        # its gradients over one clip
        {"name": "seam_back_video", "op": "seam_back", "B": 1, "T": 32760, "D": 2048, "gate": "sequence", "post": True,
         "packed": False, "dtype": "bf16"},
        # its gradients over packed sequences of different lengths, an odd channel count, fp32
        {"name": "seam_back_ragged", "op": "seam_back", "B": 41, "T": 20011, "D": 1001, "gate": "sequence", "post": False,
         "packed": True, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "read", "seam", "seam_back"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("attend", "write", "read"):
        d, Hk, page = rng.choice([64, 128, 128, 256]), _log(rng, 1, 16), rng.choice([16, 32, 64, 128, 256])
        form = rng.choice([dtype, "mxfp8", "mxfp4"])
        more = {"Hk": Hk, "d": d, "page": page, "format": form, "dtype": dtype}
        if op == "attend":
            B = _log(rng, 1, 128)
            L = min(_log(rng, 1, 131072), max(1, 2 ** 29 // (B * Hk * d * (2 if dtype == "f32" else 1))))
            window = _log(rng, 1, 8192) if rng.random() < 0.3 else 0
            return {"op": op, "B": B, "L": L, "Hq": Hk * rng.choice([1, 2, 4, 6, 8, 16]), "window": window,
                    "sinks": rng.randrange(0, 100) if window else 0, **more}
        rows = max(1, min(_log(rng, 1, 65536), 2 ** 27 // (Hk * d)))
        packed = rng.random() < 0.5
        B = _log(rng, 1, 64) if packed else rng.choice([1, 2, 3, 8, 64])
        T = rows if packed else max(1, rows // B)
        return {"op": op, "B": B, "T": T, "L": T + rng.randrange(0, 2000), "packed": packed, **more}
    D, rows = _log(rng, 64, 8192), _log(rng, 1, 65536)
    rows = max(1, min(rows, 2 ** (28 if op == "seam" else 27) // (D * SIZE[dtype])))
    packed = rng.random() < 0.4
    B = _log(rng, 1, 64) if packed else rng.choice([1, 2, 3, 8, 64])
    return {"op": op, "B": B, "T": rows if packed else max(1, rows // B), "D": D,
            "gate": rng.choice(["none", "channel", "sequence", "sequence"]), "post": rng.random() < 0.5, "packed": packed,
            "dtype": dtype}


# ---- inputs -----------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _lengths(case):
    """Cached tokens of each sequence: spread evenly up to the longest."""
    B, L = case["B"], case["L"]
    return [max(1, L * (i + 1) // B) for i in range(B)]


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


# A block of 32 channels in few bits: a power of two, the least with which the block's largest magnitude is in range
# (but not below 2^-110), as a byte (exponent + 127), and each channel over it, rounded to the nearest e4m3 or e2m1 value.

def _two_to(e):
    """2^e in fp32 from its bits (powers computed on a GPU may be a rounding off)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, form):
    """x [..., d] fp32 -> (codes: e4m3 [..., d], or e2m1 pairs, even channel low, [..., d / 2]; scale bytes [..., d / 32])."""
    top, room = (8, 0.875) if form == "mxfp8" else (2, 0.75)
    y = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(y.abs().amax(-1))
    e = torch.where(m == 0, -110, (e - 1 - top + (m > room).int()).clamp(min=-110))
    y = (y * _two_to(-e)[..., None]).flatten(-2)
    scales = (e + 127).to(torch.uint8)
    if form == "mxfp8":
        return y.to(torch.float8_e4m3fn), scales
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], scales


def _decode(codes, scales, form):
    """The values (fp32) that codes and scale bytes stand for."""
    if form == "mxfp8":
        v = codes.float()
    else:
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    return (v.unflatten(-1, (-1, 32)) * _two_to(scales.int() - 127)[..., None]).flatten(-2)


def _pool(values, form):
    return _encode(values.float(), form) if form in ("mxfp8", "mxfp4") else (values, None)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 29)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, device=dev, dtype=dtype).normal_(mean, std, generator=g)

    op, B = case["op"], case["B"]
    s = {"case": dict(case)}
    if op in ("attend", "write", "read"):
        Hk, d, page, form = case["Hk"], case["d"], case["page"], case["format"]
        off = _offsets(case, seed) if op != "attend" else None
        order = list(range(B))
        random.Random(seed * 31 + 5).shuffle(order)
        if op == "attend":
            lens = [_lengths(case)[i] for i in order]
        else:  # each sequence's rows go behind (or come from behind) what it holds before
            new = [b - a for a, b in zip(off[:-1], off[1:])]
            start = [min(case["L"] - n, order[i] * 37 % 501) for i, n in enumerate(new)]
            s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
            s["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
            lens = [a + n for a, n in zip(start, new)]
        used = [-(-n // page) for n in lens]
        width = max(max(used), 1)
        pages = sum(used) + 3
        perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = perm[at: at + n]
            at += n
        s["table"] = table
        # keys with a few strong channels, as projections have them
        strong = torch.exp(0.5 * normal(Hk, 1, d, dtype=torch.float32))
        k, ks = _pool((normal(pages, Hk, page, d) * strong).to(dt), form)
        v, vs = _pool(normal(pages, Hk, page, d), form)
        s["cache"] = (k, v, ks, vs)
        if op == "attend":
            s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
            s["q"] = normal(B, case["Hq"], d)
        elif op == "write":
            lead = (case["T"],) if case["packed"] else (B, case["T"])
            rows = normal(*lead, 3 * Hk, d)  # q, k and v of one projection
            s["k"], s["v"] = rows[..., Hk: 2 * Hk, :], rows[..., 2 * Hk:, :]
        return s
    D = case["D"]
    lead = (case["T"],) if case["packed"] else (B, case["T"])
    s["offsets"] = torch.tensor(_offsets(case, seed), dtype=torch.int32, device=dev)
    s["x"], s["y"] = normal(*lead, D, std=3.0), normal(*lead, D)
    s["weight"] = normal(D, std=0.1, mean=1.0, dtype=torch.float32)
    s["post"] = normal(D, std=0.1, mean=1.0, dtype=torch.float32) if case["post"] else None
    shape = {"none": None, "channel": (D,), "sequence": (B, D)}[case["gate"]]
    s["gate"] = normal(*shape, std=0.5, mean=0.5, dtype=torch.float32) if shape else None
    if op == "seam_back":
        s["dh"], s["dn"] = normal(*lead, D), normal(*lead, D)
    return s


# ---- one pass ---------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return OWN[op](s)
    return PLAIN[op](s)


EPS = 1e-6


def _rows_at(s):
    """For each new row its place in the pools: page and row in the page."""
    off, table = s["offsets"], s["table"]
    rows = s["case"]["T"] if s["case"]["packed"] else s["case"]["B"] * s["case"]["T"]
    r = torch.arange(rows, device=off.device)
    seq = torch.searchsorted(off, r.to(off.dtype), right=True) - 1
    pos = r - off[seq] + s["start"][seq]
    page = s["case"]["page"]
    return table[seq, pos // page].long(), pos % page


def _gather(pool, scales, at, form):
    """Rows [n, Hk, d] (fp32) of a pool."""
    page, row = at
    if scales is None:
        return pool[page, :, row].float()
    codes = pool.view(torch.uint8)[page, :, row]  # (indexing knows bytes)
    return _decode(codes.view(torch.float8_e4m3fn) if form == "mxfp8" else codes, scales[page, :, row], form)


def _shaped(rows, s):
    c = s["case"]
    return rows.to(DTYPES[c["dtype"]]).view(*((c["T"],) if c["packed"] else (c["B"], c["T"])), c["Hk"], c["d"])


def plain_attend(s):
    c = s["case"]
    B, Hk, d, page = c["B"], c["Hk"], c["d"], c["page"]
    table, lens = s["table"], s["lengths"]
    p = torch.arange(table.shape[1] * page, device=table.device)
    k, v, ks, vs = s["cache"]
    outs, lses = [], []
    group = max(1, 2 ** 28 // (p.numel() * Hk * d))  # sequences at once
    for b in range(0, B, group):
        t, n = table[b: b + group].long().clamp(min=0), lens[b: b + group, None]
        seen = p < n
        if c["window"]:
            seen &= (p >= n - c["window"]) | (p < c["sinks"])

        def rows(pool, scales):  # [b, Hk, tokens, d]
            if scales is None:
                x = pool[t].float()
            else:
                codes = pool.view(torch.uint8)[t]
                x = _decode(codes.view(torch.float8_e4m3fn) if c["format"] == "mxfp8" else codes, scales[t], c["format"])
            return x.transpose(1, 2).flatten(2, 3)

        q = s["q"][b: b + group].float().unflatten(1, (Hk, -1)) * d ** -0.5
        x = torch.matmul(q, rows(k, ks).transpose(-1, -2).contiguous())
        x = x.masked_fill(~seen[:, None, None], float("-inf"))
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1, keepdim=True)
        # (values behind a sequence's end may hold anything)
        y = torch.matmul(e, rows(v, vs).masked_fill(~seen[:, None, :, None], 0.0)) / z
        outs.append(y.flatten(1, 2))
        lses.append((m + torch.log(z)).flatten(1))
    return torch.cat(outs).to(s["q"].dtype), torch.cat(lses)


def plain_write(s):
    c = s["case"]
    at = _rows_at(s)
    for x, pool, scales in zip((s["k"], s["v"]), s["cache"][:2], s["cache"][2:]):
        x = x.reshape(-1, c["Hk"], c["d"])
        if scales is None:
            pool[at[0], :, at[1]] = x
        else:
            codes, sc = _encode(x.float(), c["format"])
            pool.view(torch.uint8)[at[0], :, at[1]] = codes.view(torch.uint8)
            scales[at[0], :, at[1]] = sc
    if c["format"] in DTYPES:
        return s["cache"][:2]
    return plain_read(s)  # what is in 8 or 4 bits, as the values it stands for


def plain_read(s):
    at = _rows_at(s)
    k, v, ks, vs = s["cache"]
    form = s["case"]["format"]
    return _shaped(_gather(k, ks, at, form), s), _shaped(_gather(v, vs, at, form), s)


def _per_row(gate, s):
    """The gate of every row: [rows, D], or [D]."""
    if gate is None or gate.dim() == 1:
        return gate
    rows = s["x"].numel() // s["case"]["D"]
    r = torch.arange(rows, device=gate.device, dtype=torch.int32)
    return gate[torch.searchsorted(s["offsets"], r, right=True) - 1]


def _seam(s):
    D = s["case"]["D"]
    x, y, gate = s["x"].reshape(-1, D).float(), s["y"].reshape(-1, D).float(), _per_row(s["gate"], s)
    ry = yhat = None
    u = y
    if s["post"] is not None:
        ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        yhat = y * ry
        u = yhat * s["post"]
    h = x + (u if gate is None else u * gate)
    rh = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    return gate, ry, yhat, u, h, rh


def plain_seam(s):
    *_, h, rh = _seam(s)
    dt, shape = s["x"].dtype, s["x"].shape
    return h.to(dt).view(shape), (h * rh * s["weight"]).to(dt).view(shape)


def plain_seam_back(s):
    c = s["case"]
    D, B = c["D"], c["B"]
    gate, ry, yhat, u, h, rh = _seam(s)
    dh, dn = s["dh"].reshape(-1, D).float(), s["dn"].reshape(-1, D).float()
    hhat = h * rh
    a = dn * s["weight"]
    dx = dh + rh * (a - hhat * (a * hhat).mean(-1, keepdim=True))
    out = {"dweight": (dn * hhat).sum(0)}
    du = dx
    if gate is not None:
        per = dx * u
        if gate.dim() == 1:
            out["dgate"] = per.sum(0)
        elif not c["packed"]:
            out["dgate"] = per.view(B, -1, D).sum(1)
        else:  # 64 bits for the running sums, whose differences are the sequences'
            run_ = torch.cat([per.new_zeros((1, D), dtype=torch.float64), per.double().cumsum(0)])[s["offsets"].long()]
            out["dgate"] = (run_[1:] - run_[:-1]).float()
        du = dx * gate
    dy = du
    if s["post"] is not None:
        out["dpost"] = (du * yhat).sum(0)
        b = du * s["post"]
        dy = ry * (b - yhat * (b * yhat).mean(-1, keepdim=True))
    dt, shape = s["x"].dtype, s["x"].shape
    return {"dx": dx.to(dt).view(shape), "dy": dy.to(dt).view(shape), **out}


PLAIN = {"attend": plain_attend, "write": plain_write, "read": plain_read, "seam": plain_seam, "seam_back": plain_seam_back}


def own_attend(s):
    import gated_delta_rule_scan_amd as gdn

    c = s["case"]
    lse = torch.empty(s["q"].shape[:2], device=s["q"].device)
    y = gdn.attention_step(s["q"], s["cache"], s["table"], s["lengths"], window=c["window"], sinks=c["sinks"], lse=lse)
    return y, lse


def own_write(s):
    import gated_delta_rule_scan_amd as gdn

    c = s["case"]
    gdn.kv_write(s["k"], s["v"], s["cache"], s["table"], s["start"], seq_offsets=s["offsets"] if c["packed"] else None)
    if c["format"] in DTYPES:
        return s["cache"][:2]
    return own_read(s)


def own_read(s):
    import gated_delta_rule_scan_amd as gdn

    c = s["case"]
    return gdn.kv_read(s["cache"], s["table"], c["T"], s["start"], seq_offsets=s["offsets"] if c["packed"] else None,
                       dtype=DTYPES[c["dtype"]])


def own_seam(s):
    import gated_delta_rule_scan_amd as gdn

    return gdn.residual_norm(s["x"], s["y"], gate=s["gate"], post_weight=s["post"], weight=s["weight"], eps=EPS,
                             seq_offsets=s["offsets"] if s["case"]["packed"] else None)


def own_seam_back(s):
    import gated_delta_rule_scan_amd as gdn

    got = gdn.residual_norm_backward(s["dh"], s["dn"], s["x"], s["y"], gate=s["gate"], post_weight=s["post"],
                                     weight=s["weight"], eps=EPS, seq_offsets=s["offsets"] if s["case"]["packed"] else None)
    return {k: v for k, v in zip(("dx", "dy", "dgate", "dpost", "dweight"), got) if v is not None}


OWN = {"attend": own_attend, "write": own_write, "read": own_read, "seam": own_seam, "seam_back": own_seam_back}


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op, es, B = case["op"], SIZE[case["dtype"]], case["B"]
    if op == "attend":
        Hq, Hk, d, W = case["Hq"], case["Hk"], case["d"], case["window"]
        tokens = 0
        for n in _lengths(case):
            tokens += n if not W else min(n, W) + min(case["sinks"], max(n - W, 0))
        return {"bytes": tokens * Hk * 2 * ROW[case["format"]](d) + B * Hq * (2 * d * es + 4), "flops": 4 * tokens * Hq * d}
    rows = case["T"] if case["packed"] else B * case["T"]
    if op in ("write", "read"):
        n = rows * case["Hk"] * 2
        held, given = n * ROW[case["format"]](case["d"]), n * case["d"] * es
        both = op == "write" and case["format"] not in DTYPES
        return {"bytes": (held + given) * (2 if both else 1), "flops": 4 * n * case["d"]}
    D = case["D"]
    params = (2 + case["post"]) * D * 4 + (B * D * 4 if case["gate"] == "sequence" else 0)
    if op == "seam":
        return {"bytes": 4 * rows * D * es + params, "flops": rows * D * (10 if case["post"] else 6)}
    return {"bytes": 6 * rows * D * es + 2 * params, "flops": rows * D * (28 if case["post"] else 18)}


# ---- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def _power(e):
    """2^e in 64 bits, exactly, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values(pool, scales, form):
    """A pool's rows in 64 bits."""
    if scales is None:
        return pool.double()
    s = _power(scales.long() - 127).repeat_interleave(32, -1)
    if form == "mxfp8":
        c = pool.view(torch.uint8).long()
        e, m = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _power(e - 7))
        return torch.where(c >= 128, -v, v) * s
    c = torch.stack([pool % 16, pool // 16], -1).flatten(-2).long()
    v = torch.tensor(E2M1, dtype=torch.float64, device=pool.device)[c % 8]
    return torch.where(c >= 8, -v, v) * s


def _rounded(x, form):
    """x in 64 bits as 8 or 4 bits hold it."""
    most, low, bits = (448.0, -6, 3) if form == "mxfp8" else (6.0, 0, 1)
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    # the least power of two with which the largest magnitude is in range: a guess, put right
    e = torch.log2((top / most).clamp(min=2.0 ** -110)).round().long()
    e = torch.where(top > most * _power(e), e + 1, e)
    e = torch.where((top <= most * _power(e - 1)) & (e > -110), e - 1, e)
    a = b.abs() / _power(e)
    ulp = _power((torch.frexp(a).exponent - 1).clamp(min=low) - bits)
    return (torch.sign(b) * torch.round(a / ulp) * ulp * _power(e)).reshape(x.shape)


def exact_attend(s):
    c = s["case"]
    Hq, Hk, d, page = c["Hq"], c["Hk"], c["d"], c["page"]
    k, v, ks, vs = s["cache"]
    y = torch.zeros((c["B"], Hq, d), dtype=torch.float64, device=k.device)
    lse = torch.zeros((c["B"], Hq), dtype=torch.float64, device=k.device)
    for b, n in enumerate(s["lengths"].tolist()):
        at = list(range(n)) if not c["window"] else [p for p in range(n) if p >= n - c["window"] or p < c["sinks"]]
        at = torch.tensor(at, device=k.device)
        pages, rows = s["table"][b].long()[at // page], at % page
        for h in range(Hk):
            def of(pool, scales):
                if scales is None:
                    return pool[pages, h, rows].double()
                return _values(pool.view(torch.uint8)[pages, h, rows], scales[pages, h, rows], c["format"])
            g = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            x = of(k, ks) @ s["q"][b, g].double().t().contiguous() / math.sqrt(d)  # [tokens, heads]
            lse[b, g] = torch.logsumexp(x, 0)
            y[b, g] = torch.softmax(x, 0).t().contiguous() @ of(v, vs)
    return y, lse


def exact_write(s):
    c = s["case"]
    off, start, page = s["offsets"].tolist(), s["start"].tolist(), c["page"]
    rows = [x.reshape(-1, c["Hk"], c["d"]) for x in (s["k"], s["v"])]
    if c["format"] not in DTYPES:
        shape = s["k"].shape
        return tuple(_rounded(x, c["format"]).view(shape) for x in rows)
    pools = [p.double() for p in s["cache"][:2]]
    for b in range(c["B"]):
        p = torch.arange(start[b], start[b] + off[b + 1] - off[b], device=rows[0].device)
        pages = s["table"][b].long()[p // page]
        for x, pool in zip(rows, pools):
            pool[pages, :, p % page] = x[off[b]: off[b + 1]].double()
    return tuple(pools)


def exact_read(s):
    c = s["case"]
    off, start, page = s["offsets"].tolist(), s["start"].tolist(), c["page"]
    outs = []
    for pool, scales in zip(s["cache"][:2], s["cache"][2:]):
        parts = []
        for b in range(c["B"]):
            p = torch.arange(start[b], start[b] + off[b + 1] - off[b], device=pool.device)
            pages = s["table"][b].long()[p // page]
            raw = pool if scales is None else pool.view(torch.uint8)
            parts.append(_values(raw[pages, :, p % page], None if scales is None else scales[pages, :, p % page], c["format"]))
        lead = (c["T"],) if c["packed"] else (c["B"], c["T"])
        outs.append(torch.cat(parts).view(*lead, c["Hk"], c["d"]))
    return tuple(outs)


def _exact_rows(s, lo, hi, gate):
    """h and n of rows lo..hi in 64 bits, from leaves that want gradients."""
    D = s["case"]["D"]
    leaf = lambda t: None if t is None else t.double().detach().requires_grad_(True)
    v = {"x": leaf(s["x"].reshape(-1, D)[lo:hi]), "y": leaf(s["y"].reshape(-1, D)[lo:hi]), "gate": leaf(gate),
         "post": leaf(s["post"]), "weight": leaf(s["weight"])}
    norm = lambda t, w: w * t / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS)
    u = v["y"] if v["post"] is None else norm(v["y"], v["post"])
    h = v["x"] + (u if v["gate"] is None else v["gate"] * u)
    return v, h, norm(h, v["weight"])


def _exact_spans(s):
    """Row ranges of a few thousand rows at most, each of one sequence, with that sequence."""
    off = s["offsets"].tolist()
    for b in range(len(off) - 1):
        for lo in range(off[b], off[b + 1], 8192):
            yield b, lo, min(lo + 8192, off[b + 1])


def exact_seam(s):
    hs, ns = [], []
    for b, lo, hi in _exact_spans(s):
        gate = s["gate"] if s["gate"] is None or s["gate"].dim() == 1 else s["gate"][b]
        _, h, n = _exact_rows(s, lo, hi, gate)
        hs.append(h.detach())
        ns.append(n.detach())
    return torch.cat(hs).view(s["x"].shape), torch.cat(ns).view(s["x"].shape)


def exact_seam_back(s):
    D = s["case"]["D"]
    zero = lambda t: None if t is None else torch.zeros(t.shape, dtype=torch.float64, device=t.device)
    dx, dy = zero(s["x"].reshape(-1, D)), zero(s["y"].reshape(-1, D))
    sums = {"dgate": zero(s["gate"]), "dpost": zero(s["post"]), "dweight": zero(s["weight"])}
    for b, lo, hi in _exact_spans(s):
        each = s["gate"] is not None and s["gate"].dim() == 2
        v, h, n = _exact_rows(s, lo, hi, s["gate"][b] if each else s["gate"])
        torch.autograd.backward([h, n], [s[k].reshape(-1, D)[lo:hi].double() for k in ("dh", "dn")])
        dx[lo:hi], dy[lo:hi] = v["x"].grad, v["y"].grad
        for k in ("gate", "post", "weight"):
            if v[k] is not None:
                (sums["dgate"][b] if each and k == "gate" else sums["d" + k]).add_(v[k].grad)
    out = {"dx": dx.view(s["x"].shape), "dy": dy.view(s["y"].shape), **sums}
    return {k: t for k, t in out.items() if t is not None}


EXACT = {"attend": exact_attend, "write": exact_write, "read": exact_read, "seam": exact_seam, "seam_back": exact_seam_back}
