"""Measured cases of the attention-side operators: per-head norm + rotation of queries and keys,
the NVFP4 key/value cache (written, read back), and attention to keys and values of another
length, in bf16 or in the cache.

A case is a plain dict.  `run` computes it in elementary torch operations, or, where `own` is
set, through the package's entry points.  `exact` evaluates the definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6


# ---- cases --------------------------------------------------------------------------------
def listed():
    return [
        # one new token of one sequence: latency
        dict(name="qk_one_token", op="qk", B=1, T=1, Hq=8, Hkv=1, D=256, R=256, pairs="half", pos=1000),
        # the backbone's prompt (3 x 256 image + 200 text tokens), its QKV output 2560 wide
        dict(name="qk_prompt", op="qk", B=1, T=968, Hq=8, Hkv=1, D=256, R=256, pairs="half", pos=0),
        # a batch of prompts, many heads, interleaved pairs, far positions
        dict(name="qk_batch", op="qk", B=16, T=968, Hq=16, Hkv=8, D=128, R=128, pairs="inter", pos=30000),
        # the action chunk's 50 rows appended behind the prompt's
        dict(name="store_chunk", op="store", B=1, T=50, C=1024, Hq=8, Hkv=1, D=256, R=256, pairs="half", pos=968),
        # the prompt's rows of a batch, written as the prompt is processed
        dict(name="store_prompts", op="store", B=16, T=968, C=1024, Hq=8, Hkv=1, D=256, R=256, pairs="half", pos=0),
        # a long cache read back to bf16
        dict(name="read_long", op="read", B=8, C=16384, Hkv=1, D=256),
        # one short one, heads of 48
        dict(name="read_short", op="read", B=1, C=304, Hkv=32, D=48),
        # action expert: 50 queries over prompt + chunk in the cache
        dict(name="attend_chunk", op="attend", B=1, T=50, S=1018, C=1024, Hq=8, Hkv=1, D=256, kv="cache", mask=False,
             spread=0),
        # DiT: 41 queries to an encoder's states, some of them masked, 32 heads of 48
        dict(name="attend_cross", op="attend", B=1, T=41, S=301, C=304, Hq=32, Hkv=32, D=48, kv="bf16", mask=True,
             spread=0),
        # the prompt to itself, four at a time
        dict(name="attend_prompts", op="attend", B=4, T=968, S=968, C=968, Hq=8, Hkv=1, D=256, kv="bf16", mask=False,
             spread=0),
        # single tokens over long caches of unequal lengths
        dict(name="attend_tokens", op="attend", B=8, T=1, S=32701, C=32704, Hq=8, Hkv=1, D=256, kv="cache",
             mask=False, spread=1500),
        # the largest: long queries to a longer encoder
        dict(name="attend_long", op="attend", B=8, T=2048, S=4096, C=4096, Hq=16, Hkv=4, D=128, kv="bf16", mask=False,
             spread=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    Hkv = rng.choice([1, 1, 2, 4, 8, 16])
    return Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv


def draw(rng):
    most = {"qk": 4.8e7, "store": 4.8e7, "read": 6.8e7, "attend": 5.4e11}
    while True:
        op = rng.choice(["qk", "store", "read", "attend", "attend", "attend"])
        B, T = _log(rng, 1, 16), _log(rng, 1, 2048)
        Hq, Hkv = _heads(rng)
        D = rng.choice([48, 64, 80, 96, 128, 128, 256, 256])
        if op in ("qk", "store"):
            pos = _log(rng, 1, 30000) - 1
            c = dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([D, D, 32]),
                     pairs=rng.choice(["half", "inter"]), pos=pos)
            if op == "store":
                c["pos"] = pos % 2000
                c["C"] = (c["pos"] + T + rng.randrange(64)) // 16 * 16 + 16
            cost = B * T * (Hq + 2 * Hkv) * D
        elif op == "read":
            c = dict(op=op, B=B, C=16 * _log(rng, 1, 2048), Hkv=Hkv, D=D)
            cost = 2 * B * c["C"] * Hkv * D
        else:
            T = rng.choice([1, 1, T, T])
            S = _log(rng, 1, 32768)
            c = dict(op=op, B=B, T=T, S=S, C=(S + 15) // 16 * 16, Hq=Hq, Hkv=Hkv, D=D,
                     kv=rng.choice(["bf16", "cache"]), mask=rng.random() < 0.3,
                     spread=rng.choice([0, 0, S // 17, S // 5 + 1]))
            cost = 4 * B * T * Hq * S * D
            # the plain form's scores and the keys' bytes stay within what the largest case takes
            if B * Hq * T * S > 1.1e9 or B * Hkv * S * D > 6.8e7:
                continue
        if cost <= most[op]:
            return c


def _lens(c):
    """Keys of each sequence: S, less for the later ones of an uneven batch, none for the last of some."""
    return [max(0, c["S"] - b * c["spread"]) for b in range(c["B"])]


# ---- inputs -------------------------------------------------------------------------------
def _table(first, count, R, device):
    """Rotation table (cos | sin) of positions 0 .. first + count - 1; the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    a = torch.arange(first + count, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c, d = case, "cuda"
    g = torch.Generator(device=d).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device=d) * std + mean).bfloat16()

    def codes(B, H, C, D):
        # a filled cache: any code, scales of values around 1
        return (torch.randint(0, 256, (B, H, C, D // 2), generator=g, device=d, dtype=torch.uint8),
                torch.randint(0x18, 0x38, (B, H, C, D // 16), generator=g, device=d, dtype=torch.uint8))

    s = {"case": c}
    if c["op"] in ("qk", "store"):
        B, T, Hq, Hkv, D = (c[n] for n in ("B", "T", "Hq", "Hkv", "D"))
        # the QKV output: q, k and v of a token side by side
        qkv = normal(B, T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["qg"], s["kg"] = normal(D, std=0.1, mean=1.0), normal(D, std=0.1, mean=1.0)
        s["table"] = _table(c["pos"], T, c["R"], d)
        if c["op"] == "qk":
            s["positions"] = (c["pos"] + torch.arange(T, device=d, dtype=torch.int32)).repeat(B, 1)
        else:
            s["start"] = torch.full((B,), c["pos"], device=d, dtype=torch.int32)
            s["cache"] = [torch.zeros((B, Hkv, c["C"], D // n), device=d, dtype=torch.uint8) for n in (2, 16, 2, 16)]
    elif c["op"] == "read":
        s["cache"] = [t for _ in range(2) for t in codes(c["B"], c["Hkv"], c["C"], c["D"])]
    else:
        B, T, S, Hq, Hkv, D = (c[n] for n in ("B", "T", "S", "Hq", "Hkv", "D"))
        s["q"] = normal(B, T, Hq, D, std=1.5)
        if c["kv"] == "cache":
            s["cache"] = [t for _ in range(2) for t in codes(B, Hkv, c["C"], D)]
        else:
            # the encoder's K and V projections side by side
            kv = normal(B, S, 2 * Hkv, D)
            s["k"], s["v"] = kv[:, :, :Hkv], kv[:, :, Hkv:]
        s["kv_len"] = torch.tensor(_lens(c), device=d, dtype=torch.int32)
        s["mask"] = None
        if c["mask"]:
            # an image that is missing, and single padded places
            m = torch.rand((B, S), generator=g, device=d) > 0.1
            m[:, S // 4:S // 2] = False
            s["mask"] = m
    return s


# ---- plain forms --------------------------------------------------------------------------
def _rotate(n, table, pos, R, pairs):
    """n fp32 [B, T, H, D]; pos int [B, T]."""
    t = table[pos.long()][:, :, None]
    cos, sin = t[..., :R // 2], t[..., R // 2:]
    if pairs == "half":
        a, b = n[..., :R // 2], n[..., R // 2:R]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, n[..., R:]], -1)
    a, b = n[..., 0:R:2], n[..., 1:R:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), n[..., R:]], -1)


def _norm(x, gamma):
    # the mean of squares in 64 bits, as the quantized values that follow sit next to borders
    r = (x.double().square().mean(-1, keepdim=True) + EPS).rsqrt().float()
    return (x.float() * r) * gamma.float()


def _nearest(v):
    """fp32 -> the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code, sign kept."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=6.0), v)


def _quantized(y):
    """fp32 [..., D] -> the values that the NVFP4 codes and scales of blocks of 16 stand for."""
    b = y.unflatten(-1, (-1, 16))
    a = b.abs().amax(-1, keepdim=True)
    # divided by a tensor: a division by a number may be a product with its reciprocal, which misses ties
    s = torch.clamp(a / torch.full_like(a, 6.0), max=448.0).to(torch.float8_e4m3fn).float()
    r = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    return (_nearest(b * r) * s).flatten(-2).bfloat16()


def _values(codes, sf):
    """Codes [B, H, C, D/2] and scales [B, H, C, D/16] -> fp32 [B, H, C, D]."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    return (v.unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _valid(s):
    c = s["case"]
    ok = torch.arange(c["S"], device=s["q"].device)[None] < s["kv_len"][:, None]
    return ok & s["mask"] if s["mask"] is not None else ok


def _plain(s):
    c = s["case"]
    if c["op"] in ("qk", "store"):
        if c["op"] == "qk":
            pos = s["positions"]
        else:
            pos = s["start"][:, None] + torch.arange(c["T"], device=s["q"].device, dtype=torch.int32)
        q = _rotate(_norm(s["q"], s["qg"]), s["table"], pos, c["R"], c["pairs"]).bfloat16()
        k = _rotate(_norm(s["k"], s["kg"]), s["table"], pos, c["R"], c["pairs"])
        return (q, k.bfloat16()) if c["op"] == "qk" else (q, _quantized(k), _quantized(s["v"].float()))
    if c["op"] == "read":
        kc, ks, vc, vs = s["cache"]
        return tuple(_values(a, b).transpose(1, 2).bfloat16() for a, b in ((kc, ks), (vc, vs)))
    B, T, S, Hq, Hkv, D = (c[n] for n in ("B", "T", "S", "Hq", "Hkv", "D"))
    if c["kv"] == "cache":
        kc, ks, vc, vs = s["cache"]
        k, v = _values(kc, ks)[:, :, :S], _values(vc, vs)[:, :, :S]
    else:
        k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    # the queries of a key head's group are rows of one product
    q = s["q"].float().transpose(1, 2).reshape(B, Hkv, Hq // Hkv * T, D)
    x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~_valid(s)[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    del x
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, Hq, T, D).transpose(1, 2).bfloat16()


# ---- the package's entry points -----------------------------------------------------------
def _own(s):
    from vla_action_head_b200 import nvfp4
    c = s["case"]
    if c["op"] == "qk":
        return nvfp4.qk_norm_rope(s["q"], s["k"], s["qg"], s["kg"], table=s["table"], positions=s["positions"],
                                  eps=EPS, pairs=c["pairs"])
    if c["op"] == "store":
        cache = nvfp4.KVCache(*s["cache"])
        q, _ = nvfp4.qk_norm_rope(s["q"], s["k"], s["qg"], s["kg"], table=s["table"], eps=EPS, pairs=c["pairs"],
                                  v=s["v"], cache=cache, start=s["start"])
        return (q,) + nvfp4.kv_read(cache, start=s["start"], length=c["T"])
    if c["op"] == "read":
        return nvfp4.kv_read(nvfp4.KVCache(*s["cache"]))
    if c["kv"] == "cache":
        return nvfp4.attention(s["q"], cache=nvfp4.KVCache(*s["cache"], length=c["S"]), kv_len=s["kv_len"],
                               key_mask=s["mask"])
    return nvfp4.attention(s["q"], s["k"], s["v"], kv_len=s["kv_len"], key_mask=s["mask"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    c = case
    if c["op"] in ("qk", "store"):
        rows, D = c["B"] * c["T"], c["D"]
        table = 4.0 * c["T"] * c["R"]
        moved = 4.0 * rows * (c["Hq"] + c["Hkv"]) * D
        if c["op"] == "store":  # k and v: read, written at 9/16 byte, read back, returned
            moved = 4.0 * rows * c["Hq"] * D + (2 + 2 * 0.5625 + 2) * rows * 2 * c["Hkv"] * D
        return {"bytes": moved + table, "flops": 8.0 * rows * (c["Hq"] + 2 * c["Hkv"]) * D}
    if c["op"] == "read":
        n = 2.0 * c["B"] * c["C"] * c["Hkv"] * c["D"]
        return {"bytes": n * (0.5625 + 2), "flops": n}
    keys = sum(_lens(c))
    each = 0.5625 if c["kv"] == "cache" else 2.0
    return {"bytes": 4.0 * c["B"] * c["T"] * c["Hq"] * c["D"] + 2 * each * keys * c["Hkv"] * c["D"],
            "flops": 4.0 * c["T"] * c["Hq"] * c["D"] * keys}


# ---- the definition in 64 bits ------------------------------------------------------------
def _decoded(codes, sf):
    """E2M1 codes and E4M3 scales by their bit fields, fp64."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    sign = torch.where(n >= 8, -1.0, 1.0).double()
    m = n % 8
    e = torch.div(m, 2, rounding_mode="floor")
    mag = torch.where(e > 0, (2 + m % 2) * 2.0 ** (e - 2), (m % 2) * 0.5)
    b = sf.double() % 128
    se = torch.div(b, 8, rounding_mode="floor")
    scale = torch.where(se > 0, (8 + b % 8) * 2.0 ** (se - 10), (b % 8) * 2.0 ** -9)
    return sign * mag * scale.repeat_interleave(16, -1)


def _code_values(y):
    """fp64 [..., D] -> quantized values: scale = amax / 6 on the E4M3 grid, each element times
    the scale's fp32 reciprocal (a step of the format, rounded once) on the E2M1 grid."""
    a = y.reshape(*y.shape[:-1], -1, 16)
    t = a.abs().amax(-1, keepdim=True)
    t = (t / torch.full_like(t, 6)).clamp(max=448)
    m = torch.frexp(t.clamp(min=2.0 ** -60))[0]  # t = m 2^x, m in [1/2, 1): four bits, above the subnormals
    s = torch.where(t >= 2.0 ** -6, torch.round(m * 16) * (t / m) / 16, torch.round(t * 512) / 512)
    r = torch.where(s > 0, (1 / s.clamp(min=2.0 ** -9)).float().double(), torch.zeros_like(s))
    w = (a * r).float().double()
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=y.device)
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.bucketize(w.abs(), mid)
    tie = (w.abs() == mid[i.clamp(max=6)]) & (i < 7)
    i = torch.where(tie & (i % 2 == 1), i + 1, i)
    return (torch.sign(w) * grid[i] * s).reshape(y.shape)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("qk", "store"):
        R, P = c["R"], c["pos"] + torch.arange(c["T"], device="cuda")
        w = torch.complex(s["table"][P, :R // 2].double(), s["table"][P, R // 2:].double())[None, :, None]

        def turned(x, gamma):
            x = x.double()
            n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.double()
            h = n[..., :R]
            z = torch.complex(*(h.chunk(2, -1) if c["pairs"] == "half" else (h[..., 0::2], h[..., 1::2]))) * w
            parts = torch.cat([z.real, z.imag], -1) if c["pairs"] == "half" else torch.view_as_real(z).flatten(-2)
            return torch.cat([parts, n[..., R:]], -1)

        q, k = turned(s["q"], s["qg"]), turned(s["k"], s["kg"])
        return (q, k) if c["op"] == "qk" else (q, _code_values(k), _code_values(s["v"].double()))
    if c["op"] == "read":
        kc, ks, vc, vs = s["cache"]
        return _decoded(kc, ks).transpose(1, 2), _decoded(vc, vs).transpose(1, 2)
    B, T, S, Hq, Hkv, D = (c[n] for n in ("B", "T", "S", "Hq", "Hkv", "D"))
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    ok = _valid(s)
    for b in range(B):
        for h in range(Hkv):
            at = ok[b].nonzero()[:, 0]
            if not len(at):
                continue
            if c["kv"] == "cache":
                kc, ks, vc, vs = (t[b, h][at] for t in s["cache"])
                k, v = _decoded(kc, ks), _decoded(vc, vs)
            else:
                k, v = s["k"][b, at, h].double(), s["v"][b, at, h].double()
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                out[b, :, g] = torch.softmax(s["q"][b, :, g].double() @ k.T / math.sqrt(D), -1) @ v
    return out
