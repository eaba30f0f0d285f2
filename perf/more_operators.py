"""A decode step on a cache held in 4 bits, and the pass that feeds a cache: what is measured, and
the operators' plain forms.

A serving step takes the projections' query, key and value rows and

    rotate   normalises queries and keys for each head, rotates them by their positions (one axis,
             or time, height and width) and writes keys and values into their pages, in one pass
    store    quantises new rows into a 4-bit cache (a step and a lowest value for each token and
             kv head) and reads the sequences back into contiguous 16-bit rows, as a prompt that
             comes in chunks does before it attends over its cached part
    read     the read-back alone, of 8- and 4-bit caches
    decode   attention of the new tokens over a 4-bit cache

`run` computes one of them, in its plain form or, where `own` is true, by the framework's calls.

A row x of a 4-bit cache is held as codes c in 0 .. 15, two a byte (the even channel in the low half),
and a pair (step, low) of the queries' type:

    low = the largest such number <= min(x),  step = the least such number >= (max(x) - low) / 15,
    c = round((x - low) / step), ties to even (0 for step 0),  x ~ low + step c
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
PAGES = (16, 32, 64, 128, 256, 512, 1024)
EPS = 1e-6


# ---- cases -------------------------------------------------------------------------------
def listed():
    return [
        # The new token of each of a batch of chats: grouped-query heads, one fused projection.
        dict(name="rotate_step_b32_h32_kv8_d128_bs16", kind="rotate", batch=32, sq=1, hq=32, hkv=8, d=128,
             bs=16, prior_lo=511, prior_hi=4095, dtype="bf16", kv="16", rd=128, axes=1, pairs=False,
             norm=True, fused=True),
        # Four draft tokens a step into an 8-bit cache with a scale for each token.
        dict(name="rotate_step_b64_h16_kv1_d128_bs1024_sq4_fp8", kind="rotate", batch=64, sq=4, hq=16, hkv=1,
             d=128, bs=1024, prior_lo=8188, prior_hi=16380, dtype="bf16", kv="8", rd=64, axes=1, pairs=True,
             norm=False, fused=False),
        # Prompts with images, of uneven lengths: positions have a time, a height and a width.
        dict(name="rotate_prompt_b8_h32_kv8_d128_bs16_axes3", kind="rotate", batch=8, sq=4096, hq=32, hkv=8,
             d=128, bs=16, prior_lo=0, prior_hi=200, dtype="bf16", kv="16", rd=128, axes=3, pairs=False,
             norm=True, fused=True),
        # Draft tokens of a step, with the short sequences that they join.
        dict(name="store_step_b32_kv8_d128_bs16_sq4", kind="store", batch=32, sq=4, hkv=8, d=128, bs=16,
             prior_lo=60, prior_hi=252, dtype="bf16"),
        # A chunk of each prompt behind its cached part.
        dict(name="store_chunk_b8_kv8_d128_bs64_sq512", kind="store", batch=8, sq=512, hkv=8, d=128, bs=64,
             prior_lo=1, prior_hi=3584, dtype="bf16"),
        # Long contexts of an 8-bit cache with a scale for each token, in large pages.
        dict(name="read_b64_kv1_d128_bs1024_fp8token", kind="read", batch=64, hkv=1, d=128, bs=1024,
             ctx_lo=8192, ctx_hi=16384, dtype="bf16", kv="8token"),
        # Long contexts of a 4-bit cache, many wide heads, small pages.
        dict(name="read_b8_kv16_d256_bs32_int4", kind="read", batch=8, hkv=16, d=256, bs=32,
             ctx_lo=2048, ctx_hi=16384, dtype="bf16", kv="4"),
        # One short request: latency.
        dict(name="decode_b1_h16_kv1_d128_bs128", kind="decode", batch=1, sq=1, hq=16, hkv=1, d=128, bs=128,
             ctx_lo=512, ctx_hi=512, causal=False, dtype="bf16"),
        # A few very long contexts: their one unit of work each has to be split.
        dict(name="decode_b4_h16_kv1_d128_bs1024_long", kind="decode", batch=4, sq=1, hq=16, hkv=1, d=128,
             bs=1024, ctx_lo=32768, ctx_hi=131072, causal=True, dtype="bf16"),
        # A batch of chats, grouped-query heads, small pages.
        dict(name="decode_b32_h32_kv8_d128_bs16", kind="decode", batch=32, sq=1, hq=32, hkv=8, d=128, bs=16,
             ctx_lo=512, ctx_hi=4096, causal=False, dtype="bf16"),
        # The same with four draft tokens each.
        dict(name="decode_b32_h32_kv8_d128_bs16_sq4", kind="decode", batch=32, sq=4, hq=32, hkv=8, d=128, bs=16,
             ctx_lo=512, ctx_hi=4096, causal=True, dtype="bf16"),
        # One kv head for each query head, wide heads, long contexts.
        dict(name="decode_b32_h16_kv16_d256_bs32", kind="decode", batch=32, sq=1, hq=16, hkv=16, d=256, bs=32,
             ctx_lo=2048, ctx_hi=16384, causal=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng, kind):
    dtype = rng.choice(("bf16", "fp16"))
    d = rng.choice((64, 128, 256))
    hkv = rng.choice((1, 2, 3, 4, 8, 16))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    bs = rng.choice(PAGES)
    prior_lo, prior_hi = rng.randrange(0, 100), _log(rng, 100, 4000)
    if kind == "rotate":
        rd = rng.choice((d, d, d // 2, d // 4))
        axes = rng.choice((1, 1, 3)) if rd >= 32 else 1
        return dict(kind=kind, batch=_log(rng, 1, 128), sq=_log(rng, 1, 4096), hq=hkv * group, hkv=hkv, d=d,
                    bs=bs, prior_lo=prior_lo, prior_hi=prior_hi, dtype=dtype, kv=rng.choice(("16", "16", "8")),
                    rd=rd, axes=axes, pairs=rng.random() < 0.3, norm=rng.random() < 0.7, fused=rng.random() < 0.6)
    if kind == "store":
        return dict(kind=kind, batch=_log(rng, 1, 64), sq=_log(rng, 1, 2048), hkv=hkv, d=d, bs=bs,
                    prior_lo=prior_lo, prior_hi=prior_hi, dtype=dtype)
    ctx_hi = _log(rng, 64, 131072)
    ctx_lo = max(16, int(ctx_hi * rng.uniform(0.05, 1.0)))
    if kind == "read":
        return dict(kind=kind, batch=_log(rng, 1, 128), hkv=hkv, d=d, bs=bs, ctx_lo=ctx_lo, ctx_hi=max(16, ctx_hi),
                    dtype=dtype, kv=rng.choice(("4", "4", "8token", "8tensor", "8block")))
    return dict(kind=kind, batch=_log(rng, 1, 64), sq=rng.choice((1, 1, 1, 2, 3, 4, 8)), hq=hkv * group, hkv=hkv,
                d=d, bs=bs, ctx_lo=ctx_lo, ctx_hi=max(16, ctx_hi), causal=rng.random() < 0.5, dtype=dtype)


def _held_bytes(c):
    """About what the plain form's largest temporaries and the inputs take, in 32 bits."""
    if c["kind"] == "rotate":
        return c["batch"] * (c["sq"] * (c["hq"] + 2 * c["hkv"]) * 12 + (c["sq"] + c["prior_hi"] + c["bs"]) * c["hkv"] * 4) * c["d"]
    longest = c["prior_hi"] + c["sq"] if c["kind"] == "store" else c["ctx_hi"]
    tokens = c["batch"] * (-(-longest // c["bs"])) * c["bs"]
    logits = tokens * c["sq"] * c["hq"] * 4 if c["kind"] == "decode" else 0
    return tokens * c["hkv"] * c["d"] * 16 + 3 * logits


def draw(rng):
    kind = rng.choice(("rotate", "store", "read", "decode", "decode"))
    most = max(work(x)["bytes"] for x in listed() if x["kind"] == kind)
    ops = max(work(x)["flops"] for x in listed() if x["kind"] == kind)
    c = _drawn(rng, kind)
    while work(c)["bytes"] > most or work(c)["flops"] > ops or _held_bytes(c) > 6e9:  # no more than the largest listed
        c = _drawn(rng, kind)
    return c


# ---- what a case cannot do without ---------------------------------------------------------
def _lens(case, lo, hi):
    """The batch's lengths, evenly spread from lo to hi: the same ones for every seed."""
    b = case["batch"]
    return [lo + (hi - lo) * j // max(1, b - 1) for j in range(b)] if b > 1 else [hi]


def _new(c):
    """Each sequence's cached tokens, and its new ones."""
    q = _lens(c, 1, c["sq"]) if c["sq"] > 8 else [c["sq"]] * c["batch"]
    return _lens(c, c["prior_lo"], c["prior_hi"]), q


def _row_bytes(c, kv):
    """A cached K or V row of a token and kv head: values, and what belongs to the token."""
    return {"16": 2 * c["d"], "8": c["d"] + 4, "8token": c["d"] + 4, "4": c["d"] // 2 + 4}.get(kv, c["d"])


def work(case):
    c = case
    if c["kind"] == "rotate":
        prior, q = _new(c)
        rows = sum(q)
        table = (max(q) if c["sq"] > 8 else rows) * c["rd"] * 4  # prompts share their positions' angles
        return dict(bytes=rows * (c["hq"] * c["d"] * 4 + c["hkv"] * (c["d"] * 4 + 2 * _row_bytes(c, c["kv"]))) + table,
                    flops=rows * (c["hq"] + c["hkv"]) * (4 * c["d"] + 3 * c["rd"]))
    if c["kind"] == "store":
        prior, q = _new(c)
        new, old = sum(q) * c["hkv"], sum(prior) * c["hkv"]
        return dict(bytes=2 * (new * (2 * c["d"] + _row_bytes(c, "4")) + old * _row_bytes(c, "4") + (new + old) * 2 * c["d"]),
                    flops=2 * c["d"] * (5 * new + 2 * (new + old)))
    lens = _lens(c, c["ctx_lo"], c["ctx_hi"])
    tokens = sum(lens) * c["hkv"]
    tables = sum(-(-n // c["bs"]) for n in lens) * (4 + (8 * c["hkv"] if c.get("kv") == "8block" else 0))
    if c["kind"] == "read":
        return dict(bytes=2 * tokens * (_row_bytes(c, c["kv"]) + 2 * c["d"]) + tables, flops=4 * tokens * c["d"])
    rows = c["batch"] * c["sq"] * c["hq"]
    return dict(bytes=2 * tokens * _row_bytes(c, "4") + tables + rows * (c["d"] * 4 + 4),
                flops=4 * sum(lens) * c["sq"] * c["hq"] * c["d"])


# ---- inputs ----------------------------------------------------------------------------------
def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _codes8(shape, g):
    """E4M3 codes of rows that were quantised over their largest value."""
    return (_randn(shape, g, torch.float16) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache4(pool, hkv, bs, d, t, g):
    """A 4-bit cache: codes, and each row's step and low (keys have an offset of their own)."""
    codes = torch.randint(0, 256, (pool, bs, hkv, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    step = torch.rand((pool, hkv, bs), generator=g, device="cuda") * 0.15 + 0.25
    low = -7.5 * step + _randn((pool, hkv, bs), g, torch.float32) * 0.2
    return codes, torch.stack((step, low), -1).to(t).contiguous()


def _table(pages, columns, pool, g):
    """Block tables of sequences with `pages` pages each, out of a shuffled pool; -1 behind."""
    perm = torch.randperm(pool, generator=g, device="cuda")
    start = torch.cumsum(pages, 0) - pages
    col = torch.arange(columns, device="cuda")
    at = (start[:, None] + col).clamp(max=pool - 1)
    return torch.where(col < pages[:, None], perm[at], -1).to(torch.int32)


def _axis_pairs(c):
    """How many of the rotated pairs follow each axis: half the time, the rest height and width."""
    half = c["rd"] // 2
    if c["axes"] == 1:
        return [half]
    side = half * 3 // 8
    return [half - 2 * side, side, side]


def _prepare_rotate(c, s, g):
    b, sq, hq, hkv, d, t = c["batch"], c["sq"], c["hq"], c["hkv"], c["d"], TYPES[c["dtype"]]
    if c["fused"]:  # slices of one projection's output
        qkv = _randn((b, sq, hq + 2 * hkv, d), g, t)
        s.update(qx=qkv[:, :, :hq], k=qkv[:, :, hq:hq + hkv], v=qkv[:, :, hq + hkv:])
    else:
        s.update(qx=_randn((b, sq, hq, d), g, t), k=_randn((b, sq, hkv, d), g, t), v=_randn((b, sq, hkv, d), g, t))
    if c["norm"]:
        s.update(wq=1 + 0.2 * _randn((d,), g, t), wk=1 + 0.2 * _randn((d,), g, t))
    # cosines and sines of every position, from angles in 64 bits
    rows = c["prior_hi"] + sq
    freq = 10000.0 ** (-torch.arange(0, c["rd"], 2, dtype=torch.float64, device="cuda") / c["rd"])
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    s.update(cs=torch.cat((angle.cos(), angle.sin()), 1).float(), pos=None, qo=torch.zeros(b, sq, hq, d, dtype=t, device="cuda"))
    if c["axes"] == 3:
        # a text token has its place three times; an image's patches share a time and lie on a grid
        at = (s["ctx"] - s["q"])[:, None] + torch.arange(sq, device="cuda")
        i = at % 1024
        side = torch.stack((at - i, at - i + i // 32, at - i + i % 32))
        image = (at // 1024 % 2 == 1) & (at < s["ctx"][:, None])
        s["pos"] = torch.where(image, side, at).clamp(max=rows - 1).to(torch.int32).contiguous()
    eight = c["kv"] == "8"
    shape = (s["pool"] + 1, c["bs"], hkv, d)  # (one page more than the pool has)
    kc, vc = (_codes8(shape, g), _codes8(shape, g)) if eight else (_randn(shape, g, t), _randn(shape, g, t))
    s.update(kc=kc, vc=vc, ks=None, vs=None)
    if eight:
        s.update(ks=torch.rand(shape[:3], generator=g, device="cuda") * 0.01 + 0.005,
                 vs=torch.rand(shape[:3], generator=g, device="cuda") * 0.01 + 0.005)
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, b, bs, hkv, d, t = c["kind"], c["batch"], c["bs"], c["hkv"], c["d"], TYPES[c["dtype"]]
    at = torch.randperm(b, generator=g, device="cuda")
    if kind in ("rotate", "store"):
        prior, q = _new(c)
        lens = [m + n for m, n in zip(prior, q)]
        q = torch.tensor(q, dtype=torch.int32, device="cuda")[at]
        longest = max(lens)
    else:
        lens = _lens(c, c["ctx_lo"], c["ctx_hi"])
        longest, sq = c["ctx_hi"], c.get("sq", 1)
        q = torch.tensor([min(n, sq) for n in lens], dtype=torch.int32, device="cuda")[at]
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")[at]
    pool = sum(-(-n // bs) for n in lens) + 3
    s = dict(case=c, ctx=ctx, q=q, pool=pool, total=sum(lens), longest=longest,
             bt=_table((ctx + bs - 1) // bs, -(-longest // bs), pool, g))
    if kind == "rotate":
        return _prepare_rotate(c, s, g)
    if kind in ("store", "read"):
        s.update(ko=torch.zeros(s["total"], hkv, d, dtype=t, device="cuda"),
                 vo=torch.zeros(s["total"], hkv, d, dtype=t, device="cuda"))
    if kind == "read" and c["kv"] != "4":
        shape = {"8token": (pool, bs, hkv), "8block": (pool, hkv), "8tensor": (1,)}[c["kv"]]
        s.update(kc=_codes8((pool, bs, hkv, d), g), vc=_codes8((pool, bs, hkv, d), g),
                 ks=torch.rand(shape, generator=g, device="cuda") * 0.01 + 0.005,
                 vs=torch.rand(shape, generator=g, device="cuda") * 0.01 + 0.005)
        return s
    (kc, ks), (vc, vs) = _cache4(pool, hkv, bs, d, t, g), _cache4(pool, hkv, bs, d, t, g)
    s.update(kc=kc, vc=vc, ks=ks, vs=vs)
    if kind == "store":
        gain = torch.where(torch.rand((1, 1, hkv, d), generator=g, device="cuda") < 1 / 32, 6.0, 1.0)  # outlying channels
        s.update(k=(_randn((b, c["sq"], hkv, d), g, torch.float32) * gain).to(t), v=_randn((b, c["sq"], hkv, d), g, t))
    if kind == "decode":
        s.update(qx=_randn((b, c["sq"], c["hq"], d), g, t), scale=1.0 / math.sqrt(d))
        s.update(out=torch.empty_like(s["qx"]), lse=torch.empty(s["qx"].shape[:3], dtype=torch.float32, device="cuda"))
    return s


# ---- the plain forms -----------------------------------------------------------------------------
def _slots(s, sq):
    """[B, Sq]: where each new row goes among the pool's slots; the last page's for a padding row."""
    bs, i = s["case"]["bs"], torch.arange(sq, device="cuda")
    pos = (s["ctx"] - s["q"])[:, None] + i
    page = s["bt"].gather(1, (pos // bs).clamp(max=s["bt"].shape[1] - 1).long())
    return torch.where(i < s["q"][:, None], page.long() * bs + pos % bs, s["pool"] * bs)


def _rotated(s, x, weight):
    """Rows [B, Sq, H, D] normalised (weight) and rotated, in 32 bits."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    half = c["rd"] // 2
    pos = s["pos"]
    if pos is None:
        pos = ((s["ctx"] - s["q"])[:, None] + torch.arange(c["sq"], device="cuda"))[None]
    axis = torch.repeat_interleave(torch.arange(len(_axis_pairs(c)), device="cuda"), torch.tensor(_axis_pairs(c), device="cuda"), output_size=half)
    row = pos.clamp(max=s["cs"].shape[0] - 1).long()[axis].permute(1, 2, 0)  # [B, Sq, half]
    pair = torch.arange(half, device="cuda")
    cos, sin = s["cs"][row, pair][:, :, None], s["cs"][row, pair + half][:, :, None]
    if c["pairs"]:
        a, b = x[..., 0:c["rd"]:2], x[..., 1:c["rd"]:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:c["rd"]]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., c["rd"]:]), -1)


def _plain_rotate(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    at = _slots(s, c["sq"]).reshape(-1)
    real = (torch.arange(c["sq"], device="cuda") < s["q"][:, None])[..., None, None]
    s["qo"].copy_(torch.where(real, _rotated(s, s["qx"], s.get("wq")).to(t), s["qo"]))
    out = dict(q=s["qo"])
    for name, x in (("k", _rotated(s, s["k"], s.get("wk"))), ("v", s["v"].float())):
        x = x.reshape(-1, *x.shape[2:])
        cache, scale = s[name + "c"], s[name + "s"]
        if c["kv"] == "8":
            big = x.abs().amax(-1)
            to = torch.where(big > 0, big / torch.full_like(big, E4M3_MAX), 1)
            x = (x / to[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            scale.flatten(0, 1).index_copy_(0, at, to)
            out[name + "_scale"] = scale[:-1]
        else:
            x = x.to(t)
        cache.flatten(0, 1).index_copy_(0, at, x)
        out[name] = cache[:-1].view(torch.float8_e4m3fn) if c["kv"] == "8" else cache[:-1]
    return out


def _nudged(x, t, up):
    """fp32 x in type t, rounded up or down."""
    y = x.to(t)
    step = torch.where((y.float() < x) if up else (y.float() > x), 1, 0).to(torch.int16)
    bits = y.view(torch.int16)
    # the next number away from zero, or towards it, is the next integer of the bits
    away = (bits >= 0) if up else (bits < 0)
    moved = torch.where(away, bits + step, bits - step).view(t)
    # below zero's smallest magnitudes: a positive number rounded to +0 steps down to the least negative
    least = torch.tensor([-32767 if not up else 1], dtype=torch.int16, device=x.device).view(t)
    return torch.where((y == 0) & (step > 0), least, moved)


def _quantised(x, t):
    """Codes [.., D] and (step, low) [.., 2] of rows."""
    x = x.float()
    low = _nudged(x.amin(-1), t, False)
    wide = x.amax(-1) - low.float()
    step = _nudged(wide / torch.full_like(wide, 15.0), t, True)
    lo, st = low.float()[..., None], step.float()[..., None]
    code = torch.where(st > 0, torch.round((x - lo) / torch.where(st > 0, st, 1)), 0).clamp(0, 15)
    return code.to(torch.uint8), torch.stack((step, low), -1)


def _values4(codes, pairs):
    """fp32 values of packed codes [.., D / 2] and their rows' (step, low) [.., 2]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    return c * pairs[..., :1].float() + pairs[..., 1:].float()


def _cached(s, name, at):
    """fp32 values [.., bs, Hkv, D] of the pages `at`."""
    cache, scale, kv = s[name + "c"][at], s[name + "s"], s["case"].get("kv", "4")
    if kv == "4":
        return _values4(cache, scale[at].transpose(-2, -3))
    x = cache.view(torch.float8_e4m3fn).float()
    if kv == "8tensor":
        return x * scale
    return x * (scale[at][..., None] if kv == "8token" else scale[at][..., None, :, None])


def _plain_read(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    # the token and the sequence of every contiguous row
    ctx = s["ctx"].long()
    end = torch.cumsum(ctx, 0)
    row = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(end, row, right=True)
    pos = row - (end - ctx)[seq]
    blk, slot = s["bt"][seq, pos // c["bs"]].long(), pos % c["bs"]
    out = {}
    for name, to in (("k", s["ko"]), ("v", s["vo"])):
        cache, scale, kv = s[name + "c"][blk, slot], s[name + "s"], c.get("kv", "4")
        if kv == "4":
            x = _values4(cache, scale[blk, :, slot])
        else:
            x = cache.view(torch.float8_e4m3fn).float()
            x = x * (scale if kv == "8tensor" else (scale[blk, slot] if kv == "8token" else scale[blk])[..., None])
        out[name] = to.copy_(x.to(t))
    return out


def _plain_store(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    bs = c["bs"]
    at = _slots(s, c["sq"]).reshape(-1)
    out = {}
    for name in "kv":
        code, pair = _quantised(s[name].reshape(-1, c["hkv"], c["d"]), t)
        cache, scale = s[name + "c"], s[name + "s"]
        # a padding row goes to a slot behind the pool, which is dropped
        flat = torch.cat((cache.flatten(0, 1), cache[0, :1]))
        flat.index_copy_(0, at, code[..., 0::2] | (code[..., 1::2] << 4))
        cache.copy_(flat[:-1].reshape(cache.shape))
        flat = torch.cat((scale.transpose(1, 2).flatten(0, 1), scale[0].transpose(0, 1)[:1]))
        flat.index_copy_(0, at, pair)
        scale.copy_(flat[:-1].reshape(s["pool"], bs, c["hkv"], 2).transpose(1, 2))
        out[name + "_scale"] = scale
    return dict(_plain_read(s), **out)


def _plain_decode(s):
    c = s["case"]
    b, sq, hkv, d, t = c["batch"], c["sq"], c["hkv"], c["d"], TYPES[c["dtype"]]
    at = s["bt"].clamp(min=0).long()
    k = _cached(s, "k", at).reshape(b, -1, hkv, d).permute(0, 2, 3, 1)
    v = _cached(s, "v", at).reshape(b, -1, hkv, d).permute(0, 2, 1, 3)
    x = s["qx"].float().reshape(b, sq, hkv, -1, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    i = torch.arange(sq, device="cuda")
    n, ql = s["ctx"][:, None], s["q"][:, None]
    seen = torch.where(i < ql, n - ql + i + 1 if c["causal"] else n, 0)[:, None, :, None, None]
    logits = (x @ k * s["scale"]).reshape(b, hkv, sq, -1, k.shape[-1])
    logits = torch.where(torch.arange(k.shape[-1], device="cuda") < seen, logits, -math.inf)
    logits = logits.reshape(b, hkv, -1, k.shape[-1])
    big = logits.amax(-1, keepdim=True)
    big = torch.where(big.isfinite(), big, 0)
    p = torch.exp(logits - big)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0)
    lse = (big + torch.log(total))[..., 0]
    out = out.reshape(b, hkv, sq, -1, d).permute(0, 2, 1, 3, 4).reshape(b, sq, -1, d)
    return dict(out=out.to(t), lse=lse.reshape(b, hkv, sq, -1).permute(0, 2, 1, 3).reshape(b, sq, -1))


# ---- the framework's calls ---------------------------------------------------------------------
def _config(s, pa):
    """The problem's pa_config, which a user's program keeps."""
    if "cfg" not in s:
        c = s["case"]
        code = {"bf16": pa.BF16, "fp16": pa.FP16}[c["dtype"]]
        kv, mode = {"16": (code, pa.SCALE_NONE), "8": (pa.FP8_E4M3, pa.SCALE_PER_TOKEN),
                    "8token": (pa.FP8_E4M3, pa.SCALE_PER_TOKEN), "8block": (pa.FP8_E4M3, pa.SCALE_PER_BLOCK),
                    "8tensor": (pa.FP8_E4M3, pa.SCALE_PER_TENSOR), "4": (pa.INT4, pa.SCALE_AFFINE)}[c.get("kv", "4")]
        s["cfg"] = pa.PaConfig(
            batch=c["batch"], max_q_len=c.get("sq", 1), num_q_heads=c.get("hq", c["hkv"]), num_kv_heads=c["hkv"],
            head_dim=c["d"], block_size=c["bs"], max_blocks_per_seq=s["bt"].shape[1], num_blocks=s["pool"],
            q_dtype=code, kv_dtype=kv, kv_scale_mode=mode, causal=int(c.get("causal", False)),
            sm_scale=s.get("scale", 1.0))
    return s["cfg"]


def _own(s):
    import paged_kv_cache_work_gb300 as pa

    c, cfg = s["case"], _config(s, pa)
    kind = c["kind"]
    if kind == "rotate":
        pa.append_rotated(cfg, s["qx"], s["k"], s["v"], s["bt"], s["ctx"], s["q"], s["qo"], s["kc"], s["vc"],
                          s["ks"], s["vs"], cos_sin=s["cs"], interleaved=c["pairs"], positions=s["pos"],
                          axis_pairs=_axis_pairs(c), q_weight=s.get("wq"), k_weight=s.get("wk"), eps=EPS)
        if c["kv"] == "8":
            return dict(q=s["qo"], k=s["kc"][:-1].view(torch.float8_e4m3fn), v=s["vc"][:-1].view(torch.float8_e4m3fn),
                        k_scale=s["ks"][:-1], v_scale=s["vs"][:-1])
        return dict(q=s["qo"], k=s["kc"][:-1], v=s["vc"][:-1])
    if kind == "decode":
        if "ws" not in s:
            s["ws"] = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device="cuda")
        pa.plan(cfg, s["bt"], s["ctx"], s["q"], s["ws"])
        pa.decode(cfg, s["qx"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], s["q"], s["out"], s["lse"], s["ws"])
        pa.reduce(cfg, s["out"], s["lse"], s["ws"])
        return dict(out=s["out"], lse=s["lse"])
    if kind == "store":
        pa.append_kv(cfg, s["k"], s["v"], s["bt"], s["ctx"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"])
    pa.dequant_kv(cfg, s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], s["ko"], s["vo"])
    if kind == "store":
        return dict(k=s["ko"], v=s["vo"], k_scale=s["ks"], v_scale=s["vs"])
    return dict(k=s["ko"], v=s["vo"])


_PLAIN = dict(rotate=_plain_rotate, store=_plain_store, read=_plain_read, decode=_plain_decode)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ---- from the definition, in 64 bits -----------------------------------------------------------
F64 = torch.float64


def _exact_rotate(c, s):
    d, rd, half, bs = c["d"], c["rd"], c["rd"] // 2, c["bs"]
    out = {name: s[name].to(F64) for name in ("qo",)}
    caches = {}
    for name in "kv":
        x = s[name + "c"][:-1]
        caches[name] = x.view(torch.float8_e4m3fn).to(F64) if c["kv"] == "8" else x.to(F64)
        if c["kv"] == "8":
            caches[name + "_scale"] = s[name + "s"][:-1].to(F64)
    first = [(2 * p if c["pairs"] else p) for p in range(half)]
    second = [(2 * p + 1 if c["pairs"] else p + half) for p in range(half)]
    axis = [a for a, m in enumerate(_axis_pairs(c)) for _ in range(m)]
    table = torch.complex(s["cs"][:, :half].to(F64), s["cs"][:, half:].to(F64))
    ctx, ql, bt = s["ctx"].tolist(), s["q"].tolist(), s["bt"].long()

    def turned(x, weight, angle):
        x = x.to(F64)
        if weight is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * weight.to(F64)
        z = torch.complex(x[..., first], x[..., second]) * angle[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    for b in range(c["batch"]):
        m = ql[b]
        pos = torch.arange(ctx[b] - m, ctx[b], device="cuda")
        where = [s["pos"][a, b, :m].long() if s["pos"] is not None else pos for a in range(c["axes"])]
        angle = torch.stack([table[where[axis[p]], p] for p in range(half)], -1)
        out["qo"][b, :m] = turned(s["qx"][b, :m], s.get("wq"), angle)
        for name, rows in (("k", turned(s["k"][b, :m], s.get("wk"), angle)), ("v", s["v"][b, :m].to(F64))):
            blk, slot = bt[b, pos // bs], pos % bs
            if c["kv"] == "8":
                to = rows.abs().amax(-1) / E4M3_MAX
                caches[name + "_scale"][blk, slot] = to
                rows = rows / to[..., None]
            caches[name][blk, slot] = rows
    return dict(q=out["qo"], **caches)


def _pages_of(s, name, b):
    """64-bit values [tokens, Hkv, D] of sequence b's pages, token after token."""
    c, kv = s["case"], s["case"].get("kv", "4")
    blk = s["bt"][b, :-(-int(s["ctx"][b]) // c["bs"])].long()
    codes, scale = s[name + "c"][blk], s[name + "s"]
    if kv == "4":
        x = torch.empty(*codes.shape[:-1], c["d"], dtype=F64, device="cuda")
        x[..., 0::2], x[..., 1::2] = (codes % 16).to(F64), (codes // 16).to(F64)
        pair = scale[blk].to(F64).permute(0, 2, 1, 3)
        x = x * pair[..., :1] + pair[..., 1:]
    else:
        x = codes.view(torch.float8_e4m3fn).to(F64)
        if kv == "8tensor":
            x = x * scale.to(F64)
        elif kv == "8token":
            x = x * scale[blk].to(F64)[..., None]
        else:
            x = x * scale[blk].to(F64)[:, None, :, None]
    return x.flatten(0, 1)[:int(s["ctx"][b])]


def _exact_type(x, t, up):
    """The least (largest) number of type t that is not below (above) the 64-bit x."""
    bits, least = {torch.bfloat16: (7, -126), torch.float16: (10, -14)}[t]
    part = torch.frexp(x).mantissa
    power = torch.where(part == 0, 0, x / part)  # 2^e with |x| in [2^(e - 1), 2^e)
    place = (power / 2).clamp(min=2.0 ** least) * 2.0 ** -bits
    return torch.ceil(x / place) * place if up else torch.floor(x / place) * place


def _exact_store(c, s):
    t, out = TYPES[c["dtype"]], {}
    for name in "kv":
        scale, rows = s[name + "s"].to(F64), []
        for b in range(c["batch"]):
            n, m = int(s["ctx"][b]), int(s["q"][b])
            x = s[name][b, :m].to(F64)
            low = _exact_type(x.amin(-1), t, False)
            step = _exact_type((x.amax(-1) - low) / 15, t, True)
            value = low[..., None] + step[..., None] * torch.round(((x - low[..., None]) / step[..., None]).nan_to_num(0))
            pos = torch.arange(n - m, n, device="cuda")
            blk, slot = s["bt"][b, pos // c["bs"]].long(), pos % c["bs"]
            scale[blk, :, slot] = torch.stack((step, low), -1)
            rows.append(torch.cat((_pages_of(s, name, b)[:n - m], value)))
        out[name], out[name + "_scale"] = torch.cat(rows), scale
    return dict(k=out["k"], v=out["v"], k_scale=out["k_scale"], v_scale=out["v_scale"])


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "rotate":
        return _exact_rotate(c, s)
    if c["kind"] == "store":
        return _exact_store(c, s)
    if c["kind"] == "read":
        if s["total"] * c["hkv"] * c["d"] > 4e8:  # (gigabytes of 64-bit rows)
            return None
        return {name: torch.cat([_pages_of(s, name, b) for b in range(c["batch"])]) for name in "kv"}
    b, sq, hq, hkv, d = c["batch"], c["sq"], c["hq"], c["hkv"], c["d"]
    group = hq // hkv
    out = torch.zeros(b, sq, hq, d, dtype=F64, device="cuda")
    lse = torch.full((b, sq, hq), -math.inf, dtype=F64, device="cuda")
    for n in range(b):
        k, v = _pages_of(s, "k", n), _pages_of(s, "v", n)
        for i in range(int(s["q"][n])):
            seen = int(s["ctx"][n]) - int(s["q"][n]) + i + 1 if c["causal"] else int(s["ctx"][n])
            for g in range(hkv):
                at = slice(g * group, (g + 1) * group)
                logits = s["qx"][n, i, at].to(F64) @ k[:seen, g].T * s["scale"]
                lse[n, i, at] = torch.logsumexp(logits, -1)
                out[n, i, at] = torch.softmax(logits, -1) @ v[:seen, g]
    return dict(out=out, lse=lse)
