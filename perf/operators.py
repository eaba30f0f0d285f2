"""The serving operators around the paged decode: what is measured, and their plain forms.

A decode step over a paged cache, when the cache is held in 8 bits with one scale for each
(page, kv head) and a step attends only over the pages that a cheap score selects, is

    tables   the requests' new lengths become block tables and slot maps, on the GPU
    append   the step's new K/V rows go into their pages; each page's scale and each page's
             channel bounds of K follow
    score    every page's bounds against the query: an upper bound of the page's logits
    select   each row's best pages, in ascending order
    sparse   attention over the selected pages
    decode   attention over all pages (8-bit cache with a scale for each page and head)

`run` computes one of them, in its plain form or, where `own` is true, by the framework's calls.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest normal fp32: the least scale of a page
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
PAGES = (16, 32, 64, 128, 256, 512, 1024)


# ---- cases -------------------------------------------------------------------------------
def listed():
    return [
        # One decode step of a batch of chats: a few rows grow into a new page, some requests
        # end and give theirs back, some rejected draft tokens are rolled back.
        dict(name="tables_step_b64_sq4_bs16", kind="tables", batch=64, sq=4, bs=16,
             ctx_lo=512, ctx_hi=4096, fresh=False),
        # A batch of prompts of uneven lengths that starts from nothing: long slot maps.
        dict(name="tables_prompt_b48_bs32", kind="tables", batch=48, sq=16384, bs=32,
             ctx_lo=2048, ctx_hi=16384, fresh=True),
        # The new rows of one decode step; grouped-query cache.
        dict(name="append_step_b32_kv8_d128_bs16", kind="append", batch=32, sq=1, hkv=8, d=128,
             bs=16, prior_lo=511, prior_hi=4095, dtype="bf16"),
        # Prompts written in one call behind a cached prefix that ends inside a page.
        dict(name="append_prompt_b8_kv8_d128_bs64", kind="append", batch=8, sq=4096, hkv=8, d=128,
             bs=64, prior_lo=1, prior_hi=200, dtype="bf16"),
        # One new token for each sequence over long contexts in large pages.
        dict(name="decode_b64_h16_kv1_d128_bs1024_sq1", kind="decode", batch=64, sq=1, hq=16, hkv=1,
             d=128, bs=1024, ctx_lo=8192, ctx_hi=16384, causal=False, dtype="bf16"),
        # Four draft tokens a step, grouped-query heads, small pages.
        dict(name="decode_b32_h32_kv8_d128_bs16_sq4", kind="decode", batch=32, sq=4, hq=32, hkv=8,
             d=128, bs=16, ctx_lo=512, ctx_hi=4096, causal=True, dtype="bf16"),
        # Scores of a chat batch's pages: short rows, many heads.
        dict(name="score_b32_h32_kv8_d128_bs16", kind="score", batch=32, sq=1, hq=32, hkv=8, d=128,
             bs=16, ctx_lo=512, ctx_hi=4096, causal=False, dtype="bf16"),
        # Scores over very long contexts.
        dict(name="score_b32_h32_kv8_d128_bs64_long", kind="score", batch=32, sq=1, hq=32, hkv=8,
             d=128, bs=64, ctx_lo=32768, ctx_hi=131072, causal=False, dtype="bf16"),
        # A chat batch's selection.
        dict(name="select_b32_kv8_n256_k32", kind="select", batch=32, sq=1, hkv=8, bs=16,
             ctx_lo=512, ctx_hi=4096, top_k=32, first=1, last=2, causal=False, ties=False),
        # A long context's selection with draft tokens, scores that were kept in 16 bits (ties).
        dict(name="select_b32_kv8_sq4_n2048_k128", kind="select", batch=32, sq=4, hkv=8, bs=64,
             ctx_lo=32768, ctx_hi=131072, top_k=128, first=1, last=4, causal=True, ties=True),
        # The selected pages of a chat batch, 16-bit cache.
        dict(name="sparse_b32_h32_kv8_d128_bs16_k64", kind="sparse", batch=32, sq=1, hq=32, hkv=8,
             d=128, bs=16, ctx_lo=4096, ctx_hi=16384, top_k=64, causal=False, dtype="bf16", kv="16"),
        # One request over a very long context, 8-bit cache: few rows, latency.
        dict(name="sparse_b4_h16_kv1_d128_bs64_k32_fp8", kind="sparse", batch=4, sq=1, hq=16, hkv=1,
             d=128, bs=64, ctx_lo=32768, ctx_hi=131072, top_k=32, causal=True, dtype="bf16", kv="8"),
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
    ctx_hi = _log(rng, 64, 131072)
    ctx_lo = max(1, int(ctx_hi * rng.uniform(0.05, 1.0)))
    if kind == "tables":
        bs = rng.choice(PAGES[:5])
        fresh = rng.random() < 0.4
        ctx_hi = _log(rng, 64, 16384)
        sq = ctx_hi if fresh else _log(rng, 1, 16)
        return dict(kind=kind, batch=_log(rng, 1, 1000), sq=sq, bs=bs,
                    ctx_lo=max(16, int(ctx_hi * rng.uniform(0.1, 1.0))), ctx_hi=max(16, ctx_hi),
                    fresh=fresh)
    if kind == "append":
        return dict(kind=kind, batch=_log(rng, 1, 128), sq=_log(rng, 1, 4096), hkv=hkv, d=d, bs=bs,
                    prior_lo=rng.randrange(0, 100), prior_hi=_log(rng, 100, 4000), dtype=dtype)
    if kind == "decode":
        return dict(kind=kind, batch=_log(rng, 1, 64), sq=rng.choice((1, 1, 2, 3, 4, 8)),
                    hq=hkv * group, hkv=hkv, d=d, bs=bs, ctx_lo=max(16, ctx_lo),
                    ctx_hi=max(16, ctx_hi), causal=rng.random() < 0.5, dtype=dtype)
    if kind == "score":
        return dict(kind=kind, batch=_log(rng, 1, 64), sq=rng.choice((1, 1, 2, 4, 7)),
                    hq=hkv * group, hkv=hkv, d=d, bs=bs, ctx_lo=max(16, ctx_lo),
                    ctx_hi=max(16, ctx_hi), causal=rng.random() < 0.5, dtype=dtype)
    if kind == "select":
        first, last = rng.randrange(0, 4), rng.randrange(0, 6)
        return dict(kind=kind, batch=_log(rng, 1, 64), sq=rng.choice((1, 1, 2, 4, 7)), hkv=hkv,
                    bs=rng.choice(PAGES[:5]), ctx_lo=max(16, ctx_lo), ctx_hi=max(16, ctx_hi),
                    top_k=max(first + last, _log(rng, 1, 512)), first=first, last=last,
                    causal=rng.random() < 0.5, ties=rng.random() < 0.3)
    return dict(kind=kind, batch=_log(rng, 1, 64), sq=rng.choice((1, 1, 2, 3, 4)), hq=hkv * group,
                hkv=hkv, d=d, bs=rng.choice(PAGES[:5]), ctx_lo=max(16, ctx_lo),
                ctx_hi=max(16, ctx_hi), top_k=_log(rng, 1, 256), causal=rng.random() < 0.5,
                dtype=dtype, kv=rng.choice(("16", "8")))


def _held_bytes(c):
    """About what prepare() puts on the card, and the plain form's largest temporary, in 32 bits."""
    if c["kind"] in ("tables", "select"):
        return c["batch"] * c["sq"] * 8 * (c["ctx_hi"] // c["bs"] if c["kind"] == "select" else 4)
    if c["kind"] == "append":
        return 3 * c["batch"] * (c["sq"] + c["prior_hi"] + 2 * c["bs"]) * c["hkv"] * c["d"] * 8
    tokens = c["batch"] * (-(-c["ctx_hi"] // c["bs"])) * c["bs"]
    if c["kind"] == "score":
        return tokens // c["bs"] * c["hkv"] * c["d"] * 16
    logits = tokens * c["sq"] * c["hq"] * 4
    if c["kind"] == "decode":
        return tokens * c["hkv"] * c["d"] * 10 + 3 * logits
    per = c["batch"] * c["sq"] * c["hkv"] * c["top_k"] * c["bs"] * c["d"] * 10
    return tokens * c["hkv"] * c["d"] * 6 + per


def draw(rng):
    kind = rng.choice(("tables", "append", "decode", "score", "select", "sparse"))
    most = {c["kind"]: max(work(x)["bytes"] for x in listed() if x["kind"] == c["kind"]) for c in listed()}
    c = _drawn(rng, kind)
    while work(c)["bytes"] > most[kind] or _held_bytes(c) > 4e9:  # no more than the largest listed
        c = _drawn(rng, kind)
    return c


# ---- what a case cannot do without ---------------------------------------------------------
def _lens(case, lo, hi):
    """The batch's lengths, evenly spread from lo to hi: the same ones for every seed."""
    b = case["batch"]
    return [lo + (hi - lo) * j // max(1, b - 1) for j in range(b)] if b > 1 else [hi]


def work(case):
    c = case
    kind, b, bs, sq = c["kind"], c["batch"], c["bs"], c["sq"]
    if kind == "append":
        q = _lens(c, 1, sq)
        rows = sum(q) * c["hkv"]
        pages = sum(-(-(n % bs + m) // bs) for n, m in zip(_lens(c, c["prior_lo"], c["prior_hi"]), q)) * c["hkv"]
        # new K and V rows in, their codes out; a page's two scales and its bounds out
        return dict(bytes=rows * c["d"] * (2 * 2 + 2) + pages * (8 + 4 * c["d"]), flops=rows * c["d"] * 8)
    lens = _lens(c, c["ctx_lo"], c["ctx_hi"])
    pages = sum(-(-n // bs) for n in lens)
    if kind == "tables":
        moved = pages if c["fresh"] else b
        return dict(bytes=b * sq * 8 + moved * 8 + b * 16, flops=0)
    rows = b * sq
    if kind == "score":
        out = rows * c["hkv"] * -(-max(lens) // bs) * 4
        return dict(bytes=pages * c["hkv"] * c["d"] * 4 + rows * c["hq"] * c["d"] * 2 + out + pages * 4,
                    flops=4 * pages * sq * c["hq"] * c["d"])
    if kind == "select":
        return dict(bytes=(pages * sq * 4 + rows * (c["top_k"] + 1) * 4) * c["hkv"], flops=pages * sq * c["hkv"])
    io = rows * c["hq"] * (c["d"] * 4 + 4)
    if kind == "decode":
        return dict(bytes=sum(lens) * c["hkv"] * c["d"] * 2 + pages * (c["hkv"] * 8 + 4) + io,
                    flops=4 * sum(lens) * sq * c["hq"] * c["d"])
    tokens = sum(min(n, c["top_k"] * bs) for n in lens) * sq
    wide = 2 if c["kv"] == "16" else 1
    chosen = sum(min(-(-n // bs), c["top_k"]) for n in lens) * sq * c["hkv"]
    return dict(bytes=tokens * c["hkv"] * c["d"] * 2 * wide + chosen * (8 + 8 * (2 - wide)) + io,
                flops=4 * tokens * c["hq"] * c["d"])


# ---- inputs ----------------------------------------------------------------------------------
def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _codes(shape, g):
    """E4M3 codes of a page that was quantised over its largest value."""
    return (_randn(shape, g, torch.float16) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(shape, g):
    return (torch.rand(shape, generator=g, device="cuda") * 0.6 + 0.7) * 0.01


def _permuted(values, g):
    at = torch.randperm(len(values), generator=g, device="cuda")
    return torch.tensor(values, dtype=torch.int32, device="cuda")[at]


def _tables(pages, columns, pool, g):
    """Block tables of sequences with `pages` pages each, out of a shuffled pool; -1 behind."""
    perm = torch.randperm(pool, generator=g, device="cuda")
    start = torch.cumsum(pages, 0) - pages
    col = torch.arange(columns, device="cuda")
    at = (start[:, None] + col).clamp(max=pool - 1)
    return torch.where(col < pages[:, None], perm[at], -1).to(torch.int32), perm


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, b, bs, sq = c["kind"], c["batch"], c["bs"], c["sq"]
    s = dict(case=c)
    if kind == "append":
        q = _permuted(_lens(c, 1, sq), g)
        ctx = _permuted(_lens(c, c["prior_lo"], c["prior_hi"]), g) + q
    else:
        ctx = _permuted(_lens(c, c["ctx_lo"], c["ctx_hi"]), g)
        q = ctx.clamp(max=sq)
    if kind == "tables":
        if not c["fresh"]:
            # one in eight requests ended, one in eight rejected some draft tokens, one in
            # eight took fewer tokens than the others
            part = torch.arange(b, device="cuda") % 8
            before = torch.where(part == 6, ctx + sq + bs, ctx - q)
            ctx = torch.where(part == 7, 0, ctx)
            q = torch.where(part == 7, 0, torch.where(part == 5, q // 2, q))
        else:
            before = torch.zeros_like(ctx)
        held = (before + bs - 1) // bs
        columns = -(-(c["ctx_hi"] + 2 * bs + sq) // bs)
        pool = b * columns + 64
        bt, perm = _tables(held, columns, pool, g)
        used = held.sum()
        at = (used + torch.arange(pool, device="cuda")).clamp(max=pool - 1)
        s.update(ctx=ctx.to(torch.int32), q=q.to(torch.int32), held=held.to(torch.int32), bt=bt,
                 free=perm[at].to(torch.int32), count=(pool - used).to(torch.int32).reshape(1),
                 new_held=torch.empty_like(held, dtype=torch.int32),
                 new_count=torch.empty(1, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(b, sq, dtype=torch.int64, device="cuda"), pool=pool)
        return s
    s.update(ctx=ctx, q=q)
    longest = c["prior_hi"] + sq if kind == "append" else c["ctx_hi"]
    columns = -(-longest // bs)
    pages = (ctx + bs - 1) // bs
    if kind == "select":
        rows = (b, sq, c["hkv"])
        x = _randn((*rows, columns), g, torch.float32) * 3 + _randn((*rows, 1), g, torch.float32)
        s.update(scores=x.to(torch.bfloat16).float() if c["ties"] else x, columns=columns,
                 sel=torch.empty(*rows, c["top_k"], dtype=torch.int32, device="cuda"),
                 num=torch.empty(rows, dtype=torch.int32, device="cuda"))
        return s
    hkv, d, t = c["hkv"], c["d"], TYPES[c["dtype"]]
    lens = [x + m for x, m in zip(sorted(_lens(c, c["prior_lo"], c["prior_hi"])), _lens(c, 1, sq))] if kind == "append" else _lens(c, c["ctx_lo"], c["ctx_hi"])
    pool = sum(-(-n // bs) for n in lens) + (b if kind == "append" else 0) + 3
    bt, _ = _tables(pages, columns, pool, g)
    s.update(bt=bt, pool=pool)
    if kind == "append":
        # a row in sixteen is an outlier: it raises the scale of the page it falls into
        gain = torch.where(torch.rand((b, sq, 1, 1), generator=g, device="cuda") < 1 / 16, 4.0, 1.0)
        lo = _randn((pool, hkv, d), g, torch.float32)
        s.update(k=(_randn((b, sq, hkv, d), g, torch.float32) * gain).to(t),
                 v=(_randn((b, sq, hkv, d), g, torch.float32) * gain).to(t),
                 kc=_codes((pool, bs, hkv, d), g), vc=_codes((pool, bs, hkv, d), g),
                 ks=_scales((pool, hkv), g), vs=_scales((pool, hkv), g),
                 bounds=torch.stack((lo - 1.5, lo + 1.5), 2).to(t).contiguous())
        return s
    hq = c["hq"]
    s.update(qx=_randn((b, sq, hq, d), g, torch.float32).to(t), scale=1.0 / math.sqrt(d))
    if kind == "score":
        mid = _randn((pool, hkv, d), g, torch.float16) * 0.5
        wide = torch.rand((pool, hkv, d), generator=g, device="cuda", dtype=torch.float16) * 2 + 0.5
        s.update(bounds=torch.stack((mid - wide, mid + wide), 2).to(t).contiguous(),
                 scores=torch.empty(b, sq, hkv, columns, dtype=torch.float32, device="cuda"))
        return s
    wide = kind == "sparse" and c["kv"] == "16"
    if wide:
        s.update(kc=_randn((pool, bs, hkv, d), g, t), vc=_randn((pool, bs, hkv, d), g, t), ks=None, vs=None)
    else:
        s.update(kc=_codes((pool, bs, hkv, d), g), vc=_codes((pool, bs, hkv, d), g),
                 ks=_scales((pool, hkv), g), vs=_scales((pool, hkv), g))
    s.update(out=torch.empty_like(s["qx"]), lse=torch.empty(b, sq, hq, dtype=torch.float32, device="cuda"))
    if kind == "sparse":
        # distinct pages of the sequence in ascending order, the newest always among them
        k = min(c["top_k"], columns)
        key = torch.rand((b, sq, hkv, columns), generator=g, device="cuda")
        col = torch.arange(columns, device="cuda")
        n = pages[:, None, None, None]
        key = torch.where(col == n - 1, 2.0, torch.where(col < n, key, -1.0))
        best = key.topk(k, -1)
        sel = torch.where(best.values >= 0, best.indices, columns).sort(-1).values
        num = pages.clamp(max=c["top_k"])[:, None, None].expand(b, sq, hkv).contiguous()
        sel = torch.where(torch.arange(k, device="cuda") < num[..., None], sel, -1).to(torch.int32)
        s.update(sel=torch.nn.functional.pad(sel, (0, c["top_k"] - k), value=-1).contiguous(), num=num)
    return s


# ---- the plain forms -----------------------------------------------------------------------------
def _seen(s, rows):
    """[B, rows]: the keys that each new-token row sees (0 for padding rows)."""
    i = torch.arange(rows, device="cuda")
    n, q = s["ctx"][:, None], s["q"][:, None]
    return torch.where(i < q, n - q + i + 1 if s["case"]["causal"] else n, 0)


def _plain_tables(s):
    c = s["case"]
    bs, bt, held, pool = c["bs"], s["bt"], s["held"][:, None], s["pool"]
    n, q, count = s["ctx"], s["q"], s["count"]
    need = ((n + bs - 1) // bs)[:, None]
    col = torch.arange(bt.shape[1], device="cuda")
    give, take = (col >= need) & (col < held), (col >= held) & (col < need)
    given, taken = give.sum(1, keepdim=True), take.sum(1, keepdim=True)
    at = count + torch.cumsum(given, 0) - given + col - need
    stack = torch.cat((s["free"], s["free"][:1]))
    stack.scatter_(0, torch.where(give, at, pool).reshape(-1), bt.reshape(-1))
    top = count + given.sum()
    at = top - 1 - (torch.cumsum(taken, 0) - taken + col - held)
    new_bt = torch.where(take, stack[at.clamp(0, pool)], bt)
    left = top - taken.sum()
    free = torch.where(torch.arange(pool, device="cuda") < left, stack[:pool], s["free"])
    i = torch.arange(c["sq"], device="cuda")
    pos = (n - q)[:, None] + i
    page = new_bt.gather(1, (pos // bs).clamp(0, bt.shape[1] - 1))
    slots = torch.where(i < q[:, None], page.to(torch.int64) * bs + pos % bs, -1)
    return dict(tables=new_bt, free=free, held=need[:, 0].to(torch.int32), count=left.to(torch.int32), slots=slots)


def _paged_rows(s, x):
    """New rows [B, Sq, ...] laid out by the pages they go to: [B, P, bs, ...], and which are new."""
    c = s["case"]
    bs = c["bs"]
    prior = (s["ctx"] - s["q"])[:, None]
    pages = (bs - 1 + c["sq"] + bs - 1) // bs
    t = torch.arange(pages * bs, device="cuda")
    i = t - prior % bs
    new = (i >= 0) & (i < s["q"][:, None])
    rows = x[torch.arange(c["batch"], device="cuda")[:, None], i.clamp(0, c["sq"] - 1)]
    return rows.reshape(c["batch"], pages, bs, *x.shape[2:]), new.reshape(c["batch"], pages, bs)


def _touched(s, pages):
    """[B, P]: the blocks of the touched pages, and whether there is such a page."""
    bs = s["case"]["bs"]
    first = ((s["ctx"] - s["q"]) // bs)[:, None]
    j = torch.arange(pages, device="cuda") + first
    there = (j * bs < s["ctx"][:, None]) & (s["q"][:, None] > 0)
    return torch.where(there, s["bt"].gather(1, j.clamp(max=s["bt"].shape[1] - 1)), 0), there


def _put(pool, blk, there, pages):
    """The pool with the touched pages in their blocks."""
    n = pool.shape[0]
    of = torch.full((n + 1,), -1, dtype=torch.int64, device="cuda")
    of.scatter_(0, torch.where(there, blk, n).reshape(-1), torch.arange(blk.numel(), device="cuda"))
    of = of[:n]
    new = pages.reshape(-1, *pool.shape[1:])[of.clamp(min=0)]
    return torch.where((of >= 0).reshape(-1, *([1] * (pool.dim() - 1))), new, pool)


def _plain_quantised(s, x, codes, scale):
    rows, new = _paged_rows(s, x.float())
    blk, there = _touched(s, rows.shape[1])
    is_new = new[..., None, None]
    big = torch.where(is_new & rows.isfinite(), rows.abs(), 0).amax((2, 4))  # [B, P, Hkv]
    want = torch.where(big > 0, (big / E4M3_MAX).clamp(min=TINY), 0)
    old_scale = scale[blk]
    to = torch.where(new[:, :, :1], torch.where(want > 0, want, 1), torch.maximum(old_scale, want))
    old = codes[blk].view(torch.float8_e4m3fn).float()
    wide, was = to[:, :, None, :, None], old_scale[:, :, None, :, None]
    kept = torch.where(to > old_scale, 1, 0)[:, :, None, :, None] > 0
    value = torch.where(is_new, rows / wide, torch.where(kept, old * was / wide, old))
    value = value.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    # what stands behind the newest token of a page, or before a fresh page's first, is left as it was
    t = torch.arange(s["case"]["bs"], device="cuda")
    end = (s["ctx"][:, None] - ((s["ctx"] - s["q"]) // s["case"]["bs"] * s["case"]["bs"])[:, None]
           - torch.arange(rows.shape[1], device="cuda") * s["case"]["bs"])
    value = torch.where((t < end[..., None])[..., None, None], value, codes[blk])
    return _put(codes, blk, there, value).view(torch.float8_e4m3fn), _put(scale, blk, there, to)


def _plain_bounds(s):
    rows, new = _paged_rows(s, s["k"])
    blk, there = _touched(s, rows.shape[1])
    is_new = new[..., None, None]
    lo = torch.where(is_new, rows, math.inf).amin(2)
    hi = torch.where(is_new, rows, -math.inf).amax(2)
    old = s["bounds"][blk]
    fresh = new[:, :, 0, None, None]
    lo = torch.where(fresh, lo, torch.minimum(lo, old[:, :, :, 0]))
    hi = torch.where(fresh, hi, torch.maximum(hi, old[:, :, :, 1]))
    return _put(s["bounds"], blk, there, torch.stack((lo, hi), 3))


def _plain_append(s):
    k, ks = _plain_quantised(s, s["k"], s["kc"], s["ks"])
    v, vs = _plain_quantised(s, s["v"], s["vc"], s["vs"])
    return dict(k=k, v=v, k_scale=ks, v_scale=vs, bounds=_plain_bounds(s))


def _plain_score(s):
    c = s["case"]
    b, sq, hkv, d = c["batch"], c["sq"], c["hkv"], c["d"]
    x = s["qx"].float().reshape(b, sq, hkv, -1, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    y = s["bounds"][s["bt"].clamp(min=0)].float().permute(0, 2, 3, 4, 1)  # [B, Hkv, 2, D, pages]
    # max(q lo, q hi) is q hi for a positive q and q lo for a negative one
    dot = x.clamp(min=0) @ y[:, :, 1] + x.clamp(max=0) @ y[:, :, 0]
    best = (dot * s["scale"]).reshape(b, hkv, sq, -1, y.shape[-1]).amax(3).permute(0, 2, 1, 3)
    pages = (_seen(s, sq) + c["bs"] - 1) // c["bs"]
    col = torch.arange(y.shape[-1], device="cuda")
    return torch.where(col < pages[:, :, None, None], best, -math.inf).contiguous()


def _plain_select(s):
    c = s["case"]
    n = ((_seen(s, c["sq"]) + c["bs"] - 1) // c["bs"])[:, :, None, None]
    col = torch.arange(s["columns"], device="cuda")
    # forced pages above every score, pages out of the row's reach below; a stable descending
    # sort leaves the lowest index first among equals
    x = torch.where((col < c["first"]) | (col >= n - c["last"]), math.inf, s["scores"])
    x = torch.where(col < n, x, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    k = min(c["top_k"], s["columns"])
    num = n[..., 0].clamp(max=c["top_k"]).expand(-1, -1, c["hkv"])
    j = torch.arange(k, device="cuda")
    sel = torch.where(j < num[..., None], order[..., :k], s["columns"]).sort(-1).values
    sel = torch.where(j < num[..., None], sel, -1).to(torch.int32)
    return dict(pages=torch.nn.functional.pad(sel, (0, c["top_k"] - k), value=-1), num=num.to(torch.int32))


def _attend(s, logits, v):
    """Softmax over the last axis (all masked: zero) and the weighted sum: rows [..., R, T] on [..., T, D]."""
    big = logits.amax(-1, keepdim=True)
    big = torch.where(big.isfinite(), big, 0)
    p = torch.exp(logits - big)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0)
    return out, (big + torch.log(total))[..., 0]


def _values(s, cache, scale):
    """Cache rows [..., bs, Hkv, D] with their pages' scales [..., Hkv] as fp32."""
    if scale is None:
        return cache.float()
    return cache.view(torch.float8_e4m3fn).float() * scale[..., None, :, None]


def _plain_decode(s):
    c = s["case"]
    b, sq, hkv, d, t = c["batch"], c["sq"], c["hkv"], c["d"], TYPES[c["dtype"]]
    at = s["bt"].clamp(min=0)
    k = _values(s, s["kc"][at], s["ks"][at]).reshape(b, -1, hkv, d).permute(0, 2, 3, 1)
    v = _values(s, s["vc"][at], s["vs"][at]).reshape(b, -1, hkv, d).permute(0, 2, 1, 3)
    x = s["qx"].float().reshape(b, sq, hkv, -1, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    seen = _seen(s, sq)[:, None, :, None, None]
    logits = (x @ k * s["scale"]).reshape(b, hkv, sq, -1, k.shape[-1])
    logits = torch.where(torch.arange(k.shape[-1], device="cuda") < seen, logits, -math.inf)
    out, lse = _attend(s, logits.reshape(b, hkv, -1, k.shape[-1]), v)
    out = out.reshape(b, hkv, sq, -1, d).permute(0, 2, 1, 3, 4).reshape(b, sq, -1, d)
    return dict(out=out.to(t), lse=lse.reshape(b, hkv, sq, -1).permute(0, 2, 1, 3).reshape(b, sq, -1))


def _plain_sparse(s):
    c = s["case"]
    b, sq, hkv, d, bs, t = c["batch"], c["sq"], c["hkv"], c["d"], c["bs"], TYPES[c["dtype"]]
    sel, num = s["sel"].clamp(min=0), s["num"]
    blk = s["bt"].gather(1, sel.reshape(b, -1)).reshape(sel.shape).clamp(min=0)  # [B, Sq, Hkv, K]
    head = torch.arange(hkv, device="cuda")[:, None]
    wide = c["kv"] == "16"
    k = s["kc"].permute(0, 2, 1, 3)[blk, head]  # [B, Sq, Hkv, K, bs, D]
    v = s["vc"].permute(0, 2, 1, 3)[blk, head]
    k = k.float() if wide else k.view(torch.float8_e4m3fn).float() * s["ks"][blk, head][..., None, None]
    v = v.float() if wide else v.view(torch.float8_e4m3fn).float() * s["vs"][blk, head][..., None, None]
    k, v = k.reshape(b, sq, hkv, -1, d), v.reshape(b, sq, hkv, -1, d)
    pos = sel[..., None] * bs + torch.arange(bs, device="cuda")
    ok = (pos < _seen(s, sq)[:, :, None, None, None]) & (torch.arange(sel.shape[-1], device="cuda") < num[..., None])[..., None]
    x = s["qx"].float().reshape(b, sq, hkv, -1, d)
    logits = x @ k.transpose(-1, -2) * s["scale"]
    logits = torch.where(ok.reshape(b, sq, hkv, 1, -1), logits, -math.inf)
    out, lse = _attend(s, logits, v)
    return dict(out=out.reshape(b, sq, -1, d).to(t), lse=lse.reshape(b, sq, -1))


# ---- the framework's calls ---------------------------------------------------------------------
def _config(s, pa):
    """The problem's pa_config, which a user's program keeps."""
    if "cfg" not in s:
        c = s["case"]
        code = {"bf16": pa.BF16, "fp16": pa.FP16}[c.get("dtype", "bf16")]
        kind = c["kind"]
        eight = kind in ("append", "decode") or c.get("kv") == "8"
        hkv = c.get("hkv", 1)
        columns = s["scores"].shape[-1] if kind == "select" else s["bt"].shape[1]
        s["cfg"] = pa.PaConfig(
            batch=c["batch"], max_q_len=c["sq"], num_q_heads=c.get("hq", hkv), num_kv_heads=hkv,
            head_dim=c.get("d", 128), block_size=c["bs"], max_blocks_per_seq=columns,
            num_blocks=s.get("pool", 1), q_dtype=code, kv_dtype=pa.FP8_E4M3 if eight else code,
            kv_scale_mode=pa.SCALE_PER_BLOCK if eight else pa.SCALE_NONE,
            causal=int(c.get("causal", False)), sm_scale=s.get("scale", 1.0))
    return s["cfg"]


def _own(s):
    import paged_kv_cache_work_gb300 as pa

    c, cfg = s["case"], _config(s, pa)
    kind = c["kind"]
    if kind == "tables":
        pa.build_tables(cfg, s["ctx"], s["q"], s["held"], s["bt"], s["free"], s["count"],
                        s["new_held"], s["new_count"], s["slots"])
        return dict(tables=s["bt"], free=s["free"], held=s["new_held"], count=s["new_count"], slots=s["slots"])
    if kind == "append":
        pa.append_kv(cfg, s["k"], s["v"], s["bt"], s["ctx"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"])
        pa.update_bounds(cfg, s["k"], s["bt"], s["ctx"], s["q"], s["bounds"])
        return dict(k=s["kc"].view(torch.float8_e4m3fn), v=s["vc"].view(torch.float8_e4m3fn),
                    k_scale=s["ks"], v_scale=s["vs"], bounds=s["bounds"])
    if kind == "score":
        pa.score_blocks(cfg, s["qx"], s["bounds"], s["bt"], s["ctx"], s["q"], s["scores"])
        return s["scores"]
    if kind == "select":
        pa.select_blocks(cfg, s["scores"], s["ctx"], s["q"], c["first"], c["last"], s["sel"], s["num"])
        return dict(pages=s["sel"], num=s["num"])
    if kind == "sparse":
        pa.decode_selected(cfg, s["qx"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], s["q"],
                           s["sel"], s["num"], s["out"], s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if "ws" not in s:
        s["ws"] = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device="cuda")
    pa.plan(cfg, s["bt"], s["ctx"], s["q"], s["ws"])
    pa.decode(cfg, s["qx"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], s["q"], s["out"], s["lse"], s["ws"])
    pa.reduce(cfg, s["out"], s["lse"], s["ws"])
    return dict(out=s["out"], lse=s["lse"])


_PLAIN = dict(tables=_plain_tables, append=_plain_append, decode=_plain_decode, score=_plain_score,
              select=_plain_select, sparse=_plain_sparse)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ---- from the definition, in 64 bits -----------------------------------------------------------
def _exact_append(c, s):
    """Token by token: each page's largest value, and every value over its page's scale."""
    bs, f64 = c["bs"], torch.float64
    res = {}
    n, q, bt = s["ctx"].tolist(), s["q"].tolist(), s["bt"].tolist()
    tabs = [(b, p) for b in range(c["batch"]) for p in range((n[b] - q[b]) // bs, -(-n[b] // bs))]
    for name, x, codes, scale in (("k", s["k"], s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        value, to = codes.view(torch.float8_e4m3fn).to(f64), scale.to(f64).clone()
        for b, p in tabs:
            old = n[b] - q[b]
            lo, hi = max(p * bs, old), min((p + 1) * bs, n[b])
            rows = x[b, lo - old:hi - old].to(f64)
            want = (rows.abs().amax((0, 2)) / E4M3_MAX).clamp(min=TINY)
            blk = bt[b][p]
            if lo > p * bs:
                was = to[blk].clone()
                want = torch.maximum(was, want)
                value[blk, :lo - p * bs] *= (was / want)[None, :, None]
            value[blk, lo - p * bs:hi - p * bs] = rows / want[None, :, None]
            to[blk] = want
        res[name], res[name + "_scale"] = value, to
    bounds = s["bounds"].to(f64)
    for b, p in tabs:
        old = n[b] - q[b]
        lo, hi = max(p * bs, old), min((p + 1) * bs, n[b])
        rows = s["k"][b, lo - old:hi - old].to(f64)
        least, most = rows.amin(0), rows.amax(0)
        blk = bt[b][p]
        if lo > p * bs:
            least, most = torch.minimum(least, bounds[blk, :, 0]), torch.maximum(most, bounds[blk, :, 1])
        bounds[blk, :, 0], bounds[blk, :, 1] = least, most
    return dict(res, bounds=bounds)


def exact(case, seed):
    c = case
    kind = c["kind"]
    if kind in ("tables", "select"):
        return None
    if kind == "append" and c["batch"] * (c["sq"] // c["bs"] + 1) > 20000:
        return None
    s = prepare(case, seed)
    if kind == "append":
        return _exact_append(c, s)
    f64, b, sq, hq, hkv, d, bs = torch.float64, c["batch"], c["sq"], c["hq"], c["hkv"], c["d"], c["bs"]
    group = hq // hkv
    ctx, q = s["ctx"].tolist(), s["q"].tolist()
    if kind == "score":
        out = torch.full(s["scores"].shape, -math.inf, dtype=f64, device="cuda")
        for n in range(b):
            box = s["bounds"][s["bt"][n, :-(-ctx[n] // bs)].long()].to(f64)  # [pages, Hkv, 2, D]
            for i in range(q[n]):
                pages = -(-(ctx[n] - q[n] + i + 1 if c["causal"] else ctx[n]) // bs)
                for g in range(hkv):
                    ends = [s["qx"][n, i, g * group + h].to(f64) * box[:pages, g] for h in range(group)]
                    out[n, i, g, :pages] = torch.stack([e.amax(1).sum(1) for e in ends]).amax(0) * s["scale"]
        return out
    out = torch.zeros(b, sq, hq, d, dtype=f64, device="cuda")
    lse = torch.full((b, sq, hq), -math.inf, dtype=f64, device="cuda")
    for n in range(b):
        for i in range(q[n]):
            seen = ctx[n] - q[n] + i + 1 if c["causal"] else ctx[n]
            for g in range(hkv):
                if kind == "sparse":
                    pages = s["sel"][n, i, g, :int(s["num"][n, i, g])].long()
                else:
                    pages = torch.arange(-(-seen // bs), device="cuda")
                blk = s["bt"][n, pages].long()
                k, v = s["kc"][blk, :, g], s["vc"][blk, :, g]
                if s["ks"] is not None:
                    k = k.view(torch.float8_e4m3fn).to(f64) * s["ks"][blk, g].to(f64)[:, None, None]
                    v = v.view(torch.float8_e4m3fn).to(f64) * s["vs"][blk, g].to(f64)[:, None, None]
                token = (pages[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
                k, v = k.to(f64).reshape(-1, d)[token < seen], v.to(f64).reshape(-1, d)[token < seen]
                at = slice(g * group, (g + 1) * group)
                logits = s["qx"][n, i, at].to(f64) @ k.T * s["scale"]
                lse[n, i, at] = torch.logsumexp(logits, -1)
                out[n, i, at] = torch.softmax(logits, -1) @ v
    return dict(out=out, lse=lse)
