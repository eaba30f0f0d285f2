"""Plain implementations, row by row, of the table, append, bounds, score, select and sparse
decode calls: integers and Python loops, fp32 where the call defines its rounding, 64 bits
everywhere else.  They share no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3_MAX = 448.0


def pages(n, bs):
    return -(-n // bs)


def seen(ctx, ql, i, causal):
    """Keys that new-token row i of a sequence sees."""
    if i >= ql:
        return 0
    return ctx - ql + i + 1 if causal else ctx


def build_tables(ctx, ql, held, bt, free, count, bs, sq):
    """(tables, free list, held, count, slots) after the call; needs enough free pages."""
    bt, free = [list(r) for r in bt], list(free)
    stack = free[:count]
    need = [pages(n, bs) for n in ctx]
    for b, n in enumerate(need):
        stack += bt[b][n:held[b]]
    for b, n in enumerate(need):
        for p in range(held[b], n):
            bt[b][p] = stack.pop()
    free[:len(stack)] = stack
    slots = [[-1] * sq for _ in ctx]
    for b in range(len(ctx)):
        for i in range(ql[b]):
            pos = ctx[b] - ql[b] + i
            slots[b][i] = bt[b][pos // bs] * bs + pos % bs
    return bt, free, need, len(stack), slots


def _e4m3(x):
    return torch.from_numpy(np.clip(x, -E4M3_MAX, E4M3_MAX)).to(torch.float8_e4m3fn).view(torch.uint8)


def append_block(new, codes, scale, ctx, ql, bt, bs):
    """Codes and scales (copies) after appending rows `new` [B, Sq, Hkv, D] one page at a time;
    every step in fp32 as the call defines it."""
    codes, scale = codes.clone(), scale.clone()
    x = new.float()
    for b in range(new.shape[0]):
        first = ctx[b] - ql[b]
        for page in range(first // bs, pages(ctx[b], bs)):
            lo, hi = max(page * bs, first), min((page + 1) * bs, ctx[b])
            if lo >= hi:
                continue
            blk = bt[b][page]
            for g in range(new.shape[2]):
                rows = x[b, lo - first:hi - first, g].numpy()
                a = np.abs(rows[np.isfinite(rows)]).max(initial=np.float32(0))
                w = max(np.float32(a) / np.float32(E4M3_MAX), np.float32(2.0 ** -126)) if a > 0 else np.float32(0)
                fresh = lo == page * bs
                old = np.float32(scale[blk, g])
                s = (w if w > 0 else np.float32(1)) if fresh else max(old, w)
                if not fresh and s > old:
                    kept = codes[blk, :lo - page * bs, g].view(torch.float8_e4m3fn).float().numpy()
                    codes[blk, :lo - page * bs, g] = _e4m3(kept * old / s)
                scale[blk, g] = float(s)
                with np.errstate(invalid="ignore", over="ignore"):
                    codes[blk, lo - page * bs:hi - page * bs, g] = _e4m3(rows / s)
    return codes, scale


def update_bounds(new, bounds, ctx, ql, bt, bs):
    bounds = bounds.clone()
    for b in range(new.shape[0]):
        first = ctx[b] - ql[b]
        for page in range(first // bs, pages(ctx[b], bs)):
            lo, hi = max(page * bs, first), min((page + 1) * bs, ctx[b])
            if lo >= hi:
                continue
            blk = bt[b][page]
            rows = new[b, lo - first:hi - first].float()
            least, most = rows.amin(0), rows.amax(0)  # both keep NaN
            if lo > page * bs:
                least = torch.minimum(least, bounds[blk, :, 0].float())
                most = torch.maximum(most, bounds[blk, :, 1].float())
            bounds[blk, :, 0], bounds[blk, :, 1] = least.to(bounds.dtype), most.to(bounds.dtype)
    return bounds


def score(q, bounds, ctx, ql, bt, bs, causal, sm_scale, hkv, nblocks):
    """(scores, the sum of the magnitudes that enter each: what its rounding is measured by)."""
    B, sq, hq, d = q.shape
    group, cols = hq // hkv, len(bt[0])
    out = np.full((B, sq, hkv, cols), -np.inf)
    size = np.zeros((B, sq, hkv, cols))
    x, box = q.double().numpy(), bounds.double().numpy()
    for b in range(B):
        for i in range(ql[b]):
            for p in range(pages(seen(ctx[b], ql[b], i, causal), bs)):
                blk = bt[b][p]
                if not 0 <= blk < nblocks:
                    continue
                for g in range(hkv):
                    rows = x[b, i, g * group:(g + 1) * group]
                    with np.errstate(invalid="ignore"):
                        up, dn = np.maximum(rows, 0) * box[blk, g, 1], np.minimum(rows, 0) * box[blk, g, 0]
                        out[b, i, g, p] = np.max((up + dn).sum(1)) * sm_scale  # NaN wins
                    size[b, i, g, p] = np.max((np.abs(up) + np.abs(dn)).sum(1)) * abs(sm_scale)
    return out, size


def select(scores, ctx, ql, bs, causal, top_k, first, last):
    B, sq, hkv, _ = scores.shape
    sel = np.full((B, sq, hkv, top_k), -1, np.int32)
    num = np.zeros((B, sq, hkv), np.int32)
    for b in range(B):
        for i in range(sq):
            n = pages(seen(ctx[b], ql[b], i, causal), bs)
            for g in range(hkv):
                def rank(p):
                    if p < first or p >= n - last:
                        return (0, 0.0, p)
                    x = float(scores[b, i, g, p])
                    return (1, 0.0, p) if math.isnan(x) else (2, -x, p)
                best = sorted(sorted(range(n), key=rank)[:top_k])
                sel[b, i, g, :len(best)] = best
                num[b, i, g] = len(best)
    return sel, num


def values(cache, scale, mode):
    """A cache's values [nb, bs, Hkv, D] in 64 bits."""
    if cache.dtype != torch.uint8:
        return cache.double().numpy()
    v = cache.view(torch.float8_e4m3fn).double().numpy()
    if mode == "tensor":
        return v * float(scale[0])
    if mode == "token":
        return v * scale.double().numpy()[..., None]
    if mode == "block":
        return v * scale.double().numpy()[:, None, :, None]
    return v


def attend(q, k, v, bt, lists, ctx, ql, causal, sm_scale):
    """Softmax attention of each row over the tokens of its pages `lists(b, i, g)`; also sum_j p_j
    |v_j|, which the rounding of the weights is measured by.  k, v: [nb, bs, Hkv, D], 64 bits."""
    B, sq, hq, d = q.shape
    bs, hkv = k.shape[1], k.shape[2]
    group = hq // hkv
    out, size = np.zeros((B, sq, hq, d)), np.zeros((B, sq, hq, d))
    lse = np.full((B, sq, hq), -np.inf)
    x = q.double().numpy()
    for b in range(B):
        for i in range(sq):
            lim = seen(ctx[b], ql[b], i, causal)
            for g in range(hkv):
                at = [(bt[b][p], p * bs + t, t) for p in lists(b, i, g) for t in range(bs) if p * bs + t < lim]
                if not at:
                    continue
                blk, slot = np.array([a[0] for a in at]), np.array([a[2] for a in at])
                kk, vv = k[blk, slot, g], v[blk, slot, g]
                for h in range(g * group, (g + 1) * group):
                    s = kk @ x[b, i, h] * sm_scale
                    m = s.max()
                    p = np.exp(s - m)
                    lse[b, i, h] = m + math.log(p.sum())
                    out[b, i, h] = p @ vv / p.sum()
                    size[b, i, h] = p @ np.abs(vv) / p.sum()
    return out, lse, size


def check_attention(out, lse, ref, ref_lse, size, dtype, weight_eps, slack=2e-5):
    """Each weight p_j is rounded once (half a step of its type: weight_eps), the output once (half
    a step of its own type); logits, sums and the merge are fp32 (slack, relative to the sum of
    magnitudes: logits of this size move by about 1e-6, and exp2 and log2 are good to 2^-22)."""
    eps = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    got = out.detach().double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = (weight_eps + slack) * size + eps * (np.abs(ref) + (weight_eps + slack) * size) + 2.0 ** -24
    worst = np.abs(got - ref) / tol
    assert worst.max(initial=0) <= 1, f"{worst.max():.3f} of the tolerance at {np.unravel_index(worst.argmax(), worst.shape)}"
    if lse is not None:
        gl = lse.detach().double().cpu().numpy()
        fin = np.isfinite(ref_lse)
        assert np.array_equal(gl[~fin], ref_lse[~fin])
        assert (np.abs(gl[fin] - ref_lse[fin]) <= slack * (1 + np.abs(ref_lse[fin]))).all()
