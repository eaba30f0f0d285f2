"""Plain implementations of the 4-bit cache's calls and of the rotating append: rows one by one, fp32
where a call defines its rounding, 64 bits everywhere else.  They share no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

from plain64 import pages, seen

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BITS = {torch.bfloat16: (7, -126), torch.float16: (10, -14)}


def to_type(x, t, up):
    """The least number of type t that is >= x (up), or the largest that is <= x."""
    mant, emin = BITS[t]
    if x == 0 or not math.isfinite(x):
        return x
    place = 2.0 ** (max(math.frexp(x)[1] - 1, emin) - mant)
    y = (math.ceil(x / place) if up else math.floor(x / place)) * place
    return y if abs(y) <= float(torch.finfo(t).max) else math.copysign(math.inf, y)


def quantise(row, t):
    """Codes, step and low of a row (fp32 numpy values)."""
    row = row.astype(np.float32)
    with np.errstate(all="ignore"):
        low = to_type(float(row.min()), t, False) if np.isfinite(row).all() else math.nan
        span = np.float32(row.max()) - np.float32(low)
        if not np.isfinite(span):
            return np.zeros(row.shape, np.uint8), math.nan, low
        step = to_type(float(span / np.float32(15)), t, True)
        if step == 0:
            return np.zeros(row.shape, np.uint8), 0.0, low
        q = (row - np.float32(low)) / np.float32(step)
    return np.rint(q).astype(np.uint8), step, low


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(codes):
    c = np.asarray(codes)
    return np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)


def append(new, codes, pair, ctx, ql, bt, bs):
    """(codes, pairs) after appending rows `new` [B, Sq, Hkv, D]; entries where a row may be all NaN
    have any low."""
    codes, pair = codes.clone(), pair.clone()
    for b in range(new.shape[0]):
        for i in range(ql[b]):
            pos = ctx[b] - ql[b] + i
            blk, slot = int(bt[b][pos // bs]), pos % bs
            for g in range(new.shape[2]):
                c, step, low = quantise(new[b, i, g].float().numpy(), new.dtype)
                codes[blk, slot, g] = torch.from_numpy(pack(c))
                pair[blk, g, slot] = torch.tensor([step, low], dtype=torch.float64).to(pair.dtype)
    return codes, pair


def values(codes, pair):
    """64-bit values [nb, bs, Hkv, D]."""
    p = pair.double().numpy().transpose(0, 2, 1, 3)
    return unpack(codes.numpy()) * p[..., :1] + p[..., 1:]


def attend(q, kv, vv, vmag, bt, ctx, ql, causal, sm_scale, nblocks):
    """out, lse and sum_j p_j vmag_j (what the rounding of the weights is measured by); pages outside
    the pool hold no keys."""
    B, sq, hq, d = q.shape
    bs, hkv = kv.shape[1], kv.shape[2]
    group = hq // hkv
    out, size = np.zeros((B, sq, hq, d)), np.zeros((B, sq, hq, d))
    lse = np.full((B, sq, hq), -np.inf)
    x = q.double().numpy()
    for b in range(B):
        n = int(ctx[b])
        tok = np.arange(n)
        blk = np.array([bt[b][t // bs] for t in tok], dtype=np.int64)
        ok = (blk >= 0) & (blk < nblocks)
        tok, blk = tok[ok], blk[ok]
        for i in range(int(ql[b])):
            lim = seen(n, int(ql[b]), i, causal)
            use = tok < lim
            if not use.any():
                continue
            for h in range(hq):
                g = h // group
                kk, v = kv[blk[use], tok[use] % bs, g], vv[blk[use], tok[use] % bs, g]
                s = kk @ x[b, i, h] * sm_scale
                m = s.max()
                p = np.exp(s - m)
                lse[b, i, h] = m + math.log(p.sum())
                out[b, i, h] = p @ v / p.sum()
                size[b, i, h] = p @ vmag[blk[use], tok[use] % bs, g] / p.sum()
    return out, lse, size


def rotate(x, weight, eps, cos_sin, pos, axis_pairs, interleaved):
    """A token's heads [H, D] in 64 bits, normalised and rotated; pos: its position on each axis."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    if cos_sin is None:
        return x
    half = cos_sin.shape[1] // 2
    y = x.copy()
    p = 0
    for a, count in enumerate(axis_pairs):
        for _ in range(count):
            c, s = float(cos_sin[pos[a], p]), float(cos_sin[pos[a], p + half])
            i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
            y[:, i], y[:, j] = x[:, i] * c - x[:, j] * s, x[:, j] * c + x[:, i] * s
            p += 1
    return y


def tables(rng, ctx, bs, spare=2):
    """(block tables, pool size): pages out of a shuffled pool, -1 behind a sequence's last."""
    need = [pages(int(n), bs) for n in ctx]
    nblocks, maxb = sum(need) + spare, max(1, max(need))
    ids, at = rng.permutation(nblocks), 0
    bt = np.full((len(ctx), maxb), -1, np.int32)
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt, nblocks
