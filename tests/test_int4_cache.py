"""4-bit caches: the append's codes and pairs bit for bit, the read-back of every quantised cache, and
the decode against 64 bits for all head groupings, sizes, splits and masks; flags, refusals, equal bits
on equal calls; and append, decode and read-back together."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_work_gb300 as pa
import plain64
import plain_int4 as plain

KINDS = {"bf16": (torch.bfloat16, pa.BF16), "fp16": (torch.float16, pa.FP16)}


def config(B, sq, hq, hkv, d, bs, maxb, nblocks, dtype="bf16", causal=0, kv=None, mode=None, **kw):
    kv = pa.INT4 if kv is None else kv
    mode = pa.SCALE_AFFINE if mode is None else mode
    return pa.PaConfig(batch=B, max_q_len=sq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                       max_blocks_per_seq=maxb, num_blocks=nblocks, q_dtype=KINDS[dtype][1], kv_dtype=kv,
                       kv_scale_mode=mode, causal=causal, sm_scale=d ** -0.5, **kw)


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# ---- append ---------------------------------------------------------------------------------
ODD_ROWS = ("zeros", "constant", "negative", "tiny", "wide", "huge", "nan", "inf", "two values", "minus inf")


def odd_row(kind, d, t, rng):
    x = torch.from_numpy(rng.standard_normal(d))
    big = float(torch.finfo(t).max)
    if kind == "zeros":
        x = torch.zeros(d)
    elif kind == "constant":
        x = torch.full((d,), -3.25)
    elif kind == "negative":
        x = -x.abs() - 7
    elif kind == "tiny":  # subnormal steps
        x = x * float(torch.finfo(t).smallest_normal) * (4 if t == torch.float16 else 2.0 ** 8)
    elif kind == "wide":
        x[3] = 1000.0
    elif kind == "huge":
        x = x.clamp(-1, 1) * big * 0.49
    elif kind == "nan":
        x[d - 1] = float("nan")
    elif kind == "inf":
        x[0] = float("inf")
    elif kind == "minus inf":
        x[5] = float("-inf")
    else:
        x = torch.where(x > 0, 1.0, -2.0)
    return x.to(t)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [2026, 2029])
@pytest.mark.parametrize("B,sq,hkv,d,bs,dtype", [
    (3, 5, 2, 128, 16, "bf16"), (4, 1, 8, 128, 16, "fp16"), (2, 40, 1, 64, 16, "bf16"), (2, 7, 3, 256, 32, "bf16"),
    (2, 3, 1, 256, 1024, "fp16"), (5, 33, 3, 64, 64, "fp16"), (70, 2, 2, 128, 16, "bf16")])
def test_append_bit_for_bit(seed, B, sq, hkv, d, bs, dtype, cuda_device, pa):
    rng = np.random.default_rng(seed)
    t = KINDS[dtype][0]
    ql = rng.integers(0, sq + 1, B)
    ql[0] = sq
    ctx = ql + rng.integers(0, 3 * bs, B)
    bt, nblocks = plain.tables(rng, ctx, bs)
    new = [torch.from_numpy(rng.standard_normal((B, sq, hkv, d)) * rng.choice([0.01, 1, 50], (B, sq, hkv, 1))).to(t)
           for _ in "kv"]
    for j, kind in enumerate(ODD_ROWS):
        b, i = j % B, (j // B) % sq
        if i < ql[b]:
            new[j % 2][b, i, j % hkv] = odd_row(kind, d, t, rng)
    codes = [torch.from_numpy(rng.integers(0, 256, (nblocks, bs, hkv, d // 2)).astype(np.uint8)) for _ in "kv"]
    pairs = [torch.from_numpy(rng.standard_normal((nblocks, hkv, bs, 2))).to(t) for _ in "kv"]
    cfg = config(B, sq, hkv, hkv, d, bs, bt.shape[1], nblocks, dtype)
    dc, dp = [c.to(cuda_device) for c in codes], [p.to(cuda_device) for p in pairs]
    flags = ints([0], cuda_device)
    pa.append_kv(cfg, new[0].to(cuda_device), new[1].to(cuda_device), ints(bt, cuda_device), ints(ctx, cuda_device),
                 ints(ql, cuda_device), *dc, *dp, flags)
    assert int(flags.item()) == 0
    for n, c, p, gc, gp in zip(new, codes, pairs, dc, dp):
        rc, rp = plain.append(n, c, p, ctx.tolist(), ql.tolist(), bt, bs)
        assert torch.equal(gc.cpu(), rc)
        got, lost = gp.cpu(), torch.isnan(rp[..., 0])
        assert torch.equal(torch.isnan(got[..., 0]), lost)
        assert torch.equal(got[~lost], rp[~lost])  # (numbers: -0 is 0)


@pytest.mark.gpu
def test_append_flags(cuda_device, pa):
    rng = np.random.default_rng(5)
    ctx, ql = np.array([20, 40, 33]), np.array([3, 3, 2])
    bt, nblocks = plain.tables(rng, ctx, 16)
    new = torch.from_numpy(rng.standard_normal((3, 3, 2, 128))).to(torch.bfloat16)
    codes = torch.zeros((nblocks, 16, 2, 64), dtype=torch.uint8)
    pairs = torch.ones((nblocks, 2, 16, 2), dtype=torch.bfloat16)
    bad_bt, bad_ql = bt.copy(), ql.copy()
    bad_bt[0, 1], bad_ql[1] = nblocks, 4  # a page outside the pool, a length past Sq
    cfg = config(3, 3, 2, 2, 128, 16, bt.shape[1], nblocks)
    dc, dp = [codes.to(cuda_device) for _ in "kv"], [pairs.to(cuda_device) for _ in "kv"]
    flags = ints([0], cuda_device)
    pa.append_kv(cfg, new.to(cuda_device), new.to(cuda_device), ints(bad_bt, cuda_device), ints(ctx, cuda_device),
                 ints(bad_ql, cuda_device), *dc, *dp, flags)
    assert int(flags.item()) == pa.FLAG_BAD_BLOCK_ID | pa.FLAG_BAD_LENGTHS
    only = new.clone()
    rc, rp = plain.append(only, codes, pairs, [ctx[0] - 3, ctx[1], ctx[2]], [0, 0, 2], bt, 16)
    # (sequence 0's three rows are positions 17 .. 19, all in the bad page)
    assert torch.equal(dc[0].cpu(), rc) and torch.equal(dp[1].cpu(), rp)


# ---- read-back -------------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["4", "8none", "8tensor", "8token", "8block"])
@pytest.mark.parametrize("B,hkv,d,bs,longest,dtype", [
    (3, 2, 128, 16, 100, "bf16"), (5, 1, 64, 16, 40, "fp16"), (2, 3, 256, 64, 300, "fp16"), (1, 1, 128, 1024, 1, "bf16"),
    (40, 8, 64, 32, 90, "bf16"), (2, 16, 256, 128, 513, "bf16")])
def test_read_back(kv, B, hkv, d, bs, longest, dtype, cuda_device, pa):
    rng = np.random.default_rng(11)
    t = KINDS[dtype][0]
    ctx = rng.integers(0, longest + 1, B)
    ctx[B // 2] = longest
    bt, nblocks = plain.tables(rng, ctx, bs)
    ref, dc, ds = [], [], []
    for _ in "kv":
        if kv == "4":
            c = torch.from_numpy(rng.integers(0, 256, (nblocks, bs, hkv, d // 2)).astype(np.uint8))
            s = torch.from_numpy(rng.standard_normal((nblocks, hkv, bs, 2))).to(t)
            ref.append(plain.values(c, s))
        else:
            c = torch.from_numpy(rng.standard_normal((nblocks, bs, hkv, d)) * 60).clamp(-448, 448)
            c = c.to(torch.float8_e4m3fn).view(torch.uint8)
            size = {"8tensor": (1,), "8token": (nblocks, bs, hkv), "8block": (nblocks, hkv)}.get(kv)
            s = None if size is None else torch.from_numpy(rng.uniform(0.005, 0.02, size).astype(np.float32))
            ref.append(plain64.values(c, s, kv[1:]))
        dc.append(c.to(cuda_device))
        ds.append(None if s is None else s.to(cuda_device))
    mode = {"4": pa.SCALE_AFFINE, "8none": 0, "8tensor": 1, "8token": 2, "8block": 3}[kv]
    cfg = config(B, 1, hkv, hkv, d, bs, bt.shape[1], nblocks, dtype, kv=pa.INT4 if kv == "4" else pa.FP8_E4M3, mode=mode)
    total = int(ctx.sum())
    out = [torch.full((total + 3, hkv, d), 7.0, dtype=t, device=cuda_device) for _ in "kv"]
    off, flags = ints(np.full(B + 1, -1), cuda_device), ints([0], cuda_device)
    pa.dequant_kv(cfg, *dc, *ds, ints(bt, cuda_device), ints(ctx, cuda_device), *out, row_offsets=off, flags=flags)
    assert int(flags.item()) == 0
    start = np.concatenate(([0], np.cumsum(ctx)))
    assert off.cpu().tolist() == start.tolist()
    # one rounding to the type (half a step, at least half of the least subnormal), of an fp32 value
    half = torch.finfo(t).eps / 2
    for got, v in zip(out, ref):
        got = got.double().cpu().numpy()
        assert (got[total:] == 7.0).all()  # rows behind the last sequence
        for b in range(B):
            tok = np.arange(ctx[b])
            want = v[bt[b, tok // bs], tok % bs] if len(tok) else np.zeros((0, hkv, d))
            mag = np.abs(want)
            tol = half * mag * (1 + 2.0 ** -20) + 2.0 ** -23 * (mag + 60) + torch.finfo(t).smallest_normal * half
            assert (np.abs(got[start[b]:start[b + 1]] - want) <= tol).all()


@pytest.mark.gpu
def test_read_back_flags(cuda_device, pa):
    """A page outside the pool is left out, a bad length counts as empty, and rows that do not fit are
    not written at all."""
    rng = np.random.default_rng(3)
    ctx = np.array([20, 1000, 30])
    bt, nblocks = plain.tables(rng, [20, 16, 30], 16)
    c = torch.from_numpy(rng.integers(0, 256, (nblocks, 16, 2, 64)).astype(np.uint8))
    s = torch.from_numpy(rng.standard_normal((nblocks, 2, 16, 2))).to(torch.float16)
    v = plain.values(c, s)
    bad = bt.copy()
    bad[2, 0] = -1
    cfg = config(3, 1, 2, 2, 128, 16, bt.shape[1], nblocks, "fp16")
    dev = cuda_device
    args = (cfg, c.to(dev), c.to(dev), s.to(dev), s.to(dev), ints(bad, dev), ints(ctx, dev))
    out = [torch.full((50, 2, 128), 7.0, dtype=torch.float16, device=dev) for _ in "kv"]
    flags = ints([0], dev)
    pa.dequant_kv(*args, *out, flags=flags)
    assert int(flags.item()) == pa.FLAG_BAD_LENGTHS | pa.FLAG_BAD_BLOCK_ID
    got = out[0].double().cpu().numpy()
    assert (got[20:36] == 7.0).all()
    want = v[bt[2, 1], :14]
    assert np.abs(got[36:] - want).max() <= 2.0 ** -11 * np.abs(want).max() + 1e-5
    out = [torch.full((50, 2, 128), 7.0, dtype=torch.float16, device=dev) for _ in "kv"]
    flags = ints([0], dev)
    pa.dequant_kv(*args, *out, max_rows=49, flags=flags)
    assert int(flags.item()) & pa.FLAG_BAD_LENGTHS and all((o == 7.0).all().item() for o in out)


# ---- decode ----------------------------------------------------------------------------------
def problem(seed, B, sq, hq, hkv, d, bs, ctx, ql, dtype="bf16", spread=0.0):
    """A cache whose V steps differ by up to 2^spread either way; NaN pairs behind the last token."""
    rng = np.random.default_rng(seed)
    t = KINDS[dtype][0]
    bt, nblocks = plain.tables(rng, ctx, bs)
    codes = [torch.from_numpy(rng.integers(0, 256, (nblocks, bs, hkv, d // 2)).astype(np.uint8)) for _ in "kv"]
    pairs = []
    for which in "kv":
        step = rng.uniform(0.2, 0.4, (nblocks, hkv, bs))
        if which == "v" and spread:
            step = step * 2.0 ** rng.uniform(-spread, spread, step.shape)
            step[rng.random(step.shape) < 0.1] = 0.0  # rows of one value
        low = -7.5 * step + rng.standard_normal(step.shape) * 0.3
        p = torch.from_numpy(np.stack((step, low), -1)).to(t)
        for b, n in enumerate(ctx):
            if n % bs:
                p[bt[b, n // bs], :, n % bs:] = float("nan")
        pairs.append(p)
    q = torch.from_numpy(rng.standard_normal((B, sq, hq, d))).to(t)
    return dict(ctx=np.asarray(ctx), ql=np.asarray(ql), bt=bt, nblocks=nblocks, kc=codes[0], vc=codes[1],
                ks=pairs[0], vs=pairs[1], q=q)


def reference(p, causal, d, bt=None):
    clean = [torch.nan_to_num(s, nan=0.0) for s in (p["ks"], p["vs"])]
    k, v = plain.values(p["kc"], clean[0]), plain.values(p["vc"], clean[1])
    # a weight carries its row's step and meets c - 8; what is left of the row, low + 8 step, is added
    # in fp32 (the check's slack)
    pair = clean[1].double().numpy().transpose(0, 2, 1, 3)
    mid = pair[..., 1:] + 8 * pair[..., :1]
    mag = np.abs(v - mid) + np.abs(mid)
    return plain.attend(p["q"], k, v, mag, p["bt"] if bt is None else bt, p["ctx"], p["ql"], causal,
                        float(np.float32(d ** -0.5)), p["nblocks"])


def run(p, cfg, dev, bt=None, want_flags=0, lse=True):
    g = lambda x: x.to(dev)  # noqa: E731
    q = g(p["q"])
    out = torch.full_like(q, float("nan"))
    ls = torch.full(q.shape[:3], float("nan"), device=dev) if lse else None
    ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=dev)
    args = ints(p["bt"] if bt is None else bt, dev), ints(p["ctx"], dev), ints(p["ql"], dev)
    pa.plan(cfg, *args, ws)
    pa.decode(cfg, q, g(p["kc"]), g(p["vc"]), g(p["ks"]), g(p["vs"]), *args, out, ls, ws)
    pa.reduce(cfg, out, ls, ws)
    assert pa.read_flags(ws) == want_flags
    return out, ls


def check(out, lse, ref, ref_lse, size, dtype):
    plain64.check_attention(out, lse, ref, ref_lse, size, KINDS[dtype][0], 2.0 ** -11)


CASES = [
    # Sq, Hq, Hkv, D, bs, contexts, new rows, causal, dtype, CTAs
    (1, 4, 1, 128, 16, (700, 16, 1, 0), (1, 1, 1, 0), 0, "bf16", 0), (1, 1, 1, 128, 16, (1,), (1,), 0, "bf16", 0),
    (3, 16, 2, 128, 64, (900, 65, 3), (3, 2, 3), 1, "fp16", 0), (1, 16, 1, 128, 1024, (3001, 1024), (1, 1), 1, "bf16", 0),
    (4, 4, 1, 128, 32, (129, 127), (4, 0), 1, "bf16", 5), (2, 24, 1, 128, 16, (333,), (2,), 1, "fp16", 3),
    (70, 3, 3, 128, 16, (150, 70), (70, 64), 1, "bf16", 0), (2, 10, 2, 64, 16, (500, 17), (2, 1), 1, "bf16", 0),
    (1, 80, 2, 64, 16, (200,), (1,), 1, "fp16", 7), (1, 2, 2, 64, 512, (2000, 511), (1, 1), 0, "fp16", 0),
    (2, 5, 1, 256, 32, (400, 33), (2, 2), 1, "bf16", 0), (1, 8, 1, 256, 1024, (2500,), (1,), 0, "fp16", 0),
    (3, 7, 1, 256, 16, (255, 90, 16), (3, 1, 2), 1, "bf16", 2), (1, 16, 16, 256, 32, (300, 64), (1, 1), 1, "bf16", 0),
    (1, 6, 3, 128, 128, (4000, 10, 2049), (1, 1, 1), 1, "fp16", 1), (1, 16, 1, 128, 256, (16, 32, 48, 15), (1, 1, 1, 1), 0, "bf16", 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("sq,hq,hkv,d,bs,ctx,ql,causal,dtype,ctas", CASES)
def test_decode_matches_64_bits(sq, hq, hkv, d, bs, ctx, ql, causal, dtype, ctas, cuda_device, pa):
    p = problem(7, len(ctx), sq, hq, hkv, d, bs, ctx, ql, dtype)
    cfg = config(len(ctx), sq, hq, hkv, d, bs, p["bt"].shape[1], p["nblocks"], dtype, causal, num_ctas=ctas)
    out, lse = run(p, cfg, cuda_device)
    check(out, lse, *reference(p, causal, d), dtype)
    again, lse2 = run(p, cfg, cuda_device)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    alone, _ = run(p, cfg, cuda_device, lse=False)
    assert torch.equal(out.view(torch.int16), alone.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,dtype", [(64, 4, "bf16"), (128, 16, "fp16"), (256, 8, "bf16"), (128, 4, "bf16")])
def test_decode_merges_alike(d, hq, dtype, cuda_device, pa):
    """Every grid and both places of the merge."""
    p = problem(21, 3, 1, hq, 1, d, 16, (900, 40, 333), (1, 1, 1), dtype)
    ref = reference(p, 1, d)
    for ctas in (1, 2, 9, 64, 300):
        for merge in (pa.MERGE_IN_DECODE, pa.MERGE_IN_REDUCE):
            cfg = config(3, 1, hq, 1, d, 16, p["bt"].shape[1], p["nblocks"], dtype, 1, num_ctas=ctas, split_merge=merge)
            out, lse = run(p, cfg, cuda_device)
            check(out, lse, *ref, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [3, 12, 25])
@pytest.mark.parametrize("d,hq,sq,dtype", [(128, 4, 1, "bf16"), (64, 16, 2, "bf16"), (256, 3, 2, "bf16")])
def test_decode_steps_far_apart(spread, d, hq, sq, dtype, cuda_device, pa):
    """V steps up to 2^50 apart, zeros among them: a weight keeps its bits beside any of them."""
    p = problem(5, 2, sq, hq, 1, d, 16, (400, 77), (sq, sq), dtype, spread=spread)
    cfg = config(2, sq, hq, 1, d, 16, p["bt"].shape[1], p["nblocks"], dtype, 1)
    out, lse = run(p, cfg, cuda_device)
    check(out, lse, *reference(p, 1, d), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_decode_large_and_small_queries(size, cuda_device, pa):
    """A bf16 query beyond f16's range, with keys that bring the logits back."""
    p = problem(6, 2, 2, 8, 2, 128, 16, (100, 50), (2, 2))
    p["q"] = (p["q"].double() * size).to(torch.bfloat16)
    p["ks"] = (p["ks"].double() / size).to(torch.bfloat16)
    cfg = config(2, 2, 8, 2, 128, 16, p["bt"].shape[1], p["nblocks"], causal=1)
    out, lse = run(p, cfg, cuda_device)
    check(out, lse, *reference(p, 1, 128), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("sm_scale", [0.0, -0.11, 1e-30])
def test_decode_any_logit_scale(sm_scale, cuda_device, pa):
    """Zero weighs all seen keys alike; a negative one favours the smallest products."""
    p = problem(14, 2, 3, 12, 2, 128, 16, (90, 33), (3, 2))
    cfg = config(2, 3, 12, 2, 128, 16, p["bt"].shape[1], p["nblocks"], causal=1)
    cfg.sm_scale = sm_scale
    out, lse = run(p, cfg, cuda_device)
    clean = [torch.nan_to_num(s, nan=0.0) for s in (p["ks"], p["vs"])]
    k, v = plain.values(p["kc"], clean[0]), plain.values(p["vc"], clean[1])
    pair = clean[1].double().numpy().transpose(0, 2, 1, 3)
    mid = pair[..., 1:] + 8 * pair[..., :1]
    ref = plain.attend(p["q"], k, v, np.abs(v - mid) + np.abs(mid), p["bt"], p["ctx"], p["ql"], 1,
                       float(np.float32(sm_scale)), p["nblocks"])
    check(out, lse, *ref, "bf16")


@pytest.mark.gpu
def test_decode_rows_apart(cuda_device, pa):
    """A NaN or infinite query element reaches its own row alone, padding rows among its tile's."""
    p = problem(15, 2, 4, 4, 1, 64, 16, (100, 40), (4, 1))
    p["q"][0, 1, 2, 5], p["q"][0, 2, 0, 60] = float("nan"), float("inf")
    p["q"][1, 1:] = float("nan")  # (rows behind the sequence's last)
    cfg = config(2, 4, 4, 1, 64, 16, p["bt"].shape[1], p["nblocks"], causal=1)
    out, _ = run(p, cfg, cuda_device)
    bad = torch.isnan(out.float()).any(-1)
    assert bad[0, 1, 2] and bad[0, 2, 0] and int(bad.sum()) == 2
    assert (out[1, 1:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("d,hq,hkv,ctas", [(64, 8, 2, 0), (128, 4, 1, 3), (128, 32, 8, 0), (256, 6, 1, 5)])
def test_decode_padded_batches(d, hq, hkv, ctas, causal, cuda_device, pa):
    """Sequences with fewer new rows than the batch's most: the rows behind, whatever their queries hold,
    are zero with lse -inf, in whole and split units."""
    p = problem(18, 5, 4, hq, hkv, d, 16, (900, 1200, 33, 640, 512), (1, 3, 4, 0, 2))
    ref = reference(p, causal, d)
    for b, n in enumerate(p["ql"]):
        p["q"][b, n:] = (float("nan"), float("inf"), 1e30, 3.0, float("-inf"))[b]
    cfg = config(5, 4, hq, hkv, d, 16, p["bt"].shape[1], p["nblocks"], causal=causal, num_ctas=ctas)
    out, lse = run(p, cfg, cuda_device)
    check(out, lse, *ref, "bf16")
    assert all((out[b, n:] == 0).all() for b, n in enumerate(p["ql"]))


@pytest.mark.gpu
def test_pages_shared_by_sequences(cuda_device, pa):
    """A common prefix: the same pages in several tables."""
    p = problem(16, 3, 1, 8, 2, 128, 16, (200, 200, 200), (1, 1, 1))
    p["bt"][1, :12], p["bt"][2, :12] = p["bt"][0, :12], p["bt"][0, :12]
    p["q"][1:] = p["q"][:1]
    p["bt"][1] = p["bt"][0]
    cfg = config(3, 1, 8, 2, 128, 16, p["bt"].shape[1], p["nblocks"])
    out, lse = run(p, cfg, cuda_device)
    check(out, lse, *reference(p, 0, 128), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_bad_blocks_and_lengths(d, cuda_device, pa):
    """A page outside the pool holds no keys; a bad length stops the step."""
    p = problem(8, 3, 2, 8, 2, d, 16, (200, 16, 90), (2, 1, 2))
    cfg = config(3, 2, 8, 2, d, 16, p["bt"].shape[1], p["nblocks"], causal=1)
    bt = p["bt"].copy()
    bt[0, 3], bt[0, 12], bt[1, 0], bt[2, 5] = p["nblocks"], -1, -7, 2 ** 30
    out, lse = run(p, cfg, cuda_device, bt, pa.FLAG_BAD_BLOCK_ID)
    check(out, lse, *reference(p, 1, d, bt), "bf16")
    p["ql"][1] = 3
    _, _ = run(p, cfg, cuda_device, None, pa.FLAG_BAD_LENGTHS)


@pytest.mark.gpu
def test_decode_nan_stays_nan(cuda_device, pa):
    """A key's NaN pair reaches the rows that see it, and no other."""
    p = problem(9, 2, 2, 4, 1, 128, 16, (64, 40), (2, 2))
    p["ks"][p["bt"][0, 3], 0, 15] = float("nan")  # position 63 of sequence 0: its last row alone
    cfg = config(2, 2, 4, 1, 128, 16, p["bt"].shape[1], p["nblocks"], causal=1)
    out, _ = run(p, cfg, cuda_device)
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [(float("nan"), 0.5), (0.25, float("nan")), (0.25, float("inf")), (float("inf"), 0.5)])
@pytest.mark.parametrize("d,hq,dtype", [(64, 4, "bf16"), (128, 4, "fp16"), (128, 9, "bf16"), (256, 8, "fp16")])
def test_decode_values_that_are_none(d, hq, dtype, bad, cuda_device, pa):
    """A value's pair that is not finite reaches the rows that see it, and no other: those get what they
    got without it."""
    p = problem(17, 2, 3, hq, 1, d, 16, (64, 40), (3, 3), dtype)
    cfg = config(2, 3, hq, 1, d, 16, p["bt"].shape[1], p["nblocks"], dtype, causal=1)
    ref, ref_lse, size = reference(p, 1, d)
    p["vs"][p["bt"][0, 3], 0, 14] = torch.tensor(bad).to(p["vs"].dtype)  # position 62: the last two rows
    out, lse = run(p, cfg, cuda_device)
    assert not torch.isfinite(out[0, 1:]).any()
    out[0, 1:] = torch.from_numpy(ref[0, 1:]).to(out)
    check(out, lse, ref, ref_lse, size, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("merge", [pa.MERGE_IN_DECODE, pa.MERGE_IN_REDUCE])
@pytest.mark.parametrize("ctas", [1, 2, 9, 40])
@pytest.mark.parametrize("d,hq", [(128, 4), (256, 10), (64, 2)])
def test_decode_nan_survives_merges(d, hq, ctas, merge, cuda_device, pa):
    """However a unit is split and wherever it is merged (4,200 tokens come to 33 pieces), a NaN query
    and a key's NaN pair are NaN in out and lse of the rows that they reach, and in no other's."""
    p = problem(19, 3, 2, hq, 1, d, 16, (4200, 4200, 150), (2, 2, 2))
    ref, ref_lse, size = reference(p, 1, d)
    p["q"][0, 1, hq - 1, 7] = float("nan")
    p["ks"][p["bt"][1, 4199 // 16], 0, 4199 % 16] = float("nan")  # the last position: the last row's alone
    cfg = config(3, 2, hq, 1, d, 16, p["bt"].shape[1], p["nblocks"], causal=1, num_ctas=ctas, split_merge=merge)
    out, lse = run(p, cfg, cuda_device)
    lost = np.zeros((3, 2, hq), bool)
    lost[0, 1, hq - 1] = lost[1, 1] = True
    assert (torch.isnan(out.float()).all(-1).cpu().numpy() == lost).all()
    assert (torch.isnan(lse).cpu().numpy() == lost).all()
    mask = torch.from_numpy(lost).to(out.device)
    out[mask], lse[mask] = torch.from_numpy(ref).to(out)[mask], torch.from_numpy(ref_lse).to(lse)[mask]
    check(out, lse, ref, ref_lse, size, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("d,hq,dtype", [(64, 3, "bf16"), (64, 16, "fp16"), (128, 4, "bf16"), (128, 13, "bf16"),
                                        (256, 8, "fp16"), (256, 16, "bf16"), (256, 9, "fp16")])
def test_decode_looks_up_pages_again(d, hq, dtype, bs, cuda_device, pa):
    """Items whose warps pass their 32nd and 64th chunk of 16 tokens, where a lane's next pages are looked
    up: as they are, and with pages outside the pool in the chunks on both sides of the first turn."""
    ctx = (4300, 4231)
    p = problem(33, 2, 1, hq, 1, d, bs, ctx, (1, 1), dtype)
    cfg = config(2, 1, hq, 1, d, bs, p["bt"].shape[1], p["nblocks"], dtype, num_ctas=1)
    out, lse = run(p, cfg, cuda_device)
    check(out, lse, *reference(p, 0, d), dtype)
    bt = p["bt"].copy()
    # a warp's 32nd and 33rd chunk: of warps 0 and 3, in tiles of two chunks (121 and 128, 127 and 134)
    # and of one (124 and 128, 127 and 131)
    for chunk in (121, 124, 127, 128, 131, 134):
        bt[:, chunk * 16 // bs] = (p["nblocks"], -1)
    out, lse = run(p, cfg, cuda_device, bt, pa.FLAG_BAD_BLOCK_ID)
    check(out, lse, *reference(p, 0, d, bt), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq", [(64, 2), (128, 20), (256, 8)])
def test_decode_of_nothing(d, hq, cuda_device, pa):
    """A batch without a single token, behind a batch with some on the same workspace."""
    p = problem(35, 3, 2, hq, 1, d, 16, (0, 0, 0), (0, 0, 0))
    cfg = config(3, 2, hq, 1, d, 16, p["bt"].shape[1], p["nblocks"])
    out, lse = run(p, cfg, cuda_device)
    assert (out == 0).all() and (lse == float("-inf")).all()


@pytest.mark.gpu
def test_paged_attention_takes_a_4_bit_cache(cuda_device, pa):
    """The step on a problem laid out as the workloads are, its config made from it."""
    from types import SimpleNamespace
    p = problem(34, 3, 2, 8, 2, 128, 16, (300, 17, 64), (2, 1, 2))
    g = lambda t: t.to(cuda_device)  # noqa: E731
    inp = dict(workload=SimpleNamespace(batch=3, max_q_len=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                                        q_dtype="bf16", kv_dtype="int4", scale_mode="none", causal=True),
               q=g(p["q"]), k_cache=g(p["kc"]), v_cache=g(p["vc"]), k_scale=g(p["ks"]), v_scale=g(p["vs"]),
               block_tables=ints(p["bt"], cuda_device), context_lens=ints(p["ctx"], cuda_device),
               q_lens=ints(p["ql"], cuda_device), sm_scale=128 ** -0.5)
    out, lse, ws = pa.paged_attention(inp)
    assert pa.read_flags(ws) == 0
    check(out, lse, *reference(p, 1, 128), "bf16")


# ---- together --------------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("d,bs,dtype", [(128, 16, "bf16"), (64, 64, "fp16"), (256, 32, "bf16")])
def test_append_then_decode_then_read(d, bs, dtype, cuda_device, pa):
    """Three steps of a growing batch in one captured graph each, against the plain append and 64 bits;
    then the whole batch read back."""
    rng = np.random.default_rng(31)
    t, dev = KINDS[dtype][0], cuda_device
    B, sq, hq, hkv = 3, 2, 8, 2
    end = np.array([90, 2 * bs + 6, 6])
    bt, nblocks = plain.tables(rng, end, bs)
    zeros = [torch.zeros((nblocks, bs, hkv, d // 2), dtype=torch.uint8) for _ in "kv"]
    ones = [torch.zeros((nblocks, hkv, bs, 2), dtype=t) for _ in "kv"]
    codes, pairs = [z.clone() for z in zeros], [o.clone() for o in ones]
    most = int(end.max())
    cfg = config(B, most, hq, hkv, d, bs, bt.shape[1], nblocks, dtype, 1)
    dc, dp = [c.to(dev) for c in codes], [p.to(dev) for p in pairs]
    dbt, dctx, dql = ints(bt, dev), ints([0] * B, dev), ints([0] * B, dev)
    first = end - 2 * sq

    def append(ctx, ql, n):
        new = [torch.from_numpy(rng.standard_normal((B, n, hkv, d))).to(t) for _ in "kv"]
        dctx.copy_(ints(ctx, dev))
        dql.copy_(ints(ql, dev))
        for j in range(2):
            codes[j], pairs[j] = plain.append(new[j], codes[j], pairs[j], list(ctx), list(ql), bt, bs)
        return [x.to(dev) for x in new]

    new = append(first, first, most)
    pa.append_kv(cfg, *new, dbt, dctx, dql, *dc, *dp)
    cfg = config(B, sq, hq, hkv, d, bs, bt.shape[1], nblocks, dtype, 1)
    q = torch.from_numpy(rng.standard_normal((B, sq, hq, d))).to(t)
    dq, out, lse = q.to(dev), torch.empty_like(q, device=dev), torch.empty(q.shape[:3], device=dev)
    ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=dev)
    held = [torch.empty(B, sq, hkv, d, dtype=t, device=dev) for _ in "kv"]

    def step():
        pa.append_kv(cfg, *held, dbt, dctx, dql, *dc, *dp)
        pa.plan(cfg, dbt, dctx, dql, ws)
        pa.decode(cfg, dq, *dc, *dp, dbt, dctx, dql, out, lse, ws)
        pa.reduce(cfg, out, lse, ws)

    graph = None
    for turn in range(2):
        ctx, ql = first + sq * (turn + 1), np.array([sq, sq, sq])
        for h, n in zip(held, append(ctx, ql, sq)):
            h.copy_(n)
        if graph is None:
            saved = [x.clone() for x in dc + dp]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            for x, y in zip(dc + dp, saved):
                x.copy_(y)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay()
        torch.cuda.synchronize()
        for j in range(2):
            assert torch.equal(dc[j].cpu(), codes[j]) and torch.equal(dp[j].cpu(), pairs[j])
        p = dict(q=q, kc=codes[0], vc=codes[1], ks=pairs[0], vs=pairs[1], bt=bt, ctx=ctx, ql=ql, nblocks=nblocks)
        check(out, lse, *reference(p, 1, d), dtype)
        static, slse = torch.empty_like(out), torch.empty_like(lse)
        pa.decode_step_static(cfg, dq, *dc, *dp, dbt, dctx, dql, static, slse)
        assert torch.equal(static.view(torch.int16), out.view(torch.int16)) and torch.equal(slse, lse)
    total = int(end.sum())
    rows = [torch.empty(total, hkv, d, dtype=t, device=dev) for _ in "kv"]
    pa.dequant_kv(cfg, *dc, *dp, dbt, dctx, *rows)
    for j in range(2):
        v = plain.values(codes[j], pairs[j])
        want = np.concatenate([v[bt[b, np.arange(end[b]) // bs], np.arange(end[b]) % bs] for b in range(B)])
        assert np.abs(rows[j].double().cpu().numpy() - want).max() <= torch.finfo(t).eps / 2 * np.abs(want).max() * 1.01


@pytest.mark.gpu
def test_blocks_past_32_bits(cuda_device, pa):
    """Codes at byte offsets past 2^32: append, decode and read-back give what a small pool gives."""
    rng = np.random.default_rng(40)
    dev, t, hq, hkv, d, bs = cuda_device, torch.bfloat16, 16, 16, 256, 1024
    high = 2 ** 32 // (bs * hkv * d // 2) + 3
    new = [torch.from_numpy(rng.standard_normal((1, 40, hkv, d))).to(t).to(dev) for _ in "kv"]
    q = torch.from_numpy(rng.standard_normal((1, 1, hq, d))).to(t).to(dev)
    ctx, ql = ints([40], dev), ints([40], dev)
    res = []
    for nblocks, blk in ((2, 1), (high + 1, high)):
        codes = [torch.empty((nblocks, bs, hkv, d // 2), dtype=torch.uint8, device=dev) for _ in "kv"]
        pairs = [torch.empty((nblocks, hkv, bs, 2), dtype=t, device=dev) for _ in "kv"]
        bt = ints([[blk]], dev)
        cfg = config(1, 40, hq, hkv, d, bs, 1, nblocks)
        pa.append_kv(cfg, *new, bt, ctx, ql, *codes, *pairs)
        one = config(1, 1, hq, hkv, d, bs, 1, nblocks)
        out, lse = torch.empty_like(q), torch.empty(1, 1, hq, device=dev)
        ws = torch.empty(pa.workspace_size(one), dtype=torch.uint8, device=dev)
        args = bt, ctx, ints([1], dev)
        pa.plan(one, *args, ws)
        pa.decode(one, q, *codes, *pairs, *args, out, lse, ws)
        pa.reduce(one, out, lse, ws)
        assert pa.read_flags(ws) == 0
        rows = [torch.empty(40, hkv, d, dtype=t, device=dev) for _ in "kv"]
        pa.dequant_kv(one, *codes, *pairs, bt, ctx, *rows)
        res.append([x.clone() for x in (out, lse, *rows)])
        del codes, pairs
    assert torch.isfinite(res[0][0].float()).all()
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_two_graphs_on_one_workspace(cuda_device, pa):
    """Two captured steps that share a workspace, replayed in turn on one stream."""
    dev = cuda_device
    ps = [problem(50 + i, 2, 1, 8, 2, 128, 16, c, (1, 1)) for i, c in enumerate(((300, 20), (64, 500)))]
    want = []
    for p in ps:
        cfg = config(2, 1, 8, 2, 128, 16, p["bt"].shape[1], p["nblocks"])
        want.append(run(p, cfg, dev))
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=dev)
    graphs, keep = [], []
    for p in ps:
        cfg = config(2, 1, 8, 2, 128, 16, p["bt"].shape[1], p["nblocks"])
        x = [p[n].to(dev) for n in ("q", "kc", "vc", "ks", "vs")]
        args = ints(p["bt"], dev), ints(p["ctx"], dev), ints(p["ql"], dev)
        out, lse = torch.empty_like(x[0]), torch.empty(x[0].shape[:3], device=dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.plan(cfg, *args, ws)
            pa.decode(cfg, *x, *args, out, lse, ws)
            pa.reduce(cfg, out, lse, ws)
        graphs.append(g)
        keep.append((cfg, x, args, out, lse))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (_, _, _, out, lse), (o, l) in zip(keep, want):
        assert torch.equal(out.view(torch.int16), o.view(torch.int16)) and torch.equal(lse, l)


@pytest.mark.gpu
def test_another_stream(cuda_device, pa):
    p = problem(12, 2, 1, 8, 2, 128, 16, (500, 90), (1, 1))
    cfg = config(2, 1, 8, 2, 128, 16, p["bt"].shape[1], p["nblocks"], causal=1)
    want, _ = run(p, cfg, cuda_device)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got, _ = run(p, cfg, cuda_device)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# ---- refusals (no GPU) -------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_cache_work_gb300.build import build
        build()
    return pa.load()


def small(**kw):
    return config(**{**dict(B=2, sq=1, hq=8, hkv=2, d=128, bs=16, maxb=8, nblocks=32, num_ctas=4), **kw})


@pytest.mark.parametrize("kw,expect", [
    ({}, pa.OK), (dict(dtype="fp16"), pa.OK), (dict(d=64), pa.OK), (dict(d=256, bs=1024), pa.OK),
    (dict(mode=pa.SCALE_NONE), pa.ERR_UNSUPPORTED), (dict(mode=pa.SCALE_PER_TOKEN), pa.ERR_UNSUPPORTED),
    (dict(mode=pa.SCALE_PER_BLOCK), pa.ERR_UNSUPPORTED), (dict(kv=pa.FP8_E4M3), pa.ERR_INVALID_ARG),
    (dict(kv=pa.BF16), pa.ERR_INVALID_ARG), (dict(kv=4), pa.ERR_INVALID_ARG), (dict(mode=5), pa.ERR_INVALID_ARG),
    (dict(d=96), pa.ERR_UNSUPPORTED), (dict(bs=8), pa.ERR_UNSUPPORTED), (dict(hq=7), pa.ERR_UNSUPPORTED)])
def test_workspace_refusals(lib, kw, expect):
    n = ctypes.c_size_t(0)
    cfg = small(**kw)
    assert lib.pa_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == expect
    assert (n.value > 0) == (expect == pa.OK)


@pytest.mark.parametrize("kv,mode", [(pa.INT4, pa.SCALE_AFFINE), (pa.BF16, pa.SCALE_NONE), (pa.FP8_E4M3, pa.SCALE_PER_BLOCK)])
@pytest.mark.parametrize("B,hkv,sq", [(65536, 32, 1 << 15), (65536, 64, 1 << 20), (1 << 16, 1 << 15, 1), (1 << 20, 1 << 12, 1)])
def test_more_units_than_an_index_holds(lib, kv, mode, B, hkv, sq):
    """Products that pass 32 bits, some of them to zero."""
    for maxb, bs in ((1, 16), (1 << 16, 16), (2 ** 31 - 1, 1024)):
        cfg = small(B=B, hq=hkv, hkv=hkv, sq=sq, maxb=maxb, bs=bs, nblocks=1 << 20, kv=kv, mode=mode)
        n = ctypes.c_size_t(0)
        assert lib.pa_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == pa.ERR_UNSUPPORTED
        assert n.value == 0


def test_config_of_a_4_bit_workload():
    from types import SimpleNamespace
    w = SimpleNamespace(batch=3, max_q_len=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, q_dtype="fp16",
                        kv_dtype="int4", scale_mode="none", causal=True)
    inp = dict(workload=w, q=torch.zeros(1), k_cache=torch.zeros(7, 1), block_tables=torch.zeros(3, 5), sm_scale=0.5)
    cfg = pa.config_for(inp, num_ctas=4)
    assert (cfg.kv_dtype, cfg.kv_scale_mode, cfg.q_dtype) == (pa.INT4, pa.SCALE_AFFINE, pa.FP16)
    assert (cfg.num_blocks, cfg.max_blocks_per_seq, cfg.causal) == (7, 5, 1) and pa.workspace_size(cfg) > 0


def test_a_query_of_4_bits_is_refused(lib):
    cfg, n = small(), ctypes.c_size_t(0)
    cfg.q_dtype = pa.INT4
    assert lib.pa_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == pa.ERR_UNSUPPORTED


def test_calls_refused_before_any_launch(lib):
    fake = 1 << 20  # never dereferenced: every call below is rejected on the host
    cfg = small()
    n = ctypes.c_size_t(0)
    assert lib.pa_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == pa.OK
    dec = lambda ks=fake, vs=fake, c=cfg: lib.pa_decode(  # noqa: E731
        ctypes.byref(c), fake, fake, fake, ks, vs, fake, fake, fake, fake, None, fake, n.value, None)
    assert dec(ks=None) == pa.ERR_INVALID_ARG and dec(vs=None) == pa.ERR_INVALID_ARG
    assert dec(ks=fake + 4) == pa.ERR_INVALID_ARG  # pairs are copied 16 bytes at a time
    app = lambda ks=fake, vs=fake, c=cfg: lib.pa_append_kv(  # noqa: E731
        ctypes.byref(c), fake, fake, fake, fake, fake, fake, fake, ks, vs, None, None)
    assert app(ks=None) == pa.ERR_INVALID_ARG and app(vs=fake + 8) == pa.ERR_INVALID_ARG
    assert app(c=small(mode=pa.SCALE_NONE)) == pa.ERR_UNSUPPORTED
    assert app(c=small(kv=pa.BF16)) == pa.ERR_INVALID_ARG
    assert lib.pa_decode_selected(ctypes.byref(cfg), fake, fake, fake, fake, fake, fake, fake, fake, fake, fake, 4,
                                  fake, None, None, None) == pa.ERR_UNSUPPORTED
    assert lib.pa_gather_kv(ctypes.byref(cfg), fake, fake, fake, fake, fake, fake, 10, None, None,
                            None) == pa.ERR_UNSUPPORTED
    read = lambda c=cfg, kc=fake, ks=fake, bt=fake, ko=fake, rows=10, off=None: lib.pa_dequant_kv(  # noqa: E731
        ctypes.byref(c), kc, fake, ks, fake, bt, fake, ko, fake, rows, off, None, None)
    for kw in (dict(kc=None), dict(bt=None), dict(ko=None), dict(ks=None), dict(kc=fake + 8), dict(ko=fake + 2),
               dict(ks=fake + 4), dict(rows=-1), dict(off=fake + 1)):
        assert read(**kw) == pa.ERR_INVALID_ARG, kw
    assert read(c=small(kv=pa.BF16, mode=0)) == pa.ERR_UNSUPPORTED  # a copy is pa_gather_kv's
    assert read(c=small(d=96)) == pa.ERR_UNSUPPORTED and read(c=small(bs=24)) == pa.ERR_UNSUPPORTED
    assert read(c=small(B=8193)) == pa.ERR_UNSUPPORTED and read(c=small(B=0)) == pa.ERR_INVALID_ARG


def test_binding_refuses_arrays_that_do_not_fit():
    """(no GPU: any tensor is on the wrong device; types and sizes are looked at the same way)"""
    cfg = small()
    cpu = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(pa.PaError):
        pa.dequant_kv(cfg, cpu, cpu, cpu, cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(pa.PaError):
        pa.append_kv(cfg, cpu, cpu, cpu, cpu, cpu, cpu, cpu, cpu, cpu)
