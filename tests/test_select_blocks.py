"""Channel bounds of the pages' keys, scores from them and the selection of the best pages, each
against a plain implementation; together: the bounds hold for the keys that were appended."""
import ctypes
import os

import numpy as np
import pytest
import torch

import paged_kv_cache_work_gb300 as pa
import plain64

KINDS = {"bf16": (torch.bfloat16, pa.BF16), "fp16": (torch.float16, pa.FP16)}


def config(B, sq, hq, hkv, d, bs, maxb, nblocks, dtype="bf16", causal=0, sm=None):
    return pa.PaConfig(batch=B, max_q_len=sq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                       max_blocks_per_seq=maxb, num_blocks=nblocks, q_dtype=KINDS[dtype][1], kv_dtype=KINDS[dtype][1],
                       kv_scale_mode=0, causal=causal, sm_scale=d ** -0.5 if sm is None else sm)


def lengths(rng, B, sq, longest):
    ctx = rng.integers(0, longest + 1, B)
    ctx[0] = longest
    ql = np.minimum(ctx, rng.integers(0, sq + 1, B))
    ql[0] = min(sq, longest)
    return ctx, ql


def tables(rng, ctx, bs, columns=None):
    need = [plain64.pages(n, bs) for n in ctx]
    nblocks, maxb = sum(need) + 2, max(1, max(need), columns or 0)
    ids, at = rng.permutation(nblocks), 0
    bt = np.full((len(ctx), maxb), -1, np.int32)
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt, nblocks, maxb


def gpu(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# ---- bounds -----------------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,hkv,d,bs,longest,dtype", [
    (3, 1, 2, 128, 16, 90, "bf16"), (2, 50, 3, 64, 16, 100, "fp16"), (2, 300, 1, 256, 128, 700, "bf16"),
    (5, 7, 4, 64, 32, 40, "bf16"), (2, 1100, 1, 128, 1024, 2300, "fp16")])
def test_bounds_match_a_plain_minimum(B, sq, hkv, d, bs, longest, dtype, cuda_device, pa):
    rng = np.random.default_rng(sq)
    ctx, ql = lengths(rng, B, sq, longest)
    bt, nblocks, maxb = tables(rng, ctx, bs)
    x = rng.standard_normal((B, sq, hkv, d))
    for v in (np.inf, -np.inf, np.nan, 0.0, -0.0):
        x[tuple(rng.integers(0, n, 6) for n in x.shape)] = v
    new = torch.from_numpy(x).to(KINDS[dtype][0])
    old = torch.sort(torch.from_numpy(rng.standard_normal((nblocks, hkv, 2, d))), 2).values.to(KINDS[dtype][0])
    want = plain64.update_bounds(new, old, ctx.tolist(), ql.tolist(), bt, bs)
    flags, got = gpu([0], cuda_device), old.to(cuda_device).clone()
    pa.update_bounds(config(B, sq, hkv, hkv, d, bs, maxb, nblocks, dtype), new.to(cuda_device), gpu(bt, cuda_device),
                     gpu(ctx, cuda_device), gpu(ql, cuda_device), got, flags)
    assert int(flags.item()) == 0
    assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=12345.0), torch.nan_to_num(want.float(), nan=12345.0))


@pytest.mark.gpu
def test_bounds_flags_and_skips(cuda_device, pa):
    rng = np.random.default_rng(1)
    ctx, ql = np.array([40, 20, 5]), np.array([20, 20, 5])
    bt, nblocks, maxb = tables(rng, ctx, 16)
    new = torch.from_numpy(rng.standard_normal((3, 20, 2, 64))).bfloat16()
    old = torch.zeros(nblocks, 2, 2, 64, dtype=torch.bfloat16)
    bad_bt, bad_ctx = bt.copy(), ctx.copy()
    bad_bt[0, 1] = -1
    bad_ctx[1] = 19
    want = plain64.update_bounds(new, old, [40, 0, 5], [20, 0, 5], bt, 16)
    want[bt[0, 1]] = 0
    flags, got = gpu([0], cuda_device), old.to(cuda_device).clone()
    pa.update_bounds(config(3, 20, 2, 2, 64, 16, maxb, nblocks), new.to(cuda_device), gpu(bad_bt, cuda_device),
                     gpu(bad_ctx, cuda_device), gpu(ql, cuda_device), got, flags)
    assert int(flags.item()) == pa.FLAG_BAD_LENGTHS | pa.FLAG_BAD_BLOCK_ID
    assert torch.equal(got.cpu(), want)


# ---- scores -----------------------------------------------------------------------------------
SCORE = [
    # B, Sq, Hq, Hkv, D, bs, longest, causal, dtype
    (3, 1, 4, 1, 128, 16, 700, 0, "bf16"), (2, 3, 10, 2, 64, 16, 3000, 1, "fp16"), (2, 1, 16, 1, 256, 64, 900, 0, "bf16"),
    (2, 2, 24, 1, 128, 16, 500, 1, "bf16"), (1, 5, 256, 2, 64, 32, 400, 1, "bf16"), (2, 70, 3, 3, 128, 16, 200, 1, "fp16"),
    (4, 40, 7, 1, 64, 128, 1000, 0, "bf16"), (1, 1, 1, 1, 128, 16, 1, 0, "bf16"), (1, 4, 9, 1, 256, 1024, 5000, 1, "fp16"),
    (1, 2, 150, 1, 64, 16, 100, 1, "bf16"), (70000, 1, 1, 1, 64, 16, 16, 0, "bf16"),
]


def score_problem(seed, B, sq, hq, hkv, d, bs, longest, dtype):
    rng = np.random.default_rng(seed)
    ctx, ql = lengths(rng, B, sq, longest)
    bt, nblocks, maxb = tables(rng, ctx, bs, 3)
    q = torch.from_numpy(rng.standard_normal((B, sq, hq, d))).to(KINDS[dtype][0])
    mid, wide = rng.standard_normal((nblocks, hkv, d)), rng.random((nblocks, hkv, d)) * 2
    bounds = torch.from_numpy(np.stack((mid - wide, mid + wide), 2)).to(KINDS[dtype][0])
    return rng, ctx, ql, bt, nblocks, maxb, q, bounds


def run_scores(pa_mod, cfg, q, bounds, bt, ctx, ql, dev, want_flags=0):
    flags = gpu([0], dev)
    scores = torch.full((cfg.batch, cfg.max_q_len, cfg.num_kv_heads, cfg.max_blocks_per_seq), float("nan"), device=dev)
    pa_mod.score_blocks(cfg, q.to(dev), bounds.to(dev), gpu(bt, dev), gpu(ctx, dev), gpu(ql, dev), scores, flags)
    assert int(flags.item()) == want_flags
    return scores


def check_scores(got, want, size, d):
    """2 D products (exact: 16-bit factors in fp32) are summed and scaled: 2 D + 1 roundings, each
    (truncation in the MMA's adder included) at most 2^-23 of the sum of magnitudes."""
    got = got.double().cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = ~fin & ~np.isnan(want)
    assert np.array_equal(got[inf], want[inf])
    assert (np.abs(got[fin] - want[fin]) <= (2 * d + 1) * 2.0 ** -23 * size[fin]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,hq,hkv,d,bs,longest,causal,dtype", SCORE)
def test_scores_match_64_bits(B, sq, hq, hkv, d, bs, longest, causal, dtype, cuda_device, pa):
    _, ctx, ql, bt, nblocks, maxb, q, bounds = score_problem(2, B, sq, hq, hkv, d, bs, longest, dtype)
    cfg = config(B, sq, hq, hkv, d, bs, maxb, nblocks, dtype, causal)
    got = run_scores(pa, cfg, q, bounds, bt, ctx, ql, cuda_device)
    want, size = plain64.score(q, bounds, ctx, ql, bt, bs, causal, float(np.float32(d ** -0.5)), hkv, nblocks)
    check_scores(got, want, size, d)


@pytest.mark.gpu
def test_scores_of_odd_values_bad_pages_and_lengths(cuda_device, pa):
    rng, ctx, ql, bt, nblocks, maxb, q, bounds = score_problem(3, 4, 2, 6, 2, 128, 16, 500, "bf16")
    ctx[1], ql[1] = 60, 2
    ctx[2], ql[2] = 3, 5                      # bad lengths
    bt[0, 3], bt[0, 4] = nblocks, -5          # bad pages
    for p, v in ((5, np.inf), (6, np.nan), (7, -np.inf)):
        bounds[bt[0, p], 0, 1, 9] = v
    q[1, 1, 2, 4] = float("nan")
    cfg = config(4, 2, 6, 2, 128, 16, maxb, nblocks, causal=1)
    got = run_scores(pa, cfg, q, bounds, bt, ctx, ql, cuda_device, pa.FLAG_BAD_LENGTHS | pa.FLAG_BAD_BLOCK_ID)
    ok = ql.copy()
    ok[2] = 0
    want, size = plain64.score(q, bounds, ctx, ok, bt, 16, 1, float(np.float32(128 ** -0.5)), 2, nblocks)
    check_scores(got, want, size, 128)


# ---- selection --------------------------------------------------------------------------------
SELECT = [
    # B, Sq, Hkv, bs, longest, top_k, first, last, causal, values
    (3, 1, 2, 16, 900, 8, 0, 0, 0, "plain"), (2, 4, 1, 16, 3000, 33, 2, 3, 1, "ties"), (2, 2, 3, 64, 500, 100, 1, 1, 1, "plain"),
    (1, 1, 1, 16, 40000, 128, 1, 4, 0, "ties"), (2, 1, 1, 16, 20000, 1000, 0, 0, 0, "odd"), (2, 3, 2, 16, 300, 1, 0, 1, 1, "odd"),
    (2, 1, 2, 16, 5000, 5, 2, 3, 0, "equal"), (1, 1, 1, 1024, 1, 4, 1, 1, 0, "plain"), (2, 1, 1, 16, 600, 37, 0, 0, 0, "equal"),
    (1, 1, 2, 16, 70000, 300, 3, 3, 0, "plain"), (1, 1, 1, 16, 900000, 64, 1, 1, 0, "ties"), (1, 1, 1, 16, 900000, 55000, 1, 1, 0, "odd"),
    (40, 1, 4, 16, 33000, 128, 1, 4, 0, "plain"), (20, 4, 2, 16, 100000, 300, 2, 4, 1, "odd"),  # more rows than SMs, long ones
    (40, 1, 5, 16, 150000, 64, 0, 1, 0, "ties"), (2, 1, 1, 16, 528, 32, 0, 0, 0, "plain"), (2, 1, 1, 16, 512, 32, 0, 0, 0, "plain"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,hkv,bs,longest,top_k,first,last,causal,values", SELECT)
def test_selection_is_that_of_a_sort(B, sq, hkv, bs, longest, top_k, first, last, causal, values, cuda_device, pa):
    rng = np.random.default_rng(longest)
    ctx, ql = lengths(rng, B, sq, longest)
    maxb = plain64.pages(longest, bs) + 3
    x = rng.standard_normal((B, sq, hkv, maxb)).astype(np.float32)
    if values == "ties":
        x = np.round(x * 4) / 4 * np.where(rng.random(x.shape) < 0.5, 1, -1).astype(np.float32)  # (both zeros)
    elif values == "equal":
        x[:] = 1.5
    elif values == "odd":
        for v in (np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-45, -1e-45):
            x[rng.random(x.shape) < 0.05] = v
    for b in range(B):  # what lies out of a row's reach is not looked at
        x[b, :, :, plain64.pages(ctx[b], bs):] = np.nan
    cfg = config(B, sq, hkv, hkv, 128, bs, maxb, 1, causal=causal)
    sel = torch.full((B, sq, hkv, top_k), -9, dtype=torch.int32, device=cuda_device)
    num = torch.full((B, sq, hkv), -9, dtype=torch.int32, device=cuda_device)
    flags = gpu([0], cuda_device)
    pa.select_blocks(cfg, torch.from_numpy(x).to(cuda_device), gpu(ctx, cuda_device), gpu(ql, cuda_device), first, last,
                     sel, num, flags)
    want, count = plain64.select(x, ctx.tolist(), ql.tolist(), bs, causal, top_k, first, last)
    assert int(flags.item()) == 0
    assert np.array_equal(num.cpu().numpy(), count)
    assert np.array_equal(sel.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [255, 256, 257, 300, 2000])
@pytest.mark.parametrize("values", ["whole range", "neighbours", "subnormal", "one finite", "no finite", "outlier", "halves"])
def test_selection_from_odd_ranges(n, values, cuda_device, pa):
    """Ranges whose width overflows, vanishes or is that of one far value: every rank's page is a sort's."""
    rng = np.random.default_rng(n)
    top = np.finfo(np.float32).max
    x = rng.standard_normal((1, 1, 6, n)).astype(np.float32)
    if values == "whole range":
        x = (x / np.abs(x).max() * top).astype(np.float32)
        x[0, 0, 1, 3:5] = top, -top
        x[0, 0, 2, 3:6] = np.inf, -np.inf, np.nan
    elif values == "neighbours":
        x = (np.float32(1).view(np.int32) + rng.integers(0, 3, x.shape)).astype(np.int32).view(np.float32)
    elif values == "subnormal":
        x = (rng.integers(0, 1000, x.shape).astype(np.int32) | rng.choice([0, -2**31], x.shape).astype(np.int32)).view(np.float32)
    elif values == "one finite":
        x = rng.choice(np.float32([np.inf, -np.inf, np.nan]), x.shape)
        x[..., n // 2] = -3.0
    elif values == "no finite":
        x = rng.choice(np.float32([np.inf, -np.inf, np.nan]), x.shape)
    elif values == "outlier":
        x[0, 0, :, n - 9] = 1e30
        x[0, 0, 3:, 7] = -1e38
    else:
        x = np.where(rng.random(x.shape) < 0.5, x, np.float32(-0.0))
    for k in (1, 2, n // 3, n - 1):
        cfg = config(1, 1, 6, 6, 128, 16, n, 1)
        sel = torch.full((1, 1, 6, k), -9, dtype=torch.int32, device=cuda_device)
        num = torch.full((1, 1, 6), -9, dtype=torch.int32, device=cuda_device)
        pa.select_blocks(cfg, torch.from_numpy(x).to(cuda_device), gpu([n * 16], cuda_device), gpu([1], cuda_device), 0, 1,
                         sel, num)
        want, count = plain64.select(x, [n * 16], [1], 16, 0, k, 0, 1)
        assert np.array_equal(num.cpu().numpy(), count)
        assert np.array_equal(sel.cpu().numpy(), want)


@pytest.mark.gpu
def test_selection_of_bad_lengths_is_empty(cuda_device, pa):
    cfg = config(3, 2, 2, 2, 128, 16, 8, 1)
    x = torch.randn(3, 2, 2, 8, device=cuda_device)
    sel = torch.full((3, 2, 2, 4), -9, dtype=torch.int32, device=cuda_device)
    num = torch.full((3, 2, 2), -9, dtype=torch.int32, device=cuda_device)
    flags = gpu([0], cuda_device)
    pa.select_blocks(cfg, x, gpu([100, 8 * 16 + 1, 40], cuda_device), gpu([2, 1, 3], cuda_device), 0, 0, sel, num, flags)
    assert int(flags.item()) == pa.FLAG_BAD_LENGTHS
    want, count = plain64.select(x.cpu().numpy(), [100, 0, 0], [2, 0, 0], 16, 0, 4, 0, 0)
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(num.cpu().numpy(), count)


@pytest.mark.gpu
def test_no_appended_key_beats_its_page(cuda_device, pa):
    """Prompts, then single tokens, appended with their bounds: no logit is above its page's score,
    and the page of the largest logit is selected whenever its score is the largest."""
    rng, bs, d, hq, hkv = np.random.default_rng(4), 16, 128, 8, 2
    start, steps = np.array([37, 100, 3]), 30
    bt, nblocks, maxb = tables(rng, start + steps, bs)
    keys = torch.from_numpy(rng.standard_normal((3, 140, hkv, d))).bfloat16().to(cuda_device)
    bounds = torch.full((nblocks, hkv, 2, d), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    table = gpu(bt, cuda_device)
    pa.update_bounds(config(3, 100, hq, hkv, d, bs, maxb, nblocks), keys[:, :100].contiguous(), table,
                     gpu(start, cuda_device), gpu(start, cuda_device), bounds)
    cfg = config(3, 1, hq, hkv, d, bs, maxb, nblocks)
    for j in range(steps):
        at = start + j
        new = torch.stack([keys[b, at[b]] for b in range(3)])[:, None].contiguous()
        ctx = gpu(at + 1, cuda_device)
        pa.update_bounds(cfg, new, table, ctx, gpu([1] * 3, cuda_device), bounds)
    q = torch.from_numpy(rng.standard_normal((3, 1, hq, d))).bfloat16().to(cuda_device)
    scores = torch.empty(3, 1, hkv, maxb, device=cuda_device)
    pa.score_blocks(cfg, q, bounds, table, ctx, gpu([1] * 3, cuda_device), scores)
    for b in range(3):
        n = int(start[b]) + steps
        x = torch.einsum("ghd,tgd->gth", q[b, 0].double().reshape(hkv, -1, d), keys[b, :n].double()) * d ** -0.5
        best = x.amax(2)  # [Hkv, n]
        for p in range(plain64.pages(n, bs)):
            assert (best[:, p * bs:(p + 1) * bs].amax(1) <= scores[b, 0, :, p].double() * (1 + 1e-5) + 1e-5).all()


# ---- refusals -----------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_cache_work_gb300.build import build
        build()
    return pa.load()


def test_bounds_and_scores_refused_on_the_host(lib):
    fake = 1 << 20  # never dereferenced: every call below is rejected on the host
    good = dict(B=2, sq=1, hq=8, hkv=2, d=128, bs=16, maxb=8, nblocks=32)

    def bounds(c=None, **kw):
        a = dict(k=fake, bt=fake, ctx=fake, q=fake, box=fake, flags=None)
        a.update(kw)
        return lib.pa_update_bounds(ctypes.byref(c or config(**good)), *a.values(), None)

    def score(c=None, **kw):
        a = dict(q=fake, box=fake, bt=fake, ctx=fake, ql=fake, scores=fake, flags=None)
        a.update(kw)
        return lib.pa_score_blocks(ctypes.byref(c or config(**good)), *a.values(), None)

    for call, wide, names in ((bounds, ("k", "box"), ("k", "bt", "ctx", "q", "box")),
                              (score, ("q", "box"), ("q", "box", "bt", "ctx", "ql", "scores"))):
        for k in names:
            assert call(**{k: None}) == pa.ERR_INVALID_ARG
            assert call(**{k: fake + (8 if k in wide else 2)}) == pa.ERR_INVALID_ARG
        assert call(flags=fake + 2) == pa.ERR_INVALID_ARG
        for kw, want in ((dict(d=96), pa.ERR_UNSUPPORTED), (dict(bs=8), pa.ERR_UNSUPPORTED), (dict(bs=48), pa.ERR_UNSUPPORTED),
                         (dict(B=0), pa.ERR_INVALID_ARG), (dict(hkv=0), pa.ERR_INVALID_ARG)):
            assert call(config(**{**good, **kw})) == want, kw
        c = config(**good)
        c.q_dtype = pa.FP8_E4M3
        assert call(c) == pa.ERR_UNSUPPORTED
    for kw in (dict(hq=9), dict(B=1 << 21, sq=1 << 11), dict(maxb=1 << 28)):
        assert score(config(**{**good, **kw})) == pa.ERR_UNSUPPORTED, kw
    assert score(config(**good, sm=float("nan"))) == pa.ERR_INVALID_ARG
    assert lib.pa_update_bounds(None, *([fake] * 5), None, None) == pa.ERR_INVALID_ARG
    assert lib.pa_score_blocks(None, *([fake] * 6), None, None) == pa.ERR_INVALID_ARG


def test_selection_refused_on_the_host(lib):
    fake = 1 << 20

    def call(c=None, **kw):
        a = dict(scores=fake, ctx=fake, ql=fake, top_k=8, first=1, last=1, sel=fake, num=fake, flags=None)
        a.update(kw)
        return lib.pa_select_blocks(ctypes.byref(c or config(2, 1, 8, 2, 128, 16, 8, 32)), *a.values(), None)

    for k in ("scores", "ctx", "ql", "sel", "num"):
        assert call(**{k: None}) == pa.ERR_INVALID_ARG
        assert call(**{k: fake + 2}) == pa.ERR_INVALID_ARG
    for kw in (dict(top_k=0), dict(first=-1), dict(last=-1), dict(first=5, last=4), dict(first=2 ** 31 - 1, last=1)):
        assert call(**kw) == pa.ERR_INVALID_ARG, kw
    assert call(config(2, 1, 8, 2, 128, 24, 8, 32)) == pa.ERR_UNSUPPORTED
    assert call(config(1 << 20, 1 << 10, 8, 8, 128, 16, 8, 32)) == pa.ERR_UNSUPPORTED
    assert call(config(2, 1, 8, 2, 128, 16, 1 << 28, 32)) == pa.ERR_UNSUPPORTED
    assert lib.pa_select_blocks(None, fake, fake, fake, 8, 0, 0, fake, fake, None, None) == pa.ERR_INVALID_ARG
