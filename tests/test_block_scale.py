"""An fp8 cache with one scale for each (page, kv head): the append bit for bit against the plain
fp32 steps, the decode (every kernel that serves such a cache) against 64 bits, both together in
a generation loop, and the refusals."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_work_gb300 as pa
import plain64

KINDS = {"bf16": (torch.bfloat16, pa.BF16), "fp16": (torch.float16, pa.FP16)}


def config(B, sq, hq, hkv, d, bs, maxb, nblocks, dtype="bf16", causal=0, **kw):
    return pa.PaConfig(batch=B, max_q_len=sq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                       max_blocks_per_seq=maxb, num_blocks=nblocks, q_dtype=KINDS[dtype][1],
                       kv_dtype=pa.FP8_E4M3, kv_scale_mode=pa.SCALE_PER_BLOCK, causal=causal,
                       sm_scale=d ** -0.5, **kw)


def cache(rng, nblocks, bs, hkv, d, spread):
    """Codes of any finite value, scales over 2^-spread .. 2^spread around 0.01."""
    codes = torch.from_numpy(rng.integers(0, 256, (nblocks, bs, hkv, d), dtype=np.uint8))
    codes = torch.where((codes & 127) == 127, codes - 1, codes)
    codes = torch.where(torch.from_numpy(rng.random(codes.shape) < 0.5), codes & 0xbf, codes)
    scale = 0.01 * 2.0 ** rng.uniform(-spread, spread, (nblocks, hkv))
    return codes, torch.from_numpy(scale.astype(np.float32))


def tables(rng, ctx, bs, extra=2):
    need = [plain64.pages(n, bs) for n in ctx]
    nblocks, maxb = sum(need) + extra, max(1, max(need))
    ids = rng.permutation(nblocks)
    bt = np.full((len(ctx), maxb), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt, nblocks, maxb


# ---- append -----------------------------------------------------------------------------------
def new_rows(rng, shape, kind, dtype):
    x = rng.standard_normal(shape) * np.where(rng.random(shape[:3] + (1,)) < 0.3, 6.0, 1.0)
    if kind == "zeros":
        x[rng.random(shape[0]) < 0.7] = 0
    elif kind == "odd":  # infinities, NaN, the least and the largest of the type
        for v in (np.inf, -np.inf, np.nan, 2.0 ** -24, 6e4):
            x[tuple(rng.integers(0, n, 20) for n in shape)] = v
    elif kind == "tiny":
        x *= 2.0 ** -131 if dtype == "bf16" else 2.0 ** -22
    return torch.from_numpy(x).to(KINDS[dtype][0])


APPEND = [
    # B, Sq, Hkv, D, bs, longest prior, dtype, kind
    (5, 1, 2, 128, 16, 60, "bf16", "plain"), (3, 1, 1, 64, 32, 0, "bf16", "plain"),
    (4, 3, 3, 256, 16, 40, "fp16", "plain"), (3, 40, 2, 128, 16, 50, "bf16", "odd"),
    (2, 300, 1, 128, 1024, 1500, "bf16", "plain"), (2, 1100, 1, 64, 1024, 300, "fp16", "odd"),
    (6, 5, 2, 128, 64, 130, "bf16", "zeros"), (4, 20, 2, 64, 16, 33, "bf16", "tiny"),
    (4, 20, 1, 128, 32, 33, "fp16", "tiny"), (9, 130, 2, 256, 64, 100, "bf16", "plain"),
]


def same_codes(a, b):
    x, y = a.cpu().view(torch.float8_e4m3fn).float(), b.cpu().view(torch.float8_e4m3fn).float()
    return bool(((x == y) | (x.isnan() & y.isnan())).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,hkv,d,bs,prior,dtype,kind", APPEND)
def test_append_matches_the_plain_steps(B, sq, hkv, d, bs, prior, dtype, kind, cuda_device, pa):
    dev = cuda_device
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        ql = rng.integers(0, sq + 1, B)
        ql[0] = sq
        ctx = rng.integers(0, prior + 1, B) + ql
        bt, nblocks, maxb = tables(rng, ctx, bs)
        kc, ks = cache(rng, nblocks, bs, hkv, d, 2)
        vc, vs = cache(rng, nblocks, bs, hkv, d, 2)
        if kind == "tiny":
            ks, vs = ks * 2.0 ** -118, vs * 2.0 ** -118
        kn, vn = (new_rows(rng, (B, sq, hkv, d), kind, dtype) for _ in "kv")
        want = [plain64.append_block(x, c, s, ctx.tolist(), ql.tolist(), bt, bs)
                for x, c, s in ((kn, kc, ks), (vn, vc, vs))]
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        got = [x.to(dev).clone() for x in (kc, vc, ks, vs)]
        flags = t([0])
        args = (config(B, sq, hkv, hkv, d, bs, maxb, nblocks, dtype), kn.to(dev), vn.to(dev), t(bt), t(ctx), t(ql),
                *got, flags)
        for again in range(2):  # the same rows once more change nothing
            pa.append_kv(*args)
            assert int(flags.item()) == 0
            assert torch.equal(got[2].cpu(), want[0][1]) and torch.equal(got[3].cpu(), want[1][1])
            assert same_codes(got[0], want[0][0]) and same_codes(got[1], want[1][0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_quotient_is_the_rounded_one(dtype, cuda_device, pa):
    """Every finite value of the type over scales of every kind of significand, small ones among
    them: the codes are those of a division."""
    dev, rng, bs, d = cuda_device, np.random.default_rng(5), 64, 256
    kind = KINDS[dtype][0]
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(kind)
    every = every[torch.isfinite(every)].float()
    pages = []
    for big in (1.0, 3.0, 1e-3, 448.0, 6e4, 1.7e-5, *rng.uniform(0.5, 900.0, 26), *(2.0 ** -np.arange(90.0, 126.0, 4) if dtype == "bf16" else ())):
        big = float(torch.tensor(big).to(kind))
        x = every[every.abs() <= big]
        x = x[torch.from_numpy(rng.permutation(len(x))[:bs * d - 1])]
        pages.append(torch.nn.functional.pad(torch.cat((x, torch.tensor([big]))), (0, bs * d - 1 - len(x))))
    n = len(pages)
    new = torch.stack(pages).reshape(n, bs, 1, d).to(kind)
    bt = np.arange(n)[:, None]
    codes, scale = torch.zeros(n, bs, 1, d, dtype=torch.uint8), torch.ones(n, 1)
    want = plain64.append_block(new, codes, scale, [bs] * n, [bs] * n, bt, bs)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    got = [codes.to(dev).clone(), codes.to(dev).clone(), scale.to(dev).clone(), scale.to(dev).clone()]
    pa.append_kv(config(n, bs, 1, 1, d, bs, 1, n, dtype), new.to(dev), new.to(dev), t(bt), t([bs] * n), t([bs] * n), *got)
    assert torch.equal(got[2].cpu(), want[1]) and torch.equal(got[3].cpu(), want[1])
    assert same_codes(got[0], want[0]) and same_codes(got[1], want[0])


@pytest.mark.gpu
def test_append_flags_and_skips(cuda_device, pa):
    dev, rng = cuda_device, np.random.default_rng(3)
    B, sq, hkv, d, bs = 4, 20, 2, 128, 16
    ctx, ql = np.array([30, 25, 40, 3]), np.array([20, 20, 20, 3])
    bt, nblocks, maxb = tables(rng, ctx, bs)
    kc, ks = cache(rng, nblocks, bs, hkv, d, 2)
    vc, vs = cache(rng, nblocks, bs, hkv, d, 2)
    kn, vn = (new_rows(rng, (B, sq, hkv, d), "plain", "bf16") for _ in "kv")
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    bad_ctx, bad_bt = ctx.copy(), bt.copy()
    bad_ctx[1] = 10          # fewer tokens than new ones: sequence 1 is skipped
    bad_bt[2, 1] = nblocks   # one page of sequence 2 is skipped
    want = []
    for x, c, s in ((kn, kc, ks), (vn, vc, vs)):
        ok = np.array([20, 0, 20, 3])
        wc, wsc = plain64.append_block(x, c, s, np.array([30, 0, 40, 3]).tolist(), ok.tolist(), bt, bs)
        wc[bt[2, 1]], wsc[bt[2, 1]] = c[bt[2, 1]], s[bt[2, 1]]
        want.append((wc, wsc))
    got = [x.to(dev).clone() for x in (kc, vc, ks, vs)]
    flags = t([0])
    pa.append_kv(config(B, sq, hkv, hkv, d, bs, maxb, nblocks), kn.to(dev), vn.to(dev), t(bad_bt), t(bad_ctx), t(ql),
                 *got, flags)
    assert int(flags.item()) == pa.FLAG_BAD_LENGTHS | pa.FLAG_BAD_BLOCK_ID
    assert torch.equal(got[2].cpu(), want[0][1]) and torch.equal(got[3].cpu(), want[1][1])
    assert same_codes(got[0], want[0][0]) and same_codes(got[1], want[1][0])


# ---- decode -----------------------------------------------------------------------------------
DECODE = [
    # B, Sq, Hq, Hkv, D, bs, longest, causal, dtype, spread, extra config
    (3, 1, 4, 1, 128, 16, 300, 0, "bf16", 2, {}), (2, 1, 16, 1, 128, 1024, 2500, 0, "bf16", 2, {}),
    (3, 2, 12, 2, 128, 64, 400, 1, "fp16", 12, {}), (2, 4, 6, 3, 256, 16, 200, 1, "bf16", 12, {}),
    (2, 8, 8, 2, 128, 32, 300, 1, "bf16", 1, {}), (3, 1, 5, 5, 64, 16, 200, 0, "bf16", 12, {}),
    (2, 3, 7, 1, 64, 128, 300, 1, "fp16", 2, {}), (2, 4, 16, 1, 128, 16, 500, 1, "bf16", 12, {}),
    (2, 4, 16, 1, 128, 1024, 3000, 1, "fp16", 2, {}), (1, 25, 8, 2, 128, 64, 600, 1, "bf16", 12, {}),
    (2, 9, 8, 2, 128, 16, 300, 0, "fp16", 2, dict(num_ctas=7)),
    (2, 1, 8, 2, 128, 16, 900, 0, "bf16", 12, dict(num_ctas=9, split_merge=1)),
    (2, 4, 16, 1, 128, 64, 900, 1, "bf16", 6, dict(num_ctas=9, split_merge=1)),
    (2, 20, 16, 8, 256, 32, 300, 1, "bf16", 2, dict(num_ctas=40)),
    (1, 1, 1, 1, 128, 16, 1, 0, "bf16", 2, {}), (2, 70, 1, 1, 256, 16, 150, 1, "fp16", 2, {}),
]


def decode_problem(seed, B, sq, hq, hkv, d, bs, longest, dtype, spread):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(max(1, longest // 3), longest + 1, B)
    ctx[0] = longest
    ql = np.minimum(ctx, rng.integers(1, sq + 1, B))
    if B > 2:
        ctx[1] = ql[1] = 0
    bt, nblocks, maxb = tables(rng, ctx, bs)
    kc, ks = cache(rng, nblocks, bs, hkv, d, min(spread, 2))
    vc, vs = cache(rng, nblocks, bs, hkv, d, spread)
    q = torch.from_numpy(rng.standard_normal((B, sq, hq, d))).to(KINDS[dtype][0])
    return dict(ctx=ctx, ql=ql, bt=bt, nblocks=nblocks, maxb=maxb, kc=kc, ks=ks, vc=vc, vs=vs, q=q)


def reference(p, causal, sm):
    k, v = plain64.values(p["kc"], p["ks"], "block"), plain64.values(p["vc"], p["vs"], "block")
    n = [plain64.pages(x, p["kc"].shape[1]) for x in p["ctx"]]
    return plain64.attend(p["q"], k, v, p["bt"], lambda b, i, g: range(n[b]), p["ctx"].tolist(), p["ql"].tolist(),
                          causal, sm)


def run_decode(pa_mod, p, cfg, dev):
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    q = p["q"].to(dev)
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device=dev)
    ws = torch.empty(pa_mod.workspace_size(cfg), dtype=torch.uint8, device=dev)
    bt, ctx, ql = t(p["bt"]), t(p["ctx"]), t(p["ql"])
    pa_mod.plan(cfg, bt, ctx, ql, ws)
    pa_mod.decode(cfg, q, p["kc"].to(dev), p["vc"].to(dev), p["ks"].to(dev), p["vs"].to(dev), bt, ctx, ql, out, lse, ws)
    pa_mod.reduce(cfg, out, lse, ws)
    assert pa_mod.read_flags(ws) == 0
    return out, lse


# Weights are rounded to f16 (half a step: 2^-11).  On the tcgen05 kernel (33 rows and more) a
# query element is off by at most 2^-19 of its row's largest (its E4M3 terms end at the least
# subnormal), so a logit by at most sm sum_d |k_d| 2^-19 max|q| = 128^-0.5 * 128 * 1.2 * 2^-19 * 4
# = 1.1e-4: that much relative to a weight.
@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,hq,hkv,d,bs,longest,causal,dtype,spread,extra", DECODE)
def test_decode_matches_64_bits(B, sq, hq, hkv, d, bs, longest, causal, dtype, spread, extra, cuda_device, pa):
    p = decode_problem(11, B, sq, hq, hkv, d, bs, longest, dtype, spread)
    cfg = config(B, sq, hq, hkv, d, bs, p["maxb"], p["nblocks"], dtype, causal, **extra)
    out, lse = run_decode(pa, p, cfg, cuda_device)
    ref, ref_lse, size = reference(p, causal, float(np.float32(d ** -0.5)))
    slack = 1.1e-4 if sq * hq // hkv > 32 else 2e-5
    plain64.check_attention(out, lse, ref, ref_lse, size, p["q"].dtype, 2.0 ** -11, slack)


@pytest.mark.gpu
@pytest.mark.parametrize("sq,hq,hkv,d", [(1, 4, 1, 128), (4, 16, 1, 128), (1, 4, 2, 64), (2, 4, 1, 256)])
def test_tiny_and_huge_scales_lose_nothing(sq, hq, hkv, d, cuda_device, pa):
    """A weight times a V scale of 1e-7 or 1e4 would leave f16: outputs stay as exact as others."""
    for factor in (1e-7, 1e6):
        p = decode_problem(5, 2, sq, hq, hkv, d, 16, 300, "bf16", 1)
        p["vs"] = p["vs"] * factor
        cfg = config(2, sq, hq, hkv, d, 16, p["maxb"], p["nblocks"])
        out, lse = run_decode(pa, p, cfg, cuda_device)
        ref, ref_lse, size = reference(p, 0, float(np.float32(d ** -0.5)))
        # (outputs of 1e-7 are compared relative to their size: no absolute term)
        scale = 1 / factor
        plain64.check_attention(out.double().cpu() * scale, lse, ref * scale, ref_lse, size * scale, torch.bfloat16,
                                2.0 ** -11, 1.1e-4)


# ---- scales that lie far apart ----------------------------------------------------------------
def far_scales(rng, p, kind, ratio):
    """Half of the pages, first ones among them, get a V scale 1 / ratio times the others' and no
    part in the output: they hold zeros ("zeros": what an append of zeros leaves, with its scale of
    1) or keys whose logits lie far below every other ("low")."""
    nblocks = p["vs"].shape[0]
    far = torch.from_numpy(rng.random(nblocks) < 0.5)
    for b in range(len(p["ctx"])):
        if p["ctx"][b]:
            far[p["bt"][b, 0]] = True
            far[p["bt"][b, plain64.pages(p["ctx"][b], p["kc"].shape[1]) - 1]] = False
    p["vs"] = torch.where(far[:, None], p["vs"] / ratio, p["vs"])
    if kind == "zeros":
        p["vc"][far] = 0
    else:  # keys of -448 * 0.03 in every channel against queries above zero: logits below -80
        p["q"] = p["q"].abs()
        p["kc"][far] = 0xfe
        p["ks"][far] = 0.03


FAR = [
    # Sq, Hq, Hkv, D, bs, dtype, longest
    (1, 8, 2, 128, 16, "bf16", 300), (2, 8, 2, 128, 32, "fp16", 300), (2, 8, 2, 64, 16, "bf16", 300),
    (1, 4, 1, 256, 16, "fp16", 200), (10, 4, 2, 256, 16, "bf16", 200), (20, 16, 8, 256, 32, "fp16", 200),
    (4, 16, 1, 128, 16, "bf16", 300), (4, 16, 1, 128, 64, "fp16", 600), (8, 16, 1, 128, 32, "bf16", 300),
]


# Weights keep f16's half step (2^-11) whatever the other pages' scales are.  On the tcgen05 kernel
# (33 rows and more) a scale 2^-32 of the item's unit leaves weights below 2^-11 of the largest to
# f16's subnormals: off by 2^-22 each, all tokens together by longest * 2^-22 of the largest weight.
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["zeros", "low"])
@pytest.mark.parametrize("sq,hq,hkv,d,bs,dtype,longest", FAR)
def test_a_page_of_far_larger_scale_costs_the_others_nothing(sq, hq, hkv, d, bs, dtype, longest, kind, cuda_device, pa):
    tensor_core = d == 128 and sq * hq // hkv > 32
    for ratio in (1e-5, 1e-7, 1e-9, *(() if tensor_core else (1e-14,))):
        rng = np.random.default_rng(21)
        p = decode_problem(13, 2, sq, hq, hkv, d, bs, longest, dtype, 1)
        far_scales(rng, p, kind, ratio)
        ref, ref_lse, size = reference(p, 1, float(np.float32(d ** -0.5)))
        slack = 1.1e-4 + longest * 2.0 ** -22 if tensor_core else 2e-5
        for ctas in (0, 3):  # an item a step, and items of many steps
            cfg = config(2, sq, hq, hkv, d, bs, p["maxb"], p["nblocks"], dtype, 1, num_ctas=ctas)
            out, lse = run_decode(pa, p, cfg, cuda_device)
            plain64.check_attention(out, lse, ref, ref_lse, size, p["q"].dtype, 2.0 ** -11, slack)


@pytest.mark.gpu
@pytest.mark.parametrize("sq,hq,hkv,d", [(1, 4, 1, 128), (2, 4, 2, 64), (1, 8, 1, 256), (5, 4, 1, 256), (10, 4, 1, 256), (4, 16, 1, 128)])
def test_queries_that_leave_f16(sq, hq, hkv, d, cuda_device, pa):
    """Queries of 1e6 or 1e-6 with keys that make up for it: as exact as any other."""
    for factor in (1e6, 1e-6):
        p = decode_problem(19, 2, sq, hq, hkv, d, 16, 300, "bf16", 1)
        p["q"] = (p["q"].float() * factor).bfloat16()
        p["ks"] = p["ks"] / factor
        cfg = config(2, sq, hq, hkv, d, 16, p["maxb"], p["nblocks"], causal=1)
        out, lse = run_decode(pa, p, cfg, cuda_device)
        ref, ref_lse, size = reference(p, 1, float(np.float32(d ** -0.5)))
        plain64.check_attention(out, lse, ref, ref_lse, size, torch.bfloat16, 2.0 ** -11, 1.1e-4 if sq * hq // hkv > 32 else 2e-5)


@pytest.mark.gpu
def test_equal_scales_are_the_per_token_cache(cuda_device, pa):
    """The same scale on every page, given per page and per token: the same attention."""
    p = decode_problem(6, 2, 1, 8, 2, 128, 16, 400, "bf16", 0)
    p["ks"][:], p["vs"][:] = 0.0078125, 0.015625
    cfg = config(2, 1, 8, 2, 128, 16, p["maxb"], p["nblocks"])
    out, lse = run_decode(pa, p, cfg, cuda_device)
    cfg.kv_scale_mode = pa.SCALE_PER_TOKEN
    p["ks"] = p["ks"][:, None].expand(-1, 16, -1).contiguous()
    p["vs"] = p["vs"][:, None].expand(-1, 16, -1).contiguous()
    out2, lse2 = run_decode(pa, p, cfg, cuda_device)
    assert torch.allclose(out.float(), out2.float(), rtol=2.0 ** -7, atol=1e-4)
    assert torch.allclose(lse, lse2, rtol=1e-5, atol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("sq,hq,hkv,d,bs", [(1, 16, 1, 128, 16), (2, 4, 1, 64, 64), (1, 8, 2, 256, 32), (3, 6, 1, 256, 16),
                                            (4, 16, 1, 128, 32)])
def test_decode_reads_nothing_else(sq, hq, hkv, d, bs, cuda_device, pa):
    """NaN codes and scales wherever no key lies change no bit; the static scratch gives the same; a
    bad page is flagged and the other sequences keep their bits; so is a plan for other lengths."""
    p = decode_problem(7, 4, sq, hq, hkv, d, bs, 700, "bf16", 2)
    p["ctx"][1] = p["ql"][1] = 1
    p["ql"][:] = np.minimum(p["ctx"], sq)
    p["bt"][1, 0] = p["nblocks"] - 1
    cfg = config(4, sq, hq, hkv, d, bs, p["maxb"], p["nblocks"], causal=1)
    out, lse = run_decode(pa, p, cfg, cuda_device)
    free = np.ones((p["nblocks"], bs), bool)
    for b in range(4):
        for t in range(p["ctx"][b]):
            free[p["bt"][b, t // bs], t % bs] = False
    for k in ("kc", "vc"):
        p[k][torch.from_numpy(free)] = 0x7f
    for k in ("ks", "vs"):
        p[k][torch.from_numpy(free.all(1))] = float("nan")
    again, lse_again = run_decode(pa, p, cfg, cuda_device)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)

    dev = cuda_device
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    args = [p[k].to(dev) for k in ("q", "kc", "vc", "ks", "vs")]
    bt, ctx, ql = t(p["bt"]), t(p["ctx"]), t(p["ql"])
    o2, l2 = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
    if pa.workspace_size(cfg) <= pa.STATIC_SCRATCH_BYTES:
        pa.decode_step_static(cfg, *args, bt, ctx, ql, o2, l2)
        assert torch.equal(o2, out) and torch.equal(l2, lse)

    ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=dev)

    def step(tables, now):
        pa.plan(cfg, bt, ctx, ql, ws)
        pa.decode(cfg, *args, tables, now, ql, o2, l2, ws)
        pa.reduce(cfg, o2, l2, ws)
        torch.cuda.synchronize()

    for bad in (-1, p["nblocks"]):
        bt_bad = bt.clone()
        bt_bad[2, 0] = bad
        step(bt_bad, ctx)
        assert pa.read_flags(ws) == pa.FLAG_BAD_BLOCK_ID
        for b in (0, 1, 3):
            assert torch.equal(o2[b], out[b]) and torch.equal(l2[b], lse[b])
    if d < 256 or sq * hq // hkv <= 16:  # (the mma.sync kernel waits for the planner)
        half = ctx.clone()
        half[0] //= 2
        step(bt, half)
        assert pa.read_flags(ws) & pa.FLAG_STALE_PLAN
    step(bt, ctx)
    assert pa.read_flags(ws) == 0 and torch.equal(o2, out)


@pytest.mark.gpu
def test_generation_appends_then_decodes(cuda_device, pa):
    """Steps of append and decode (captured, on a stream of their own, replayed) over pages that
    grow: each step's output is that of the cache the plain append left."""
    dev, rng = cuda_device, np.random.default_rng(8)
    B, hq, hkv, d, bs, steps = 3, 8, 2, 128, 16, 20
    start = np.array([0, 15, 30])
    bt, nblocks, maxb = tables(rng, start + steps, bs)
    kc, ks = cache(rng, nblocks, bs, hkv, d, 1)
    vc, vs = cache(rng, nblocks, bs, hkv, d, 1)
    cfg = config(B, 1, hq, hkv, d, bs, maxb, nblocks)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(q=torch.zeros(B, 1, hq, d, dtype=torch.bfloat16, device=dev),
             kn=torch.zeros(B, 1, hkv, d, dtype=torch.bfloat16, device=dev),
             vn=torch.zeros(B, 1, hkv, d, dtype=torch.bfloat16, device=dev), ctx=t(start + 1), ql=t([1] * B), bt=t(bt),
             kc=kc.to(dev), vc=vc.to(dev), ks=ks.to(dev), vs=vs.to(dev))
    out, lse = torch.empty_like(s["q"]), torch.empty(B, 1, hq, device=dev)
    ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=dev)

    def step():
        pa.append_kv(cfg, s["kn"], s["vn"], s["bt"], s["ctx"], s["ql"], s["kc"], s["vc"], s["ks"], s["vs"])
        pa.plan(cfg, s["bt"], s["ctx"], s["ql"], ws)
        pa.decode(cfg, s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], s["ql"], out, lse, ws)
        pa.reduce(cfg, out, lse, ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()  # sets the kernels up; its rows are zeros, taken back below
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
        for x, y in ((s["kc"], kc), (s["vc"], vc), (s["ks"], ks), (s["vs"], vs)):
            x.copy_(y)
        for j in range(steps):
            ctx = (start + j + 1).tolist()
            q = torch.from_numpy(rng.standard_normal((B, 1, hq, d))).bfloat16()
            kn, vn = (new_rows(rng, (B, 1, hkv, d), "plain", "bf16") for _ in "kv")
            kc, ks = plain64.append_block(kn, kc, ks, ctx, [1] * B, bt, bs)
            vc, vs = plain64.append_block(vn, vc, vs, ctx, [1] * B, bt, bs)
            for x, y in ((s["q"], q), (s["kn"], kn), (s["vn"], vn), (s["ctx"], t(ctx))):
                x.copy_(y)
            g.replay()
            stream.synchronize()
            assert torch.equal(s["ks"].cpu(), ks) and torch.equal(s["vs"].cpu(), vs)
            assert same_codes(s["kc"], kc) and same_codes(s["vc"], vc)
            p = dict(q=q, kc=kc, ks=ks, vc=vc, vs=vs, ctx=np.array(ctx), ql=np.array([1] * B), bt=bt)
            ref, ref_lse, size = reference(p, 0, float(np.float32(d ** -0.5)))
            plain64.check_attention(out, lse, ref, ref_lse, size, torch.bfloat16, 2.0 ** -11)
    assert pa.read_flags(ws) == 0


# ---- refusals -----------------------------------------------------------------------------------
def test_per_page_scales_refused_on_the_host():
    import os
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_cache_work_gb300.build import build
        build()
    lib = pa.load()
    fake = 1 << 20  # never dereferenced: every call below is rejected on the host
    cfg = config(2, 1, 8, 2, 128, 16, 8, 32, num_ctas=4)
    n = ctypes.c_size_t(0)
    assert lib.pa_workspace_size(ctypes.byref(cfg), ctypes.byref(n)) == pa.OK
    dec = lambda ks, vs, c=cfg: lib.pa_decode(  # noqa: E731
        ctypes.byref(c), fake, fake, fake, ks, vs, fake, fake, fake, fake, None, fake, n.value, None)
    app = lambda ks, vs, c=cfg: lib.pa_append_kv(  # noqa: E731
        ctypes.byref(c), fake, fake, fake, fake, fake, fake, fake, ks, vs, None, None)
    for call in (dec, app):
        assert call(None, fake) == pa.ERR_INVALID_ARG
        assert call(fake, None) == pa.ERR_INVALID_ARG
        assert call(fake + 2, fake) == pa.ERR_INVALID_ARG
        wide = config(2, 1, 8, 2, 128, 16, 8, 32, num_ctas=4)
        wide.kv_dtype = pa.BF16
        assert call(fake, fake, wide) == pa.ERR_UNSUPPORTED
        mode = config(2, 1, 8, 2, 128, 16, 8, 32, num_ctas=4)
        mode.kv_scale_mode = 4
        assert call(fake, fake, mode) == pa.ERR_INVALID_ARG
    many = config(1 << 16, 1 << 20, 8, 2, 128, 16, 8, 32)
    assert app(fake, fake, many) == pa.ERR_UNSUPPORTED  # more page CTAs than a grid has


@pytest.mark.parametrize("mode,count", [(pa.SCALE_PER_TENSOR, 1), (pa.SCALE_PER_TOKEN, 32 * 16 * 2), (pa.SCALE_PER_BLOCK, 32 * 2)])
def test_binding_refuses_scales_that_do_not_fit(mode, count, monkeypatch):
    """The append writes its scales and the decodes read them, as many as the mode has: an array of
    another mode, type or layout, or elsewhere than the current GPU, does not reach the library
    (a stand-in here, with host memory as its current device)."""
    calls = []

    class Library:
        def pa_status_string(self, status):
            return b"refused"

        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or 0

    monkeypatch.setattr(pa, "_lib", Library())
    here = [-1]  # get_device() of a CPU tensor
    i32, i64, f32 = (torch.int32,), (torch.int64,), (torch.float32,)
    kinds = {pa.BF16: (torch.bfloat16,), pa.FP16: (torch.float16,), pa.FP8_E4M3: (torch.uint8, torch.float8_e4m3fn)}
    monkeypatch.setattr(pa, "_type_cache", (lambda: here[0], i32, i64, f32, kinds))
    cfg = config(2, 1, 8, 2, 128, 16, 8, 32, num_ctas=4)
    cfg.kv_scale_mode = mode
    new, q = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    cache, bt, lens = torch.zeros(32, 16, 2, 128, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    run = dict(
        append=lambda ks, vs: pa.append_kv(cfg, new, new, bt, lens, lens, cache, cache, ks, vs, lens, stream=0),
        decode=lambda ks, vs: pa.decode(cfg, q, cache, cache, ks, vs, bt, lens, lens, q, None, ws, stream=0),
        static=lambda ks, vs: pa.decode_step_static(cfg, q, cache, cache, ks, vs, bt, lens, lens, q, None, stream=0))
    good = torch.ones(count)
    bad = [None, torch.ones(count - 1), good.half(), torch.ones(count, 2)[:, 0] if count > 1 else good.double(), good.int()]
    for name, call in run.items():
        for s in (good, torch.ones(count + 5), 1 << 20):
            call(s, s)
            assert len(calls) == 1 and (s if isinstance(s, int) else s.data_ptr()) in calls.pop()[1], name
        for s in bad:
            for pair in ((s, good), (good, s)):
                with pytest.raises(pa.PaError) as e:
                    call(*pair)
                assert e.value.status == pa.ERR_INVALID_ARG and not calls, (name, s)
        here[0] = 0  # the arrays lie elsewhere than the current device
        with pytest.raises(pa.PaError):
            call(good, good)
        here[0] = -1
    for k, x in ((1, new[:1]), (2, new.half()), (3, bt[:1]), (4, lens.long()), (5, lens[:1]), (6, cache[1:]), (7, cache.int()),
                 (10, lens[:0])):
        args = [cfg, new, new, bt, lens, lens, cache, cache, good, good, lens]
        args[k] = x
        with pytest.raises(pa.PaError) as e:
            pa.append_kv(*args, stream=0)
        assert e.value.status == pa.ERR_INVALID_ARG and not calls, k
    cfg.kv_scale_mode = pa.SCALE_NONE  # whatever is given is not passed on
    run["append"](None, None)
    run["decode"](good, None)
    assert [c[1][8:10] if c[0] == "pa_append_kv" else c[1][4:6] for c in calls] == [(None, None)] * 2
