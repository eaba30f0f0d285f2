"""pa_decode_selected against 64 bits over the listed pages, for every cache, head grouping and
split; lists in any order, with repeats, empty, and of pages that a row does not see; flags,
refusals, equal bits on equal calls; and the whole step: append, bounds, score, select, attend."""
import ctypes
import os

import numpy as np
import pytest
import torch

import paged_kv_cache_work_gb300 as pa
import plain64

KINDS = {"bf16": (torch.bfloat16, pa.BF16), "fp16": (torch.float16, pa.FP16)}
MODES = {"none": 0, "tensor": 1, "token": 2, "block": 3}


def config(B, sq, hq, hkv, d, bs, maxb, nblocks, dtype="bf16", kv="16", mode="none", causal=0):
    return pa.PaConfig(batch=B, max_q_len=sq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                       max_blocks_per_seq=maxb, num_blocks=nblocks, q_dtype=KINDS[dtype][1],
                       kv_dtype=KINDS[dtype][1] if kv == "16" else pa.FP8_E4M3, kv_scale_mode=MODES[mode],
                       causal=causal, sm_scale=d ** -0.5)


def problem(seed, B, sq, hq, hkv, d, bs, longest, top_k, causal, dtype="bf16", kv="16", mode="none", spread=2):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, longest + 1, B)
    ctx[0] = longest
    ql = np.minimum(ctx, rng.integers(0, sq + 1, B))
    ql[0] = min(sq, longest)
    need = [plain64.pages(n, bs) for n in ctx]
    nblocks, maxb = sum(need) + 2, max(1, max(need))
    ids, at = rng.permutation(nblocks), 0
    bt = np.full((B, maxb), -1, np.int32)
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    shape = (nblocks, bs, hkv, d)
    ks = vs = None
    if kv == "16":
        kc, vc = (torch.from_numpy(rng.standard_normal(shape)).to(KINDS[dtype][0]) for _ in "kv")
        for b in range(B):  # what lies behind a sequence's last token may hold anything
            if ctx[b] % bs:
                kc[bt[b, need[b] - 1], ctx[b] % bs:] = float("nan")
                vc[bt[b, need[b] - 1], ctx[b] % bs:] = float("inf")
    else:
        def codes():
            x = torch.from_numpy(rng.standard_normal(shape) * 60).clamp(-448, 448)
            return x.to(torch.float8_e4m3fn).view(torch.uint8)
        kc, vc = codes(), codes()
        size = {"tensor": (1,), "token": shape[:3], "block": (nblocks, hkv)}.get(mode)
        if size:
            ks = torch.from_numpy((0.02 * 2.0 ** rng.uniform(-1, 1, size)).astype(np.float32))
            vs = torch.from_numpy((0.02 * 2.0 ** rng.uniform(-spread, spread, size)).astype(np.float32))
        else:
            kc, vc = (torch.where((c & 127) > 0x40, c & 0xbf, c) for c in (kc, vc))
    q = torch.from_numpy(rng.standard_normal((B, sq, hq, d))).to(KINDS[dtype][0])
    sel = np.full((B, sq, hkv, top_k), -1, np.int32)
    num = np.zeros((B, sq, hkv), np.int32)
    for b in range(B):
        for i in range(ql[b]):
            for g in range(hkv):
                k = min(top_k, need[b])
                sel[b, i, g, :k] = rng.permutation(need[b])[:k]  # any order, pages not seen among them
                num[b, i, g] = rng.integers(0, k + 1) if rng.random() < 0.3 else k
    return dict(ctx=ctx, ql=ql, bt=bt, nblocks=nblocks, maxb=maxb, kc=kc, ks=ks, vc=vc, vs=vs, q=q, sel=sel, num=num)


def reference(p, causal, d, mode, lists=None):
    k, v = plain64.values(p["kc"], p["ks"], mode), plain64.values(p["vc"], p["vs"], mode)
    lists = lists or (lambda b, i, g: p["sel"][b, i, g, :p["num"][b, i, g]])
    return plain64.attend(p["q"], k, v, p["bt"], lists, p["ctx"].tolist(), p["ql"].tolist(), causal,
                          float(np.float32(d ** -0.5)))


def run(p, cfg, dev, want_flags=0, lse=True):
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    g = lambda x: None if x is None else x.to(dev)  # noqa: E731
    q, flags = p["q"].to(dev), t([0])
    out = torch.full_like(q, float("nan"))
    ls = torch.full(q.shape[:3], float("nan"), device=dev) if lse else None
    pa.decode_selected(cfg, q, g(p["kc"]), g(p["vc"]), g(p["ks"]), g(p["vs"]), t(p["bt"]), t(p["ctx"]), t(p["ql"]),
                       t(p["sel"]), t(p["num"]), out, ls, flags)
    assert int(flags.item()) == want_flags
    return out, ls


CASES = [
    # B, Sq, Hq, Hkv, D, bs, longest, top_k, causal, dtype, kv, mode
    (3, 1, 4, 1, 128, 16, 700, 12, 0, "bf16", "16", "none"), (2, 3, 16, 2, 128, 64, 900, 6, 1, "fp16", "16", "none"),
    (2, 2, 10, 2, 64, 16, 500, 40, 1, "bf16", "16", "none"), (2, 2, 5, 1, 256, 32, 400, 9, 1, "bf16", "16", "none"),
    (1, 1, 24, 1, 128, 16, 300, 30, 0, "bf16", "16", "none"), (1, 2, 80, 2, 64, 16, 200, 9, 1, "fp16", "16", "none"),
    (1, 1, 1, 1, 128, 16, 1, 1, 0, "bf16", "16", "none"), (2, 70, 3, 3, 128, 16, 150, 5, 1, "bf16", "16", "none"),
    (1, 1, 8, 1, 256, 1024, 5000, 4, 0, "fp16", "16", "none"), (1, 2, 16, 1, 64, 512, 9000, 20, 1, "bf16", "16", "none"),
    (3, 1, 4, 1, 128, 16, 700, 12, 0, "bf16", "8", "block"), (2, 3, 16, 2, 128, 64, 900, 6, 1, "fp16", "8", "block"),
    (2, 2, 10, 2, 64, 16, 500, 40, 1, "bf16", "8", "block"), (2, 2, 5, 1, 256, 32, 400, 9, 1, "bf16", "8", "token"),
    (1, 1, 24, 1, 128, 16, 300, 30, 0, "bf16", "8", "token"), (1, 2, 80, 2, 64, 16, 200, 9, 1, "fp16", "8", "token"),
    (2, 1, 8, 2, 128, 128, 2000, 8, 1, "bf16", "8", "tensor"), (2, 1, 8, 2, 64, 16, 300, 8, 1, "fp16", "8", "none"),
    (1, 2, 16, 1, 128, 1024, 9000, 9, 1, "bf16", "8", "block"), (2, 1, 8, 2, 256, 16, 900, 50, 0, "fp16", "8", "block"),
    (1, 1, 16, 1, 128, 16, 6000, 375, 0, "bf16", "16", "none"), (1, 1, 16, 1, 128, 16, 6001, 400, 0, "bf16", "8", "block"),
]


# Weights are rounded to the MMA's operand type: bf16 for a bf16 cache (half a step: 2^-8), f16 for
# fp16 and fp8 caches (2^-11).
def rounding(kv, dtype):
    return dict(weight_eps=2.0 ** -8 if kv == "16" and dtype == "bf16" else 2.0 ** -11)


@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,hq,hkv,d,bs,longest,top_k,causal,dtype,kv,mode", CASES)
def test_matches_64_bits(B, sq, hq, hkv, d, bs, longest, top_k, causal, dtype, kv, mode, cuda_device, pa):
    p = problem(7, B, sq, hq, hkv, d, bs, longest, top_k, causal, dtype, kv, mode)
    cfg = config(B, sq, hq, hkv, d, bs, p["maxb"], p["nblocks"], dtype, kv, mode, causal)
    out, lse = run(p, cfg, cuda_device)
    ref, ref_lse, size = reference(p, causal, d, mode)
    plain64.check_attention(out, lse, ref, ref_lse, size, p["q"].dtype, **rounding(kv, dtype))
    again, lse2 = run(p, cfg, cuda_device)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    alone, _ = run(p, cfg, cuda_device, lse=False)
    assert torch.equal(out.view(torch.int16), alone.view(torch.int16))


@pytest.mark.gpu
def test_all_pages_are_the_dense_decode(cuda_device, pa):
    p = problem(9, 3, 2, 8, 2, 128, 16, 600, 40, 1)
    for b in range(3):
        n = plain64.pages(p["ctx"][b], 16)
        p["sel"][b, :, :, :n] = np.arange(n)
        p["num"][b] = n
    cfg = config(3, 2, 8, 2, 128, 16, p["maxb"], p["nblocks"], causal=1)
    out, lse = run(p, cfg, cuda_device)
    ref, ref_lse, size = reference(p, 1, 128, "none")
    plain64.check_attention(out, lse, ref, ref_lse, size, torch.bfloat16, 2.0 ** -8)
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=cuda_device)  # noqa: E731
    q = p["q"].to(cuda_device)
    dense, dlse = torch.empty_like(q), torch.empty(q.shape[:3], device=cuda_device)
    ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=cuda_device)
    args = t(p["bt"]), t(p["ctx"]), t(p["ql"])
    pa.plan(cfg, *args, ws)
    pa.decode(cfg, q, p["kc"].to(cuda_device), p["vc"].to(cuda_device), None, None, *args, dense, dlse, ws)
    pa.reduce(cfg, dense, dlse, ws)
    fin = torch.isfinite(dlse)
    assert torch.equal(fin, torch.isfinite(lse)) and torch.allclose(lse[fin], dlse[fin], rtol=1e-5, atol=1e-5)
    assert torch.allclose(out.float(), dense.float(), rtol=2.0 ** -7, atol=2.0 ** -7)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,mode", [("16", "none"), ("8", "block")])
def test_odd_lists(kv, mode, cuda_device, pa):
    """A page listed twice counts twice; counts and pages that cannot be are clamped, skipped and
    flagged; so are bad blocks and lengths."""
    p = problem(3, 4, 2, 8, 2, 128, 16, 400, 10, 1, kv=kv, mode=mode)
    p["ctx"][2], p["ql"][2] = 3, 2  # (its lists were drawn for more pages: those are skipped)
    cfg = config(4, 2, 8, 2, 128, 16, p["maxb"], p["nblocks"], kv=kv, mode=mode, causal=1)
    p["sel"][0, 0, 0, :4] = (1, 1, 0, 1)
    p["num"][0, 0, 0] = 4

    def within(b, i, g):
        x = [int(v) for v in p["sel"][b, i, g, :max(0, min(10, p["num"][b, i, g]))]]
        return [v for v in x if 0 <= v < plain64.pages(p["ctx"][b], 16)]

    out, lse = run(p, cfg, cuda_device, pa.FLAG_BAD_SELECTION)
    ref, ref_lse, size = reference(p, 1, 128, mode, within)
    tol = rounding(kv, "bf16")
    plain64.check_attention(out, lse, ref, ref_lse, size, torch.bfloat16, **tol)

    pages = plain64.pages(p["ctx"][0], 16)
    p["num"][0, 1, 0], p["num"][0, 1, 1] = 11, -3
    p["sel"][0, 1, 0, 9] = 2
    p["sel"][0, 0, 1, :3] = (pages, -1, 3)
    p["num"][0, 0, 1] = 3
    bad = dict(p, bt=p["bt"].copy(), ctx=p["ctx"].copy())
    bad["bt"][0, 5] = p["nblocks"]
    bad["ctx"][2] = 1

    def lists(b, i, g):
        return [] if b == 2 else [v for v in within(b, i, g) if not (b == 0 and v == 5)]

    listed = any(5 in within(0, i, g) for i in range(2) for g in range(2))  # (the bad block's page)
    assert listed or kv == "8"
    out, lse = run(bad, cfg, cuda_device, pa.FLAG_BAD_SELECTION | pa.FLAG_BAD_LENGTHS | (pa.FLAG_BAD_BLOCK_ID if listed else 0))
    ref, ref_lse, size = reference(p, 1, 128, mode, lists)
    plain64.check_attention(out, lse, ref, ref_lse, size, torch.bfloat16, **tol)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,mode", [("16", "none"), ("8", "none"), ("8", "tensor"), ("8", "token"), ("8", "block")])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32), (256, 16)])
def test_a_listed_bad_block_is_skipped(d, bs, kv, mode, cuda_device, pa):
    """A listed page whose block lies outside the pool, alone in its list, first, last and between
    others: flagged and left out, and no other row changes a bit."""
    p = problem(17, 2, 2, 8, 2, d, bs, 400, 12, 1, kv=kv, mode=mode)
    p["ctx"][:], p["ql"][:] = 400, 2
    p["bt"] = np.random.default_rng(18).integers(0, p["nblocks"], (2, plain64.pages(400, bs)))
    p["maxb"] = p["bt"].shape[1]
    if kv == "16":
        for c in (p["kc"], p["vc"]):
            c[~torch.isfinite(c)] = 0.5
    bad = 5
    p["sel"][:] = -1
    for g, row in enumerate(([bad], [bad, 2, 7, 1], [3, 8, 6, bad], [0, 4, bad, 9, 3])):
        p["sel"][0, g // 2, g % 2, :len(row)] = row
        p["num"][0, g // 2, g % 2] = len(row)
    p["sel"][1, :, :, :3], p["num"][1] = (1, 2, 3), 3
    cfg = config(2, 2, 8, 2, d, bs, p["maxb"], p["nblocks"], kv=kv, mode=mode, causal=1)
    good, _ = run(p, cfg, cuda_device)
    lists = lambda b, i, g: [x for x in p["sel"][b, i, g, :p["num"][b, i, g]] if b or x != bad]  # noqa: E731
    ref, ref_lse, size = reference(p, 1, d, mode, lists)
    for block in (-1, p["nblocks"], 1 << 30):
        spoilt = dict(p, bt=p["bt"].copy())
        spoilt["bt"][0, bad] = block
        out, lse = run(spoilt, cfg, cuda_device, pa.FLAG_BAD_BLOCK_ID)
        plain64.check_attention(out, lse, ref, ref_lse, size, torch.bfloat16, **rounding(kv, "bf16"))
        assert torch.equal(out[1], good[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_ranges_that_leave_f16(d, cuda_device, pa):
    """Queries of 1e6 or 1e-6 with keys that make up for it, V scales of 1e-7 and 1e6, and scales
    that differ by 2^12 between pages: as exact as any other."""
    for factor, spread in ((1e6, 1), (1e-6, 12)):
        p = problem(5, 2, 1, 8, 2, d, 16, 400, 20, 0, kv="8", mode="block", spread=spread)
        p["q"] = (p["q"].float() * factor).bfloat16()
        p["ks"] = p["ks"] / factor
        p["vs"] = p["vs"] * factor
        cfg = config(2, 1, 8, 2, d, 16, p["maxb"], p["nblocks"], kv="8", mode="block")
        out, lse = run(p, cfg, cuda_device)
        ref, ref_lse, size = reference(p, 0, d, "block")
        plain64.check_attention(out.double().cpu() / factor, lse, ref / factor, ref_lse, size / factor, torch.bfloat16,
                                **rounding("8", "bf16"))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["zeros", "low"])
@pytest.mark.parametrize("d,bs,mode,dtype", [(128, 16, "block", "bf16"), (64, 64, "block", "fp16"), (64, 16, "block", "bf16"),
                                             (256, 16, "block", "bf16"), (128, 32, "token", "fp16"), (256, 16, "token", "bf16")])
def test_far_larger_scales_cost_the_others_nothing(d, bs, mode, dtype, kind, cuda_device, pa):
    """Half of the pages (or tokens) get a V scale 1 / ratio times the others' and no part in the
    output, as they hold zeros or keys whose logits lie far below every other: the others keep
    their weights' bits."""
    for ratio in (1e-5, 1e-7, 1e-9, 1e-14):
        p = problem(15, 2, 2, 8, 2, d, bs, 400, 20, 0, dtype, "8", mode, 1)
        rng = np.random.default_rng(16)
        far = torch.from_numpy(rng.random(p["vs"].shape[:1] if mode == "block" else p["vs"].shape[:2]) < 0.5)
        p["vs"][far] /= ratio
        if kind == "zeros":
            p["vc"][far] = 0
        else:  # keys of -448 * 0.04 in every channel against queries above zero: logits below -80
            p["q"] = p["q"].abs()
            p["kc"][far] = 0xfe
            p["ks"][far] = 0.04
            for b in range(2):  # (a row that sees far keys alone would be theirs: list some of the others)
                p["sel"][b, :, :, 0] = next(x for x in range(p["maxb"]) if not far[p["bt"][b, x]].all())
        cfg = config(2, 2, 8, 2, d, bs, p["maxb"], p["nblocks"], dtype, "8", mode)
        out, lse = run(p, cfg, cuda_device)
        ref, ref_lse, size = reference(p, 0, d, mode)
        plain64.check_attention(out, lse, ref, ref_lse, size, p["q"].dtype, **rounding("8", dtype))


@pytest.mark.gpu
def test_a_cache_past_32_bits_of_elements(cuda_device, pa):
    """Pages beyond element 2^31 of the cache (and of the fp8 one's bytes)."""
    B, hq, hkv, d, bs = 1, 4, 2, 128, 1024
    nblocks = (1 << 31) // (bs * hkv * d) + 40
    for kv, mode in (("16", "none"), ("8", "block")):
        small = problem(6, B, 1, hq, hkv, d, bs, 4 * bs - 5, 4, 0, kv=kv, mode=mode)
        kind = torch.bfloat16 if kv == "16" else torch.uint8
        at = [int(x) for x in small["bt"][0]]
        far = [nblocks - 1, 3, nblocks - 30, nblocks - 7]
        kc = torch.zeros(nblocks, bs, hkv, d, dtype=kind, device=cuda_device)
        vc = torch.zeros(nblocks, bs, hkv, d, dtype=kind, device=cuda_device)
        ks = vs = None
        if mode == "block":
            ks, vs = (torch.ones(nblocks, hkv, device=cuda_device) for _ in "kv")
        for x, y in zip(at, far):
            kc[y], vc[y] = small["kc"][x].to(cuda_device), small["vc"][x].to(cuda_device)
            if ks is not None:
                ks[y], vs[y] = small["ks"][x].to(cuda_device), small["vs"][x].to(cuda_device)
        cfg = config(B, 1, hq, hkv, d, bs, 4, nblocks, kv=kv, mode=mode)
        out, lse = run(dict(small, kc=kc, vc=vc, ks=ks, vs=vs, bt=np.array([far])), cfg, cuda_device)
        ref, ref_lse, size = reference(small, 0, d, mode)
        plain64.check_attention(out, lse, ref, ref_lse, size, torch.bfloat16, **rounding(kv, "bf16"))
        del kc, vc
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["16", "8"])
def test_a_whole_sparse_step(kv, cuda_device, pa):
    """Table growth, append, bounds, score, select and attention of a few steps, captured on a
    stream of their own and replayed: each step attends over the best pages by the plain rule."""
    dev, rng = cuda_device, np.random.default_rng(8)
    B, sq, hq, hkv, d, bs, top_k, steps = 3, 2, 8, 2, 128, 16, 6, 12
    mode = "none" if kv == "16" else "block"
    maxb, nblocks = 16, 60
    cfg = config(B, sq, hq, hkv, d, bs, maxb, nblocks, kv=kv, mode=mode, causal=1)
    i32 = dict(dtype=torch.int32, device=dev)
    t = lambda x: torch.tensor(x, **i32)  # noqa: E731
    kind = torch.bfloat16 if kv == "16" else torch.uint8
    z = dict(n=t([0] * B), q=t([0] * B), held=t([0] * B), new_held=t([0] * B), count=t([nblocks]), new_count=t([0]),
             bt=torch.full((B, maxb), -1, **i32), free=torch.randperm(nblocks).to(**i32),
             slots=torch.empty(B, sq, dtype=torch.int64, device=dev),
             kc=torch.zeros(nblocks, bs, hkv, d, dtype=kind, device=dev), bounds=torch.zeros(nblocks, hkv, 2, d, dtype=torch.bfloat16, device=dev),
             qx=torch.zeros(B, sq, hq, d, dtype=torch.bfloat16, device=dev), scores=torch.empty(B, sq, hkv, maxb, device=dev),
             sel=torch.empty(B, sq, hkv, top_k, **i32), num=torch.empty(B, sq, hkv, **i32),
             lse=torch.empty(B, sq, hq, device=dev), flags=t([0]))
    z["vc"], z["out"] = torch.zeros_like(z["kc"]), torch.empty_like(z["qx"])
    z["kn"] = torch.zeros(B, sq, hkv, d, dtype=torch.bfloat16, device=dev)
    z["vn"] = torch.zeros_like(z["kn"])
    z["ks"] = z["vs"] = None
    if mode == "block":
        z["ks"], z["vs"] = torch.ones(nblocks, hkv, device=dev), torch.ones(nblocks, hkv, device=dev)

    def step():
        f = z["flags"]
        pa.build_tables(cfg, z["n"], z["q"], z["held"], z["bt"], z["free"], z["count"], z["new_held"], z["new_count"], z["slots"], f)
        pa.append_kv(cfg, z["kn"], z["vn"], z["bt"], z["n"], z["q"], z["kc"], z["vc"], z["ks"], z["vs"], f)
        pa.update_bounds(cfg, z["kn"], z["bt"], z["n"], z["q"], z["bounds"], f)
        pa.score_blocks(cfg, z["qx"], z["bounds"], z["bt"], z["n"], z["q"], z["scores"], f)
        pa.select_blocks(cfg, z["scores"], z["n"], z["q"], 1, 1, z["sel"], z["num"], f)
        pa.decode_selected(cfg, z["qx"], z["kc"], z["vc"], z["ks"], z["vs"], z["bt"], z["n"], z["q"], z["sel"], z["num"],
                           z["out"], z["lse"], f)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    n = np.array([0, 0, 0])
    with torch.cuda.stream(stream):
        step()  # (empty sequences: sets the kernels up)
        stream.synchronize()
        assert (z["out"] == 0).all() and torch.isinf(z["lse"]).all()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
        # the prompts come in one call of their own
        long = 150
        prompt = rng.integers(20, long, B)
        big = config(B, long, hq, hkv, d, bs, maxb, nblocks, kv=kv, mode=mode, causal=1)
        kp, vp = (torch.from_numpy(rng.standard_normal((B, long, hkv, d))).bfloat16().to(dev) for _ in "kv")
        z["n"].copy_(t(prompt.tolist()))
        pa.build_tables(big, z["n"], z["n"], z["held"], z["bt"], z["free"], z["count"], z["new_held"], z["new_count"], None, z["flags"])
        pa.append_kv(big, kp, vp, z["bt"], z["n"], z["n"], z["kc"], z["vc"], z["ks"], z["vs"], z["flags"])
        pa.update_bounds(big, kp, z["bt"], z["n"], z["n"], z["bounds"], z["flags"])
        n = prompt
        for j in range(steps):
            z["held"].copy_(z["new_held"])
            z["count"].copy_(z["new_count"])
            q = rng.integers(0 if j else 1, sq + 1, B)
            n = n + q
            z["n"].copy_(t(n.tolist()))
            z["q"].copy_(t(q.tolist()))
            for k in ("kn", "vn", "qx"):
                z[k].copy_(torch.from_numpy(rng.standard_normal(tuple(z[k].shape))))
            g.replay()
            stream.synchronize()
            assert int(z["flags"].item()) == 0
            scores, sel, num = z["scores"].cpu().numpy(), z["sel"].cpu().numpy(), z["num"].cpu().numpy()
            bt = z["bt"].cpu().numpy()
            want, size = plain64.score(z["qx"].cpu(), z["bounds"].cpu(), n, q, bt, bs, 1, float(np.float32(d ** -0.5)), hkv, nblocks)
            fin = np.isfinite(want)
            assert np.array_equal(fin, np.isfinite(scores))
            assert (np.abs(scores[fin] - want[fin]) <= (2 * d + 1) * 2.0 ** -23 * size[fin]).all()
            wsel, wnum = plain64.select(scores, n.tolist(), q.tolist(), bs, 1, top_k, 1, 1)
            assert np.array_equal(sel, wsel) and np.array_equal(num, wnum)
            p = dict(q=z["qx"].cpu(), kc=z["kc"].cpu(), vc=z["vc"].cpu(), ks=z["ks"], vs=z["vs"], sel=sel, num=num, bt=bt, ctx=n, ql=q)
            if mode == "block":
                p["ks"], p["vs"] = z["ks"].cpu(), z["vs"].cpu()
            ref, ref_lse, size = reference(p, 1, d, mode)
            plain64.check_attention(z["out"], z["lse"], ref, ref_lse, size, torch.bfloat16, **rounding(kv, "bf16"))
    torch.cuda.current_stream().wait_stream(stream)


# ---- refusals -----------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_cache_work_gb300.build import build
        build()
    return pa.load()


def test_refused_on_the_host(lib):
    fake = 1 << 20  # never dereferenced: every call below is rejected on the host
    good = dict(B=2, sq=1, hq=8, hkv=2, d=128, bs=16, maxb=8, nblocks=32)

    def call(c=None, **kw):
        a = dict(q=fake, kc=fake, vc=fake, ks=None, vs=None, bt=fake, ctx=fake, ql=fake, sel=fake, num=fake, top_k=4,
                 out=fake, lse=None, flags=None)
        a.update(kw)
        return lib.pa_decode_selected(ctypes.byref(c or config(**good)), *a.values(), None)

    for k in ("q", "kc", "vc", "bt", "ctx", "ql", "sel", "num", "out"):
        assert call(**{k: None}) == pa.ERR_INVALID_ARG, k
        assert call(**{k: fake + (8 if k in ("q", "kc", "vc", "out") else 2)}) == pa.ERR_INVALID_ARG, k
    for kw in (dict(top_k=0), dict(top_k=-1), dict(lse=fake + 2), dict(flags=fake + 2)):
        assert call(**kw) == pa.ERR_INVALID_ARG, kw
    for kw, want in ((dict(d=96), pa.ERR_UNSUPPORTED), (dict(bs=8), pa.ERR_UNSUPPORTED), (dict(hq=9), pa.ERR_UNSUPPORTED),
                     (dict(B=0), pa.ERR_INVALID_ARG), (dict(kv="16", mode="block"), pa.ERR_UNSUPPORTED),
                     (dict(maxb=1 << 28), pa.ERR_UNSUPPORTED), (dict(B=1 << 20, sq=1 << 10), pa.ERR_UNSUPPORTED)):
        assert call(config(**{**good, **kw})) == want, kw
    assert call(top_k=1 << 27) == pa.ERR_UNSUPPORTED  # a list of 2^31 tokens
    for mode in ("tensor", "token", "block"):
        c = config(**good, kv="8", mode=mode)
        assert call(c) == pa.ERR_INVALID_ARG
        assert call(c, ks=fake) == pa.ERR_INVALID_ARG
        assert call(c, ks=fake, vs=fake + 2) == pa.ERR_INVALID_ARG
    assert lib.pa_decode_selected(None, *([fake] * 3), None, None, *([fake] * 5), 4, fake, None, None, None) == pa.ERR_INVALID_ARG


@pytest.mark.gpu
def test_binding_refuses_tensors_that_do_not_fit(cuda_device, pa):
    p = problem(1, 2, 1, 8, 2, 128, 16, 100, 4, 0)
    cfg = config(2, 1, 8, 2, 128, 16, p["maxb"], p["nblocks"])
    dev = cuda_device
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    good = dict(q=p["q"].to(dev), kc=p["kc"].to(dev), vc=p["vc"].to(dev), ks=None, vs=None, bt=t(p["bt"]), ctx=t(p["ctx"]),
                ql=t(p["ql"]), sel=t(p["sel"]), num=t(p["num"]), out=p["q"].to(dev))
    bad = [("q", p["q"]), ("q", good["q"].float()), ("q", good["q"].repeat(1, 1, 1, 2)[..., ::2]), ("kc", good["kc"][1:]),
           ("kc", good["kc"].half()), ("bt", good["bt"].long()), ("ctx", good["ctx"][:1]), ("sel", good["sel"][:1]),
           ("num", good["num"].flatten()[:3]), ("out", good["out"][:1]), ("vc", None), ("sel", None), ("sel", 1 << 20)]
    for k, x in bad:
        with pytest.raises(pa.PaError) as e:
            pa.decode_selected(cfg, *{**good, k: x}.values())
        assert e.value.status == pa.ERR_INVALID_ARG, k
