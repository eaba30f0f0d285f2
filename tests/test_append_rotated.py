"""pa_append_rotated against 64 bits: norms, rotations of every layout, axes, strides, caches; equality
with the separate append where the two define the same rounding; flags, refusals, graphs."""
import ctypes
import os

import numpy as np
import pytest
import torch

import paged_kv_cache_work_gb300 as pa
import plain64
import plain_int4 as plain

KINDS = {"bf16": (torch.bfloat16, pa.BF16), "fp16": (torch.float16, pa.FP16)}
CACHES = {"16": (None, pa.SCALE_NONE), "8none": (pa.FP8_E4M3, pa.SCALE_NONE), "8tensor": (pa.FP8_E4M3, pa.SCALE_PER_TENSOR),
          "8token": (pa.FP8_E4M3, pa.SCALE_PER_TOKEN), "4": (pa.INT4, pa.SCALE_AFFINE)}


def config(B, sq, hq, hkv, d, bs, maxb, nblocks, dtype="bf16", kv="16", **kw):
    kind, mode = CACHES[kv]
    return pa.PaConfig(batch=B, max_q_len=sq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
                       max_blocks_per_seq=maxb, num_blocks=nblocks, q_dtype=KINDS[dtype][1],
                       kv_dtype=KINDS[dtype][1] if kind is None else kind, kv_scale_mode=mode, sm_scale=d ** -0.5, **kw)


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def angles(rows, rd):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rd, 2) / rd)
    return torch.from_numpy(np.concatenate((np.cos(a), np.sin(a)), 1)).float()


class Problem:
    def __init__(self, seed, B, sq, hq, hkv, d, bs, dtype, kv, rd, axes, interleaved, norm, fused):
        rng = np.random.default_rng(seed)
        t = KINDS[dtype][0]
        self.__dict__.update(B=B, sq=sq, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype, kv=kv, rd=rd, interleaved=interleaved, t=t)
        self.ql = rng.integers(0, sq + 1, B)
        self.ql[0] = sq
        self.ctx = self.ql + rng.integers(0, 3 * bs, B)
        self.bt, self.nblocks = plain.tables(rng, self.ctx, bs)
        qkv = torch.from_numpy(rng.standard_normal((B, sq, hq + 2 * hkv, d)) * rng.choice([0.1, 1, 4], (B, sq, 1, 1))).to(t)
        self.fused, self.qkv = fused, qkv
        self.q, self.k, self.v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        self.wq = torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(t) if norm in ("both", "q") else None
        self.wk = torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(t) if norm in ("both", "k") else None
        rows = int(self.ctx.max()) + 1
        self.cs = angles(rows, rd) if rd else None
        half = rd // 2
        self.axis_pairs = {1: [half], 2: [half // 4, half - half // 4], 3: [half - 2 * (half // 3), half // 3, half // 3]}[axes]
        self.pos = None if axes == 1 else torch.from_numpy(rng.integers(0, rows, (axes, B, sq)).astype(np.int32))
        shape = (self.nblocks, bs, hkv, d)
        if kv == "16":
            make = lambda: torch.from_numpy(rng.standard_normal(shape)).to(t)  # noqa: E731
        elif kv == "4":
            make = lambda: torch.from_numpy(rng.integers(0, 256, (*shape[:3], d // 2)).astype(np.uint8))  # noqa: E731
        else:
            make = lambda: torch.from_numpy(rng.integers(0, 0x78, shape).astype(np.uint8))  # noqa: E731
        self.kc, self.vc = make(), make()
        self.ks = self.vs = None
        if kv == "8tensor":
            self.ks, self.vs = torch.tensor([0.03]), torch.tensor([0.02])
        elif kv == "8token":
            self.ks, self.vs = torch.ones(shape[:3]), torch.ones(shape[:3])
        elif kv == "4":
            self.ks, self.vs = torch.ones(shape[0], hkv, bs, 2, dtype=t), torch.ones(shape[0], hkv, bs, 2, dtype=t)
        self.cfg = config(B, sq, hq, hkv, d, bs, self.bt.shape[1], self.nblocks, dtype, kv)

    def on(self, dev):
        g = lambda x: None if x is None else x.to(dev)  # noqa: E731
        if self.fused:
            qkv = self.qkv.to(dev)
            q, k, v = qkv[:, :, :self.hq], qkv[:, :, self.hq:self.hq + self.hkv], qkv[:, :, self.hq + self.hkv:]
        else:
            q, k, v = (x.contiguous().to(dev) for x in (self.q, self.k, self.v))
        self.dev = dict(q=q, k=k, v=v, bt=ints(self.bt, dev), ctx=ints(self.ctx, dev), ql=ints(self.ql, dev),
                        qo=torch.full((self.B, self.sq, self.hq, self.d), 5.0, dtype=self.t, device=dev),
                        ko=torch.full((self.B, self.sq, self.hkv, self.d), 5.0, dtype=self.t, device=dev),
                        kc=g(self.kc), vc=g(self.vc), ks=g(self.ks), vs=g(self.vs), flags=ints([0], dev),
                        kw=dict(cos_sin=g(self.cs), interleaved=self.interleaved, positions=g(self.pos),
                                axis_pairs=self.axis_pairs if self.cs is not None else None, q_weight=g(self.wq),
                                k_weight=g(self.wk), eps=1e-5))
        return self.dev

    def call(self, dev, k_out=True):
        x = self.on(dev)
        pa.append_rotated(self.cfg, x["q"], x["k"], x["v"], x["bt"], x["ctx"], x["ql"], x["qo"], x["kc"], x["vc"],
                          x["ks"], x["vs"], k_out=x["ko"] if k_out else None, flags=x["flags"], **x["kw"])
        return x

    def rotated(self, b, i):
        """The token's q and k heads in 64 bits."""
        pos = [self.ctx[b] - self.ql[b] + i] * 3 if self.pos is None else self.pos[:, b, i].tolist()
        cs = None if self.cs is None else self.cs.double().numpy()
        f = lambda x, w: plain.rotate(x.double().numpy(), None if w is None else w.double().numpy(),  # noqa: E731
                                      float(np.float32(1e-5)), cs, pos, self.axis_pairs, self.interleaved)
        return f(self.q[b, i], self.wq), f(self.k[b, i], self.wk)


# fp32: a sum of D squares, a root, a division, two products and the rotation's three operations, each
# off by at most 2^-24 of the magnitudes that enter it, come to less than 16 of them for a rotated pair
FP32 = 16 * 2.0 ** -24


def off(got, want, pair_size, t):
    """Within half a step of the type t of an fp32 value."""
    half = torch.finfo(t).eps / 2
    tol = half * np.abs(want) + FP32 * pair_size * 1.01 + torch.finfo(t).smallest_normal * half
    return np.abs(got - want) <= tol * (1 + 2.0 ** -9)


def sizes(x, rd, interleaved):
    """Magnitude of the pair that each channel of [H, D] belongs to."""
    s = np.abs(x).copy()
    half = rd // 2
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        s[:, i] = s[:, j] = np.abs(x[:, i]) + np.abs(x[:, j])
    return s


CASES = [
    # B, Sq, Hq, Hkv, D, bs, dtype, cache, rotary_dim, axes, interleaved, norm, fused
    (3, 1, 8, 2, 128, 16, "bf16", "16", 128, 1, False, "both", True), (2, 5, 4, 4, 64, 16, "fp16", "16", 64, 1, True, "both", False),
    (2, 3, 3, 1, 256, 32, "bf16", "16", 256, 3, False, "both", True), (1, 40, 2, 1, 128, 64, "bf16", "16", 32, 1, False, None, True),
    (2, 4, 6, 3, 64, 128, "bf16", "16", 16, 1, False, "k", False), (2, 4, 5, 1, 256, 16, "fp16", "16", 64, 3, True, "q", True),
    (2, 2, 4, 2, 128, 16, "fp16", "16", 0, 1, False, "both", False), (2, 6, 4, 2, 128, 16, "bf16", "16", 96, 2, False, None, True),
    (3, 4, 8, 2, 128, 16, "bf16", "8token", 128, 1, False, "both", True), (2, 3, 4, 1, 64, 32, "fp16", "8token", 64, 1, True, None, False),
    (2, 3, 4, 1, 256, 1024, "bf16", "8tensor", 128, 1, False, "both", True), (2, 3, 4, 2, 128, 16, "bf16", "8none", 128, 3, False, "both", False),
    (3, 4, 8, 2, 128, 16, "bf16", "4", 128, 1, False, "both", True), (2, 7, 4, 1, 64, 32, "fp16", "4", 32, 1, True, "both", False),
    (2, 3, 4, 2, 256, 16, "bf16", "4", 256, 3, False, None, True), (1, 1, 1, 1, 128, 16, "bf16", "4", 128, 1, False, "both", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_matches_64_bits(case, cuda_device, pa):
    p = Problem(17, *case)
    x = p.call(cuda_device)
    assert int(x["flags"].item()) == 0
    qo, ko = x["qo"].double().cpu().numpy(), x["ko"].double().cpu().numpy()
    kc = x["kc"].cpu()
    for b in range(p.B):
        for i in range(p.sq):
            if i >= p.ql[b]:  # rows behind a sequence's last: as they were
                assert (qo[b, i] == 5).all() and (ko[b, i] == 5).all()
                continue
            zq, zk = p.rotated(b, i)
            assert off(qo[b, i], zq, sizes(zq, p.rd, p.interleaved), p.t).all()
            assert off(ko[b, i], zk, sizes(zk, p.rd, p.interleaved), p.t).all()
            pos = p.ctx[b] - p.ql[b] + i
            blk, slot = p.bt[b, pos // p.bs], pos % p.bs
            if p.kv == "16":
                assert torch.equal(kc[blk, slot], x["ko"][b, i].cpu())
                assert torch.equal(x["vc"][blk, slot].cpu(), p.v[b, i])
                continue
            # half a step of the cache's codes around the 64-bit key, and the fp32 error of the key
            for g in range(p.hkv):
                want, slack = zk[g], FP32 * sizes(zk, p.rd, p.interleaved)[g] * 1.01
                if p.kv == "4":
                    step, low = (float(f) for f in x["ks"][blk, g, slot])
                    got = plain.unpack(kc[blk, slot, g].numpy()) * step + low
                    rs, rl = plain.to_type((want.max() - low) / 15, p.t, True), plain.to_type(want.min(), p.t, False)
                    unit = torch.finfo(p.t).eps
                    assert abs(step - rs) <= unit * rs and abs(low - rl) <= unit * abs(rl)
                    assert (np.abs(got - want) <= step / 2 + slack + 2.0 ** -22 * (abs(low) + 15 * step)).all()
                else:
                    scale = {"8none": 1.0, "8tensor": 0.03}.get(p.kv) or float(x["ks"][blk, slot, g])
                    scale = float(np.float32(scale))
                    if p.kv == "8token":
                        assert abs(scale - np.abs(want).max() / 448) <= scale * 2.0 ** -20
                    got = kc[blk, slot, g].view(torch.float8_e4m3fn).double().numpy() * scale
                    clip = np.clip(want, -448 * scale, 448 * scale)
                    assert (np.abs(got - clip) <= 2.0 ** -4 * np.abs(clip) * 1.001 + scale * 2.0 ** -10 + slack).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in CASES if c[7] != "16"] + [CASES[0], CASES[3]])
def test_values_as_the_append_writes_them(case, cuda_device, pa):
    """V rows, and K rows where nothing turns or normalises them, are pa_append_kv's bit for bit; what
    no new row belongs to is left as it was."""
    case = list(case)
    case[8], case[9], case[11] = 0, 1, None
    p = Problem(23, *case)
    x = p.call(cuda_device, k_out=False)
    g = lambda t: None if t is None else t.to(cuda_device)  # noqa: E731
    kc, vc, ks, vs = g(p.kc), g(p.vc), g(p.ks), g(p.vs)
    pa.append_kv(p.cfg, p.k.contiguous().to(cuda_device), p.v.contiguous().to(cuda_device), x["bt"], x["ctx"], x["ql"],
                 kc, vc, ks, vs)
    assert torch.equal(x["kc"].view(torch.uint8), kc.view(torch.uint8))
    assert torch.equal(x["vc"].view(torch.uint8), vc.view(torch.uint8))
    if ks is not None:
        assert torch.equal(x["ks"], ks) and torch.equal(x["vs"], vs)


@pytest.mark.gpu
def test_rotates_in_place_and_without_pages(cuda_device, pa):
    """q_out and k_out may be q and k; without caches nothing else is touched; the keys then go into
    pages with one scale by pa_append_kv, whose bounds they give too."""
    p = Problem(3, 2, 4, 8, 2, 128, 16, "bf16", "16", 128, 1, False, "both", False)
    x = p.call(cuda_device)
    q, k = p.q.contiguous().to(cuda_device), p.k.contiguous().to(cuda_device)
    pa.append_rotated(p.cfg, q, k, None, None, x["ctx"], x["ql"], q, None, None, k_out=k, flags=x["flags"], **x["kw"])
    for b in range(p.B):
        n = p.ql[b]
        assert torch.equal(q[b, :n], x["qo"][b, :n]) and torch.equal(k[b, :n], x["ko"][b, :n])
        assert torch.equal(q[b, n:].cpu(), p.q[b, n:]) and torch.equal(k[b, n:].cpu(), p.k[b, n:])


@pytest.mark.gpu
def test_flags(cuda_device, pa):
    p = Problem(4, 3, 4, 4, 2, 128, 16, "bf16", "4", 64, 3, False, "both", True)
    clean = p.call(cuda_device)
    assert int(clean["flags"].item()) == 0
    kept = {n: clean[n].clone() for n in ("qo", "ko", "kc", "vc")}
    # a position outside the table: that token is not written at all
    p.pos[1, 0, 1] = p.cs.shape[0]
    x = p.call(cuda_device)
    assert int(x["flags"].item()) == pa.FLAG_BAD_POSITION
    assert (x["qo"][0, 1] == 5).all() and (x["ko"][0, 1] == 5).all()
    assert torch.equal(x["qo"][0, 0], kept["qo"][0, 0]) and torch.equal(x["qo"][1:], kept["qo"][1:])
    pos = int(p.ctx[0] - p.ql[0] + 1)
    blk, slot = int(p.bt[0, pos // 16]), pos % 16
    assert torch.equal(x["kc"][blk, slot].cpu(), p.kc[blk, slot])
    p.pos[1, 0, 1] = -1
    assert int(p.call(cuda_device)["flags"].item()) == pa.FLAG_BAD_POSITION
    p.pos[1, 0, 1] = 0
    # a page outside the pool: queries are rotated all the same
    first = int(p.ctx[0] - p.ql[0]) // 16
    was = p.bt.copy()
    p.bt[0, first] = p.nblocks
    x = p.call(cuda_device)
    assert int(x["flags"].item()) == pa.FLAG_BAD_BLOCK_ID
    assert torch.equal(x["qo"][0, 0], kept["qo"][0, 0]) and torch.equal(x["ko"][0, 0], kept["ko"][0, 0])
    # a bad length: nothing of that sequence
    p.bt, p.ql[2] = was, 5
    x = p.call(cuda_device)
    assert int(x["flags"].item()) == pa.FLAG_BAD_LENGTHS
    assert (x["qo"][2] == 5).all() and torch.equal(x["qo"][1], kept["qo"][1])


@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,hq,hkv,d", [(1, 1, 1, 1, 64), (1, 2000, 9, 3, 128), (700, 1, 7, 7, 64), (2, 1500, 2, 1, 256)])
@pytest.mark.parametrize("kv", ["16", "4"])
def test_every_split_of_a_tokens_rows(B, sq, hq, hkv, d, kv, cuda_device, pa):
    """Few tokens and many (a token's rows on many warps or one), odd head counts: queries and keys
    against fp32 torch, and pages as the append writes them."""
    rng = np.random.default_rng(9)
    t, dev, bs = torch.bfloat16, cuda_device, 64
    ql = rng.integers(0, sq + 1, B)
    ql[0] = sq
    ctx = ql + rng.integers(0, 100, B)
    bt, nblocks = plain.tables(rng, ctx, bs)
    cfg = config(B, sq, hq, hkv, d, bs, bt.shape[1], nblocks, "bf16", kv)
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((B, sq, hq + 2 * hkv, d), generator=g, device=dev).to(t)
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    w = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(t)
    cs = angles(int(ctx.max()) + 1, d).to(dev)
    byte = kv == "4"
    shape = (nblocks, bs, hkv, d // 2 if byte else d)
    fresh = lambda: (torch.zeros(shape, dtype=torch.uint8 if byte else t, device=dev),  # noqa: E731
                     torch.zeros((nblocks, hkv, bs, 2), dtype=t, device=dev) if byte else None)
    (kc, ks), (vc, vs), (rk, rks), (rv, rvs) = (fresh() for _ in range(4))
    qo, ko = torch.zeros(B, sq, hq, d, dtype=t, device=dev), torch.zeros(B, sq, hkv, d, dtype=t, device=dev)
    args, flags = (ints(bt, dev), ints(ctx, dev), ints(ql, dev)), ints([0], dev)
    pa.append_rotated(cfg, q, k, v, *args, qo, kc, vc, ks, vs, cos_sin=cs, q_weight=w, k_weight=w, k_out=ko, flags=flags)
    assert int(flags.item()) == 0
    i = torch.arange(sq, device=dev)
    real = i < args[2][:, None]
    pos = ((args[1] - args[2])[:, None] + i).clamp(max=cs.shape[0] - 1)
    c, s = (a[:, :, None].double() for a in cs[pos].chunk(2, -1))

    def turned(y):
        y = y.double()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        a, b = y.chunk(2, -1)
        z = torch.cat((a * c - b * s, b * c + a * s), -1)
        return z, torch.cat((a.abs() + b.abs(),) * 2, -1)

    for got, src in ((qo, q), (ko, k)):
        z, size = turned(src)
        tol = 2.0 ** -8 * z.abs() + FP32 * size * 1.01
        ok = (got.double() - z).abs() <= tol * (1 + 2.0 ** -9)
        assert bool((ok | ~real[..., None, None]).all()) and bool((got[~real] == 0).all())
    # the pages: values as the append writes them, keys (16 bits) as k_out has them
    pa.append_kv(cfg, ko, v.contiguous(), *args, rk, rv, rks, rvs)
    assert torch.equal(vc, rv) and (vs is None or torch.equal(vs, rvs))
    assert byte or torch.equal(kc, rk)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_zeros_keep_their_signs(d, dtype, cuda_device, pa):
    """fp8 codes of zeros, and of what a code cannot hold, have the sign of the value, by the plain append
    and by the rotating one."""
    t, dev = KINDS[dtype][0], cuda_device
    x = torch.randn(2, 3, 2, d, generator=torch.Generator().manual_seed(5)).to(t)
    x[..., ::5], x[..., 1::5], x[..., 2::5] = -0.0, 0.0, -float(torch.finfo(t).smallest_normal)
    want = (x.float() / (x.float().abs().amax(-1, keepdim=True) / 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert (want[..., 0] == 0x80).all() and (want[..., 1] == 0).all()
    cfg = config(2, 3, 2, 2, d, 16, 1, 2, dtype, "8token")
    x, bt, n = x.to(dev), ints([[0], [1]], dev), ints([3, 3], dev)
    for rotated in (False, True):
        cache = [torch.zeros(2, 16, 2, d, dtype=torch.uint8, device=dev) for _ in "kv"]
        scale = [torch.zeros(2, 16, 2, device=dev) for _ in "kv"]
        if rotated:
            pa.append_rotated(cfg, x, x, x, bt, n, n, torch.empty_like(x), *cache, *scale)
        else:
            pa.append_kv(cfg, x, x, bt, n, n, *cache, *scale)
        for c in cache:
            assert torch.equal(c[:, :3].cpu(), want)


@pytest.mark.gpu
def test_replays_in_a_graph(cuda_device, pa):
    p = Problem(8, 3, 2, 8, 2, 128, 16, "bf16", "8token", 128, 1, False, "both", True)
    want = {n: t.clone() for n, t in p.call(cuda_device).items() if n in ("qo", "kc", "vc", "ks")}
    x = p.on(cuda_device)
    call = lambda: pa.append_rotated(p.cfg, x["q"], x["k"], x["v"], x["bt"], x["ctx"], x["ql"], x["qo"], x["kc"],  # noqa: E731
                                     x["vc"], x["ks"], x["vs"], flags=x["flags"], **x["kw"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        x["qo"].fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in want.items():
            assert torch.equal(x[n].view(torch.uint8), t.view(torch.uint8)), n


@pytest.mark.gpu
@pytest.mark.parametrize("kv,dtype", [("16", "bf16"), ("8token", "bf16"), ("4", "bf16"), ("4", "fp16")])
def test_prompt_then_step(kv, dtype, cuda_device, pa):
    """A prompt and a step of draft tokens through rotation, pages and decode, against 64 bits on the
    values that the cache holds; scores depend on the distance of positions alone."""
    dev, B, hq, hkv, d, bs = cuda_device, 2, 8, 2, 128, 16
    t = KINDS[dtype][0]
    rng = np.random.default_rng(2)
    end = np.array([60, 37])
    bt, nblocks = plain.tables(rng, end, bs)
    cs = angles(64, d)
    kind, _ = CACHES[kv]
    byte = kind is not None
    shape = (nblocks, bs, hkv, d // 2 if kv == "4" else d)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8 if byte else t, device=dev) for _ in "kv")
    scale = {"8token": (shape[:3], torch.float32), "4": ((nblocks, hkv, bs, 2), t)}.get(kv)
    ks, vs = (None if scale is None else torch.zeros(scale[0], dtype=scale[1], device=dev) for _ in "kv")
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(d)).to(t).to(dev)
    dbt = ints(bt, dev)
    for sq, ql in ((56, end - 4), (4, np.array([4, 4]))):
        ctx = ql if sq == 56 else end
        cfg = config(B, sq, hq, hkv, d, bs, bt.shape[1], nblocks, dtype, kv, causal=1)
        qkv = torch.from_numpy(rng.standard_normal((B, sq, hq + 2 * hkv, d))).to(t).to(dev)
        q = torch.zeros(B, sq, hq, d, dtype=t, device=dev)
        args = dbt, ints(ctx, dev), ints(ql, dev)
        pa.append_rotated(cfg, qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], *args, q, kc, vc, ks, vs,
                          cos_sin=cs.to(dev), q_weight=w, k_weight=w)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=dev)
        ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=dev)
        pa.plan(cfg, *args, ws)
        pa.decode(cfg, q, kc, vc, ks, vs, *args, out, lse, ws)
        pa.reduce(cfg, out, lse, ws)
        if kv == "4":
            k64, v64 = plain.values(kc.cpu(), ks.cpu()), plain.values(vc.cpu(), vs.cpu())
            pair = vs.cpu().double().numpy().transpose(0, 2, 1, 3)
            mid = pair[..., 1:] + 8 * pair[..., :1]
            mag = np.abs(v64 - mid) + np.abs(mid)
        else:
            k64, v64 = (plain64.values(c.cpu(), None if s is None else s.cpu(), kv[1:]) for c, s in ((kc, ks), (vc, vs)))
            mag = np.abs(v64)
        ref = plain.attend(q.cpu(), k64, v64, mag, bt, ctx, ql, 1, float(np.float32(d ** -0.5)), nblocks)
        # f16 weights, but bf16 ones for a bf16 cache; 33 rows and more of an fp8 cache have their query
        # in E4M3 terms, good to about 2^-9 of the logits' magnitudes: the prompt there is not compared
        if not (kv == "8token" and sq == 56):
            plain64.check_attention(out, lse, *ref, t, 2.0 ** -8 if kv == "16" and dtype == "bf16" else 2.0 ** -11)


# ---- refusals (no GPU) ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_cache_work_gb300.build import build
        build()
    return pa.load()


FAKE = 1 << 20  # never dereferenced: every call below is rejected on the host


def rotary(**kw):
    r = pa.PaRotary(q_weight=FAKE, k_weight=FAKE, eps=1e-6, rotary_dim=128, interleaved=0, cos_sin=FAKE, table_rows=100,
                    positions=None, num_axes=1)
    r.axis_pairs[0] = 64
    for n, v in kw.items():
        if n == "axis_pairs":
            r.axis_pairs[:] = v
        else:
            setattr(r, n, v)
    return r


def call(lib, cfg, r, **kw):
    a = dict(q=FAKE, k=FAKE + 65536, v=FAKE, bt=FAKE, ctx=FAKE, ql=FAKE, qo=FAKE + 4096, ko=None, kc=FAKE, vc=FAKE,
             ks=None, vs=None, flags=None, stream=None)
    a.update(kw)
    return lib.pa_append_rotated(ctypes.byref(cfg) if cfg else None, ctypes.byref(r) if r else None, *a.values())


def base(kv="16", **kw):
    return config(2, 1, 8, 2, 128, 16, 8, 32, kv=kv, **kw)


@pytest.mark.parametrize("kw", [
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rotary_dim=-16), dict(interleaved=2),
    dict(cos_sin=None), dict(table_rows=0), dict(num_axes=0), dict(num_axes=4), dict(axis_pairs=(63, 0, 0)),
    dict(num_axes=2, axis_pairs=(65, -1, 0)), dict(q_stride=-8), dict(q_stride=8), dict(k_stride=257), dict(v_stride=128),
    dict(q_weight=FAKE + 2), dict(cos_sin=FAKE + 4), dict(positions=FAKE + 2)])
def test_bad_rotary(lib, kw):
    assert call(lib, base(), rotary(**kw)) == pa.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rotary_dim=24, axis_pairs=(12, 0, 0)), dict(rotary_dim=144, axis_pairs=(72, 0, 0))])
def test_unsupported_rotary(lib, kw):
    assert call(lib, base(), rotary(**kw)) == pa.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(ctx=None), dict(ql=None), dict(qo=None),
    dict(kc=None), dict(vc=None), dict(kc=None, vc=None), dict(q=FAKE + 8), dict(qo=FAKE + 2), dict(vc=FAKE + 4),
    dict(flags=FAKE + 1), dict(ko=FAKE + 8)])
def test_bad_pointers(lib, kw):
    assert call(lib, base(), rotary(), **kw) == pa.ERR_INVALID_ARG


def test_other_refusals(lib):
    r = rotary()
    assert call(lib, None, r) == pa.ERR_INVALID_ARG and call(lib, base(), None) == pa.ERR_INVALID_ARG
    for kv in ("8token", "8tensor", "4"):
        assert call(lib, base(kv), r) == pa.ERR_INVALID_ARG  # no scales
        assert call(lib, base(kv), r, ks=FAKE, vs=FAKE + 2) == pa.ERR_INVALID_ARG
    assert call(lib, base("4"), r, ks=FAKE, vs=FAKE + 8) == pa.ERR_INVALID_ARG
    c = base("8token")
    c.kv_scale_mode = pa.SCALE_PER_BLOCK
    assert call(lib, c, r, ks=FAKE, vs=FAKE) == pa.ERR_UNSUPPORTED
    for n, v, want in (("head_dim", 96, pa.ERR_UNSUPPORTED), ("block_size", 24, pa.ERR_UNSUPPORTED), ("batch", 0, pa.ERR_INVALID_ARG),
                       ("num_q_heads", 7, pa.ERR_UNSUPPORTED), ("kv_dtype", pa.FP16, pa.ERR_UNSUPPORTED),
                       ("q_dtype", pa.INT4, pa.ERR_UNSUPPORTED), ("kv_scale_mode", 9, pa.ERR_INVALID_ARG)):
        c = base()
        setattr(c, n, v)
        assert call(lib, c, r) == want, n
    # in place only where the rows lie dense
    assert call(lib, base(), rotary(q_stride=2048), qo=FAKE) == pa.ERR_INVALID_ARG
    assert call(lib, base(), rotary(k_stride=2048), ko=FAKE + 65536) == pa.ERR_INVALID_ARG


def test_binding_refuses_rows_that_do_not_fit():
    cfg = base()
    x = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    for bad in (x.transpose(2, 3), x[:, :, :4], x.float(), x[..., ::2]):
        with pytest.raises(pa.PaError):
            pa.append_rotated(cfg, bad, x, x, x, x, x, x, None, None, k_out=x)


def test_binding_refuses_rows_that_are_one_row():
    """An expanded tensor's tokens share one row, which the strides of a call cannot say (0 is dense)."""
    x = torch.zeros(4, 1, 8, 128, dtype=torch.bfloat16)
    for t, tokens in ((x[:1].expand(4, 1, 8, 128), 4), (x[:1].expand(1, 1, 8, 128).expand(4, 1, 8, 128), 2),
                      (x[:1, :1].expand(1, 3, 8, 128), 3), (x[:1, :1].expand(2, 3, 8, 128), 6)):
        with pytest.raises(pa.PaError):
            pa._rows("pa_append_rotated", -1, tokens, 8, 128, t, (torch.bfloat16,))
    assert pa._rows("pa_append_rotated", -1, 4, 8, 128, x, (torch.bfloat16,)) == (x.data_ptr(), 1024)
    assert pa._rows("pa_append_rotated", -1, 1, 8, 128, x[:1], (torch.bfloat16,))[0] == x.data_ptr()


def test_binding_refuses_positions_without_angles(monkeypatch):
    """Positions or axes say how to turn: without cos_sin nothing turns, and the call is refused."""
    class Lib:
        calls = 0

        def pa_append_rotated(self, *args):
            Lib.calls += 1
            return pa.OK

        def pa_status_string(self, status):
            return b"refused"

    monkeypatch.setattr(pa, "load", Lib)
    rows = lambda **kw: pa.append_rotated(base(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,  # noqa: E731
                                          stream=0, **kw)
    for kw in (dict(positions=FAKE), dict(axis_pairs=(64,)), dict(positions=FAKE, axis_pairs=(32, 32))):
        with pytest.raises(pa.PaError) as e:
            rows(**kw)
        assert e.value.status == pa.ERR_INVALID_ARG
    assert Lib.calls == 0
    rows(), rows(interleaved=True)
    assert Lib.calls == 2


@pytest.mark.gpu
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_any_scale_of_a_tensor(dtype, rotated, cuda_device, pa):
    """Codes under a tensor's scale are those of IEEE quotients, whatever the scale and the elements are."""
    t, dev, d = KINDS[dtype][0], cuda_device, 128
    g = torch.Generator().manual_seed(6)
    x = torch.randn(1, 64, 1, d, generator=g).float() * 2.0 ** torch.randint(-90, 90, (1, 64, 1, d), generator=g)
    x = x.clamp(-float(torch.finfo(t).max), float(torch.finfo(t).max)).to(t)
    edge = [0.0, -0.0, float("inf"), float("-inf"), float("nan"), float(torch.finfo(t).max), -float(torch.finfo(t).max),
            float(torch.finfo(t).smallest_normal), -float(torch.finfo(t).smallest_normal) / 4, 448.0, -464.0, 2.0 ** -10]
    x[0, 0, 0, :len(edge)] = torch.tensor(edge).to(t)
    cfg = config(1, 64, 1, 1, d, 64, 1, 1, dtype, "8tensor")
    dx, bt, n = x.to(dev), ints([[0]], dev), ints([64], dev)
    for s in (0.03, 1.0, 0.7, 2.0 ** -60, 2.0 ** 60, 1.5 * 2.0 ** -61, 2.0 ** 61, 3.1e-30, 1e-38, 1e38, -0.3, 0.0, float("inf"),
              float("nan")):
        scale = torch.tensor([s])
        q = x.float() / scale
        want = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        none = torch.isnan(q)
        cache = [torch.zeros(1, 64, 1, d, dtype=torch.uint8, device=dev) for _ in "kv"]
        args = bt, n, n
        if rotated:
            pa.append_rotated(cfg, dx, dx, dx, *args, torch.empty_like(dx), *cache, scale.to(dev), scale.to(dev))
        else:
            pa.append_kv(cfg, dx, dx, *args, *cache, scale.to(dev), scale.to(dev))
        for c in cache:
            c = c.cpu()
            assert torch.equal(c[~none], want[~none]), s
            assert ((c[none] & 0x7f) == 0x7f).all(), s


@pytest.mark.gpu
@pytest.mark.parametrize("exp", [-30, -1, 0, 7])
def test_scale_of_all_ones(exp, cuda_device, pa):
    """Divisors just below a power of two: the quotient of a power of two lies half a step past one, and
    past the tie of the least code with zero, where one correction step has no bit to spare."""
    dev, d = cuda_device, 64
    s = (2 - 2.0 ** -23) * 2.0 ** exp
    x = (2.0 ** (exp + 1 + torch.arange(-16.0, 16.0)).repeat(2)).view(1, 1, 1, d).to(torch.bfloat16)
    x[..., 32:] = -x[..., 32:]
    scale = torch.tensor([s], dtype=torch.float32)
    want = (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert int(want[0, 0, 0, 6]) == 1  # 2^-10 and a little
    cfg = config(1, 1, 1, 1, d, 16, 1, 1, "bf16", "8tensor")
    cache = [torch.zeros(1, 16, 1, d, dtype=torch.uint8, device=dev) for _ in "kv"]
    pa.append_kv(cfg, x.to(dev), x.to(dev), ints([[0]], dev), ints([1], dev), ints([1], dev), *cache, scale.to(dev), scale.to(dev))
    for c in cache:
        assert torch.equal(c[0, 0].cpu(), want[0, 0])


@pytest.mark.gpu
def test_keys_past_the_type_of_their_pairs(cuda_device, pa):
    """fp16 keys that a norm's weights take past 65504: those whose low or step does not fit read back as
    NaN, with codes 0, and so do the rows that see them; others keep their codes."""
    dev, d, bs = cuda_device, 256, 16
    x = torch.zeros(1, 4, 1, d)
    x[0, 0, 0, 5], x[0, 1, 0, 6], x[0, 2, 0, 7] = -1.0, 1.0, 1.0  # 16 in size once normalised
    x[0, 3] = torch.randn(1, d, generator=torch.Generator().manual_seed(1))
    w = torch.ones(d)
    w[5], w[6], w[7] = 8000.0, 8000.0, 65000.0  # -128,000; 128,000 (a step of 8,534); 1,040,000 (69,334)
    x, w = x.half().to(dev), w.half().to(dev)
    cfg = config(1, 4, 1, 1, d, bs, 1, 1, "fp16", "4", causal=1)
    codes = [torch.full((1, bs, 1, d // 2), 255, dtype=torch.uint8, device=dev) for _ in "kv"]
    pairs = [torch.zeros(1, 1, bs, 2, dtype=torch.float16, device=dev) for _ in "kv"]
    bt, n, flags, q = ints([[0]], dev), ints([4], dev), ints([0], dev), torch.empty_like(x)
    pa.append_rotated(cfg, x, x, x, bt, n, n, q, *codes, *pairs, k_weight=w, eps=0.0, flags=flags)
    assert int(flags.item()) == 0
    step, low = pairs[0][0, 0, :4].float().cpu().T
    y = plain.rotate(x[0, :, 0].double().cpu().numpy(), w.double().cpu().numpy(), 0.0, None, None, None, False)
    beyond = (y.min(1) < -65504) | ((y.max(1) - y.min(1)) / 15 > 65504)
    assert beyond.tolist() == [True, False, True, True]  # (row 3's element 7 is -100,572)
    assert torch.isnan(step).tolist() == beyond.tolist()
    c = plain.unpack(codes[0][0, :4, 0].cpu().numpy())
    assert (c[beyond] == 0).all()
    assert float(low[1]) == 0 and 127999 / 15 <= float(step[1]) <= 128000 / 15 * (1 + 2.0 ** -10)
    assert c[1, 6] == 15 and c[1].sum() == 15
    assert torch.isfinite(pairs[1][0, 0, :4]).all()
    k, v = (torch.empty(4, 1, d, dtype=torch.float16, device=dev) for _ in "kv")
    pa.dequant_kv(cfg, *codes, *pairs, bt, n, k, v)
    assert torch.isnan(k[[0, 2, 3]]).all() and not torch.isnan(k[1]).any() and torch.isfinite(v).all()
    for rows, lost in (([1], False), ([0], True), ([2], True), ([3, 1], True)):  # the seen keys, one or two
        bt2 = ints([[0]], dev)
        cc, pp = [torch.zeros_like(t) for t in codes], [torch.zeros_like(t) for t in pairs]
        for a, b in zip(cc + pp, codes + pairs):
            for i, r in enumerate(rows):
                if a.dtype == torch.uint8:
                    a[0, i] = b[0, r]
                else:
                    a[0, 0, i] = b[0, 0, r]
        one = config(1, 1, 1, 1, d, bs, 1, 1, "fp16", "4")
        out, lse = torch.empty(1, 1, 1, d, dtype=torch.float16, device=dev), torch.empty(1, 1, 1, device=dev)
        pa.decode_step_static(one, q[:, 3:].contiguous(), *cc, *pp, bt2, ints([len(rows)], dev), ints([1], dev), out, lse)
        assert bool(torch.isnan(out).all()) == lost and bool(torch.isnan(lse).all()) == lost
