"""One plan a step, kept over the layers: each layer's queries and rows are appended between the plan and
the decode that reads them, back to back and in a captured graph, and give what a plan behind each append
gives with a wait after every call."""
import numpy as np
import pytest
import torch

import paged_kv_cache_work_gb300 as pa
import plain_int4 as plain

B, LAYERS = 48, 5
KINDS = {"16": (pa.BF16, pa.SCALE_NONE), "8token": (pa.FP8_E4M3, pa.SCALE_PER_TOKEN),
         "8block": (pa.FP8_E4M3, pa.SCALE_PER_BLOCK), "4": (pa.INT4, pa.SCALE_AFFINE)}


def layer_cache(kv, nblocks, bs, hkv, d, dev):
    """(k_cache, v_cache, k_scale, v_scale) of a layer, empty."""
    shape = (nblocks, bs, hkv, d // 2 if kv == "4" else d)
    cache = [torch.zeros(shape, dtype=torch.bfloat16 if kv == "16" else torch.uint8, device=dev) for _ in "kv"]
    size = {"8token": (nblocks, bs, hkv), "8block": (nblocks, hkv), "4": (nblocks, hkv, bs, 2)}.get(kv)
    if size is None:
        return [*cache, None, None]
    return cache + [torch.ones(size, dtype=torch.bfloat16 if kv == "4" else torch.float32, device=dev) for _ in "kv"]


@pytest.mark.gpu
@pytest.mark.parametrize("rotated", [True, False])
@pytest.mark.parametrize("kv,sq,hq,hkv,d", [
    ("4", 1, 32, 8, 128), ("4", 4, 16, 1, 128), ("4", 2, 8, 1, 256), ("4", 1, 8, 2, 64),  # the 4-bit decode
    ("16", 12, 4, 1, 128), ("8token", 12, 4, 1, 128),  # the tcgen05 decode (48 rows)
    ("8block", 2, 8, 1, 128)])  # the streaming decode
def test_layers_on_one_plan(kv, sq, hq, hkv, d, rotated, cuda_device, pa):
    dev, bs, steps = cuda_device, 16, 3
    rng = np.random.default_rng(77)
    start = rng.integers(1, 300, B)
    most = int(start.max())
    end = start + steps * sq
    bt, nblocks = plain.tables(rng, end, bs)
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    kind, mode = KINDS[kv]
    make = lambda n: pa.PaConfig(  # noqa: E731
        batch=B, max_q_len=n, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
        max_blocks_per_seq=bt.shape[1], num_blocks=nblocks, q_dtype=pa.BF16, kv_dtype=kind, kv_scale_mode=mode,
        causal=1, sm_scale=d ** -0.5)
    cfg = make(sq)
    g = torch.Generator(device=dev).manual_seed(3)
    rows = lambda n, h: torch.randn((B, n, h, d), generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    angle = torch.arange(int(end.max()), device=dev)[:, None] * 1e4 ** (-torch.arange(0, d, 2, device=dev) / d)
    cs = torch.cat((angle.cos(), angle.sin()), 1).float()
    dbt, ctx, ql = ints(bt), ints(start), ints(start)
    empty = [layer_cache(kv, nblocks, bs, hkv, d, dev) for _ in range(LAYERS)]
    for cache in empty:
        pa.append_kv(make(most), rows(most, hkv), rows(most, hkv), dbt, ctx, ql, *cache)
    ql.fill_(sq)
    qkv = [torch.empty((B, sq, hq + 2 * hkv, d), dtype=torch.bfloat16, device=dev) for _ in range(LAYERS)]
    inputs = [[rows(sq, hq + 2 * hkv) for _ in range(LAYERS)] for _ in range(steps)]
    ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=dev)

    class Run:
        """A model's buffers: its layers' caches, and queries and new keys that every layer writes anew."""
        def __init__(self):
            self.cache = [[None if t is None else t.clone() for t in c] for c in empty]
            self.q = torch.zeros((B, sq, hq, d), dtype=torch.bfloat16, device=dev)
            self.k = torch.zeros((B, sq, hkv, d), dtype=torch.bfloat16, device=dev)
            self.out = [torch.zeros_like(self.q) for _ in range(LAYERS)]
            self.lse = [torch.zeros((B, sq, hq), device=dev) for _ in range(LAYERS)]

        def step(self, kept, wait=lambda: None):
            if kept:
                pa.plan(cfg, dbt, ctx, ql, ws)
            for x, cache, out, lse in zip(qkv, self.cache, self.out, self.lse):
                q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
                wait()
                if not rotated:  # (what the decode reads of the queries is the layer's own)
                    k, v, q = k.contiguous(), v.contiguous(), q.contiguous()
                    pa.append_kv(cfg, k, v, dbt, ctx, ql, *cache)
                elif kv == "8block":  # a page's one scale needs all its new rows
                    pa.append_rotated(cfg, q, k, None, None, ctx, ql, self.q, None, None, cos_sin=cs, k_out=self.k)
                    v, q = v.contiguous(), self.q
                    pa.append_kv(cfg, self.k, v, dbt, ctx, ql, *cache)
                else:
                    pa.append_rotated(cfg, q, k, v, dbt, ctx, ql, self.q, *cache, cos_sin=cs)
                    q = self.q
                wait()
                if not kept:
                    pa.plan(cfg, dbt, ctx, ql, ws)
                    wait()
                pa.decode(cfg, q, *cache, dbt, ctx, ql, out, lse, ws)
                wait()
                pa.reduce(cfg, out, lse, ws)
                wait()

        def state(self):
            return [t.clone() for t in self.out + self.lse] + [t.clone() for c in self.cache for t in c if t is not None]

    def give(turn):
        ctx.copy_(ints(start + (turn + 1) * sq))
        for x, new in zip(qkv, inputs[turn]):
            x.copy_(new)

    want, run = [], Run()
    for turn in range(steps):
        give(turn)
        run.step(False, torch.cuda.synchronize)
        want.append(run.state())

    def same(run, turn):
        torch.cuda.synchronize()
        for a, b in zip(run.state(), want[turn]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

    run = Run()
    for turn in range(steps):
        give(turn)
        run.step(True)
        same(run, turn)
        assert pa.read_flags(ws) == 0
    graph, run = torch.cuda.CUDAGraph(), Run()
    with torch.cuda.graph(graph):
        run.step(True)
    for again in range(4):
        for c, e in zip(run.cache, empty):
            for t, u in zip(c, e):
                if t is not None:
                    t.copy_(u)
        for turn in range(steps):
            give(turn)
            graph.replay()
            same(run, turn)


@pytest.mark.gpu
@pytest.mark.parametrize("merge", [pa.MERGE_IN_DECODE, pa.MERGE_IN_REDUCE])
@pytest.mark.parametrize("kv,hq,d", [("4", 4, 128), ("4", 16, 256), ("16", 48, 128), ("8block", 8, 64)])
def test_decodes_of_split_units_on_one_plan(kv, hq, d, merge, cuda_device, pa):
    """Two caches and queries in turn on one plan, their units in many pieces, in a captured graph: the
    merges start anew with every decode, and read its own pieces."""
    dev, bs, hkv, n = cuda_device, 32, 1, (3000, 40, 1111)
    kind, mode = KINDS[kv]
    bt, nblocks = plain.tables(np.random.default_rng(5), np.asarray(n), bs)
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    make = lambda sq: pa.PaConfig(  # noqa: E731
        batch=3, max_q_len=sq, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs,
        max_blocks_per_seq=bt.shape[1], num_blocks=nblocks, q_dtype=pa.BF16, kv_dtype=kind, kv_scale_mode=mode,
        sm_scale=d ** -0.5, num_ctas=70, split_merge=merge)
    g = torch.Generator(device=dev).manual_seed(8)
    args, cfg, cases = (ints(bt), ints(n), ints([1, 1, 1])), make(1), []
    for _ in range(2):
        cache = layer_cache(kv, nblocks, bs, hkv, d, dev)
        new = [torch.randn((3, max(n), hkv, d), generator=g, device=dev).to(torch.bfloat16) for _ in "kv"]
        pa.append_kv(make(max(n)), *new, args[0], args[1], args[1], *cache)
        q = torch.randn((3, 1, hq, d), generator=g, device=dev).to(torch.bfloat16)
        cases.append((q, cache, torch.empty_like(q), torch.empty((3, 1, hq), device=dev)))
    ws = torch.empty(pa.workspace_size(cfg), dtype=torch.uint8, device=dev)

    def step(fresh):
        if not fresh:
            pa.plan(cfg, *args, ws)
        for q, cache, out, lse in cases:
            if fresh:
                pa.plan(cfg, *args, ws)
            pa.decode(cfg, q, *cache, *args, out, lse, ws)
            pa.reduce(cfg, out, lse, ws)
            if fresh:
                torch.cuda.synchronize()

    step(True)
    want = [(out.clone(), lse.clone()) for _, _, out, lse in cases]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(False)
        step(False)
    for _ in range(5):
        for _, _, out, lse in cases:
            out.fill_(7), lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert pa.read_flags(ws) == 0
        for (_, _, out, lse), (o, l) in zip(cases, want):
            assert torch.equal(out.view(torch.int16), o.view(torch.int16)) and torch.equal(lse, l)
