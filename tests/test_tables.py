"""pa_build_tables against a stack in plain Python: growth, requests that end, rejected tokens,
prompts from nothing, pages given and taken in one call, sizes past one CTA and past one thread a
sequence, refusals, flags, and a captured graph."""
import ctypes
import os

import numpy as np
import pytest
import torch

import paged_kv_cache_work_gb300 as pa
import plain64


def config(B, sq, bs, maxb, nblocks):
    return pa.PaConfig(batch=B, max_q_len=sq, num_q_heads=1, num_kv_heads=1, head_dim=128, block_size=bs,
                       max_blocks_per_seq=maxb, num_blocks=nblocks, q_dtype=pa.BF16, kv_dtype=pa.BF16,
                       kv_scale_mode=0, causal=0, sm_scale=1.0)


def problem(seed, B, sq, bs, longest, fresh=False, spare=8):
    """Random growth, shrinkage and ends; at least as many free pages as are taken."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, longest + 1, B)
    n[rng.random(B) < 0.15] = 0
    q = np.minimum(n, rng.integers(0, sq + 1, B))
    before = np.where(rng.random(B) < 0.3, rng.integers(0, longest + 1, B), n - q)
    held = np.zeros(B, int) if fresh else -(-before // bs)
    maxb = max(1, -(-longest // bs))
    need = -(-n // bs)
    used = int(held.sum())
    count = max(0, int(np.maximum(need - held, 0).sum() - np.maximum(held - need, 0).sum())) + spare
    nblocks = used + count
    ids = rng.permutation(nblocks)
    bt = np.full((B, maxb), -1, np.int64)
    at = 0
    for b in range(B):
        bt[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(nblocks, -7)
    free[:count] = ids[at:]
    return dict(n=n, q=q, held=held, bt=bt, free=free, count=count, nblocks=nblocks, maxb=maxb)


def plain(p, bs, sq):
    return plain64.build_tables(p["n"].tolist(), p["q"].tolist(), p["held"].tolist(), p["bt"].tolist(),
                                p["free"].tolist(), p["count"], bs, sq)


def on_gpu(p, dev):
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    return {k: t(p[k]) for k in ("n", "q", "held", "bt", "free")} | {"count": t([p["count"]])}


def call(pa_mod, p, sq, bs, dev, d=None, flags=None, slots=True):
    d = d or on_gpu(p, dev)
    B = len(p["n"])
    new_held = torch.full((B,), -5, dtype=torch.int32, device=dev)
    new_count = torch.full((1,), -5, dtype=torch.int32, device=dev)
    slot_map = torch.full((B, sq), -9, dtype=torch.int64, device=dev) if slots else None
    pa_mod.build_tables(config(B, sq, bs, p["maxb"], p["nblocks"]), d["n"], d["q"], d["held"], d["bt"],
                        d["free"], d["count"], new_held, new_count, slot_map, flags)
    return d, new_held, new_count, slot_map


CASES = [
    # B, Sq, bs, longest, fresh
    (1, 1, 16, 1, True), (1, 1, 16, 40, False), (3, 4, 16, 100, False), (64, 4, 16, 700, False),
    (37, 5, 32, 333, False), (5, 300, 64, 300, True), (9, 2000, 16, 2000, True), (700, 3, 16, 90, False),
    (1025, 1, 128, 400, False), (4096, 2, 16, 50, False), (2, 1, 1024, 5000, False), (48, 700, 32, 900, False),
    (3, 2047, 16, 2047, True), (33, 33, 16, 4000, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,sq,bs,longest,fresh", CASES)
def test_tables_match_a_plain_stack(B, sq, bs, longest, fresh, cuda_device, pa):
    for seed in (1, 2):
        p = problem(seed, B, sq, bs, longest, fresh)
        flags = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        bt, free, held, count, slots = plain(p, bs, sq)
        d, nh, nc, sm = call(pa, p, sq, bs, cuda_device, flags=flags)
        for again in range(2):  # a second call on the same inputs gives the same
            assert int(flags.item()) == 0
            assert d["bt"].cpu().tolist() == bt
            assert d["free"].cpu().tolist()[:count] == free[:count]
            assert nh.cpu().tolist() == held and int(nc.item()) == count
            assert sm.cpu().tolist() == slots
            d, nh, nc, sm = call(pa, p, sq, bs, cuda_device, d=d, flags=flags)


@pytest.mark.gpu
def test_every_given_page_is_taken_again(cuda_device, pa):
    """No free page at all: what some rows give is what others take."""
    p = dict(n=np.array([0, 64, 16]), q=np.array([0, 30, 16]), held=np.array([3, 2, 0]),
             bt=np.array([[4, 0, 2, -1], [1, 3, -1, -1], [-1] * 4]), free=np.zeros(5, int), count=0, nblocks=5, maxb=4)
    bt, _, held, count, slots = plain(p, 16, 30)
    d, nh, nc, sm = call(pa, p, 30, 16, cuda_device)
    given = d["bt"].cpu().tolist()
    assert given[1:] == bt[1:] and nh.cpu().tolist() == held
    assert int(nc.item()) == count == 0 and sm.cpu().tolist() == slots


@pytest.mark.gpu
def test_rows_without_a_slot_map(cuda_device, pa):
    p = problem(3, 20, 4, 16, 200)
    bt, _, held, count, _ = plain(p, 16, 4)
    d, nh, nc, _ = call(pa, p, 4, 16, cuda_device, slots=False)
    assert d["bt"].cpu().tolist() == bt and nh.cpu().tolist() == held and int(nc.item()) == count


def _spoil(p, what):
    if what == "short":
        p["count"] = int((-(-p["n"] // 16)).sum()) - 1
    elif what == "q > n":
        p["n"][2], p["q"][2] = 1, 2
    elif what == "q < 0":
        p["q"][2] = -1
    elif what == "n > cap":
        p["n"][2] = p["maxb"] * 16 + 1
    elif what == "held > columns":
        p["held"][2] = p["maxb"] + 1
    elif what == "count < 0":
        p["count"] = -1
    elif what == "count > pool":
        p["count"] = p["nblocks"] + 1


@pytest.mark.gpu
@pytest.mark.parametrize("what,flag", [
    ("short", "NO_FREE_BLOCKS"), ("q > n", "BAD_LENGTHS"), ("q < 0", "BAD_LENGTHS"), ("n > cap", "BAD_LENGTHS"),
    ("held > columns", "BAD_FREE_LIST"), ("count < 0", "BAD_FREE_LIST"), ("count > pool", "BAD_FREE_LIST")])
def test_bad_inputs_change_nothing(what, flag, cuda_device, pa):
    p = problem(5, 12, 4, 16, 300, fresh=True)
    _spoil(p, what)
    flags = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    d, nh, nc, sm = call(pa, p, 4, 16, cuda_device, flags=flags)
    assert int(flags.item()) == getattr(pa, "FLAG_" + flag)
    assert d["bt"].cpu().tolist() == p["bt"].tolist() and d["free"].cpu().tolist() == p["free"].tolist()
    assert nh.cpu().tolist() == p["held"].tolist() and int(nc.item()) == p["count"]
    assert (sm.cpu() == -1).all()


@pytest.mark.gpu
def test_a_page_outside_the_pool_gets_no_slot(cuda_device, pa):
    p = problem(6, 6, 8, 16, 200, fresh=True)
    p["n"][0], p["q"][0] = 8, 8
    p["free"][p["count"] - 1] = p["nblocks"] + 3  # the first page taken: row 0's
    flags = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    slots = plain(p, 16, 8)[4]
    _, _, _, sm = call(pa, p, 8, 16, cuda_device, flags=flags)
    limit = p["nblocks"] * 16
    assert any(s >= limit for r in slots for s in r)
    assert sm.cpu().tolist() == [[s if s < limit else -1 for s in r] for r in slots]
    assert int(flags.item()) == pa.FLAG_BAD_BLOCK_ID


@pytest.mark.gpu
@pytest.mark.parametrize("slots", [True, False])
@pytest.mark.parametrize("bad", [-1, 5, 1 << 30])
@pytest.mark.parametrize("how", ["freed", "handed on", "taken"])
def test_a_page_outside_the_pool_is_flagged_where_it_moves(how, bad, slots, cuda_device, pa):
    """Given back to the free list, given to another row, or taken from the free list by a row
    without new tokens: each is flagged, with and without a slot map."""
    p = dict(n=np.array([16, 0]), q=np.array([0, 0]), held=np.array([3, 0]), bt=np.array([[4, 0, 2], [-1] * 3]),
             free=np.array([1, 3, -7, -7, -7]), count=2, nblocks=5, maxb=3)
    if how == "taken":
        p["free"][1] = bad
        p["held"][0], p["n"][1] = 1, 30
    else:
        p["bt"][0, 1 if how == "freed" else 2] = bad
        p["n"][1] = 0 if how == "freed" else 20  # (row 1 takes the pages pushed last)
    want = plain(p, 16, 1)
    moved = want[0][1][:want[2][1]] + want[1][:want[3]]
    assert bad in moved and (how == "freed") == (bad not in want[0][1][:want[2][1]])
    flags = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    d, nh, nc, _ = call(pa, p, 1, 16, cuda_device, flags=flags, slots=slots)
    assert int(flags.item()) == pa.FLAG_BAD_BLOCK_ID
    assert d["bt"].cpu().tolist() == want[0] and nh.cpu().tolist() == want[2] and int(nc.item()) == want[3]
    assert d["free"].cpu().tolist()[:want[3]] == want[1][:want[3]]


@pytest.mark.gpu
def test_captured_and_replayed_with_other_lengths(cuda_device, pa):
    p = problem(7, 30, 4, 16, 300, spare=300)
    d = on_gpu(p, cuda_device)
    cfg = config(30, 4, 16, p["maxb"], p["nblocks"])
    nh = torch.empty(30, dtype=torch.int32, device=cuda_device)
    nc = torch.empty(1, dtype=torch.int32, device=cuda_device)
    sm = torch.empty(30, 4, dtype=torch.int64, device=cuda_device)
    args = (cfg, d["n"], d["q"], d["held"], d["bt"], d["free"], d["count"], nh, nc, sm)
    call(pa, p, 4, 16, cuda_device)  # (sets the kernel up before the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.build_tables(*args)
    bt, free, held, count = p["bt"].tolist(), p["free"].tolist(), p["held"].tolist(), p["count"]
    n, q = p["n"].tolist(), p["q"].tolist()
    for step in range(5):
        want = plain64.build_tables(n, q, held, bt, free, count, 16, 4)
        g.replay()
        torch.cuda.synchronize()
        assert d["bt"].cpu().tolist() == want[0] and sm.cpu().tolist() == want[4]
        assert nh.cpu().tolist() == want[2] and int(nc.item()) == want[3]
        bt, free, held, count = want[0], d["free"].cpu().tolist(), want[2], want[3]
        d["held"].copy_(nh)
        d["count"].copy_(nc)
        n = [0 if (b + step) % 9 == 0 else min(x + 3, 300) for b, x in enumerate(n)]
        q = [min(x, 3) for x in n]
        d["n"].copy_(torch.tensor(n, dtype=torch.int32))
        d["q"].copy_(torch.tensor(q, dtype=torch.int32))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_cache_work_gb300.build import build
        build()
    return pa.load()


def test_refused_on_the_host(lib):
    fake = 1 << 20  # never dereferenced: every call below is rejected on the host
    names = ("ctx", "q", "held", "bt", "free", "count", "new_held", "new_count", "slots", "flags")

    def call(cfg=None, **kw):
        a = {k: fake + 65536 * j for j, k in enumerate(names)}
        a.update(kw)
        c = cfg or config(4, 2, 16, 8, 32)
        return lib.pa_build_tables(ctypes.byref(c), *(a[k] for k in names), None)

    for k in names[:8]:
        assert call(**{k: None}) == pa.ERR_INVALID_ARG, k
    for k in names:
        assert call(**{k: fake + 2}) == pa.ERR_INVALID_ARG, k
    assert call(slots=fake + 8) == pa.ERR_INVALID_ARG
    assert call(new_held=fake + 65536 * 2) == pa.ERR_INVALID_ARG       # this call's held_blocks
    assert call(new_held=fake + 65536 * 2 + 12) == pa.ERR_INVALID_ARG  # overlaps them
    assert call(new_count=fake + 65536 * 5) == pa.ERR_INVALID_ARG
    assert lib.pa_build_tables(None, *([fake] * 10), None) == pa.ERR_INVALID_ARG
    for kw, want in ((dict(B=0), pa.ERR_INVALID_ARG), (dict(sq=0), pa.ERR_INVALID_ARG),
                     (dict(maxb=0), pa.ERR_INVALID_ARG), (dict(nblocks=0), pa.ERR_INVALID_ARG),
                     (dict(bs=24), pa.ERR_UNSUPPORTED), (dict(bs=8), pa.ERR_UNSUPPORTED),
                     (dict(B=4097), pa.ERR_UNSUPPORTED), (dict(sq=1 << 30), pa.ERR_UNSUPPORTED),
                     (dict(maxb=1 << 29), pa.ERR_UNSUPPORTED)):
        assert call(config(**{**dict(B=4, sq=2, bs=16, maxb=8, nblocks=32), **kw})) == want, kw


def test_binding_refuses_tensors_that_do_not_fit(lib):
    cfg = config(4, 2, 16, 8, 32)
    i32 = torch.zeros(64, dtype=torch.int32)
    with pytest.raises(pa.PaError) as e:  # CPU tensors
        pa.build_tables(cfg, i32, i32, i32, i32, i32, i32, i32, i32)
    assert e.value.status == pa.ERR_INVALID_ARG
