"""Attention over a cache at the shapes that decide between its kernels and
inside them: rows per key head around every tile size, row tiles that are
alone in their unit next to pairs, pages of every box height, units cut by
many blocks and many units per block, batches of more sequences than threads,
shared pages, shared workspaces, concurrent threads, and the guard build."""
import random
import threading

import numpy as np
import pytest
import torch

import oracle
from _cache import Setup, TORCH, attention_reference, check, int32, random_tree, values
from test_gpu_cache import attend, compare_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("int8", "f16")])
@pytest.mark.parametrize("G,T", [(1, 16), (1, 17), (3, 11), (8, 6), (7, 7), (1, 64), (5, 13), (1, 128), (3, 43), (4, 64),
                                 (1, 257), (4, 75)])
def test_rows_around_the_tiles(gpu_lib, D, cache, dtype, G, T):
    """G * T from 16 to 300: one to four tiles of 16 rows, 64 and 65, 128, a
    pair of tiles, a pair and a tile alone."""
    ta = gpu_lib
    kv = [T + 3, T + 200]
    st = Setup(ta, kv, 2, 16, D, dtype, cache, 41)
    q = values(3, (2, 2 * G, T, D), dtype, 1.3)
    rng = random.Random(G * 100 + T)
    ql = [T, max(1, T - 2)]
    for tr in (None, np.stack([random_tree(rng, T) for _ in range(2)])):
        o, lse = attend(ta, st, q, ql, tr, torch.zeros_like(q).cuda(), torch.zeros(2, 2 * G, T, device="cuda"))
        assert ta.sync_status() == "TA_OK"
        compare_attention(st, q, o, lse, ql, tr)


@pytest.mark.parametrize("page", [1, 7, 8, 16, 24, 32, 40, 96, 256])
@pytest.mark.parametrize("cache,dtype,D", [("bf16", "bf16", 128), ("int8", "bf16", 32), ("e4m3", "f16", 64)])
def test_page_sizes(gpu_lib, page, cache, dtype, D):
    """Pages that hold a tile, end inside one, and (1 and 7) have no box."""
    ta = gpu_lib
    T, G = 50, 3
    st = Setup(ta, [50, 130, 391], 1, page, D, dtype, cache, 17)
    q = values(3, (3, G, T, D), dtype)
    tr = np.stack([random_tree(random.Random(2), T)])
    o, lse = attend(ta, st, q, None, tr)
    assert ta.sync_status() == "TA_OK"
    compare_attention(st, q, o, lse, None, tr)


@pytest.mark.parametrize("cache,dtype,D", [("bf16", "bf16", 128), ("f16", "f16", 64), ("e4m3", "bf16", 128),
                                           ("int8", "f16", 64)])
def test_many_units_of_both_kinds(gpu_lib, cache, dtype, D):
    """Sequences whose rows fill pairs of tiles, tiles alone and a few rows, in
    one call with several units per block: blocks go from one kind to the
    other, finish units and leave cut ones."""
    ta = gpu_lib
    Hkv, G, T = 5, 4, 75
    ql = [75, 3, 40, 75, 1, 33, 64, 0, 75, 20]
    kv = [n + x for n, x in zip(ql, [900, 5, 0, 333, 2000, 127, 128, 10, 1500, 60])]
    st = Setup(ta, kv, Hkv, 16, D, dtype, cache, 23)
    q = values(3, (len(kv), Hkv * G, T, D), dtype)
    rng = random.Random(9)
    trees = np.stack([random_tree(rng, T) for _ in kv])
    for tr in (None, trees):
        o, lse = attend(ta, st, q, ql, tr, torch.full_like(q, 2.0).cuda(), torch.full((len(kv), Hkv * G, T), 2.0, device="cuda"))
        assert ta.sync_status() == "TA_OK"
        compare_attention(st, q, o, lse, ql, tr, seqs=[0, 1, 2, 4, 6, 9])
        for b, n in enumerate(ql):
            assert (o[b, :, n:] == 2).all() and (lse[b, :, n:] == 2).all()


@pytest.mark.parametrize("T,G", [(1, 4), (40, 4)])
def test_more_sequences_than_threads(gpu_lib, T, G):
    ta = gpu_lib
    B, D = 700, 16
    rng = random.Random(4)
    kv = [T + rng.randrange(0, 60) for _ in range(B)]
    ql = [rng.choice([T, T, max(0, T - 1), 0]) for _ in range(B)]
    st = Setup(ta, kv, 1, 8, D, "bf16", "int8", 3)
    q = values(3, (B, G, T, D), "bf16")
    o, lse = attend(ta, st, q, ql, None, torch.zeros_like(q).cuda(), torch.zeros(B, G, T, device="cuda"))
    assert ta.sync_status() == "TA_OK"
    compare_attention(st, q, o, lse, ql, None, seqs=[0, 1, 2, 127, 128, 129, 333, 511, 512, 698, 699])


@pytest.mark.parametrize("cache,dtype,T,G", [("bf16", "bf16", 1, 8), ("e4m3", "bf16", 1, 8), ("f16", "f16", 40, 4),
                                             ("int8", "f16", 100, 1)])
def test_one_long_sequence_over_every_block(gpu_lib, cache, dtype, T, G):
    """A single unit cut by every border of the line."""
    ta = gpu_lib
    D, N = 64, 20000
    page = 64
    P = (N + page - 1) // page
    c = ta.kv_cache(P, 1, page, D, TORCH[cache])
    k, v = (values(i, (1, 1, N, D), dtype).cuda() for i in (1, 2))
    pages = int32(reversed(range(P))).view(1, P)
    ta.cache_append(c, k, v, pages, int32([N]))
    kr, vr = ta.cache_read(c, pages, int32([N]), N, dtype=TORCH[dtype])
    q = values(3, (1, G, T, D), dtype, 2.0)
    o, lse = ta.attn_cache_fwd(q.cuda(), c, pages, int32([N]), int32([T]))
    assert ta.sync_status() == "TA_OK"
    kn, vn, vs = kr[0, 0].double().cpu().numpy(), vr[0, 0].double().cpu().numpy(), None
    if cache in ("e4m3", "int8"):  # what the codes stand for, unrounded
        (kc, ks), (vc, vs) = (oracle.cache_quantise(x[0, 0].cpu(), cache) for x in (k, v))
        kn, vn, vs = kc * ks[:, None].astype(np.float64), vc * vs[:, None].astype(np.float64), vs.astype(np.float64)
    O, L, bO, bL = attention_reference(q[0], kn, vn, None, cache, dtype, vs)
    check("O", o[0], O, bO)
    check("L", lse[0], L, bL)


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("int8", "f16")])
@pytest.mark.parametrize("T,G", [(1, 4), (3, 8), (80, 2)])
@pytest.mark.parametrize("junk", [0, 1, 0x7F, 0x80, 0xFF, 0x3C])
def test_memory_behind_the_end_holds_anything(gpu_lib, cache, dtype, T, G, junk):
    """Codes, values and scales of rows behind a sequence's end, in its last page
    and in others: zeros, denormals, infinities, NaN, ordinary numbers."""
    ta = gpu_lib
    kv = [T + 5, T + 61, T + 133]
    st = Setup(ta, kv, 1, 32, 64, dtype, cache, 3)
    q = values(3, (3, G, T, 64), dtype)
    o, lse = attend(ta, st, q)
    compare_attention(st, q, o, lse, None, None)
    owned = torch.zeros(st.cache.shape[0], 32, dtype=torch.bool)
    for b, n in enumerate(kv):
        for i in range(n):
            owned[oracle.cache_slot(st.table[b], 32, i)] = True
    free = (~owned).cuda()
    for t in (st.cache.k, st.cache.v, st.cache.k_scale, st.cache.v_scale):
        if t is not None:
            raw = t.view(torch.uint8).view(t.shape[0], 32, -1)  # one head
            raw[free] = junk
    o2, lse2 = attend(ta, st, q)
    assert ta.sync_status() == "TA_OK"
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_sequences_share_pages(gpu_lib):
    """A common prompt's pages in two page tables."""
    ta = gpu_lib
    D = 64
    c = ta.kv_cache(12, 2, 16, D, torch.bfloat16)
    k, v = (values(i, (1, 2, 48, D), "bf16").cuda() for i in (1, 2))
    ta.cache_append(c, k, v, int32([3, 5, 7]).view(1, 3), int32([48]))
    pages, lens = int32([3, 5, 7, 1, 3, 5, 7, 2]).view(2, 4), int32([52, 50])
    nk, nv = (values(i, (2, 2, 4, D), "bf16").cuda() for i in (3, 4))
    ql = int32([4, 2])
    ta.cache_append(c, nk, nv, pages, lens, ql)
    for G in (2, 20):
        q = values(5, (2, 2 * G, 4, D), "bf16")
        o, lse = ta.attn_cache_fwd(q.cuda(), c, pages, lens, ql)
        assert ta.sync_status() == "TA_OK"
        for b, n in enumerate((4, 2)):
            for h in range(2):
                kk, vv = (torch.cat([x[0, h], y[b, h, :n]]).double().cpu().numpy() for x, y in ((k, nk), (v, nv)))
                O, L, bO, bL = attention_reference(q[b, h * G:(h + 1) * G, :n], kk, vv, None, "bf16", "bf16")
                check("O", o[b, h * G:(h + 1) * G, :n], O, bO)
                check("L", lse[b, h * G:(h + 1) * G, :n], L, bL)


def test_graphs_that_share_a_workspace(gpu_lib):
    """Two captured calls of different shapes with one workspace, replayed in
    turn: nothing of one is left for the other."""
    ta = gpu_lib
    D = 64
    a = Setup(ta, [700, 30, 9], 2, 16, D, "bf16", "bf16", 3)
    b = Setup(ta, [1500], 1, 16, D, "bf16", "e4m3", 4)
    qa, qb = values(1, (3, 8, 2, D), "bf16").cuda(), values(2, (1, 4, 40, D), "bf16").cuda()
    kva, kvb = a.kv_lens, b.kv_lens
    n = max(ta.attn_cache_workspace_bytes(3, 8, 2, 2, 800, D, torch.bfloat16),
            ta.attn_cache_workspace_bytes(1, 4, 1, 40, 1600, D, torch.bfloat16, torch.float8_e4m3fn))
    ws = torch.empty(n, device="cuda", dtype=torch.uint8)
    ref = [attend(ta, a, qa), attend(ta, b, qb)]
    out = [[torch.zeros_like(t) for t in r] for r in ref]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for st, q, (o, lse) in ((a, qa, out[0]), (b, qb, out[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            ta.attn_cache_fwd(q, st.cache, st.pages, st.kv_lens, o=o, lse=lse, ws=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        ws.fill_(0xFF)  # NaN partial states, impossible records
        for t in out[i]:
            t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out[i], ref[i]))
    assert ta.sync_status() == "TA_OK"
    assert kva is a.kv_lens and kvb is b.kv_lens


def test_host_threads(gpu_lib):
    """Calls from several threads, each with its own stream and buffers, equal
    the same calls one at a time."""
    ta = gpu_lib
    jobs = [(Setup(ta, [300, 41], 2, 16, 64, "bf16", c, 5), values(7, (2, 2 * G, T, 64), "bf16").cuda())
            for c, G, T in (("bf16", 2, 1), ("e4m3", 4, 9), ("int8", 4, 41), ("bf16", 8, 41))]
    ref = [attend(ta, st, q) for st, q in jobs]
    torch.cuda.synchronize()
    out, errors = [None] * len(jobs), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    out[i] = attend(ta, *jobs[i])
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors and ta.sync_status() == "TA_OK"
    for r, o in zip(ref, out):
        assert all(torch.equal(x, y) for x, y in zip(r, o))


def test_refusals(gpu_lib):
    """The binding's checks on CUDA tensors, before anything is launched."""
    ta = gpu_lib
    c = ta.kv_cache(4, 2, 16, 64, torch.bfloat16)
    pages, lens = int32([0, 1]).view(2, 1), int32([5, 6])
    q = torch.zeros(2, 4, 3, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 3, 64, device="cuda", dtype=torch.bfloat16)
    tree = torch.ones(2, 3, 3, dtype=torch.bool, device="cuda")
    bad = [
        lambda: ta.attn_cache_fwd(q.float(), c, pages, lens),
        lambda: ta.attn_cache_fwd(q[..., ::2], c, pages, lens),
        lambda: ta.attn_cache_fwd(q[:1], c, pages, lens),
        lambda: ta.attn_cache_fwd(q.cpu(), c, pages, lens),
        lambda: ta.attn_cache_fwd(q, c, pages.long(), lens),
        lambda: ta.attn_cache_fwd(q, c, pages[:1], lens),
        lambda: ta.attn_cache_fwd(q, c, pages, lens, lens.cpu()),
        lambda: ta.attn_cache_fwd(q, c, pages, lens, tree=tree[:, :2]),
        lambda: ta.attn_cache_fwd(q, c, pages, lens, tree=tree.float()),
        lambda: ta.attn_cache_fwd(q, c, pages, lens, tree=tree.transpose(1, 2)),
        lambda: ta.attn_cache_fwd(q, c, pages, lens, o=q[:, :1].expand(2, 4, 3, 64)),
        lambda: ta.attn_cache_fwd(q, c, pages, lens, lse=torch.zeros(2, 4, 2, device="cuda")),
        lambda: ta.cache_append(c, k, k[:, :1], pages, lens),
        lambda: ta.cache_append(c, k, k.half(), pages, lens),
        lambda: ta.cache_read(c, pages, lens, 8, dtype=torch.float32),
        lambda: ta.cache_read(c, pages, lens, 8, k=torch.zeros(2, 2, 9, 64, device="cuda", dtype=torch.bfloat16)),
        lambda: ta.cache_keep(c, pages, lens, lens, pages, lens[:1]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: ta.attn_cache_fwd(q[:, :3], c, pages, lens),              # 3 query heads, 2 key heads
                 lambda: ta.attn_cache_fwd(q.half(), c, pages, lens),              # a bf16 cache
                 lambda: ta.cache_append(c, k.half(), k.half(), pages, lens),
                 lambda: ta.attn_cache_fwd(q, c, pages, lens, ws=torch.zeros(64, device="cuda", dtype=torch.uint8))):
        with pytest.raises(ta.TAError):
            call()
    assert ta.sync_status() == "TA_OK"


@pytest.fixture
def guarded(gpu_lib):
    """The binding, pointed at the library with the device-side checks."""
    from tiled_attention_tcgen05_gb300 import build
    ta = gpu_lib
    saved, ta._lib = ta._lib, None
    try:
        assert ta.load(build.build(guard=True)).ta_guard_build() == 1
        yield ta
    finally:
        ta._lib = saved


@pytest.mark.parametrize("cache,dtype,D", [("bf16", "bf16", 128), ("f16", "f16", 32), ("e4m3", "bf16", 64),
                                           ("int8", "f16", 128), ("e4m3", "f16", 16)])
def test_guard_build(guarded, cache, dtype, D):
    """Every check of the operands passes where shapes have their edges."""
    ta = guarded
    for Hkv, G, T, kv, ql, page in ((2, 3, 1, [1, 300], None, 16), (3, 4, 75, [75, 500], [75, 9], 24),
                                    (1, 2, 40, [41, 129, 0], [40, 1, 0], 8)):
        st = Setup(ta, kv, Hkv, page, D, dtype, cache, 3)
        q = values(3, (len(kv), Hkv * G, T, D), dtype)
        k = values(4, (len(kv), Hkv, T, D), dtype).cuda()
        o, lse = attend(ta, st, q, ql, None, torch.zeros_like(q).cuda(), torch.zeros(len(kv), Hkv * G, T, device="cuda"))
        assert ta.sync_status() == "TA_OK", ta.load().ta_guard_last()
        compare_attention(st, q, o, lse, ql, None)
        lists = None if ql is None else int32(ql)
        ta.cache_append(st.cache, k, k, st.pages, st.kv_lens, lists)
        ta.cache_read(st.cache, st.pages, st.kv_lens, max(kv) + 5, dtype=TORCH[dtype])
        ta.cache_keep(st.cache, st.pages, st.kv_lens, lists, int32([0] * len(kv) * T).view(len(kv), T),
                      int32([min(1, n) for n in (ql or [T] * len(kv))]))
        assert ta.sync_status() == "TA_OK", ta.load().ta_guard_last()
