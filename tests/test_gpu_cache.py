"""The key/value cache on the GPU against plain definitions in 64 bits:
append (quantising), read, keep, and attention of new tokens over the cache, at
the sizes and contents where they can go wrong."""
import random

import numpy as np
import pytest
import torch

import oracle
from _cache import Setup, TORCH, attention_reference, check, int32, page_table, random_tree, values
from _parity import ROUND_U, to_np

pytestmark = pytest.mark.gpu

NAN = float("nan")


def raw(t):
    """Bytes of a tensor, for comparisons that tell NaN and -0 apart."""
    return t.contiguous().view(torch.uint8).cpu()


# ------------------------------------------------------------------ append
APPEND = [
    # B, Hkv, page, D, T, kv_lens, q_lens (None: T each), dtype, cache, strided
    (1, 1, 16, 128, 1, [1], None, "bf16", "bf16", False),
    (3, 2, 16, 128, 1, [17, 16, 500], None, "bf16", "e4m3", True),
    (3, 5, 24, 64, 7, [7, 30, 100], [0, 7, 3], "f16", "int8", True),
    (2, 3, 1, 32, 5, [9, 5], [5, 4], "bf16", "int8", False),
    (4, 1, 33, 16, 40, [40, 66, 67, 0], [40, 33, 1, 0], "f16", "e4m3", True),
    (2, 2, 128, 128, 300, [300, 1000], None, "f16", "f16", True),
    (65, 4, 8, 64, 2, list(range(2, 67)), None, "bf16", "e4m3", False),
]


@pytest.mark.parametrize("B,Hkv,page,D,T,kv,ql,dtype,cache,strided", APPEND)
def test_append(gpu_lib, B, Hkv, page, D, T, kv, ql, dtype, cache, strided):
    ta = gpu_lib
    st = Setup(ta, kv, Hkv, page, D, dtype, cache, 5)
    before = [raw(t) for t in (st.cache.k, st.cache.v)]
    shape = (B, T, Hkv, D) if strided else (B, Hkv, T, D)
    x = [values(11 + i, shape, dtype, 3.0) for i in range(2)]
    for t in x:
        flat = t.view(-1, D)
        flat[0] = 0
        flat[-1] *= 2.0 ** -12
    g = [t.cuda() for t in x]
    if strided:
        x, g = [t.transpose(1, 2) for t in x], [t.transpose(1, 2) for t in g]
    ta.cache_append(st.cache, g[0], g[1], st.pages, st.kv_lens, None if ql is None else int32(ql))
    assert ta.sync_status() == "TA_OK"
    q = [T] * B if ql is None else ql
    for i, (name, t, sc) in enumerate((("k", st.cache.k, st.cache.k_scale), ("v", st.cache.v, st.cache.v_scale))):
        want = st.cpu[name].clone()
        wscale = None if sc is None else st.scale[name].clone()
        for b in range(B):
            if not q[b]:
                continue
            if sc is None:
                code = x[i][b, :, :q[b]]
            else:
                c, s = oracle.cache_quantise(x[i][b, :, :q[b]], cache)
                code = torch.from_numpy(c).float().to(want.dtype)
            for j in range(q[b]):
                pg, r = oracle.cache_slot(st.table[b], page, kv[b] - q[b] + j)
                want.view(torch.uint8)[pg, :, r] = code[:, j].contiguous().view(torch.uint8).reshape(Hkv, -1)
                if sc is not None:
                    wscale[pg, :, r] = torch.from_numpy(s)[:, j]
        # every byte: the rows written, and all others as they were
        assert torch.equal(raw(t), raw(want)), f"{name} differs"
        if sc is not None:
            assert torch.equal(raw(sc), raw(wscale)), f"{name}_scale differs"
    assert len(before) == 2


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_extreme_rows(gpu_lib, cache, dtype):
    """Zeros, the type's largest and smallest values, infinities, NaN, and
    values that lie halfway between two codes."""
    ta = gpu_lib
    D, T = 64, 12
    fi = torch.finfo(TORCH[dtype])
    x = values(1, (1, 1, T, D), dtype)
    x[0, 0, 0] = 0
    x[0, 0, 1] = fi.max
    x[0, 0, 2] = fi.smallest_normal
    x[0, 0, 3, 5] = float("inf")
    x[0, 0, 4, 6] = -float("inf")
    x[0, 0, 5, 7] = NAN
    x[0, 0, 6, 8], x[0, 0, 6, 9] = NAN, float("inf")
    x[0, 0, 7] = -0.0
    x[0, 0, 8] = (torch.arange(D) - 31.5).to(x.dtype)
    x[0, 0, 8, 0] = oracle.CACHE_QMAX[cache]  # scale 1 (e4m3: 448 exactly): ties stay ties
    x[0, 0, 9] = torch.finfo(TORCH[dtype]).tiny / 4
    x[0, 0, 10] = 1
    c = ta.kv_cache(1, 1, 16, D, TORCH[cache])
    pages, lens = int32([0]).view(1, 1), int32([T])
    ta.cache_append(c, x.cuda(), x.cuda(), pages, lens)
    k, v = ta.cache_read(c, pages, lens, T + 2, dtype=TORCH[dtype])
    assert ta.sync_status() == "TA_OK"
    code, scale = oracle.cache_quantise(x[0, 0], cache)
    assert np.array_equal(c.k[0, 0, :T].float().cpu().double().numpy(), code)
    assert np.array_equal(c.k_scale[0, 0, :T].cpu().numpy(), scale, equal_nan=True)
    back = torch.from_numpy(code * scale.astype(np.float64)[:, None]).to(TORCH[dtype])
    for t in (k, v):
        assert np.array_equal(to_np(t[0, 0, :T]), to_np(back), equal_nan=True)
        assert (t[0, 0, T:] == 0).all()


# -------------------------------------------------------------------- read
@pytest.mark.parametrize("Hkv,page,D,kv,N,dtype,cache", [
    (1, 16, 128, [1], 1, "bf16", "bf16"),
    (2, 24, 64, [0, 100, 23, 24], 101, "f16", "int8"),
    (3, 1, 16, [5, 40], 30, "bf16", "e4m3"),        # N inside a sequence
    (2, 64, 32, [300, 7], 333, "f16", "f16"),
    (4, 128, 128, [513], 600, "f16", "e4m3"),
])
def test_read(gpu_lib, Hkv, page, D, kv, N, dtype, cache):
    ta = gpu_lib
    st = Setup(ta, kv, Hkv, page, D, dtype, cache, 9)
    k, v = ta.cache_read(st.cache, st.pages, st.kv_lens, N, dtype=TORCH[dtype])
    assert ta.sync_status() == "TA_OK"
    for t, name in ((k, "k"), (v, "v")):
        want = np.zeros((len(kv), Hkv, N, D))
        for b, n in enumerate(kv):
            want[b, :, :min(n, N)] = st.rows[name][b][:, :N]
        got = to_np(t)
        assert got.shape == want.shape
        # one rounding of the product: half a step, plus half fp16's smallest step; fp32's own rounding before it
        u = ROUND_U[dtype] * (1 + 2.0 ** -12)
        assert (np.abs(got - want) <= u * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 0)).all()


# -------------------------------------------------------------------- keep
@pytest.mark.parametrize("Hkv,page,D,dtype,cache,T,kv,ql,keep", [
    (1, 16, 128, "bf16", "bf16", 4, [4], None, [[0, 2, 3]]),
    (3, 5, 64, "f16", "int8", 9, [30, 9, 12], [9, 8, 0], [[8], [0, 1, 2, 3, 4, 5, 6, 7], []]),
    (2, 32, 128, "bf16", "e4m3", 64, [64, 100, 65], None, [list(range(0, 64, 2)), [0, 3, 9, 27], list(range(1, 64))]),
    (2, 1, 16, "f16", "e4m3", 5, [7], None, [[1, 2, 4]]),
    # more rows than one round moves: every source lies where a later round has written already or will
    (1, 16, 128, "bf16", "bf16", 300, [310], None, [list(range(1, 300))]),
    (1, 8, 16, "bf16", "int8", 2000, [2000], None, [[i for i in range(2000) if i % 3]]),
])
def test_keep(gpu_lib, Hkv, page, D, dtype, cache, T, kv, ql, keep):
    ta = gpu_lib
    st = Setup(ta, kv, Hkv, page, D, dtype, cache, 13)
    B = len(kv)
    q = [T] * B if ql is None else ql
    kt = torch.full((B, T), -7, dtype=torch.int32)
    for b, p in enumerate(keep):
        kt[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    new = ta.cache_keep(st.cache, st.pages, st.kv_lens, None if ql is None else int32(ql), kt.cuda(),
                        int32(len(p) for p in keep))
    assert ta.sync_status() == "TA_OK"
    assert new.tolist() == [n - m + len(p) for n, m, p in zip(kv, q, keep)]
    for name, t, sc in (("k", st.cache.k, st.cache.k_scale), ("v", st.cache.v, st.cache.v_scale)):
        want = st.cpu[name].clone().view(torch.uint8)
        ws = None if sc is None else st.scale[name].clone()
        for b, p in enumerate(keep):
            first = kv[b] - q[b]
            for i, j in enumerate(p):
                (dp, dr), (sp, sr) = (oracle.cache_slot(st.table[b], page, first + x) for x in (i, j))
                want[dp, :, dr] = st.cpu[name].view(torch.uint8)[sp, :, sr]
                if ws is not None:
                    ws[dp, :, dr] = st.scale[name][sp, :, sr]
        assert torch.equal(raw(t).view(-1), want.reshape(-1)), f"{name} differs"
        if ws is not None:
            assert torch.equal(raw(sc), raw(ws))


# --------------------------------------------------------------- attention
def attend(ta, st, q, ql=None, tree=None, o=None, lse=None, **kw):
    return ta.attn_cache_fwd(q.cuda() if not q.is_cuda else q, st.cache, st.pages, st.kv_lens,
                             None if ql is None else int32(ql),
                             tree=None if tree is None else torch.from_numpy(np.asarray(tree)).cuda(), o=o, lse=lse,
                             **kw)


def compare_attention(st, q, o, lse, ql, tree, seqs=None, sm_scale=None):
    """Every row of the given sequences against the oracle."""
    B, Hq, T, D = q.shape
    G = Hq // st.Hkv
    for b in range(B) if seqs is None else seqs:
        n = T if ql is None else ql[b]
        if n == 0:
            continue
        tr = None if tree is None else np.asarray(tree)[b if len(tree) > 1 else 0][:n, :n]
        for h in range(st.Hkv):
            vs = None
            if st.scale["v"] is not None:
                vs = np.array([st.scale["v"][pg, h, r] for pg, r in
                               (oracle.cache_slot(st.table[b], st.page, i) for i in range(st.kv[b]))], dtype=np.float64)
            O, L, bO, bL = attention_reference(q[b, h * G:(h + 1) * G, :n], st.rows["k"][b][h], st.rows["v"][b][h], tr,
                                               st.kind, st.dtype, vs, sm_scale, G * T)
            check(f"O[{b},{h}]", o[b, h * G:(h + 1) * G, :n], O, bO)
            check(f"L[{b},{h}]", lse[b, h * G:(h + 1) * G, :n], L, bL)


ATTN = [
    # Hkv, G, page, D, T, kv_lens, q_lens, dtype, cache, tree
    (1, 1, 16, 128, 1, [1], None, "bf16", "bf16", False),              # one key
    (2, 4, 16, 128, 1, [1, 2, 63, 64, 65, 700], None, "bf16", "bf16", False),
    (2, 7, 24, 128, 1, [15, 16, 17, 300], None, "f16", "f16", False),
    (1, 16, 64, 64, 1, [129, 1000], None, "bf16", "e4m3", False),
    (3, 17, 16, 64, 1, [40, 333], None, "f16", "int8", False),         # rows past one tile
    (2, 2, 1, 32, 3, [3, 100, 31], [3, 1, 2], "bf16", "int8", False),
    (5, 1, 33, 16, 1, [500, 1], None, "f16", "e4m3", False),
    (2, 3, 16, 128, 9, [9, 50, 200], [9, 0, 5], "bf16", "e4m3", True),
    (2, 4, 32, 64, 33, [33, 34, 161], None, "f16", "int8", True),
    (1, 8, 16, 128, 16, [16, 400], None, "bf16", "bf16", True),
    (2, 1, 128, 128, 130, [130, 517], [129, 130], "f16", "f16", False),
    (1, 4, 16, 32, 70, [70, 90], None, "bf16", "bf16", True),
    (1, 2, 8, 16, 65, [65, 300], [64, 65], "f16", "f16", True),
    (2, 4, 64, 64, 200, [200, 456], None, "bf16", "bf16", False),
    (1, 5, 16, 128, 100, [777, 100], [100, 99], "bf16", "int8", False),
    (1, 2, 16, 128, 257, [300], None, "f16", "e4m3", True),
    (4, 2, 16, 64, 1, [2000] + [3] * 40, None, "bf16", "e4m3", False),  # one long among short
]


@pytest.mark.parametrize("Hkv,G,page,D,T,kv,ql,dtype,cache,tree", ATTN)
def test_attention(gpu_lib, Hkv, G, page, D, T, kv, ql, dtype, cache, tree):
    ta = gpu_lib
    B = len(kv)
    st = Setup(ta, kv, Hkv, page, D, dtype, cache, 21)
    q = values(3, (B, Hkv * G, T, D), dtype, 1.5)
    rng = random.Random(7)
    tr = np.stack([random_tree(rng, T) for _ in range(B)]) if tree else None
    o = torch.full_like(q, 7.0).cuda()
    lse = torch.full((B, Hkv * G, T), 7.0, device="cuda")
    attend(ta, st, q, ql, tr, o, lse)
    assert ta.sync_status() == "TA_OK"
    compare_attention(st, q, o, lse, ql, tr)
    if ql is not None:  # rows behind a sequence's new tokens are left as they were
        for b, n in enumerate(ql):
            assert (o[b, :, n:] == 7).all() and (lse[b, :, n:] == 7).all()


def test_attention_layouts_and_scale(gpu_lib):
    """Queries and results as projections lay them out, an expanded query, a
    given scale, a tree shared by the batch: the same bits as contiguous."""
    ta = gpu_lib
    B, Hkv, G, T, D = 3, 2, 3, 4, 64
    st = Setup(ta, [40, 70, 4], Hkv, 16, D, "bf16", "bf16", 4)
    q = values(3, (B, Hkv * G, T, D), "bf16").cuda()
    tree = random_tree(random.Random(1), T)[None]
    o, lse = attend(ta, st, q, None, tree, sm_scale=0.3)
    compare_attention(st, q.cpu(), o, lse, None, tree, sm_scale=0.3)
    wide = torch.empty(B, T, Hkv * G + 2, D, device="cuda", dtype=q.dtype)
    qs = wide[:, :, 1:-1].transpose(1, 2)
    qs.copy_(q)
    o2 = torch.zeros(B, T, Hkv * G, D, device="cuda", dtype=q.dtype).transpose(1, 2)
    attend(ta, st, qs, None, np.repeat(tree, B, 0), o=o2, sm_scale=0.3)
    assert torch.equal(o, o2)
    one = q[:, :1, :, :].expand(B, Hkv * G, T, D)
    oe, le = attend(ta, st, one, None, tree)
    oc, lc = attend(ta, st, one.contiguous(), None, tree)
    assert torch.equal(oe, oc) and torch.equal(le, lc) and oe.is_contiguous()
    assert ta.sync_status() == "TA_OK"


@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("int8", "f16")])
@pytest.mark.parametrize("T,G", [(4, 1), (4, 4), (40, 4)])
def test_rows_that_see_nothing_and_hidden_non_finite(gpu_lib, cache, dtype, T, G):
    """A draft with no tokens before it: rows whose mask is empty give O = 0,
    L = -inf; keys and values with infinities and NaN reach exactly the rows
    that see them."""
    ta = gpu_lib
    D, Hkv = 64, 2
    st = Setup(ta, [T, T + 20], Hkv, 16, D, dtype, cache, 6)
    bad = values(8, (2, Hkv, T, D), dtype)
    bad[:, :, 1, 3] = float("inf")
    bad[:, :, 2, 5] = NAN
    ta.cache_append(st.cache, values(9, (2, Hkv, T, D), dtype).cuda(), bad.cuda(), st.pages, st.kv_lens)
    tree = np.tril(np.ones((T, T), dtype=bool))
    tree[:, 1:3] = False      # nobody sees the two ...
    tree[3, 1] = True         # ... but one row the infinity
    tree[0] = False           # and one row nothing at all
    tree = np.stack([tree, tree])
    q = values(3, (2, Hkv * G, T, D), dtype).cuda()
    o, lse = attend(ta, st, q, None, tree)
    assert ta.sync_status() == "TA_OK"
    assert (o[0, :, 0] == 0).all() and torch.isneginf(lse[0, :, 0]).all()
    hit = torch.zeros(T, dtype=torch.bool)
    hit[3] = True
    assert torch.isfinite(o[:, :, ~hit].float()).all()
    assert torch.isfinite(lse[:, :, ~hit & (torch.arange(T) > 0)]).all()
    if cache in ("e4m3", "int8"):
        assert torch.isnan(o[:, :, 3].float()).all()  # the row reads back as NaN whole
        assert torch.isnan(lse[:, :, 3]).all()
    else:
        f = o[:, :, 3].float()
        assert torch.isinf(f[..., 3]).all()
        assert torch.isfinite(torch.cat([f[..., :3], f[..., 4:]], -1)).all()
    # the other rows are those of a cache without the bad values
    clean = torch.where(torch.isfinite(bad.float()), bad, torch.zeros_like(bad))
    ta.cache_append(st.cache, values(9, (2, Hkv, T, D), dtype).cuda(), clean.cuda(), st.pages, st.kv_lens)
    o2, _ = attend(ta, st, q, None, tree)
    assert torch.equal(o[:, :, ~hit], o2[:, :, ~hit])


def test_scores_of_extreme_size(gpu_lib):
    """Scores far outside the exponential's range, both signs, and a key type's
    largest values: the softmax stays a softmax."""
    ta = gpu_lib
    D = 64
    for cache, dtype in (("bf16", "bf16"), ("e4m3", "bf16"), ("int8", "f16")):
        st = Setup(ta, [300], 1, 16, D, dtype, cache, 31, gain=20.0)
        q = values(3, (1, 4, 1, D), dtype, 30.0)
        o, lse = attend(ta, st, q)
        assert ta.sync_status() == "TA_OK"
        compare_attention(st, q, o, lse, None, None)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_value_rows_of_very_different_size(gpu_lib, cache, order, T):
    """Values from 2^-25 to 2^18 (and a row of zeros) beside each other: the
    scales' range does not cost the small ones their weight in the sum."""
    ta = gpu_lib
    D, N = 64, 700
    st = Setup(ta, [N], 1, 16, D, "bf16", cache, 2)
    k = values(1, (1, 1, N, D), "bf16")
    v = values(2, (1, 1, N, D), "bf16")
    # tile by tile larger (or smaller), and every size inside each
    steps = torch.arange(N) // 50
    size = (steps if order > 0 else steps.flip(0)) + torch.arange(N) % 31 - 25.0
    v = v * torch.exp2(size)[None, None, :, None].to(v.dtype)
    v[0, 0, 7] = 0
    k[0, 0, 7] = 3.0
    ta.cache_append(st.cache, k.cuda(), v.cuda(), st.pages, st.kv_lens)
    for name, x in (("k", k), ("v", v)):
        c, s = oracle.cache_quantise(x[0], cache)
        st.rows[name] = [c * s.astype(np.float64)[..., None]]
        for i in range(N):
            pg, r = oracle.cache_slot(st.table[0], 16, i)
            st.scale[name][pg, :, r] = torch.from_numpy(s)[:, i]
    q = values(3, (1, 3, T, D), "bf16", 2.0)
    q[0, 0] = 2.0  # prefers the row of zeros
    o, lse = attend(ta, st, q)
    assert ta.sync_status() == "TA_OK"
    compare_attention(st, q, o, lse, None, None)


# ------------------------------------------------------- used together
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int8"])
def test_prompt_steps_draft_and_keep(gpu_lib, cache):
    """A prompt in two chunks, a step, a draft verified and cut to its accepted
    path, the next step: each attention equals attention over what the cache
    holds by then, and what is read back is what the cache attends to."""
    ta = gpu_lib
    B, Hkv, G, D, page = 2, 2, 3, 64, 16
    P = 30
    rng = random.Random(5)
    c = ta.kv_cache(P, Hkv, page, D, TORCH[cache])
    table, _ = page_table(rng, [12, 12])
    pages = table.cuda()
    held = [0, 0]

    def new(T, ql, seed):
        q = values(seed, (B, Hkv * G, T, D), "bf16").cuda()
        k, v = (values(seed + i, (B, T, Hkv, D), "bf16").cuda().transpose(1, 2) for i in (1, 2))
        for b in range(B):
            held[b] += ql[b]
        lens, qls = int32(held), int32(ql)
        ta.cache_append(c, k, v, pages, lens, qls)
        return q, lens, qls

    def verify(q, ql, o, lse, tree=None):
        N = max(held)
        k, v = ta.cache_read(c, pages, int32(held), N, dtype=torch.bfloat16)
        for b in range(B):
            n = ql[b]
            for h in range(Hkv):
                O, L = oracle.cache_attention(to_np(q[b, h * G:(h + 1) * G, :n]), to_np(k[b, h, :held[b]]),
                                              to_np(v[b, h, :held[b]]), None if tree is None else tree[b][:n, :n])
                # read back rounded to bf16 where the cache's rows are not: 2^-8 of scores and values
                err = 2.0 ** -6 if cache == "bf16" else 2.0 ** -4
                assert np.abs(to_np(o[b, h * G:(h + 1) * G, :n]) - O).max() <= err
                assert np.abs(to_np(lse[b, h * G:(h + 1) * G, :n]) - L).max() <= err

    for T, ql, seed in ((50, [50, 37], 1), (20, [11, 20], 11), (1, [1, 1], 21)):
        q, lens, qls = new(T, ql, seed)
        o, lse = ta.attn_cache_fwd(q, c, pages, lens, qls)
        verify(q, ql, o, lse)
    T = 12
    trees = np.stack([random_tree(rng, T, 0.0) for _ in range(B)])
    q, lens, qls = new(T, [12, 9], 31)
    o, lse = ta.attn_cache_fwd(q, c, pages, lens, qls, tree=torch.from_numpy(trees).cuda())
    verify(q, [12, 9], o, lse, trees)
    paths = [np.flatnonzero(trees[0, 11]).tolist(), np.flatnonzero(trees[1, 8]).tolist()]
    keep = torch.zeros(B, T, dtype=torch.int32)
    for b, p in enumerate(paths):
        keep[b, :len(p)] = torch.tensor(p)
    k0, v0 = ta.cache_read(c, pages, lens, max(held))
    lens2 = ta.cache_keep(c, pages, lens, qls, keep.cuda(), int32(len(p) for p in paths))
    k1, v1 = ta.cache_read(c, pages, lens2, max(held))
    for b, p in enumerate(paths):
        first = held[b] - [12, 9][b]
        rows = list(range(first)) + [first + j for j in p]
        assert lens2[b] == len(rows)
        assert torch.equal(k1[b, :, :len(rows)], k0[b][:, rows]) and torch.equal(v1[b, :, :len(rows)], v0[b][:, rows])
        held[b] = len(rows)
    q, lens, qls = new(1, [1, 1], 41)
    o, lse = ta.attn_cache_fwd(q, c, pages, lens, qls)
    verify(q, [1, 1], o, lse)
    # the same queries over whole tensors: the framework's own forward, for one head per key head
    k, v = ta.cache_read(c, pages, lens, min(held))
    assert ta.sync_status() == "TA_OK"
    of, lf = ta.attn_fwd(q[:1, ::G].contiguous(), *(x[:1, :, :held[0]].contiguous() for x in
                                                    ta.cache_read(c, pages, lens, max(held))))
    assert (of.float() - o[:1, ::G].float()).abs().max() <= 2.0 ** -4
    assert (lf - lse[:1, ::G]).abs().max() <= 2.0 ** -4


def test_states_merge(gpu_lib):
    """Attention over two caches' keys joined by attn_merge_fwd is attention
    over both: L has the framework's convention."""
    ta = gpu_lib
    D = 128
    st = Setup(ta, [300], 2, 16, D, "bf16", "bf16", 3)
    q = values(3, (1, 8, 1, D), "bf16").cuda()
    o, lse = attend(ta, st, q)
    half = st.pages[:, 10:].contiguous()
    parts = [ta.attn_cache_fwd(q, st.cache, p, int32([n])) for p, n in ((st.pages, 160), (half, 140))]
    om, lm = ta.merge_fwd(*parts[0], *parts[1])
    assert ta.sync_status() == "TA_OK"
    assert (lm - lse).abs().max() <= 1e-4
    # three more roundings to bf16 of values up to their largest
    assert (om.float() - o.float()).abs().max() <= 3 * 2.0 ** -8 * float(o.float().abs().max())


def test_results_do_not_depend_on_the_batch_beside(gpu_lib):
    """Two runs of one call are equal bit by bit, on a busy GPU too, and a
    sequence's result moves by rounding only when others join the batch."""
    ta = gpu_lib
    st = Setup(ta, [900, 20, 411], 2, 16, 64, "bf16", "e4m3", 3)
    q = values(3, (3, 8, 1, 64), "bf16").cuda()
    o, lse = attend(ta, st, q)
    side = torch.cuda.Stream()
    x = torch.randn(2048, 2048, device="cuda")
    for _ in range(5):
        with torch.cuda.stream(side):
            x = x @ x * 1e-3
        o2, lse2 = attend(ta, st, q)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    torch.cuda.synchronize()
    assert ta.sync_status() == "TA_OK"


# ----------------------------------------------- streams, graphs, bad pages
def test_other_stream_and_graph(gpu_lib):
    """Append, attention and keep captured on a side stream; a replay computes
    on what the captured buffers hold then: new lengths, tokens and pages."""
    ta = gpu_lib
    B, Hkv, G, D, T, page = 2, 2, 4, 128, 3, 16
    c = ta.kv_cache(40, Hkv, page, D, torch.int8)
    c.k.zero_(), c.v.zero_(), c.k_scale.fill_(1), c.v_scale.fill_(1)
    rng = random.Random(3)
    pages = page_table(rng, [15, 15])[0].cuda()
    lens, ql = int32([3, 3]), int32([3, 2])
    q = values(1, (B, Hkv * G, T, D), "bf16").cuda()
    k, v = (values(i, (B, Hkv, T, D), "bf16").cuda() for i in (2, 3))
    tree = torch.from_numpy(np.stack([random_tree(rng, T)] * B)).cuda()
    keep, kl = int32([0, 2, 0, 1, 0, 0]).view(B, T), int32([2, 1])
    o, lse = torch.zeros_like(q), torch.zeros(B, Hkv * G, T, device="cuda")
    ws = torch.empty(ta.attn_cache_workspace_bytes(B, Hkv * G, Hkv, T, 16 * page, D, torch.bfloat16, torch.int8),
                     device="cuda", dtype=torch.uint8)

    def step(stream=None):
        ta.cache_append(c, k, v, pages, lens, ql, stream=stream)
        ta.attn_cache_fwd(q, c, pages, lens, ql, tree=tree, o=o, lse=lse, ws=ws, stream=stream)
        return ta.cache_keep(c, pages, lens, ql, keep, kl, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    step(side)  # given as an argument, with another stream current
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        new = step()
    for i in range(4):
        state = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
        if i:
            lens.copy_(new + ql)
            q.copy_(values(10 + i, q.shape, "bf16"))
            k.copy_(values(20 + i, k.shape, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, lse, new, c.k, c.v, c.k_scale, c.v_scale)]
        for t, s in zip((c.k, c.v, c.k_scale, c.v_scale), state):
            t.copy_(s)
        n = step()
        for a, b in zip(got, (o, lse, n, c.k, c.v, c.k_scale, c.v_scale)):
            assert torch.equal(a, b)
    assert ta.sync_status() == "TA_OK"


def test_bad_pages_and_lengths_are_reported(gpu_lib):
    """Page ids and lengths outside the cache: skipped, reported, and the other
    sequences' results unharmed."""
    ta = gpu_lib
    D, T = 64, 2
    for cache in ("bf16", "int8"):
        st = Setup(ta, [40, 40, 40], 1, 16, D, "bf16", cache, 3)
        q = values(1, (3, 2, T, D), "bf16").cuda()
        k = values(2, (3, 1, T, D), "bf16").cuda()
        o, lse = attend(ta, st, q)
        good, gl = o.clone(), lse.clone()
        assert ta.sync_status() == "TA_OK"
        pages = st.pages.clone()
        P = st.cache.shape[0]
        for wrong in (P, -1, 2 ** 31 - 1, -2 ** 31):
            pages[1, 2] = wrong
            before = [raw(t) for t in (st.cache.k, st.cache.v)]
            o, lse = ta.attn_cache_fwd(q, st.cache, pages, st.kv_lens)
            assert ta.sync_status() == "TA_ERR_INDEX" and ta.sync_status() == "TA_OK"
            assert torch.equal(o[::2], good[::2]) and torch.equal(lse[::2], gl[::2])
            assert torch.isfinite(o.float()).all()
            kr, _ = ta.cache_read(st.cache, pages, st.kv_lens, 40, dtype=torch.bfloat16)
            assert ta.sync_status() == "TA_ERR_INDEX"
            assert (kr[1, :, 32:] == 0).all() and (kr[0, :, 32:] != 0).any()
            only = int32([0, 40, 0])
            ta.cache_append(st.cache, k, k, pages, only, int32([0, 2, 0]))  # both rows lie on the bad page
            assert ta.sync_status() == "TA_ERR_INDEX"
            ta.cache_keep(st.cache, pages, only, int32([0, 2, 0]), int32([0, 0, 1, 0, 0, 0]).view(3, 2), int32([0, 1, 0]))
            assert ta.sync_status() == "TA_ERR_INDEX"
            assert all(torch.equal(raw(t), s) for t, s in zip((st.cache.k, st.cache.v), before))
        cap = st.pages.shape[1] * 16
        for n, m in ((-1, 1), (1, 2), (40, 3), (40, -1), (cap + 1, 1), (2 ** 31 - 1, 1), (-2 ** 31, 0)):
            lens, ql = int32([40, n, 40]), int32([2, m, 2])
            o = torch.full_like(q, 5.0)
            ta.attn_cache_fwd(q, st.cache, st.pages, lens, ql, o=o)
            assert ta.sync_status() == "TA_ERR_INDEX"
            assert torch.equal(o[::2], good[::2]) and (o[1] == 5).all()
            before = [raw(t) for t in (st.cache.k, st.cache.v)]
            ta.cache_append(st.cache, k, k, st.pages, int32([0, n, 0]), int32([0, m, 0]))
            assert ta.sync_status() == "TA_ERR_INDEX"
            ta.cache_keep(st.cache, st.pages, int32([0, n, 0]), int32([0, m, 0]), int32([0] * 6).view(3, 2), int32([0, 1, 0]))
            assert ta.sync_status() == "TA_ERR_INDEX"
            assert all(torch.equal(raw(t), s) for t, s in zip((st.cache.k, st.cache.v), before))
        # lists that are not ascending, or leave the draft
        for lst, n in (([1, 0], 2), ([0, 0], 2), ([2, 0], 1), ([-1, 0], 1), ([0, 1], 3), ([0, 1], -1)):
            before = [raw(t) for t in (st.cache.k, st.cache.v)]
            new = ta.cache_keep(st.cache, st.pages, st.kv_lens, None, int32(lst * 3).view(3, 2), int32([0, n, 0]))
            assert ta.sync_status() == "TA_ERR_INDEX"
            assert new.tolist() == [38, 38, 38]
            assert all(torch.equal(raw(t), s) for t, s in zip((st.cache.k, st.cache.v), before))


def test_empty_calls(gpu_lib):
    ta = gpu_lib
    c = ta.kv_cache(4, 2, 16, 64, torch.bfloat16)
    e = torch.zeros(2, 2, 0, 64, device="cuda", dtype=torch.bfloat16)
    pages, lens = int32([0, 1, 2, 3]).view(2, 2), int32([5, 0])
    ta.cache_append(c, e, e, pages, lens)
    o, lse = ta.attn_cache_fwd(torch.zeros(2, 4, 0, 64, device="cuda", dtype=torch.bfloat16), c, pages, lens)
    assert o.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)
    none = int32([]).view(0, 2)
    z = torch.zeros(0, 2, 1, 64, device="cuda", dtype=torch.bfloat16)
    ta.cache_append(c, z, z, none, int32([]))
    assert ta.attn_cache_fwd(z, c, none, int32([]))[0].shape == z.shape
    assert ta.cache_read(c, pages, lens, 0)[0].shape == (2, 2, 0, 64)
    # sequences without new tokens only: nothing is written
    o = torch.full((2, 4, 3, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    ta.attn_cache_fwd(torch.zeros_like(o), c, pages, lens, int32([0, 0]), o=o)
    assert (o == 3).all()
    assert ta.cache_keep(c, pages, lens, int32([0, 0]), int32([]).view(2, 0), int32([0, 0])).tolist() == [5, 0]
    assert ta.sync_status() == "TA_OK"


def test_rows_past_two_to_the_thirty_one_elements(gpu_lib):
    """Pages whose elements lie more than 2^31 (and whose bytes more than 2^32)
    from the start."""
    ta = gpu_lib
    D, Hkv, page = 128, 8, 64
    P = 2 ** 31 // (D * Hkv * page) + 600
    c = ta.kv_cache(P, Hkv, page, D, torch.bfloat16)
    N, T = 300, 2
    pages = int32(range(P - 5, P)).view(1, 5)
    lens = int32([N])
    k, v = (values(i, (1, Hkv, N, D), "bf16").cuda() for i in (1, 2))
    ta.cache_append(c, k, v, pages, lens)
    kr, vr = ta.cache_read(c, pages, lens, N)
    assert torch.equal(kr, k) and torch.equal(vr, v)
    assert torch.equal(c.k[P - 5].float(), k[0, :, :page].float())
    q = values(3, (1, 16, T, D), "bf16")
    o, lse = ta.attn_cache_fwd(q.cuda(), c, pages, lens)
    assert ta.sync_status() == "TA_OK"
    for h in (0, 7):
        O, L, bO, bL = attention_reference(q[0, 2 * h:2 * h + 2], to_np(k[0, h]), to_np(v[0, h]), None, "bf16", "bf16")
        check("O", o[0, 2 * h:2 * h + 2], O, bO)
        check("L", lse[0, 2 * h:2 * h + 2], L, bL)
