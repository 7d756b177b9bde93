"""Attention over a cache whose keys and values lie far apart, or are no numbers:
infinities and NaN among older tokens and the draft's, scales of very different
size, queries of very different size, values that a row does not see."""
import numpy as np
import pytest
import torch

import oracle
from _cache import Setup, attention_reference, check, int32, values
from _parity import to_np
from test_gpu_cache import attend

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def put(ta, st, b, k, v):
    """Writes sequence b of the setup anew: k, v [Hkv, n, D] on the host."""
    n = st.kv[b]
    ta.cache_append(st.cache, k[None].cuda(), v[None].cuda(), st.pages[b:b + 1], int32([n]))
    for name, x in (("k", k), ("v", v)):
        if st.scale[name] is None:
            st.rows[name][b] = x.double().numpy()
            continue
        c, s = oracle.cache_quantise(x, st.kind)
        st.rows[name][b] = c * s.astype(np.float64)[..., None]
        slots = [oracle.cache_slot(st.table[b], st.page, i) for i in range(n)]
        pg, r = (torch.tensor(z) for z in zip(*slots))
        st.scale[name][pg, :, r] = torch.from_numpy(s).T


def compare(st, q, o, lse, tree=None, heads=None, columns=None, rows=None, b=0):
    """Rows (default: all) and columns of O against the oracle, and L.

    The bounds are those of products on the bare codes whatever the number of
    rows: nothing in them comes from a key that a row does not see, but for the
    weights' half steps, which the row's largest contribution scales."""
    G, n = q.shape[1] // st.Hkv, q.shape[2]
    for h in range(st.Hkv) if heads is None else heads:
        vs = None
        if st.scale["v"] is not None:
            vs = np.array([st.scale["v"][pg, h, r] for pg, r in
                           (oracle.cache_slot(st.table[b], st.page, i) for i in range(st.kv[b]))], dtype=np.float64)
        v = np.where(np.isfinite(st.rows["v"][b][h]), st.rows["v"][b][h], 0.0)
        O, L, bO, bL = attention_reference(q[b, h * G:(h + 1) * G].cpu(), st.rows["k"][b][h], v, tree, st.kind, st.dtype,
                                           vs, rows=1)
        got, gl = to_np(o[b, h * G:(h + 1) * G]), to_np(lse[b, h * G:(h + 1) * G])
        r = np.arange(n) if rows is None else np.asarray(rows)
        c = np.arange(st.D) if columns is None else np.asarray(columns)
        check(f"O[{b},{h}]", got[:, r][:, :, c], O[:, r][:, :, c], bO[:, r][:, :, c])
        check(f"L[{b},{h}]", gl[:, r], L[:, r], bL[:, r])


def place(st, b, n):
    return oracle.cache_slot(st.table[b], st.page, n)


# ------------------------------------------- infinities and NaN, 16-bit caches
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("T,G", [(3, 4), (12, 8), (40, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_non_finite_values_of_older_tokens(gpu_lib, D, dtype, T, G, tree):
    """Every row sees the tokens before the new ones, those that share a key tile
    with new ones among them."""
    ta = gpu_lib
    n = 333
    st = Setup(ta, [n], 2, 16, D, dtype, dtype, 5)
    q = values(3, (1, 2 * G, T, D), dtype, 0.7)
    past = n - T
    tr = np.tril(np.ones((T, T), dtype=bool)) if tree else None
    for pos in (past - 1, past // 128 * 128, past - 129):
        pg, r = place(st, 0, pos)
        kept = st.cache.v[pg, :, r].clone()
        st.cache.v[pg, 0, r, 3] = NAN
        st.cache.v[pg, 1, r, 5] = INF
        o, lse = attend(ta, st, q, None, None if tr is None else tr[None])
        assert ta.sync_status() == "TA_OK"
        f = o.float().cpu()
        assert torch.isnan(f[0, :G, :, 3]).all(), pos
        assert not torch.isfinite(f[0, G:, :, 5]).any(), pos  # (0 * inf where a weight rounds to nothing)
        compare(st, q, o, lse, tr, heads=[0], columns=[c for c in range(D) if c != 3])
        compare(st, q, o, lse, tr, heads=[1], columns=[c for c in range(D) if c != 5])
        st.cache.v[pg, :, r] = kept


@pytest.mark.parametrize("T,G", [(3, 2), (24, 1), (40, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_non_finite_values_of_new_tokens_with_tiny_weights(gpu_lib, dtype, T, G):
    """A row that sees an infinity or a NaN gets it, however far below the row's
    maximum its score lies."""
    ta = gpu_lib
    D, n = 64, 200
    st = Setup(ta, [n], 1, 16, D, dtype, dtype, 6)
    k, v = (torch.from_numpy(st.rows[x][0]).to(q16(dtype)) for x in "kv")
    k[:, n - T + 1] = -20.0
    v[:, n - T + 1, 2], v[:, n - T + 1, 7] = NAN, INF
    put(ta, st, 0, k, v)
    q = values(3, (1, G, T, D), dtype, 0.1) + 2.0
    o, lse = attend(ta, st, q)
    assert ta.sync_status() == "TA_OK"
    f = o.float()
    assert torch.isfinite(f[:, :, 0]).all()
    assert torch.isnan(f[:, :, 1:, 2]).all() and (f[:, :, 1:, 7] == INF).all()
    compare(st, q, o, lse, columns=[c for c in range(D) if c not in (2, 7)])


def q16(dtype):
    return {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,G,T,n,high", [
    (1, 1, 32, 140, 25),      # rows of one tile, keys over a cluster's blocks
    (45, 1, 32, 140, 25),     # units cut by block borders
    (400, 1, 32, 140, 25),    # whole units
    (1, 1, 32, 19990, 25),    # one unit over all blocks
    (1, 2, 64, 150, 50),      # 128 rows, cut
    (200, 2, 64, 150, 50),    # 128 rows, whole
    (1, 1, 300, 310, 295),    # a pair of row tiles and one alone
])
def test_infinities_outlive_a_larger_maximum(gpu_lib, dtype, Hkv, G, T, n, high):
    """An infinity among the draft's first values, and a later key whose score
    lies so far above that everything before it weighs nothing."""
    ta = gpu_lib
    D = 64
    st = Setup(ta, [n], Hkv, 16, D, dtype, dtype, 6) if n < 1000 and Hkv < 100 else blank(ta, n, Hkv, D, dtype)
    k, v = values(11, (Hkv, n, D), dtype), values(12, (Hkv, n, D), dtype)
    v[:, n - T, 7] = INF
    k[:, n - T + high] = 20.0
    put(ta, st, 0, k, v)
    q = values(3, (1, Hkv * G, T, D), dtype, 0.1) + 2.0
    o, lse = attend(ta, st, q)
    assert ta.sync_status() == "TA_OK"
    f = o.float()
    assert (f[..., 7] == INF).all()
    compare(st, q, o, lse, columns=[c for c in range(D) if c != 7], heads=sorted({0, Hkv // 2, Hkv - 1}))


def blank(ta, n, Hkv, D, dtype, cache=None):
    """A setup whose one sequence put() fills (a long one's rows take the
    setup's own loop too long)."""
    st = Setup(ta, [0], Hkv, 16, D, dtype, cache or dtype, 6)
    P = (n + 15) // 16
    st.kv, st.table = [n], torch.arange(P, dtype=torch.int32).flip(0)[None].contiguous()
    st.cache = ta.kv_cache(P, Hkv, 16, D, st.cache.dtype)
    st.pages, st.kv_lens = st.table.cuda(), int32([n])
    if st.scale["v"] is not None:
        st.scale = {x: torch.zeros(P, Hkv, 16) for x in "kv"}
    return st


# ---------------------------------------------------- scales of 8-bit caches
@pytest.mark.parametrize("order", ["zeros first", "zeros last", "mixed"])
@pytest.mark.parametrize("size", [2.0 ** 30, 2.0 ** 80, 2.0 ** 118])
@pytest.mark.parametrize("Hkv,G,T", [(1, 1, 1), (1, 4, 3), (40, 1, 1), (400, 2, 1), (1, 4, 40), (200, 1, 70)])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_rows_of_zeros_beside_large_values(gpu_lib, cache, Hkv, G, T, size, order):
    """The softmax's sum does not depend on the values: keys whose values are
    zeros (their scale is 2^-60) keep their weight in it."""
    ta = gpu_lib
    D, n = 64, 300
    st = blank(ta, n, Hkv, D, "bf16", cache)
    k, v = values(11, (Hkv, n, D), "bf16"), values(12, (Hkv, n, D), "bf16")
    i = torch.arange(n)
    zero = {"zeros first": i < 170, "zeros last": i >= 130, "mixed": i % 2 == 0}[order]
    v = torch.where(zero[None, :, None], torch.zeros_like(v), v * size)
    put(ta, st, 0, k, v)
    q = values(3, (1, Hkv * G, T, D), "bf16")
    o, lse = attend(ta, st, q)
    assert ta.sync_status() == "TA_OK"
    compare(st, q, o, lse, heads=sorted({0, Hkv // 2, Hkv - 1}))


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("T,G", [(3, 4), (40, 4), (70, 2)])
@pytest.mark.parametrize("cache,dtype", [("e4m3", "bf16"), ("int8", "bf16")])
def test_large_values_that_rows_do_not_use(gpu_lib, cache, dtype, T, G, size):
    """A large value that the draft's tree hides from all rows but its own, and one
    of an older token whose weight is far below all others: the other rows'
    results are as exact as without them."""
    ta = gpu_lib
    D, n = 64, 300
    st = blank(ta, n, 1, D, dtype, cache)
    k, v = values(11, (1, n, D), dtype), values(12, (1, n, D), dtype)
    hidden = 1
    v[:, n - T + hidden] *= size
    k[:, 40], v[:, 40] = -30.0, v[:, 40] * size  # scores about -480 below
    put(ta, st, 0, k, v)
    tree = np.tril(np.ones((T, T), dtype=bool))
    tree[:, hidden] = False
    tree[hidden, hidden] = True
    q = values(3, (1, G, T, D), dtype, 0.1) + 2.0
    o, lse = attend(ta, st, q, None, tree[None])
    assert ta.sync_status() == "TA_OK"
    compare(st, q, o, lse, tree)


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("T,G", [(1, 4), (3, 4), (40, 4), (70, 2)])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_one_large_query_beside_ordinary_ones(gpu_lib, cache, T, G, size):
    ta = gpu_lib
    D, n = 128, 300
    st = blank(ta, n, 1, D, "bf16", cache)
    put(ta, st, 0, values(11, (1, n, D), "bf16"), values(12, (1, n, D), "bf16"))
    q = values(3, (1, G, T, D), "bf16")
    q[0, 1, T // 2] *= size
    q[0, 0, 0] *= 1 / size
    o, lse = attend(ta, st, q)
    assert ta.sync_status() == "TA_OK"
    compare(st, q, o, lse)


@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 118, 2.0 ** 124.5, 2.0 ** -40, 2.0 ** -50])
@pytest.mark.parametrize("T,G", [(1, 4), (3, 4), (40, 4), (70, 2)])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_large_keys_and_small_queries(gpu_lib, cache, T, G, size):
    """Keys and queries far outside fp16's range whose scores are ordinary."""
    ta = gpu_lib
    D, n = 128, 300
    st = blank(ta, n, 1, D, "bf16", cache)
    put(ta, st, 0, values(11, (1, n, D), "bf16") * size, values(12, (1, n, D), "bf16"))
    q = values(3, (1, G, T, D), "bf16") * (1 / size)
    o, lse = attend(ta, st, q)
    assert ta.sync_status() == "TA_OK"
    compare(st, q, o, lse)


@pytest.mark.parametrize("T,G", [(4, 4), (40, 4)])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_negative_value_scales_are_no_numbers(gpu_lib, cache, T, G):
    """A row that sees a value with a negative scale gets NaN; others keep
    every bit."""
    ta = gpu_lib
    D, n = 64, 150
    st = Setup(ta, [n], 1, 16, D, "bf16", cache, 6)
    tree = np.tril(np.ones((T, T), dtype=bool))
    tree[2:, 1] = False
    q = values(3, (1, G, T, D), "bf16")
    o, lse = attend(ta, st, q, None, tree[None])
    pg, r = place(st, 0, n - T + 1)
    for x in (-1.0, -2.0 ** -70, -INF):
        st.cache.v_scale[pg, 0, r] = x
        o2, lse2 = attend(ta, st, q, None, tree[None])
        assert ta.sync_status() == "TA_OK"
        own = torch.arange(T) == 1
        assert torch.isnan(o2[:, :, own].float()).all() and torch.isnan(lse2[:, :, own]).all(), x
        assert torch.equal(o2[:, :, ~own], o[:, :, ~own]) and torch.equal(lse2[:, :, ~own], lse[:, :, ~own]), x


# ------------------------------------------------------------ batches, streams
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("int8", "f16")])
@pytest.mark.parametrize("T,G", [(1, 4), (5, 4), (40, 4)])
def test_a_sequence_alone_and_in_a_batch(gpu_lib, cache, dtype, T, G):
    """Other sequences beside it move a result by rounding only (its keys are
    cut at other places, short tables go to another form of the kernel)."""
    ta = gpu_lib
    kv = [900, T + 20, 411, T] + [64 + 9 * i for i in range(40)]
    st = Setup(ta, kv, 2, 16, 64, dtype, cache, 3)
    q = values(3, (len(kv), 2 * G, T, 64), dtype)
    o, lse = attend(ta, st, q)
    for b in (0, 1, 2, 3, 43):
        need = (kv[b] + 15) // 16
        o1, l1 = ta.attn_cache_fwd(q[b:b + 1].cuda(), st.cache, st.pages[b:b + 1, :need].contiguous(), int32([kv[b]]))
        assert ta.sync_status() == "TA_OK"
        for h in range(2):
            _, _, bO, bL = attention_reference(q[b, h * G:(h + 1) * G], st.rows["k"][b][h], st.rows["v"][b][h], None, cache,
                                               dtype, None if st.scale["v"] is None else np.array(
                                                   [st.scale["v"][pg, h, r] for pg, r in
                                                    (place(st, b, i) for i in range(kv[b]))], dtype=np.float64), rows=1)
            part = slice(h * G, (h + 1) * G)
            assert (np.abs(to_np(o[b, part]) - to_np(o1[0, part])) <= 2 * bO).all()
            assert (np.abs(to_np(lse[b, part]) - to_np(l1[0, part])) <= 2 * bL).all()


def test_outputs_made_for_another_stream(gpu_lib):
    """A call on another stream makes its outputs and workspace out of that
    stream's memory: memory that the current stream has freed may still be
    written to by what runs there."""
    ta = gpu_lib
    st = Setup(ta, [64, 40], 2, 16, 64, "bf16", "int8", 3)
    q = values(3, (2, 8, 3, 64), "bf16").cuda()
    ql, keep, kl = int32([3, 3]), int32([0, 1, 2] * 2).view(2, 3), int32([2, 1])
    calls = (lambda s: ta.cache_read(st.cache, st.pages, st.kv_lens, 64, stream=s),
             lambda s: ta.attn_cache_fwd(q, st.cache, st.pages, st.kv_lens, stream=s),
             lambda s: (ta.cache_keep(st.cache, st.pages, st.kv_lens, ql, keep, kl, stream=s),))
    side = torch.cuda.Stream()
    for call in calls:
        ref = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        # what the call will allocate on the current stream, freed with writes pending
        for _ in range(3):
            pending = [torch.empty_like(t) for t in ref]
            torch.cuda._sleep(200_000_000)
            for t in pending:
                t.fill_(77)
            del pending, t
            out = call(side)
            side.synchronize()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert ta.sync_status() == "TA_OK"


def test_page_tables_without_a_column(gpu_lib):
    """Sequences that hold nothing, and so need no page."""
    ta = gpu_lib
    for cache in (torch.bfloat16, torch.int8):
        c = ta.kv_cache(2, 2, 16, 64, cache)
        pages, none = int32([]).view(2, 0), int32([0, 0])
        for T in (1, 40):
            q = torch.zeros(2, 8, T, 64, device="cuda", dtype=torch.bfloat16)
            o = torch.full_like(q, 3.0)
            ta.attn_cache_fwd(q, c, pages, none, none, o=o)
            assert (o == 3).all()
            ta.attn_cache_fwd(q, c, pages, none, int32([1, 1]), o=o)
            assert ta.sync_status() == "TA_ERR_INDEX" and (o == 3).all()
        k, _ = ta.cache_read(c, pages, none, 5)
        assert (k == 0).all() and ta.sync_status() == "TA_OK"
