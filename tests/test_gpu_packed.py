"""Attention of packed sequences with shared key heads, forward and backward,
against the fp64 oracle."""
import threading

import numpy as np
import pytest
import torch

import oracle
from _parity import to_np
from _prompt import TORCH, ints, offsets, packed_case, values, within

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def rows(cu):
    """Index of the rows that belong to a sequence."""
    return torch.arange(cu[0], cu[-1])


def make(seed, Tq, Tk, Hq, Hkv, D, dtype, fused=False, gain=1.0):
    if fused and Tq == Tk:
        x = values(seed, (Tq, Hq + 2 * Hkv, D), dtype, gain)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return (values(seed, (Tq, Hq, D), dtype, gain), values(seed + 1, (Tk, Hkv, D), dtype, gain),
            values(seed + 2, (Tk, Hkv, D), dtype))


def on_gpu(x):
    """A tensor's copy on the GPU, of the same strides for parts of a projection."""
    base = x._base if x._base is not None and x._base.dim() == 3 else None
    if base is None:
        return x.cuda()
    return torch.as_strided(base.cuda(), x.shape, x.stride(), x.storage_offset())


def run(ta, q, k, v, cu_q, cu_k, causal, do=None, sm_scale=None, **kw):
    """(o, lse (, dq, dk, dv)) written over 7s, so that untouched rows show."""
    q, k, v = (on_gpu(x) for x in (q, k, v))
    plan = ta.packed_plan(ints(cu_q), q.shape[0], q.shape[1], k.shape[1], causal, ints(cu_k), k.shape[0])
    full = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")
    o, lse = full(q), torch.full(q.shape[:2], 7.0, device="cuda")
    ta.attn_packed_fwd(q, k, v, plan, sm_scale, o=o, lse=lse, **kw)
    if do is None:
        return o, lse
    return (o, lse) + tuple(ta.attn_packed_bwd(q, k, v, o, lse, do.cuda(), plan, sm_scale, dq=full(q), dk=full(k),
                                               dv=full(v), **kw))


def check(ta, got, ref, bounds, cu_q, cu_k):
    assert ta.sync_status() == "TA_OK"
    for name, g, r, b, cu in zip(("O", "L", "dQ", "dK", "dV"), got, ref, bounds, (cu_q, cu_q, cu_q, cu_k, cu_k)):
        i = rows(cu)
        within(name, g.cpu()[i], r[i], b[i])
        rest = torch.ones(g.shape[0], dtype=torch.bool)
        rest[i] = False
        assert (g.cpu()[rest] == 7).all(), f"{name}: rows of no sequence"


def case(ta, lens, klens, Hq, Hkv, D, dtype, causal, bwd, fused=False, pad=3, seed=1, sm_scale=None):
    cu_q, cu_k = offsets(lens, pad and 2), offsets(klens, pad and 2)
    q, k, v = make(seed, cu_q[-1] + pad, cu_k[-1] + pad, Hq, Hkv, D, dtype, fused)
    do = values(seed + 7, tuple(q.shape), dtype) if bwd else None
    got = run(ta, q, k, v, cu_q, cu_k, causal, do, sm_scale)
    ref, bounds = packed_case(q, k, v, cu_q, cu_k, causal, dtype, do, sm_scale)
    check(ta, got, ref, bounds, cu_q, cu_k)


LENS = [1, 2, 0, 15, 16, 17, 127, 128, 129, 64, 200]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 4])
def test_lengths_around_the_tiles(gpu_lib, G, D, dtype, causal):
    case(gpu_lib, LENS, LENS, 2 * G, 2, D, dtype, causal, True, fused=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (10, 2), (6, 1), (7, 1), (16, 2), (33, 1), (64, 1), (71, 1),
                                    (128, 1), (9, 3)])
def test_heads_per_key_head(gpu_lib, Hq, Hkv, D):
    case(gpu_lib, [5, 70, 1, 140], [5, 70, 1, 140], Hq, Hkv, D, "bf16", True, True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 1), (3, 1)])
def test_long_sequences(gpu_lib, Hq, Hkv, D, dtype):
    """Enough tiles that every ring turns several times, ragged at the end."""
    case(gpu_lib, [1501, 900], [1501, 900], Hq, Hkv, D, dtype, True, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_keys_of_other_lengths(gpu_lib, D, G, causal):
    """More keys than queries (a prefix), fewer (rows that see nothing), none, and
    keys without queries (their gradients are zeros)."""
    case(gpu_lib, [10, 130, 300, 0, 5, 40, 257], [200, 130, 20, 60, 0, 167, 300], 2 * G, 2, D, "bf16", causal, True)


def test_scale(gpu_lib):
    case(gpu_lib, [100, 300], [100, 300], 4, 2, 64, "f16", True, True, sm_scale=0.31)
    case(gpu_lib, [100, 300], [100, 300], 4, 2, 64, "f16", True, True, sm_scale=-1.0)


def test_many_short_sequences(gpu_lib):
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 9, 1500)]
    case(gpu_lib, lens, lens, 4, 2, 64, "bf16", True, True)


def test_no_rows(gpu_lib):
    ta = gpu_lib
    for lens, klens in (([0, 0], [0, 0]), ([3, 0], [0, 0]), ([0, 0], [5, 130]), ([], [])):
        cu_q, cu_k = offsets(lens), offsets(klens)
        q, k, v = make(1, cu_q[-1], cu_k[-1], 4, 2, 64, "bf16")
        got = run(ta, q, k, v, cu_q, cu_k, True, torch.ones_like(q))
        assert ta.sync_status() == "TA_OK"
        assert not got[0].any() and not got[2].any() and not got[3].any() and not got[4].any()
        assert (got[1] == -INF).all()


def test_gradients_by_differences(gpu_lib):
    """<do, O> along random directions, by differences of the oracle's forward."""
    ta = gpu_lib
    cu = offsets([37, 1, 90])
    q, k, v = make(3, cu[-1], cu[-1], 6, 2, 64, "f16")
    do = values(9, tuple(q.shape), "f16")
    grads = run(ta, q, k, v, cu, cu, True, do)[2:]
    _, bounds = packed_case(q, k, v, cu, cu, True, "f16", do)
    x = [to_np(t) for t in (q, k, v)]
    loss = lambda *z: (to_np(do) * oracle.packed_attention(*z, cu, cu, True)[0]).sum()
    rng = np.random.default_rng(1)
    for i in range(3):
        t = rng.standard_normal(x[i].shape)
        h = 1e-4
        lo, hi = list(x), list(x)
        lo[i], hi[i] = x[i] - h * t, x[i] + h * t
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        got = (to_np(grads[i]) * t).sum()
        assert abs(got - want) <= (bounds[2 + i] * np.abs(t)).sum() + 1e-5 * abs(want)


# ------------------------------------------------ infinities and NaN, masked places
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (3, 64)])
def test_neighbours_of_no_number(gpu_lib, G, D, causal):
    """Every row around the sequences, and one whole sequence, is NaN or infinite; no
    other sequence's results or gradients know of it."""
    ta = gpu_lib
    lens = [50, 129, 33, 1, 300]
    cu = offsets(lens, 2)
    T = cu[-1] + 3
    q, k, v = make(1, T, T, 2 * G, 2, D, "bf16")
    do = values(8, tuple(q.shape), "bf16")
    ref, bounds = packed_case(q, k, v, cu, cu, causal, "bf16", do)
    bad = torch.ones(T, dtype=torch.bool)
    bad[cu[0]:cu[2]] = False
    bad[cu[3]:cu[-1]] = False
    for x, y in ((q, NAN), (k, INF), (v, NAN), (do, -INF)):
        x[bad] = y
    got = run(ta, q, k, v, cu, cu, causal, do)
    assert ta.sync_status() == "TA_OK"
    good = (~bad).nonzero()[:, 0]
    for name, g, r, b in zip(("O", "L", "dQ", "dK", "dV"), got, ref, bounds):
        within(name, g.cpu()[good], r[good], b[good])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G,D,n", [(1, 64, 300), (4, 128, 200), (8, 64, 50), (3, 128, 131), (1, 128, 520)])
def test_values_of_no_number_reach_the_rows_that_see_them(gpu_lib, G, D, n, dtype):
    ta = gpu_lib
    cu = offsets([n, 20])
    for at in sorted({0, 1, n // 2, n - 2, n - 1, 127 if n > 127 else 0, 128 if n > 128 else 0}):
        q, k, v = make(2, cu[-1], cu[-1], 2 * G, 2, D, dtype, gain=0.3)
        clean = v.clone()
        v[at, 0, 3], v[at, 1, 5], v[at, 1, 9] = NAN, INF, -INF
        clean[at, 0, 3] = clean[at, 1, 5] = clean[at, 1, 9] = 0
        o, lse = run(ta, q, k, v, cu, cu, True)
        assert ta.sync_status() == "TA_OK"
        f = o.float().cpu()
        assert torch.isnan(f[at:n, :G, 3]).all()
        assert (f[at:n, G:, 5] == INF).all() and (f[at:n, G:, 9] == -INF).all()
        ref, bounds = packed_case(q, k, clean, cu, cu, True, dtype)
        seen = np.zeros(ref[0].shape, dtype=bool)
        seen[at:n, :G, 3] = seen[at:n, G:, 5] = seen[at:n, G:, 9] = True
        within("O", np.where(seen, 0.0, to_np(o)), np.where(seen, 0.0, ref[0]), bounds[0])
        within("L", lse, ref[1], bounds[1])


def test_keys_of_no_number_reach_the_rows_that_see_them(gpu_lib):
    ta = gpu_lib
    n, at = 260, 140
    cu = offsets([n])
    q, k, v = make(2, n, n, 4, 2, 64, "bf16")
    k[at, 0, 3] = NAN
    o, lse = run(ta, q, k, v, cu, cu, True)
    assert ta.sync_status() == "TA_OK"
    assert torch.isnan(o[at:, :2]).all() and torch.isnan(lse[at:, :2]).all()
    k[at, 0, 3] = 0
    ref, bounds = packed_case(q, k, v, cu, cu, True, "bf16")
    within("O", o[:at], ref[0][:at], bounds[0][:at])
    within("O of the other key head", o[:, 2:], ref[0][:, 2:], bounds[0][:, 2:])


def test_scores_far_apart(gpu_lib):
    """A running maximum that jumps by more than the rescaling threshold, and rows
    whose other weights vanish."""
    ta = gpu_lib
    n = 400
    cu = offsets([n])
    q, k, v = make(4, n, n, 2, 1, 64, "bf16", gain=0.2)
    q += 1.0
    for at, size in ((100, 0.5), (200, 1.5), (300, 3.0)):
        k[at] = size
    do = values(8, tuple(q.shape), "bf16")
    got = run(ta, q, k, v, cu, cu, True, do)
    ref, bounds = packed_case(q, k, v, cu, cu, True, "bf16", do)
    check(ta, got, ref, bounds, cu, cu)


# --------------------------------------------------------- layouts and calls
def test_strides(gpu_lib):
    """Head-major tensors, parts of wider ones, and gradients into parts of one
    projection's gradient."""
    ta = gpu_lib
    cu = offsets([77, 200])
    T, Hq, Hkv, D = cu[-1], 6, 2, 64
    q, k, v = make(5, T, T, Hq, Hkv, D, "bf16")
    do = values(9, tuple(q.shape), "bf16")
    want = run(ta, q, k, v, cu, cu, True, do)
    plan = ta.packed_plan(ints(cu), T, Hq, Hkv)
    wide = torch.full((T, Hq + 2 * Hkv, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    qg = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)  # [heads, tokens, D] in memory
    kg = wide[:, :Hkv, :D]
    kg.copy_(k)
    vg = wide[:, 1:1 + Hkv, D:]
    vg.copy_(v)
    og = torch.full((Hq, T, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    o, lse = ta.attn_packed_fwd(qg, kg, vg, plan, o=og)
    grad = torch.full((T, Hq + 2 * Hkv + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    parts = grad[:, :Hq], grad[:, Hq:Hq + Hkv], grad[:, Hq + Hkv:-1]
    ta.attn_packed_bwd(qg, kg, vg, o, lse, do.cuda(), plan, dq=parts[0], dk=parts[1], dv=parts[2])
    assert ta.sync_status() == "TA_OK"
    for a, b in zip((o, lse) + parts, want):
        assert torch.equal(a, b)
    assert (grad[:, -1] == 7).all()


def test_same_bits_again_and_alone(gpu_lib):
    """A call's results do not depend on the order in which its tiles ran, nor a
    sequence's on the others in the batch."""
    ta = gpu_lib
    lens = [200, 31, 128, 500, 7]
    cu = offsets(lens)
    q, k, v = make(6, cu[-1], cu[-1], 8, 2, 64, "bf16")
    do = values(9, tuple(q.shape), "bf16")
    first = run(ta, q, k, v, cu, cu, True, do)
    for a, b in zip(first, run(ta, q, k, v, cu, cu, True, do)):
        assert torch.equal(a, b)
    for i, n in enumerate(lens):
        s = slice(cu[i], cu[i + 1])
        alone = run(ta, q[s].clone(), k[s].clone(), v[s].clone(), [0, n], [0, n], True, do[s])
        for a, b in zip(first, alone):
            assert torch.equal(a[s], b)


def test_equal_to_attn_fwd_up_to_rounding(gpu_lib):
    """One head per key head and equal lengths: the framework's own batched calls."""
    ta = gpu_lib
    B, H, S, D = 2, 3, 384, 128
    q, k, v = make(7, B * S, B * S, H, H, D, "bf16")
    do = values(9, tuple(q.shape), "bf16")
    cu = offsets([S] * B)
    got = run(ta, q, k, v, cu, cu, True, do)
    batch = lambda x: x.cuda().view(B, S, H, D).transpose(1, 2).contiguous()
    o, lse = ta.attn_fwd(*(batch(x) for x in (q, k, v)), True)
    grads = ta.attn_bwd(*(batch(x) for x in (q, k, v)), o, lse, batch(do), True)
    _, bounds = packed_case(q, k, v, cu, cu, True, "bf16", do)
    for name, a, b, e in zip(("O", "L", "dQ", "dK", "dV"), got, (o, lse) + tuple(grads), bounds):
        b = b.transpose(1, 2).reshape(a.shape)
        within(name, a, to_np(b), 2 * e)


def test_merged_with_another_key_set(gpu_lib):
    """Partial results over two key sets of each sequence, joined by merge_fwd."""
    ta = gpu_lib
    lens, left, right = [40, 129], [70, 10], [40, 129]
    cu, cl, cr = offsets(lens), offsets(left), offsets(right)
    q, kl, vl = make(8, cu[-1], cl[-1], 4, 2, 64, "f16")
    _, kr, vr = make(18, cu[-1], cr[-1], 4, 2, 64, "f16")
    ol, ll = run(ta, q, kl, vl, cu, cl, False)
    orr, lr = run(ta, q, kr, vr, cu, cr, True)
    o, lse = ta.merge_fwd(ol[None], ll[None], orr[None], lr[None])
    k = torch.cat([x for i in range(2) for x in (kl[cl[i]:cl[i + 1]], kr[cr[i]:cr[i + 1]])])
    v = torch.cat([x for i in range(2) for x in (vl[cl[i]:cl[i + 1]], vr[cr[i]:cr[i + 1]])])
    both = offsets([a + b for a, b in zip(left, right)])
    ref, bounds = packed_case(q, k, v, cu, both, True, "f16")
    # the parts' own roundings weigh at most as the whole's, and the merge rounds once more
    within("O", o[0], ref[0], 3 * bounds[0] + 2.0 ** -10 * np.abs(to_np(ol)).max())
    within("L", lse[0], ref[1], 3 * bounds[1])


def test_replayed_on_new_offsets(gpu_lib):
    """Plan, forward and backward captured once, replayed on other lengths; two
    captures share the inputs and have plans and workspaces of their own."""
    ta = gpu_lib
    T, Hq, Hkv, D = 400, 4, 2, 64
    q, k, v = (x.cuda() for x in make(9, T, T, Hq, Hkv, D, "bf16"))
    do = values(10, (T, Hq, D), "bf16").cuda()
    cu = ints(offsets([100, 200, 100]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        plan = ta.packed_plan(cu, T, Hq, Hkv)
        o, lse = ta.attn_packed_fwd(q, k, v, plan)
        return (o, lse) + ta.attn_packed_bwd(q, k, v, o, lse, do, plan)
    with torch.cuda.stream(side):
        step()
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(step())
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    new = offsets([1, 399, 0])
    cu.copy_(ints(new))
    q.copy_(values(11, (T, Hq, D), "bf16"))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = run(ta, q.cpu(), k.cpu(), v.cpu(), new, new, True, do.cpu())
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ta.sync_status() == "TA_OK"


def test_threads_on_streams_of_their_own(gpu_lib):
    ta = gpu_lib
    jobs = []
    for i in range(4):
        cu = offsets([30 + 50 * i, 128, 5])
        q, k, v = make(20 + i, cu[-1], cu[-1], 4, 2, 64 if i % 2 else 128, "bf16")
        jobs.append((q, k, v, cu, cu, True, values(30 + i, tuple(q.shape), "bf16")))
    want = [run(ta, *j) for j in jobs]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(3):
                got[i] = run(ta, *jobs[i], stream=s)
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_that_cannot_be(gpu_lib):
    ta = gpu_lib
    q, k, v = (x.cuda() for x in make(3, 20, 20, 2, 1, 64, "bf16"))
    for cu in ([0, 10, 21], [0, 10, 5], [-1, 10, 20], [0, 30, 20]):
        plan = ta.packed_plan(ints(cu), 20, 2, 1)
        assert ta.sync_status() == "TA_ERR_INDEX"
        o = torch.full_like(q, 7.0)
        ta.attn_packed_fwd(q, k, v, plan, o=o)
        assert ta.sync_status() == "TA_OK" and (o == 7).all()
    # a plan of other sizes than the call's
    plan, other = ta.packed_plan(ints([0, 20]), 20, 2, 1), ta.packed_plan(ints([0, 19]), 19, 2, 1)
    other.total = other.total_k = 20
    other._bytes = plan._bytes
    other._t = torch.nn.functional.pad(other._t, (0, plan._bytes - other._t.numel()))
    other._ptr = other._t.data_ptr()
    o = torch.full_like(q, 7.0)
    ta.attn_packed_fwd(q, k, v, other, o=o)
    assert ta.sync_status() == "TA_ERR_INDEX" and (o == 7).all()


def test_rows_past_two_to_the_31_elements(gpu_lib):
    ta = gpu_lib
    Hq, Hkv, D = 64, 8, 128
    T = 270000  # 2.2e9 elements of q
    lens = [50, T - 150, 100]
    cu = offsets(lens)
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    last = slice(cu[2], cu[3])
    a, b, c = make(3, 100, 100, Hq, Hkv, D, "bf16")
    q[last], k[last], v[last] = a.cuda(), b.cuda(), c.cuda()
    lse = torch.empty(T, Hq, device="cuda")
    do = torch.zeros_like(q)
    d = values(6, (100, Hq, D), "bf16")
    do[last] = d.cuda()
    # the middle sequence would take long: its queries belong to nobody here
    cu_q = torch.tensor([[0, 50], [cu[2], cu[3]]], dtype=torch.int32)
    for s in cu_q.tolist()[1:]:
        plan = ta.packed_plan(ints(s), T, Hq, Hkv)
        o, _ = ta.attn_packed_fwd(q, k, v, plan, lse=lse)
        grads = ta.attn_packed_bwd(q, k, v, o, lse, do, plan)
        assert ta.sync_status() == "TA_OK"
    one = [0, 100]
    ref, bounds = packed_case(a, b, c, one, one, True, "bf16", d)
    for name, g, r, e in zip(("O", "L", "dQ", "dK", "dV"), (o, lse) + tuple(grads), ref, bounds):
        within(name, g[last], r, e)
