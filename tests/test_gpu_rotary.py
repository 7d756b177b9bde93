"""Rotary positions, head norms with the rotation, and the write of rotated keys to a
cache, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from _parity import ROUND_U, to_np
from _prompt import TINY, TORCH, ints, partner, rotary_bound, values, within

pytestmark = pytest.mark.gpu

EPS = 1e-6


def tokens_first(x):
    """[tokens, heads, D] of a 3-D or 4-D tensor."""
    return x if x.dim() == 3 else x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])


def make(seed, layout, T, Hq, Hkv, D, dtype, gain=1.0):
    """q, k, v on the GPU: of their own, views of one projection, or [B, heads, T, D]."""
    if layout == "fused":
        x = values(seed, (T, Hq + 2 * Hkv, D), dtype, gain).cuda()
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if layout == "heads":
        B = 2 if T % 2 == 0 else 1
        return tuple(values(seed + i, (B, h, T // B, D), dtype, gain).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
    if layout == "turned":  # [B, T, heads, D] seen as [B, heads, T, D]
        B = 2 if T % 2 == 0 else 1
        return tuple(values(seed + i, (B, T // B, h, D), dtype, gain).cuda().transpose(1, 2)
                     for i, h in enumerate((Hq, Hkv, Hkv)))
    return tuple(values(seed + i, (T, h, D), dtype, gain).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))


def positions(rng, x, far):
    n = x.shape[0] if x.dim() == 3 else x.shape[0] * x.shape[2]
    p = torch.from_numpy(rng.integers(0, far, n).astype(np.int32))
    p[-1] = far - 1
    return (p if x.dim() == 3 else p.view(x.shape[0], x.shape[2])).cuda()


def weights(D, dtype, seed=9):
    g = torch.Generator().manual_seed(seed)
    return tuple((1 + 0.2 * torch.randn(D, generator=g)).to(torch.float32 if dtype == "f32" else TORCH[dtype])
                 for _ in range(2))


def check_rows(name, got, x, pos, rot, dtype, w=None, eps=EPS, back=False):
    """Rotated (and normed) rows of x against the oracle."""
    a = to_np(tokens_first(x))
    h = a if w is None else oracle.head_norm(a, to_np(w), eps)
    p = pos.reshape(-1).cpu().numpy()
    ref = oracle.rotary(h, p, rot.inv_freq, rot.interleaved, rot.scale, back)
    within(name, to_np(tokens_first(got)), ref,
           rotary_bound(h, ref, rot.dim, rot.interleaved, rot.scale, dtype, a.shape[-1], w is not None))
    return h, ref


SHAPES = [  # layout, tokens, Hq, Hkv, D, dim
    ("packed", 1, 1, 1, 128, 128),
    ("packed", 7, 5, 1, 128, 64),
    ("packed", 700, 32, 8, 128, 128),   # a warp per token
    ("fused", 33, 12, 4, 64, 64),
    ("fused", 5, 3, 3, 16, 16),
    ("fused", 40, 7, 1, 32, 16),
    ("heads", 64, 9, 3, 128, 96),
    ("turned", 10, 4, 2, 64, 24),       # halves of 12: partners read again
    ("heads", 31, 2, 1, 16, 8),         # halves of 4
    ("packed", 12, 2, 2, 32, 2),
    ("packed", 12, 2, 2, 64, 0),        # nothing turns
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout,T,Hq,Hkv,D,dim", SHAPES)
def test_rotation_and_its_backward(gpu_lib, layout, T, Hq, Hkv, D, dim, dtype, interleaved):
    ta = gpu_lib
    q, k, _ = make(3, layout, T, Hq, Hkv, D, dtype)
    rot = ta.Rotary(dim, interleaved=interleaved, scale=1.25)
    pos = positions(np.random.default_rng(5), q, 5000)
    qo, ko = ta.rotary_fwd(q, k, pos, rot)
    check_rows("q", qo, q, pos, rot, dtype)
    check_rows("k", ko, k, pos, rot, dtype)
    dq, dk = ta.rotary_bwd(q, k, pos, rot)
    check_rows("dq", dq, q, pos, rot, dtype, back=True)
    check_rows("dk", dk, k, pos, rot, dtype, back=True)
    assert ta.sync_status() == "TA_OK"
    # one side alone, and in place
    only, none = ta.rotary_fwd(q, None, pos, rot)
    assert none is None and torch.equal(only, qo)
    none, only = ta.rotary_fwd(None, k, pos, rot)
    assert none is None and torch.equal(only, ko)
    ta.rotary_fwd(q, k, pos, rot, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("scaling", [{}, dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                     dict(scaling="yarn", factor=16.0, first_len=4096)])
def test_far_positions(gpu_lib, scaling):
    """The angle's exact fraction of a turn, at positions where fp32 has lost whole turns."""
    ta = gpu_lib
    rot = ta.Rotary(128, **scaling)
    q, k, _ = make(4, "packed", 6, 3, 1, 128, "bf16")
    pos = ints([0, 1, 1000003, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1])
    qo, ko = ta.rotary_fwd(q, k, pos, rot)
    # the reference's own angles: position * f in fp64 is off by 2^-53 of up to 2^31 radians
    for name, got, x in (("q", qo, q), ("k", ko, k)):
        a = to_np(x)
        ref = oracle.rotary(a, pos.cpu().numpy(), rot.inv_freq, False, rot.scale)
        bound = rotary_bound(a, ref, 128, False, rot.scale, "bf16", 128, False)
        within(name, got, ref, bound + 2.0 ** -21 * (np.abs(a) + partner(a, 128, False)) * rot.scale)


def test_negative_positions_turn_back(gpu_lib):
    ta = gpu_lib
    rot = ta.Rotary(64)
    q, _, _ = make(4, "packed", 3, 2, 1, 64, "f16")
    a, _ = ta.rotary_fwd(q, None, ints([-5, -1, -70000]), rot)
    b, _ = ta.rotary_bwd(q, None, ints([5, 1, 70000]), rot)
    check_rows("q", a, q, ints([-5, -1, -70000]), rot, "f16")
    within("back", a, to_np(b), 2 * (rotary_bound(to_np(q), to_np(b), 64, False, 1.0, "f16", 64, False)))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,wt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("layout,T,Hq,Hkv,D,dim", SHAPES)
def test_norm_and_its_backward(gpu_lib, layout, T, Hq, Hkv, D, dim, dtype, wt, interleaved):
    ta = gpu_lib
    q, k, _ = make(6, layout, T, Hq, Hkv, D, dtype)
    wq, wk = weights(D, wt)
    rot = ta.Rotary(dim, interleaved=interleaved, scale=0.75)
    pos = positions(np.random.default_rng(6), q, 5000)
    qo, ko = ta.qk_norm_rotary_fwd(q, k, wq.cuda(), wk.cuda(), pos, rot, eps=EPS)
    check_rows("q", qo, q, pos, rot, dtype, wq)
    check_rows("k", ko, k, pos, rot, dtype, wk)
    gq, gk, _ = make(60, layout, T, Hq, Hkv, D, dtype)
    got = ta.qk_norm_rotary_bwd(gq, gk, q, k, wq.cuda(), wk.cuda(), pos, rot, eps=EPS)
    assert ta.sync_status() == "TA_OK"
    p = pos.reshape(-1).cpu().numpy()
    for name, dx, dw, x, g, w in (("q", got[0], got[2], q, gq, wq), ("k", got[1], got[3], k, gk, wk)):
        a, ga, wn = to_np(tokens_first(x)), to_np(tokens_first(g)), to_np(w)
        back = oracle.rotary(ga, p, rot.inv_freq, interleaved, rot.scale, back=True)
        ref, rw = oracle.head_norm_bwd(a, wn, EPS, back)
        r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + EPS)
        h = a * r
        # the rotated gradient as in rotary_bound, times w; h as a norm's row; their mean's D products
        size = (np.abs(ga) * max(rot.scale, 1.0) + partner(ga, dim, interleaved) * rot.scale)
        rel = 2.0 ** -21 + (2 * D + 64) * 2.0 ** -24
        mean = (size * np.abs(wn * h)).mean(-1, keepdims=True)
        within("d" + name, to_np(tokens_first(dx)), ref,
               r * rel * (size * np.abs(wn) + 2 * np.abs(h) * mean) + ROUND_U[dtype] * np.abs(ref) + TINY[dtype])
        rows = a.shape[0] * a.shape[1]
        assert dw.dtype == torch.float32
        within("dw" + name, dw, rw, (rel + rows * 2.0 ** -24) * (size * np.abs(h)).reshape(-1, D).sum(0))
    # the same bits again, and with the gradients written over
    again = ta.qk_norm_rotary_bwd(gq, gk, q, k, wq.cuda(), wk.cuda(), pos, rot, eps=EPS, dq_out=gq, dk_out=gk)
    assert all(torch.equal(x, y) for x, y in zip(got, again)) and torch.equal(gq, got[0])


def test_norm_of_extreme_rows(gpu_lib):
    """Squares past fp32's range, tiny rows, rows of zeros; an infinity or a NaN stays in its row."""
    ta = gpu_lib
    D = 64
    rot = ta.Rotary(32)
    x = values(8, (8, 1, D), "bf16")
    for i, size in enumerate((2.0 ** 100, 2.0 ** 124, 2.0 ** -100, 0.0)):
        x[i] *= size
    x[4, 0, 3], x[5, 0, 40] = float("inf"), float("nan")
    w = torch.ones(D)
    pos = ints(range(8))
    y, _ = ta.qk_norm_rotary_fwd(x.cuda(), None, w.cuda(), None, pos, rot, eps=EPS)
    good = [0, 1, 2, 3, 6, 7]
    check_rows("rows", y[good], x[good], pos[good], rot, "bf16", w)
    assert torch.isnan(y[4, 0, 3]) and torch.isnan(y[5]).all()
    g = values(9, (8, 1, D), "bf16")
    dx, _, dw, _ = ta.qk_norm_rotary_bwd(g[good].cuda(), None, x[good].cuda(), None, w.cuda(), None, pos[good], rot, eps=EPS)
    back = oracle.rotary(to_np(g[good]), pos[good].cpu().numpy(), rot.inv_freq, False, 1.0, back=True)
    ref, _ = oracle.head_norm_bwd(to_np(x[good]), np.ones(D), EPS, back)
    r = 1 / np.sqrt((to_np(x[good]) ** 2).mean(-1, keepdims=True) + EPS)
    # (gradients of rows of 2^100 and more are tiny numbers; they may flush to zero below 2^-126)
    within("dx", dx, ref, r * (4 * D) * 2.0 ** -21 + ROUND_U["bf16"] * np.abs(ref) + 2.0 ** -126)


def test_plain_rotation_keeps_infinities_in_their_pair(gpu_lib):
    ta = gpu_lib
    for interleaved, pair in ((False, (5, 21)), (True, (4, 5))):
        rot = ta.Rotary(32, interleaved=interleaved)
        x = values(8, (4, 2, 64), "f16")
        x[1, 0, 5], x[2, 1, 50] = float("inf"), float("nan")
        y, _ = ta.rotary_fwd(x.cuda(), None, ints([3, 4, 5, 6]), rot)
        bad = ~torch.isfinite(y.cpu())
        want = torch.zeros_like(bad)
        want[1, 0, list(pair)] = True
        want[2, 1, 50] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("cache", ["16", "e4m3", "int8"])
@pytest.mark.parametrize("layout,T,Hq,Hkv,D,dim,page", [
    ("fused", 1, 4, 1, 128, 128, 16), ("packed", 37, 6, 2, 64, 32, 24), ("heads", 20, 8, 8, 16, 16, 8),
    ("turned", 6, 3, 3, 32, 24, 5), ("fused", 300, 16, 4, 128, 128, 64),
])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append(gpu_lib, layout, T, Hq, Hkv, D, dim, page, dtype, cache, norm):
    ta = gpu_lib
    kind = dtype if cache == "16" else cache
    rng = np.random.default_rng(7)
    q, k, v = make(11, layout, T, Hq, Hkv, D, dtype)
    rot = ta.Rotary(dim)
    pos = positions(rng, q, 9000)
    P = -(-T // page) + 2
    slots = rng.permutation(P * page)[:T].astype(np.int32)
    if T > 3:
        slots[2] = -1
        slots[T - 1] = -7
    c = ta.kv_cache(P, Hkv, page, D, TORCH[kind])
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x55)
    for t in (c.k_scale, c.v_scale):
        if t is not None:
            t.fill_(-3.0)
    before = [None if t is None else t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    wq, wk = weights(D, dtype) if norm else (None, None)
    gpu = (lambda w: None if w is None else w.cuda())
    sl = torch.from_numpy(slots).cuda().view(pos.shape)
    qo = ta.rotary_append(c, q, k, v, pos, sl, rot, q_weight=gpu(wq), k_weight=gpu(wk), eps=EPS)
    assert ta.sync_status() == "TA_OK"
    check_rows("q", qo, q, pos, rot, dtype, wq)
    a = to_np(tokens_first(k))
    h = a if wk is None else oracle.head_norm(a, to_np(wk), EPS)
    p = pos.reshape(-1).cpu().numpy()
    kr = oracle.rotary(h, p, rot.inv_freq, False, 1.0)
    err = rotary_bound(h, kr, dim, False, 1.0, dtype, D, norm) - ROUND_U[dtype] * np.abs(kr) - TINY[dtype]
    vr = to_np(tokens_first(v))
    live = slots >= 0
    at = (torch.from_numpy(slots[live] // page).long(), torch.from_numpy(slots[live] % page).long())
    for name, t, scale, ref, e in (("k", c.k, c.k_scale, kr, err), ("v", c.v, c.v_scale, vr, 0 * vr)):
        got = to_np(t.cpu().float()[at[0], :, at[1]])
        ref, e = ref[live], e[live]
        if scale is None:
            within(name, got, ref, e + (ROUND_U[dtype] * np.abs(ref) + TINY[dtype]) * (name == "k"))
            continue
        s = to_np(scale.cpu()[at[0], :, at[1]])
        top = oracle.CACHE_QMAX[cache]
        rs = np.maximum(np.abs(ref).max(-1) / top, 2.0 ** -60)
        within(name + " scale", s, rs, e.max(-1) / top + 2.0 ** -22 * rs)
        # code * scale: half a step of the code (e4m3: 2^-4 of it, or of its least normal 2^-6), the input's
        # error, and the code's fp32 product with the rounded reciprocal
        step = s[..., None] * (0.5 if cache == "int8" else np.maximum(2.0 ** -4 * np.abs(got), 2.0 ** -10))
        within(name, got * s[..., None], ref, step * (1 + 2.0 ** -20) + e + 2.0 ** -21 * np.abs(ref))
    # nothing else was written
    for t, b in zip((c.k, c.v, c.k_scale, c.v_scale), before):
        if t is not None:
            t, b = t.clone().view(torch.uint8).view(*t.shape[:3], -1), b.view(torch.uint8).view(*t.shape[:3], -1)
            i, j = (x.cuda() for x in at)
            t[i, :, j] = b[i, :, j]
            assert torch.equal(t, b)


def test_append_of_what_is_no_number_and_of_slots_outside(gpu_lib):
    ta = gpu_lib
    c = ta.kv_cache(2, 1, 4, 64, torch.int8)
    c.k.fill_(9)
    c.k_scale.fill_(2.0)
    x = values(3, (4, 1, 64), "bf16").cuda()
    k = x.clone()
    k[1, 0, 3] = float("nan")
    k[2] = 0
    rot = ta.Rotary(64)
    ta.rotary_append(c, x, k, k, ints(range(4)), ints([0, 1, 2, 8]), rot)
    assert ta.sync_status() == "TA_ERR_INDEX" and ta.sync_status() == "TA_OK"
    assert torch.isnan(c.k_scale[0, 0, 1]) and not c.k[0, 0, 1].any()
    assert c.k_scale[0, 0, 2] == 2.0 ** -60 and not c.k[0, 0, 2].any()
    assert (c.k[0, 0, 3] == 9).all() and (c.k[1] == 9).all()


def test_values_go_to_the_cache_as_cache_append_writes_them(gpu_lib):
    ta = gpu_lib
    for ct in (torch.bfloat16, torch.float8_e4m3fn, torch.int8):
        q, k, v = make(5, "heads", 24, 4, 2, 128, "bf16")  # [2, heads, 12, D]
        a, b = ta.kv_cache(4, 2, 8, 128, ct), ta.kv_cache(4, 2, 8, 128, ct)
        for c in (a, b):
            c.k.view(torch.uint8).zero_(), c.v.view(torch.uint8).zero_()
        pages = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32).cuda()
        slots = torch.tensor([[(pages[s, n // 8] * 8 + n % 8).item() for n in range(12)] for s in range(2)],
                             dtype=torch.int32).cuda()
        ta.cache_append(a, k, v, pages, ints([12, 12]))
        ta.rotary_append(b, q, k, v, torch.zeros(2, 12, dtype=torch.int32).cuda(), slots, ta.Rotary(128))
        assert torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8))
        assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))  # position 0: nothing turns
        if ct is not torch.bfloat16:
            for s in range(2):
                i = slots[s].long()
                for x, y in ((a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
                    assert torch.equal(x[i // 8, :, i % 8], y[i // 8, :, i % 8])


def test_no_tokens(gpu_lib):
    ta = gpu_lib
    rot = ta.Rotary(64)
    q, k, p = (torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    pos = ints([])
    assert ta.rotary_fwd(q, k, pos, rot)[0].shape == (0, 4, 64)
    w = torch.ones(64, device="cuda")
    _, _, dw, dk = ta.qk_norm_rotary_bwd(q, k, q, k, w, w, pos, rot)
    assert not dw.any() and not dk.any()
    c = ta.kv_cache(1, 4, 4, 64)
    ta.rotary_append(c, q, k, p, pos, pos, rot)
    assert ta.sync_status() == "TA_OK"


def test_replayed_from_a_graph(gpu_lib):
    """A step's calls captured once and replayed on other values and positions; two
    captures of the weights' sums have workspaces of their own."""
    ta = gpu_lib
    rot = ta.Rotary(64)
    q, k, _ = make(5, "fused", 50, 8, 2, 64, "bf16")
    w = torch.ones(64, device="cuda")
    pos = ints(range(50))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs, graphs = [], []
    with torch.cuda.stream(side):
        ta.qk_norm_rotary_bwd(q, k, q, k, w, w, pos, rot)
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(ta.qk_norm_rotary_bwd(q, k, q, k, w, w, pos, rot) + ta.rotary_fwd(q, k, pos, rot))
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    q.copy_(values(77, q.shape, "bf16"))
    pos.add_(100000)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = ta.qk_norm_rotary_bwd(q, k, q, k, w, w, pos, rot) + ta.rotary_fwd(q, k, pos, rot)
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_past_two_to_the_31_elements(gpu_lib):
    ta = gpu_lib
    T, H, D = 140000, 128, 128  # 2.3e9 elements
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    rows = [0, 70000, T - 1]
    q[rows] = values(5, (3, H, D), "bf16").cuda()
    rot = ta.Rotary(128)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    y, _ = ta.rotary_fwd(q, None, pos, rot)
    check_rows("rows", y[rows], q[rows], pos[rows], rot, "bf16")
    assert not y[1:70000].any()
