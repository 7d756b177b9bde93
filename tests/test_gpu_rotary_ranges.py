"""Head norms with the rotation where a side has no heads, where a row's squares leave
fp32's range, and without eps; angles on another stream than their own."""
import numpy as np
import pytest
import torch

import oracle
from _parity import ROUND_U, to_np
from _prompt import TORCH, ints, partner, values, within
from test_gpu_rotary import EPS, check_rows, weights

pytestmark = pytest.mark.gpu


def call_c(ta, fn, cache=None, **kw):
    """A call of the C ABI on rows [tokens, heads, D] given by name, on the current stream."""
    rows = [kw.get(n) for n in ("q", "k", "v", "dq", "dk", "q_out", "k_out")]
    x = next(t for t in rows if t is not None)
    heads = [0 if t is None else t.shape[1] for t in rows[:2]]
    p = lambda n: 0 if kw.get(n) is None else kw[n].data_ptr()
    ws = kw.get("ws")
    rot, dt = kw["rotary"], 0 if x.dtype is torch.float16 else 1
    wt = next((w.dtype for w in (kw.get("q_weight"), kw.get("k_weight")) if w is not None), x.dtype)
    call = ta._ROT.pack(*[y for t in rows for y in ((0, 0, 0, 0) if t is None else ta._rows_arg(t))], p("positions"), 0, 1,
                        p("slots"), rot.turns.data_ptr(), p("q_weight"), p("k_weight"), p("dq_weight"), p("dk_weight"),
                        p("ws"), 0 if ws is None else ws.numel(), rot.dim, rot.interleaved, rot.scale, kw.get("eps", EPS), 1,
                        x.shape[0], *heads, x.shape[2], dt, 2 if wt is torch.float32 else dt)
    s = torch.cuda.current_stream().cuda_stream
    lib = ta.load()
    return getattr(lib, fn)(call, s) if cache is None else lib.attn_rotary_append(cache._ref, call, s)


@pytest.mark.parametrize("dim", [64, 32, 24])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_append_of_normed_keys_without_queries(gpu_lib, kind, dim):
    """A call with no queries norms its keys by the keys' weight."""
    ta = gpu_lib
    T, H, D, page = 21, 3, 64, 8
    rot = ta.Rotary(dim)
    q, k, v = (values(i, (T, H, D), "bf16").cuda() for i in (1, 2, 3))
    wq, wk = (w.cuda() for w in weights(D, "bf16"))
    pos = ints(range(5, 5 + T))
    slots = torch.from_numpy(np.random.default_rng(3).permutation(4 * page)[:T].astype(np.int32)).cuda()
    caches = [ta.kv_cache(4, H, page, D, TORCH[kind]) for _ in range(2)]
    for c in caches:
        for t in (c.k, c.v):
            t.view(torch.uint8).zero_()
        for t in (c.k_scale, c.v_scale):
            if t is not None:
                t.zero_()
    assert call_c(ta, "attn_rotary_append", caches[0], k=k, v=v, positions=pos, slots=slots, rotary=rot, k_weight=wk) == 0
    ta.rotary_append(caches[1], q, k, v, pos, slots, rot, wq, wk, eps=EPS)
    assert ta.sync_status() == "TA_OK"
    for x, y in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v), (caches[0].k_scale, caches[1].k_scale),
                 (caches[0].v_scale, caches[1].v_scale)):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    if kind == "bf16":
        i = slots.long()
        check_rows("k", caches[0].k[i // page, :, i % page], k, pos, rot, "bf16", wk)


def norm_case(ta, x, g, w, rot, eps, dtype="bf16"):
    """Forward and backward of rows x [tokens, heads, D] against the oracle."""
    T, H, D = x.shape
    pos = ints(range(T))
    y, _ = ta.qk_norm_rotary_fwd(x.cuda(), None, w.cuda(), None, pos, rot, eps=eps)
    check_rows("rows", y, x, pos, rot, dtype, w, eps)
    dx, _, dw, _ = ta.qk_norm_rotary_bwd(g.cuda(), None, x.cuda(), None, w.cuda(), None, pos, rot, eps=eps)
    assert ta.sync_status() == "TA_OK"
    a, ga, wn = to_np(x), to_np(g), to_np(w)
    back = oracle.rotary(ga, pos.cpu().numpy(), rot.inv_freq, rot.interleaved, rot.scale, back=True)
    ref, rw = oracle.head_norm_bwd(a, wn, eps, back)
    r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
    h = a * r
    # the rotated gradient as in rotary_bound, times w; h as a norm's row; their mean's D products
    size = np.abs(ga) + partner(ga, rot.dim, rot.interleaved)
    rel = 2.0 ** -21 + (2 * D + 64) * 2.0 ** -24
    mean = (size * np.abs(wn * h)).mean(-1, keepdims=True)
    # (a gradient below fp32's normal numbers may flush to zero)
    within("dx", dx, ref, r * rel * (size * np.abs(wn) + 2 * np.abs(h) * mean) + ROUND_U[dtype] * np.abs(ref) + 2.0 ** -126)
    within("dw", dw, rw, (rel + T * H * 2.0 ** -24) * (size * np.abs(h)).reshape(-1, D).sum(0))


@pytest.mark.parametrize("D,dim", [(16, 16), (64, 64), (128, 128), (128, 64), (64, 24)])
def test_norm_of_the_largest_rows(gpu_lib, D, dim):
    """Rows whose every element is near the type's largest number (bf16: 2^128)."""
    x = values(3, (6, 3, D), "bf16").sign() * 3.0e38
    x[3:] = values(4, (3, 3, D), "bf16") * 2.0 ** 125
    norm_case(gpu_lib, x.to(torch.bfloat16), values(5, (6, 3, D), "bf16"), weights(D, "f32")[0], gpu_lib.Rotary(dim), EPS)


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38])
@pytest.mark.parametrize("D,dim", [(16, 16), (64, 64), (128, 128), (128, 64), (64, 24)])
def test_norm_of_tiny_rows_without_eps(gpu_lib, D, dim, eps):
    """Rows whose squares fp32 does not hold, and an eps that does not outweigh them."""
    sizes = torch.tensor([2.0 ** -40, 2.0 ** -50, 2.0 ** -63, 2.0 ** -70, 2.0 ** -75, 2.0 ** -100, 2.0 ** -120, 2.0 ** -129])
    x = (values(3, (8, 4, D), "bf16").float() * sizes.view(-1, 1, 1)).to(torch.bfloat16)
    eps = float(np.float32(eps))
    # (gradients that leave the rows' ones below the type's largest number)
    norm_case(gpu_lib, x, values(5, (8, 4, D), "bf16", 2.0 ** -10), weights(D, "f32")[0], gpu_lib.Rotary(dim), eps)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,D,dim", [(1, 16, 16), (5, 128, 128), (3, 64, 64), (7, 64, 24), (1, 32, 16)])
def test_norm_without_eps_beside_rows_that_are_none(gpu_lib, H, D, dim, dtype):
    """Heads that do not fill a group of rows: what stands in the others' place is in no sum."""
    x, g = values(3, (9, H, D), dtype), values(5, (9, H, D), dtype)
    norm_case(gpu_lib, x, g, weights(D, "f32")[0], gpu_lib.Rotary(dim), 0.0, dtype)


@pytest.mark.parametrize("T", [0, 4])
def test_weights_of_no_heads_have_no_gradient(gpu_lib, T):
    ta = gpu_lib
    D = 64
    rot, pos = ta.Rotary(D), ints(range(T))
    x, none = values(3, (T, 2, D), "bf16").cuda(), torch.empty(T, 0, D, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(D, device="cuda")
    ws = torch.empty(max(1, ta.load().attn_qk_norm_rotary_bwd_workspace_bytes(D)), dtype=torch.uint8, device="cuda")
    for side in (0, 1):
        dw = torch.full((2, D), 7.0, device="cuda")
        rows = dict(k=x, dk=x.clone(), k_out=x.clone()) if side == 0 else dict(q=x, dq=x.clone(), q_out=x.clone())
        if T == 0:
            rows = dict(q=none, k=none)
        assert call_c(ta, "attn_qk_norm_rotary_bwd", positions=pos, rotary=rot, q_weight=w, k_weight=w, dq_weight=dw[0],
                      dk_weight=dw[1], ws=ws, **rows) == 0
        assert ta.sync_status() == "TA_OK"
        assert not dw[side].any()
    pair = lambda a: (x, none) if a else (none, x)
    for side in (0, 1):
        junk = [torch.full((2, D), float("nan"), device="cuda") for _ in range(8)]
        del junk
        got = ta.qk_norm_rotary_bwd(*pair(side), *pair(side), w, w, pos, rot)
        assert not got[2 + side].any() and torch.isfinite(got[3 - side]).all()


def test_angles_used_on_another_stream(gpu_lib):
    """The memory of a Rotary that is gone is given away only once the streams it was recorded on are done."""
    ta = gpu_lib
    T, H, D = 4096, 32, 128
    q, pos = values(3, (T, H, D), "bf16").cuda(), ints(range(T))
    want, _ = ta.rotary_fwd(q, None, pos, ta.Rotary(D))
    outs = [torch.empty_like(q) for _ in range(40)]
    torch.cuda.synchronize()
    makes, uses = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(makes):
        rot = ta.Rotary(D)
    uses.wait_stream(makes)
    rot.record_stream(uses)
    for o in outs:  # some milliseconds of work on the stream
        ta.rotary_fwd(q, None, pos, rot, q_out=o, stream=uses)
    del rot
    with torch.cuda.stream(makes):
        for _ in range(8):
            torch.zeros(D // 2, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    assert ta.sync_status() == "TA_OK"
    assert all(torch.equal(o, want) for o in outs)
