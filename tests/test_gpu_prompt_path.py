"""A server's steps as they are used: pages assigned, projections rotated on their way
into the cache, prompts attended packed, then tokens one by one over the cache."""
import numpy as np
import pytest
import torch

import oracle
from _parity import ROUND_U, to_np
from _prompt import ints, offsets, packed_bounds, values, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv,dim,interleaved", [(64, 8, 2, 64, False), (128, 6, 6, 64, True)])
def test_prompts_then_single_tokens(gpu_lib, D, Hq, Hkv, dim, interleaved):
    ta = gpu_lib
    page, num, width, steps = 8, 64, 12, 3
    lens = [13, 1, 40]
    B, eps = len(lens), 1e-6
    rot = ta.Rotary(dim, interleaved=interleaved)
    w = [(1 + 0.1 * values(5 + i, (D,), "bf16")).cuda() for i in range(2)]
    seqs = [values(20 + b, (n + steps, Hq + 2 * Hkv, D), "bf16") for b, n in enumerate(lens)]  # projections
    cache = ta.kv_cache(num, Hkv, page, D)
    pages = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count, kv = ints(range(num)), ints([num]), ints([0] * B)

    def split(x):
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    # the prompts, packed, with rows of padding behind them
    x = torch.cat([s[:n] for s, n in zip(seqs, lens)] + [torch.zeros(4, Hq + 2 * Hkv, D, dtype=torch.bfloat16)]).cuda()
    a = ta.cache_assign(pages, kv, ints(lens), free, count, page, x.shape[0])
    q, k, v = split(x)
    qr = ta.rotary_append(cache, q, k, v, a.positions, a.slots, rot, *w, eps=eps)
    _, kr = ta.qk_norm_rotary_fwd(None, k, None, w[1], a.positions, rot, eps=eps)
    plan = ta.packed_plan(a.cu_seqlens, x.shape[0], Hq, Hkv)
    outs = [ta.attn_packed_fwd(qr, kr, v, plan)]
    # what lies in the cache is what was attended
    ck, cv = ta.cache_read(cache, pages, a.kv_lens, max(lens))
    for b in range(B):
        s = slice(offsets(lens)[b], offsets(lens)[b + 1])
        assert torch.equal(ck[b, :, :lens[b]].transpose(0, 1), kr[s]) and torch.equal(cv[b, :, :lens[b]].transpose(0, 1), v[s])
    kv, count = a.kv_lens, a.free_count
    for i in range(steps):
        x = torch.stack([s[n + i] for s, n in zip(seqs, lens)]).cuda()
        a = ta.cache_assign(pages, kv, ints([1] * B), free, count, page, B)
        q, k, v = split(x)
        qr = ta.rotary_append(cache, q, k, v, a.positions, a.slots, rot, *w, eps=eps)
        o, lse = ta.attn_cache_fwd(qr.unsqueeze(2), cache, pages, a.kv_lens)
        outs.append((o[:, :, 0], lse[:, :, 0]))
        kv, count = a.kv_lens, a.free_count
    assert ta.sync_status() == "TA_OK"
    assert kv.tolist() == [n + steps for n in lens]

    for b, n in enumerate(lens):
        q, k, v = (to_np(t) for t in split(seqs[b]))
        pos = np.arange(n + steps)
        kw = (rot.inv_freq, interleaved, rot.scale)
        q = oracle.rotary(oracle.head_norm(q, to_np(w[0]), eps), pos, *kw)
        k = oracle.rotary(oracle.head_norm(k, to_np(w[1]), eps), pos, *kw)
        cu = [0, n + steps]
        O, L = oracle.packed_attention(q, k, v, cu, cu)
        t = [torch.from_numpy(z) for z in (q, k, v)]
        bO, bL = packed_bounds(*t, cu, cu, True, "bf16", O, L)
        # q and k are rounded to bf16 first: a score moves by 2 u s |q| |k|, O by twice that of |P| |V|
        u = ROUND_U["bf16"]
        mv = np.zeros(L.shape)
        for h in range(Hq):
            mv[:, h] = (2.1 * u * oracle.default_scale(D) * np.abs(q[:, h]) @ np.abs(k[:, h * Hkv // Hq]).T).max(1)
        bO, bL = bO + (2 * mv[..., None] + u) * np.abs(v).max(), bL + mv
        first = offsets(lens)[b]
        o = torch.cat([outs[0][0][first:first + n]] + [x[0][b:b + 1] for x in outs[1:]])
        lse = torch.cat([outs[0][1][first:first + n]] + [x[1][b:b + 1] for x in outs[1:]])
        within("O", o, O, bO)
        within("L", lse, L, bL)


def test_a_training_step(gpu_lib):
    """Norm, rotation and packed attention forward and backward, against differences
    of the whole through the oracle."""
    ta = gpu_lib
    lens, Hq, Hkv, D, eps = [30, 129, 2], 4, 2, 64, 1e-5
    cu = offsets(lens)
    T = cu[-1]
    x = values(1, (T, Hq + 2 * Hkv, D), "f16")
    do = values(2, (T, Hq, D), "f16")
    w = [(1 + 0.1 * values(5 + i, (D,), "f16")) for i in range(2)]
    pos = np.concatenate([np.arange(n) for n in lens])
    rot = ta.Rotary(D)
    g, wg, pg = x.cuda(), [t.cuda() for t in w], ints(pos)
    q, k, v = g[:, :Hq], g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:]
    plan = ta.packed_plan(ints(cu), T, Hq, Hkv)
    qr, kr = ta.qk_norm_rotary_fwd(q, k, *wg, pg, rot, eps=eps)
    o, lse = ta.attn_packed_fwd(qr, kr, v, plan)
    dx = torch.empty_like(g)
    dqr, dkr, _ = ta.attn_packed_bwd(qr, kr, v, o, lse, do.cuda(), plan, dv=dx[:, Hq + Hkv:])
    _, _, dwq, dwk = ta.qk_norm_rotary_bwd(dqr, dkr, q, k, *wg, pg, rot, eps=eps, dq_out=dx[:, :Hq],
                                           dk_out=dx[:, Hq:Hq + Hkv])
    assert ta.sync_status() == "TA_OK"

    def loss(x, wq, wk):
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        q = oracle.rotary(oracle.head_norm(q, wq, eps), pos, rot.inv_freq)
        k = oracle.rotary(oracle.head_norm(k, wk, eps), pos, rot.inv_freq)
        return (to_np(do) * oracle.packed_attention(q, k, v, cu, cu)[0]).sum()
    at = [to_np(x), to_np(w[0]), to_np(w[1])]
    rng = np.random.default_rng(3)
    h = 1e-4
    for i, got in enumerate((to_np(dx), to_np(dwq), to_np(dwk))):
        t = rng.standard_normal(at[i].shape)
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - h * t, at[i] + h * t
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        # five fp16 roundings on the way (q, k, P, dS, the gradients), each 2^-11 of its operand, random in sign
        # over the sum's terms: 8 standard deviations of their sizes
        size = np.sqrt(((got * t) ** 2).sum())
        assert abs((got * t).sum() - want) <= 8 * 5 * 2.0 ** -11 * max(size, np.abs(got).max()), (i, (got * t).sum(), want)
