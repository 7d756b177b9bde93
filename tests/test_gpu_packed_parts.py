"""Packed attention over one of several key sets, the backward with the O and L of all of
them, sequences with a single key, and infinite values whose weight has vanished."""
import numpy as np
import pytest
import torch

import oracle
from _parity import ROUND_U, to_np
from _prompt import TINY, ints, offsets, packed_case, values, within
from test_gpu_packed import INF, make, run

pytestmark = pytest.mark.gpu


def delta_bounds(q, k, v, cu, cu_k, do, u):
    """What errors of delta = <dO, O> by 3 u <|dO|, sum_j P_j |V_j|> add to dQ and dK: O's parts are each
    rounded, and their sum is, and none of them is larger than that sum of magnitudes."""
    qn, kn, vn, gn = (to_np(x) for x in (q, k, v, do))
    s, G = oracle.default_scale(q.shape[2], None), q.shape[1] // k.shape[1]
    dq, dk = np.zeros_like(qn), np.zeros_like(kn)
    for b in range(len(cu) - 1):
        a, t = slice(cu[b], cu[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(q.shape[1]):
            x, y = qn[a, h], kn[t, h // G]
            S = s * (x @ y.T)
            P = np.exp(S - S.max(1, keepdims=True))
            P /= P.sum(1, keepdims=True)
            e = 3 * u * P * (np.abs(gn[a, h]) * (P @ np.abs(vn[t, h // G]))).sum(1, keepdims=True)
            dq[a, h] += s * 1.1 * (e @ np.abs(y))
            dk[t, h // G] += s * 1.1 * (e.T @ np.abs(x))
    return dq, dk


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 1), (32, 2)])
def test_backward_over_a_part_of_the_keys(gpu_lib, D, G, dtype):
    """Gradients of one key set from O and L over two: P sums to less than one in it, also where
    it is a single key."""
    ta = gpu_lib
    lens, left, right = [3, 130, 1, 40], [1, 1, 1, 70], [5, 30, 1, 1]
    cu, cl, cr = offsets(lens), offsets(left), offsets(right)
    q, kl, vl = make(8, cu[-1], cl[-1], 2 * G, 2, D, dtype)
    _, kr, vr = make(18, cu[-1], cr[-1], 2 * G, 2, D, dtype)
    do = values(9, tuple(q.shape), dtype)
    k = torch.cat([x for i in range(4) for x in (kl[cl[i]:cl[i + 1]], kr[cr[i]:cr[i + 1]])])
    v = torch.cat([x for i in range(4) for x in (vl[cl[i]:cl[i + 1]], vr[cr[i]:cr[i + 1]])])
    both = offsets([a + b for a, b in zip(left, right)])
    at = [np.concatenate([np.arange(both[i], both[i] + left[i]) for i in range(4)]),
          np.concatenate([np.arange(both[i] + left[i], both[i + 1]) for i in range(4)])]
    parts = [run(ta, q, x, y, cu, c, False) for x, y, c in ((kl, vl, cl), (kr, vr, cr))]
    o, lse = (x[0] for x in ta.merge_fwd(*(x[None] for p in parts for x in p)))
    ref, bounds = packed_case(q, k, v, cu, both, False, dtype, do)
    more = delta_bounds(q, k, v, cu, both, do, ROUND_U[dtype])
    dqs = []
    g = do.cuda()
    for (kp, vp, cp), i in zip(((kl, vl, cl), (kr, vr, cr)), at):
        plan = ta.packed_plan(ints(cu), q.shape[0], 2 * G, 2, False, ints(cp), kp.shape[0])
        got = ta.attn_packed_bwd(q.cuda(), kp.cuda(), vp.cuda(), o, lse, g, plan)
        assert ta.sync_status() == "TA_OK"
        dqs.append(to_np(got[0]))
        # L carries two calls' errors and the merge's: three times the bounds of one call
        within("dK", got[1], ref[3][i], 3 * bounds[3][i] + more[1][i])
        within("dV", got[2], ref[4][i], 3 * bounds[4][i])
    # (each part's dQ is rounded, and may be larger than the sum: by its bounds and those of P <= 1 in it)
    size = sum(np.abs(x) for x in dqs)
    within("dQ", sum(dqs), ref[2], 3 * bounds[2] + more[0] + ROUND_U[dtype] * 1.01 * size + 2 * TINY[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 1), (16, 2), (32, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_scores_of_a_lone_key_have_no_gradient(gpu_lib, D, G, dtype, causal):
    """P = 1 whatever the score, so its gradient is zero, not what rounding leaves of dP - delta."""
    ta = gpu_lib
    lens, klens = [200, 5, 1, 130], [200, 1, 1, 1]
    cu, ck = offsets(lens), offsets(klens)
    q, k, v = make(6, cu[-1], ck[-1], 2 * G, 2, D, dtype, gain=3.0)
    v[ck[2], 0, :4] = torch.tensor([0.0, -0.0, 2.0 ** -24, -1.0])
    do = values(9, tuple(q.shape), dtype)
    got = run(ta, q, k, v, cu, ck, causal, do)
    assert ta.sync_status() == "TA_OK"
    ref, bounds = packed_case(q, k, v, cu, ck, causal, dtype, do)
    for name, g, r, b in zip(("O", "L", "dQ", "dK", "dV"), got, ref, bounds):
        within(name, g, r, b)
    dq, dk = got[2:4]
    assert not dq[cu[1]:].any() and not dk[ck[1]:].any()
    assert dq[1:cu[1]].any() and dk[:ck[1]].any()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("G,D", [(1, 64), (4, 128)])
def test_infinite_values_of_vanished_weights(gpu_lib, G, D, short, causal):
    """A row that sees an infinite value gets it, or NaN, whatever its weight; no other row knows of it."""
    ta = gpu_lib
    n = 300
    cu = offsets([n] + [1] * 4 * short)
    q, k, v = make(4, cu[-1], cu[-1], 2 * G, 2, D, "bf16", gain=0.1)
    q += 4.0
    k[0] = 40.0  # all other weights vanish
    for at in (5, 130, n - 1):
        x = v.clone()
        x[at, 0, 3] = INF
        o, _ = run(ta, q, k, x, cu, cu, causal)
        assert ta.sync_status() == "TA_OK"
        f = o.float().cpu()
        bad = ~torch.isfinite(f)
        want = torch.zeros_like(bad)
        want[at if causal else 0:n, :G, 3] = True
        assert torch.equal(bad, want)
        assert not (f == -INF).any()
