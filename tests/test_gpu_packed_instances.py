"""Packed attention's forward has an instance for few keys a sequence (up to 512 rows
of keys a sequence on average) and one for many: each on the other's sequences.  Rows
behind the last sequence count as keys, so padding reaches the second on short
sequences; sequences of one token reach the first on long ones."""
import numpy as np
import pytest
import torch

from _parity import to_np
from _prompt import offsets, packed_case, values, within
from test_gpu_packed import INF, LENS, NAN, case, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,dtype", [(32, "bf16"), (64, "f16"), (64, "bf16"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_short_sequences_among_much_padding(gpu_lib, G, D, dtype, causal):
    case(gpu_lib, LENS, LENS, 2 * G, 2, D, dtype, causal, False, pad=520 * len(LENS))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,D", [(1, 64), (3, 128), (8, 64), (8, 128)])
def test_keys_of_other_lengths_among_much_padding(gpu_lib, G, D, causal):
    case(gpu_lib, [10, 130, 300, 0, 5, 40, 257], [200, 130, 20, 60, 0, 167, 300], 2 * G, 2, D, "bf16", causal, False,
         pad=4000)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (4, 1, 128), (3, 1, 64), (2, 2, 128)])
def test_long_sequences_among_short_ones(gpu_lib, Hq, Hkv, D, dtype, causal):
    lens = [1, 1501, 1, 1, 250, 1, 400, 1, 130, 900, 1]
    case(gpu_lib, lens, lens, Hq, Hkv, D, dtype, causal, False)


@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("G,D,n", [(1, 64, 300), (8, 64, 50), (3, 128, 131), (1, 128, 700), (4, 64, 900)])
def test_values_of_no_number(gpu_lib, G, D, n, short):
    """They reach the rows that see them, in both instances and in short and long units."""
    ta, dtype = gpu_lib, "bf16"
    cu = offsets([n, 20] + [1] * 2 * short)
    T = cu[-1] + (0 if short else 512 * 2)
    assert (T <= 512 * (len(cu) - 1)) == short
    for at in sorted({0, n // 2, n - 1, min(n - 1, 127), min(n - 1, 128)}):
        q, k, v = make(2, T, T, 2 * G, 2, D, dtype, gain=0.3)
        clean = v.clone()
        v[at, 0, 3], v[at, 1, 5], v[at, 1, 9] = NAN, INF, -INF
        clean[at, 0, 3] = clean[at, 1, 5] = clean[at, 1, 9] = 0
        o, lse = (x[:cu[-1]] for x in run(ta, q, k, v, cu, cu, True))
        assert ta.sync_status() == "TA_OK"
        f = o.float().cpu()
        assert torch.isnan(f[at:n, :G, 3]).all()
        assert (f[at:n, G:, 5] == INF).all() and (f[at:n, G:, 9] == -INF).all()
        ref, bounds = ([x[:cu[-1]] for x in y[:2]] for y in packed_case(q, k, clean, cu, cu, True, dtype))
        seen = np.zeros(ref[0].shape, dtype=bool)
        seen[at:n, :G, 3] = seen[at:n, G:, 5] = seen[at:n, G:, 9] = True
        within("O", np.where(seen, 0.0, to_np(o)), np.where(seen, 0.0, ref[0]), bounds[0])
        within("L", lse, ref[1], bounds[1])


@pytest.mark.parametrize("pad", [0, 6000])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_far_apart(gpu_lib, D, pad):
    """Running maxima that jump by more than the rescaling threshold from one key tile to the next, and back."""
    lens = [256, 200, 390, 129]
    cu = offsets(lens)
    T = cu[-1] + pad
    q, k, v = make(4, T, T, 4, 2, D, "bf16")
    for b, n in enumerate(lens):
        k[cu[b]:cu[b] + 128] *= 0.05
        k[cu[b] + 128:cu[b + 1]] *= 6.0
    o, lse = run(gpu_lib, q, k, v, cu, cu, True)
    assert gpu_lib.sync_status() == "TA_OK"
    ref, bounds = packed_case(q, k, v, cu, cu, True, "bf16")
    within("O", o[:cu[-1]], ref[0][:cu[-1]], bounds[0][:cu[-1]])
    within("L", lse[:cu[-1]], ref[1][:cu[-1]], bounds[1][:cu[-1]])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 1)])
def test_a_lone_key_has_no_gradient(gpu_lib, D, G, causal):
    """P = 1 whatever the score: dQ and dK are zeros, dV is the sum of dO."""
    lens, klens = [1, 5, 1, 130, 129], [1, 1, 1, 1, 129]
    cu, ck = offsets(lens), offsets(klens)
    q, k, v = make(6, cu[-1], ck[-1], 2 * G, 2, D, "bf16")
    do = values(9, tuple(q.shape), "bf16")
    got = run(gpu_lib, q, k, v, cu, ck, causal, do)
    assert gpu_lib.sync_status() == "TA_OK"
    ref, bounds = packed_case(q, k, v, cu, ck, causal, "bf16", do)
    for name, g, r, b in zip(("O", "L", "dQ", "dK", "dV"), got, ref, bounds):
        within(name, g, r, b)
    assert (got[2][:cu[4]] == 0).all() and (got[3][:ck[4]] == 0).all()
    assert (got[2][cu[4] + 1:] != 0).any() and (got[3][ck[4]:] != 0).any()


def test_a_plan_used_on_another_stream(gpu_lib):
    ta = gpu_lib
    cu = offsets([200, 3, 90])
    q, k, v = (x.cuda() for x in make(7, cu[-1], cu[-1], 4, 2, 64, "bf16"))
    want = ta.attn_packed_fwd(q, k, v, ta.packed_plan(torch.tensor(cu, dtype=torch.int32).cuda(), cu[-1], 4, 2))
    torch.cuda.synchronize()
    makes, uses = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(makes):
        plan = ta.packed_plan(torch.tensor(cu, dtype=torch.int32).cuda(), cu[-1], 4, 2)
    uses.wait_stream(makes)
    plan.record_stream(uses)
    got = ta.attn_packed_fwd(q, k, v, plan, stream=uses)
    del plan  # its memory may go to the stream it was made on, once `uses` is past the call
    with torch.cuda.stream(makes):
        torch.full((1 << 16,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert ta.sync_status() == "TA_OK"
    assert all(torch.equal(a, b) for a, b in zip(got, want))
