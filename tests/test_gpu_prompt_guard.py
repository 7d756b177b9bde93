"""The guard build (see test_gpu_guard.py) over packed attention, the rotations and
the page bookkeeping: shapes chosen for their edges, every call with TA_OK, and
the results those of the product build bit for bit."""
import pytest
import torch

from _prompt import ints, offsets, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def builds(gpu_lib):
    """run(f) calls f() through the product library, then through the guard one."""
    from tiled_attention_tcgen05_gb300 import build
    path = build.build(guard=True)
    ta = gpu_lib
    product = ta.load()

    def run(f):
        outs = []
        try:
            for lib in (product, None):
                ta._lib = lib
                if lib is None:
                    assert ta.load(path).ta_guard_build() == 1
                outs.append(f(ta))
                st = ta.sync_status()
                assert st == "TA_OK", f"{st} at {ta.load().ta_guard_last().decode()}"
        finally:
            ta._lib = product
        for a, b in zip(*outs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    yield run
    assert ta.load().ta_guard_build() == 0


@pytest.mark.parametrize("q_lens,k_lens,Hq,Hkv,D,dtype,causal", [
    ([1, 130, 0, 257], None, 4, 2, 64, "bf16", True),
    ([200, 33, 5], [140, 300, 0], 2, 2, 128, "f16", True),
    ([129, 7], [1, 128], 8, 1, 128, "bf16", False),
    ([3, 70], None, 6, 2, 64, "f16", False),
    ([1], None, 1, 1, 64, "bf16", True),
    ([40] * 400, None, 4, 1, 64, "bf16", True),  # more units than blocks run at once
])
def test_packed_attention(builds, q_lens, k_lens, Hq, Hkv, D, dtype, causal):
    k_lens = k_lens or q_lens
    cuq, cuk = offsets(q_lens), offsets(k_lens)
    q, do = (values(i, (cuq[-1] + 3, Hq, D), dtype).cuda() for i in (1, 2))
    k, v = (values(i, (cuk[-1] + 5, Hkv, D), dtype).cuda() for i in (3, 4))

    def f(ta):
        plan = ta.packed_plan(ints(cuq), q.shape[0], Hq, Hkv, causal=causal, cu_seqlens_k=ints(cuk), total_k=k.shape[0])
        o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        ta.attn_packed_fwd(q, k, v, plan, o=o, lse=lse)
        grads = [torch.zeros_like(t) for t in (q, k, v)]
        ta.attn_packed_bwd(q, k, v, o, lse, do, plan, None, *grads)
        return [o, lse] + grads
    builds(f)


@pytest.mark.parametrize("D,dim,interleaved", [(64, 64, False), (128, 64, True)])
@pytest.mark.parametrize("T", [1, 77])
def test_rotations_and_pages(builds, D, dim, interleaved, T):
    Hq, Hkv, page, B = 4, 2, 8, 3
    x = values(7, (T, Hq + 2 * Hkv, D), "bf16").cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    w = [(1 + 0.1 * values(8 + i, (D,), "bf16")).cuda() for i in range(2)]
    new = ints([T // 2, 0, T - T // 2])

    def f(ta):
        rot = ta.Rotary(dim, interleaved=interleaved)
        cache = ta.kv_cache(40, Hkv, page, D, torch.float8_e4m3fn)
        for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            t.view(torch.uint8).zero_()
        pages = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
        a = ta.cache_assign(pages, ints([0] * B), new, ints(range(40)), ints([40]), page, T)
        plain = ta.rotary_fwd(q, k, a.positions, rot)
        back = ta.rotary_bwd(*plain, a.positions, rot)
        norm = ta.qk_norm_rotary_fwd(q, k, *w, a.positions, rot)
        grads = ta.qk_norm_rotary_bwd(*plain, q, k, *w, a.positions, rot)
        qr = ta.rotary_append(cache, q, k, v, a.positions, a.slots, rot, *w)
        return [pages, *a, *plain, *back, *norm, *grads, qr, cache.k, cache.v, cache.k_scale, cache.v_scale]
    builds(f)
