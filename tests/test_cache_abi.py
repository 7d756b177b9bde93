"""The key/value cache's entry points without a GPU: the C ABI's refusals before
any launch, and the binding's."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
F16, BF16, F32, E4M3, I8 = 0, 1, 2, 3, 4
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def ta():
    from tiled_attention_tcgen05_gb300 import build
    path = build.build()
    import tiled_attention_tcgen05_gb300 as pkg
    pkg.load(path)
    return pkg


def cache(ta, k=0x1000, v=0x2000, ks=0, vs=0, P=8, H=2, page=16, D=64, ct=BF16):
    c = ta._CacheStruct(k, v, ks, vs, P, H, page, D, ct)
    return vp(ctypes.addressof(c)), c


def strides(ta, b=2048, h=1024, t=64):
    return ta._Strides(b, h, t)


def append(ta, c, k=0x3000, v=0x4000, ks=None, vs=None, pages=0x5000, maxp=4, kv=0x6000, ql=0, B=2, T=3, dt=BF16):
    return ta.load().attn_cache_append(c, vp(k), ks or strides(ta), vp(v), vs or strides(ta), vp(pages), maxp, vp(kv),
                                       vp(ql), B, T, dt, vp(0))


def read(ta, c, k=0x3000, v=0x4000, pages=0x5000, maxp=4, kv=0x6000, B=2, N=3, dt=BF16):
    return ta.load().attn_cache_read(c, vp(pages), maxp, vp(kv), vp(k), vp(v), B, N, dt, vp(0))


def keep(ta, c, pages=0x5000, maxp=4, kv=0x6000, ql=0, kp=0x7000, kl=0x8000, new=0x9000, B=2, T=3):
    return ta.load().attn_cache_keep(c, vp(pages), maxp, vp(kv), vp(ql), vp(kp), vp(kl), vp(new), B, T, vp(0))


def attn(ta, c, q=0x3000, qs=None, pages=0x5000, maxp=4, kv=0x6000, ql=0, tree=0, ts=None, o=0x7000, os=None,
         lse=0x8000, ws=0x10000, nws=1 << 30, B=2, Hq=4, T=3, dt=BF16):
    return ta.load().attn_cache_fwd(vp(q), qs or strides(ta), c, vp(pages), maxp, vp(kv), vp(ql), vp(tree), ts, vp(o),
                                    os or strides(ta), vp(lse), vp(ws), nws, B, Hq, T, dt, -1.0, vp(0))


def test_cache_checks_shared_by_every_call(ta):
    calls = (append, read, keep, attn)
    for call in calls:
        for kw, want in (({"P": 0}, INVALID), ({"H": 0}, INVALID), ({"page": 0}, INVALID), ({"P": -1}, INVALID),
                         ({"D": 96}, UNSUPPORTED), ({"D": 256}, UNSUPPORTED), ({"ct": F32}, UNSUPPORTED),
                         ({"ct": 9}, UNSUPPORTED), ({"P": 2 ** 20, "H": 64, "page": 64}, UNSUPPORTED),
                         ({"k": 0}, INVALID), ({"v": 0x2008}, ALIGNMENT),
                         ({"ct": I8}, INVALID),                             # no scales
                         ({"ct": E4M3, "ks": 0x3001, "vs": 0x3100}, ALIGNMENT)):
            c, hold = cache(ta, **kw)
            assert call(ta, c) == want, (call.__name__, kw)
        c, hold = cache(ta)
        assert call(ta, vp(0)) == INVALID
        assert call(ta, c, B=-1) == INVALID
        assert call(ta, c, maxp=-1) == INVALID
        assert call(ta, c, pages=0) == INVALID
        assert call(ta, c, pages=0x5002) == ALIGNMENT
        assert call(ta, c, kv=0) == INVALID
        assert call(ta, c, B=0) == OK            # no work, no launch
    c, hold = cache(ta)
    for call in (append, read, attn):
        assert call(ta, c, dt=F16) == UNSUPPORTED  # a 16-bit cache holds its own type
        assert call(ta, c, dt=F32) == UNSUPPORTED
    assert append(ta, c, T=0) == OK and read(ta, c, N=0) == OK and attn(ta, c, T=0) == OK
    assert append(ta, c, T=-1) == INVALID and read(ta, c, N=-1) == INVALID and attn(ta, c, T=-1) == INVALID


def test_append_read_keep_checks(ta):
    c, hold = cache(ta)
    assert append(ta, c, k=0) == INVALID and append(ta, c, v=0x4004) == ALIGNMENT
    assert append(ta, c, ks=strides(ta, t=60)) == ALIGNMENT
    assert append(ta, c, vs=strides(ta, h=1028)) == ALIGNMENT
    assert append(ta, c, ql=0x6002) == ALIGNMENT
    assert append(ta, c, B=2 ** 16, T=2 ** 15) == UNSUPPORTED  # rows past 2^31
    assert read(ta, c, k=0) == INVALID and read(ta, c, v=0x4004) == ALIGNMENT
    assert read(ta, c, B=2 ** 16, N=2 ** 15) == UNSUPPORTED
    assert keep(ta, c, kp=0) == INVALID and keep(ta, c, kl=0) == INVALID and keep(ta, c, new=0) == INVALID
    # the new lengths over an array that other blocks still read
    assert keep(ta, c, new=0x6000) == INVALID
    assert keep(ta, c, new=0x6004) == INVALID
    assert keep(ta, c, new=0x8004) == INVALID
    assert keep(ta, c, ql=0xa000, new=0xa000) == INVALID
    assert keep(ta, c, new=0x7008) == INVALID


def test_attention_checks(ta):
    c, hold = cache(ta)
    n = ta.load().attn_cache_workspace_bytes(2, 4, 2, 3, 64, 64, BF16, BF16)
    assert n > 0
    assert attn(ta, c, nws=n - 1) == INVALID and attn(ta, c, ws=0) == INVALID and attn(ta, c, ws=0x10008) == ALIGNMENT
    assert attn(ta, c, Hq=3) == INVALID and attn(ta, c, Hq=0) == INVALID
    assert attn(ta, c, q=0) == INVALID and attn(ta, c, o=0x7008) == ALIGNMENT and attn(ta, c, lse=0x8002) == ALIGNMENT
    assert attn(ta, c, qs=strides(ta, b=2047)) == ALIGNMENT and attn(ta, c, os=strides(ta, t=65)) == ALIGNMENT
    assert attn(ta, c, tree=0x9000) == INVALID  # a tree without strides
    assert attn(ta, c, Hq=2 ** 15, T=2 ** 16) == UNSUPPORTED
    w = ta.load().attn_cache_workspace_bytes
    assert w(0, 4, 2, 3, 64, 64, BF16, BF16) == 0 and w(2, 4, 3, 3, 64, 64, BF16, BF16) == 0
    assert w(2, 4, 2, 3, 64, 96, BF16, BF16) == 0 and w(2, 4, 2, 3, 64, 64, BF16, F16) == 0
    assert w(2, 4, 2, 3, 64, 64, F16, I8) > 0


def test_status_name(ta):
    assert ta.load().ta_status_str(7) == b"TA_ERR_INDEX" and ta.STATUS[7] == "TA_ERR_INDEX"


def test_binding_refuses_host_tensors_and_wrong_caches(ta):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ta.KVCache(k, k)
    with pytest.raises(ValueError, match="CUDA"):
        ta.kv_cache(4, 2, 16, 64, torch.int8, device="cpu")
    with pytest.raises(ValueError, match="scale"):
        ta.KVCache(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(ValueError, match="scale"):
        ta.KVCache(k, k, torch.zeros(4, 2, 16), torch.zeros(4, 2, 16))
    with pytest.raises(ValueError, match="dtype"):
        ta.KVCache(k.float(), k.float())
    with pytest.raises(ValueError, match="num_pages"):
        ta.KVCache(k[0], k[0])
    lens = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: ta.cache_append(None, k, k, lens[None], lens), lambda: ta.cache_read(None, lens[None], lens, 3),
                 lambda: ta.cache_keep(None, lens[None], lens, lens, lens[None], lens),
                 lambda: ta.attn_cache_fwd(k, None, lens[None], lens)):
        with pytest.raises(ValueError, match="KVCache"):
            call()
