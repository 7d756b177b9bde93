"""Rotary positions, page assignment and packed attention without a GPU: the C ABI's
refusals before any launch, the binding's, and the angles of Rotary."""
import ctypes
import math
import re
import os
from fractions import Fraction

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
F16, BF16, F32, E4M3 = 0, 1, 2, 3
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def ta():
    from tiled_attention_tcgen05_gb300 import build
    path = build.build()
    import tiled_attention_tcgen05_gb300 as pkg
    pkg.load(path)
    return pkg


def fields(struct_name):
    """Names of a call struct's members in the header's order, rows expanded."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tattn.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + struct_name + ";", text).group(1)
    out = []
    for line in body.split(";"):
        m = re.match(r"(?:const\s+)?(\w+)\b\s*(.*)", line.strip(), flags=re.S)
        if m:
            for name in m.group(2).split(","):
                name = name.strip().lstrip("* ")
                out += [f"{name}.{x}" for x in ("p", "sb", "sh", "st")] if m.group(1) == "ta_rows" else [name]
    return out


def packer(st, names):
    def call(base, **kw):
        v = dict(base)
        for k, x in kw.items():
            k = k.replace("__", ".")
            assert k in v, k
            v[k] = x
        return st.pack(*(v[n] for n in names))
    return call


# ------------------------------------------------------------- rotary calls
def rotary(ta):
    names = fields("ta_rotary_call")
    base = {n: 0 for n in names}
    for i, r in enumerate(("q", "k", "v", "dq", "dk", "q_out", "k_out")):
        base.update({f"{r}.p": 0x10000 * (i + 1), f"{r}.sb": 4096, f"{r}.sh": 64, f"{r}.st": 512})
    base.update(positions=0x1000, pos_t=1, slots=0x2000, turns=0x3000, q_weight=0x4000, k_weight=0x5000, dq_weight=0x6000,
                dk_weight=0x7000, ws=0x8000, ws_bytes=1 << 30, dim=64, scale=1.0, eps=1e-6, B=2, T=3, Hq=4, Hkv=2, D=64,
                dt=BF16, wt=BF16)
    make = packer(ta._ROT, names)
    return lambda fn, **kw: getattr(ta.load(), fn)(make(base, **kw), vp(0))


ROTARY = ("attn_rotary_fwd", "attn_rotary_bwd", "attn_qk_norm_rotary_fwd", "attn_qk_norm_rotary_bwd")


def test_rotary_refusals(ta):
    call = rotary(ta)
    for fn in ROTARY:
        assert getattr(ta.load(), fn)(vp(0), vp(0)) == INVALID
        for kw, want in ((dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=-1), INVALID),
                         (dict(D=96), UNSUPPORTED), (dict(dt=F32), UNSUPPORTED), (dict(dt=9), UNSUPPORTED),
                         (dict(dim=66), INVALID), (dict(dim=3), INVALID), (dict(dim=-2), INVALID),
                         (dict(scale=math.inf), INVALID), (dict(positions=0), INVALID), (dict(positions=0x1002), ALIGNMENT),
                         (dict(turns=0), INVALID), (dict(turns=0x3004), ALIGNMENT), (dict(q__p=0), INVALID),
                         (dict(k__p=0x20008), ALIGNMENT), (dict(q_out__p=0), INVALID), (dict(k_out__p=0x70004), ALIGNMENT),
                         (dict(q__st=516), ALIGNMENT), (dict(k__sh=63), ALIGNMENT), (dict(k_out__sb=4), ALIGNMENT),
                         (dict(Hq=70000), UNSUPPORTED), (dict(B=2 ** 16, T=2 ** 16), UNSUPPORTED)):
            assert call(fn, **kw) == want, (fn, kw)
    for fn in ROTARY[:3]:  # nothing to do, no launch
        assert call(fn, B=0) == OK and call(fn, T=0) == OK and call(fn, Hq=0, Hkv=0) == OK
    for fn in ROTARY[2:]:
        for kw, want in ((dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(q_weight=0), INVALID),
                         (dict(k_weight=0), INVALID), (dict(wt=F16), UNSUPPORTED), (dict(q_weight=0x4001), ALIGNMENT),
                         (dict(wt=F32, k_weight=0x5002), ALIGNMENT)):
            assert call(fn, **kw) == want, (fn, kw)
    fn = ROTARY[3]
    need = ta.load().attn_qk_norm_rotary_bwd_workspace_bytes(64)
    assert need > 0 and ta.load().attn_qk_norm_rotary_bwd_workspace_bytes(65) == 0
    for kw, want in ((dict(dq__p=0), INVALID), (dict(dk__p=8), ALIGNMENT), (dict(dq_weight=0), INVALID),
                     (dict(dk_weight=0x7002), ALIGNMENT), (dict(ws=0), INVALID), (dict(ws=0x8008), ALIGNMENT),
                     (dict(ws_bytes=need - 1), INVALID)):
        assert call(fn, **kw) == want, kw


def test_outputs_on_other_operands_are_refused(ta):
    call = rotary(ta)
    at = {r: 0x10000 * (i + 1) for i, r in enumerate(("q", "k", "v", "dq", "dk", "q_out", "k_out"))}
    for fn in ROTARY:
        bwd = fn == ROTARY[3]
        for kw in [dict(q_out__p=at["k"]), dict(k_out__p=at["q"]), dict(k_out__p=at["q_out"]),
                   dict(q_out__p=at["q"], q_out__st=1024), dict(k_out__p=at["k"], k_out__sh=128)] + \
                [dict(q_out__p=at["dk"]), dict(k_out__p=at["dq"]), dict(q_out__p=at["dq"], q_out__sb=8192)] * bwd:
            assert call(fn, **kw) == INVALID, (fn, kw)
    call = packed(ta)
    at = {r: 0x10000 * (i + 1) for i, r in enumerate(("q", "k", "v", "o", "dO", "dq", "dk", "dv"))}
    for out, others in (("dq", ("q", "k", "v", "o", "dO", "dk", "dv")), ("dk", ("q", "k", "v", "o", "dO", "dv")),
                        ("dv", ("q", "k", "v", "o", "dO"))):
        for x in others:
            assert call("attn_packed_bwd", **{out + "__p": at[x]}) == INVALID, (out, x)
    for x in ("q", "k", "v"):
        assert call("attn_packed_fwd", o__p=at[x]) == INVALID, x


def test_append_refusals(ta):
    names = fields("ta_rotary_call")
    lib = ta.load()
    hold = []

    def cache(k=0x1000, v=0x2000, ks=0, vs=0, P=8, H=2, page=16, D=64, ct=BF16):
        hold.append(ta._CacheStruct(k, v, ks, vs, P, H, page, D, ct))
        return vp(ctypes.addressof(hold[-1]))
    base_call = rotary(ta)
    make = packer(ta._ROT, names)
    base = {n: 0 for n in names}
    for i, r in enumerate(("q", "k", "v", "q_out")):
        base.update({f"{r}.p": 0x10000 * (i + 1), f"{r}.sb": 4096, f"{r}.sh": 64, f"{r}.st": 512})
    base.update(positions=0x1000, pos_t=1, slots=0x2000, turns=0x3000, dim=64, scale=1.0, B=2, T=3, Hq=4, Hkv=2, D=64,
                dt=BF16, wt=BF16)
    run = lambda c, **kw: lib.attn_rotary_append(c, make(base, **kw), vp(0))
    assert run(vp(0)) == INVALID and base_call(ROTARY[0], B=0) == OK
    for c, want in ((cache(D=128), INVALID), (cache(H=4), INVALID), (cache(ct=F16), UNSUPPORTED), (cache(ct=E4M3), INVALID),
                    (cache(k=0), INVALID), (cache(P=0), INVALID)):
        assert run(c) == want
    for kw, want in ((dict(slots=0), INVALID), (dict(slots=0x2001), ALIGNMENT), (dict(v__p=0), INVALID),
                     (dict(v__st=4), ALIGNMENT), (dict(q_weight=0x4000), INVALID), (dict(k_weight=0x4000), INVALID),
                     (dict(q_weight=0x4000, k_weight=0x5000, eps=-1.0), INVALID), (dict(positions=0), INVALID)):
        assert run(cache(), **kw) == want, kw
    assert run(cache(), B=0) == OK


# --------------------------------------------------------- page assignment
def test_assign_refusals(ta):
    names = ("pages", "max_pages", "kv", "new", "free", "num", "count", "page", "kvo", "q", "cu", "pos", "slots", "cnt", "B",
             "total")
    base = dict(pages=0x10000, max_pages=4, kv=0x20000, new=0x21000, free=0x30000, num=9, count=0x22000, page=16,
                kvo=0x40000, q=0x41000, cu=0x42000, pos=0x43000, slots=0x44000, cnt=0x45000, B=3, total=5)

    def run(**kw):
        v = dict(base, **kw)
        return ta.load().attn_cache_assign(*(v[n] if n in ("max_pages", "num", "page", "B", "total") else vp(v[n])
                                             for n in names), vp(0))
    for kw, want in ((dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(num=-1), INVALID),
                     (dict(page=0), INVALID), (dict(num=2 ** 27, page=64), UNSUPPORTED), (dict(count=0), INVALID),
                     (dict(cu=0), INVALID), (dict(cnt=0x45002), ALIGNMENT), (dict(kv=0), INVALID), (dict(new=0x21001), ALIGNMENT),
                     (dict(pages=0), INVALID), (dict(free=0), INVALID), (dict(pos=0), INVALID), (dict(slots=0x44002), ALIGNMENT),
                     (dict(kvo=0x20004), INVALID),   # the new lengths over the old
                     (dict(cnt=0x22000), INVALID), (dict(q=0x41000, cu=0x41008), INVALID), (dict(pos=0x44010), INVALID),
                     (dict(pages=0x30020), INVALID), (dict(free=0x21000), INVALID)):
        assert run(**kw) == want, kw


# -------------------------------------------------------- packed attention
def packed(ta):
    names = fields("ta_packed_call")
    base = {n: 0 for n in names}
    for i, r in enumerate(("q", "k", "v", "o", "dO", "dq", "dk", "dv")):
        base.update({f"{r}.p": 0x10000 * (i + 1), f"{r}.sh": 64, f"{r}.st": 512})
    base.update(plan=0x1000, plan_bytes=1 << 30, lse=0x2000, ws=0x3000, ws_bytes=1 << 30, B=2, total_q=100, total_k=100, Hq=4,
                Hkv=2, D=64, dt=BF16, sm_scale=-1.0)
    make = packer(ta._PACKED, names)
    return lambda fn, **kw: getattr(ta.load(), fn)(make(base, **kw), vp(0))


def test_packed_refusals(ta):
    call = packed(ta)
    need = ta.load().attn_packed_plan_bytes(2, 100, 100, 4, 2)
    for fn in ("attn_packed_fwd", "attn_packed_bwd"):
        assert getattr(ta.load(), fn)(vp(0), vp(0)) == INVALID
        for kw, want in ((dict(B=-1), INVALID), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID), (dict(Hkv=0), INVALID),
                         (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Hq=258), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
                         (dict(dt=F32), UNSUPPORTED), (dict(total_q=2 ** 31 - 1), UNSUPPORTED),
                         (dict(total_q=2 ** 30, Hq=2 ** 12, Hkv=2 ** 12), UNSUPPORTED), (dict(plan=0), INVALID),
                         (dict(plan=0x1008), ALIGNMENT), (dict(plan_bytes=need - 1), INVALID), (dict(q__p=0), INVALID),
                         (dict(k__p=0x20008), ALIGNMENT), (dict(v__st=508), ALIGNMENT), (dict(o__sh=1), ALIGNMENT),
                         (dict(k__sh=0), UNSUPPORTED), (dict(q__st=-512), UNSUPPORTED), (dict(q__st=2 ** 39), UNSUPPORTED),
                         (dict(lse=0), INVALID), (dict(lse=0x2002), ALIGNMENT)):
            assert call(fn, **kw) == want, (fn, kw)
        assert call(fn, B=0) == OK and call(fn, total_q=0, total_k=0) == OK
    assert call("attn_packed_fwd", total_q=0) == OK
    for kw, want in ((dict(dO__p=0), INVALID), (dict(dk__p=0x70004), ALIGNMENT), (dict(dv__st=0), UNSUPPORTED),
                     (dict(dq__st=4), ALIGNMENT)):
        assert call("attn_packed_bwd", **kw) == want, kw


def test_plan_refusals(ta):
    lib = ta.load()
    n = lib.attn_packed_plan_bytes(2, 100, 100, 4, 2)
    # a 64-byte head and a 32-byte entry for each tile there can be: 64 tokens a tile of 2 heads
    assert n == 64 + 32 * ((100 // 128 + 2) + (100 // 64 + 2) + (100 // 128 + 2))
    assert lib.attn_packed_plan_bytes(2, 100, 100, 3, 2) == 0 and lib.attn_packed_plan_bytes(-1, 1, 1, 1, 1) == 0
    run = lambda cq=0x1000, ck=0x2000, B=2, tq=100, tk=100, Hq=4, Hkv=2, plan=0x3000, nb=n: lib.attn_packed_plan(
        vp(cq), vp(ck), B, tq, tk, Hq, Hkv, 1, vp(plan), nb, vp(0))
    assert run(cq=0) == INVALID and run(ck=0x2002) == ALIGNMENT and run(plan=0) == INVALID and run(plan=0x3008) == ALIGNMENT
    assert run(nb=n - 1) == INVALID and run(Hq=5) == INVALID and run(B=-1) == INVALID and run(B=0) == OK
    assert lib.attn_packed_bwd_workspace_bytes(100, 4) == 1792 and lib.attn_packed_bwd_workspace_bytes(0, 4) == 0
    assert lib.attn_packed_bwd_workspace_bytes(-1, 4) == 0


# ------------------------------------------------------------- the binding
def test_rotary_angles_are_fractions_of_a_turn(ta):
    r = ta.Rotary(64, device="cpu")
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    for f, t in zip(r.inv_freq, r.turns.tolist()):
        want = Fraction(f) / two_pi * 2 ** 64
        assert abs((t % 2 ** 64) - want) <= 1
    assert r.inv_freq[0] == 1.0 and abs(r.inv_freq[31] - 10000.0 ** (-62 / 64)) < 1e-18 and r.scale == 1.0
    assert ta.Rotary(8, scaling="linear", factor=4.0, device="cpu").inv_freq[0] == 0.25
    n = ta.Rotary(8, scaling="ntk", factor=8.0, device="cpu").inv_freq
    assert n[0] == 1.0 and math.isclose(n[3], (10000.0 * 8 ** (8 / 6)) ** (-6 / 8))
    y = ta.Rotary(128, scaling="yarn", factor=16.0, first_len=4096, device="cpu")
    plain = ta.Rotary(128, device="cpu").inv_freq
    assert y.inv_freq[0] == plain[0] and math.isclose(y.inv_freq[63], plain[63] / 16)
    assert math.isclose(y.scale, 0.1 * math.log(16.0) + 1)
    assert ta.Rotary(4, inv_freq=[-0.5, 7.0], scale=2.0, device="cpu").inv_freq == (-0.5, 7.0)
    assert ta.Rotary(2, device="cpu").inv_freq == (1.0,) and ta.Rotary(0, device="cpu").inv_freq == ()


def test_rotary_refuses(ta):
    for kw in (dict(dim=3), dict(dim=130), dict(dim=-2), dict(dim=8, base=0.0), dict(dim=8, factor=-1.0),
               dict(dim=8, scaling="other"), dict(dim=8, scaling="yarn"), dict(dim=8, inv_freq=[1.0]),
               dict(dim=2, inv_freq=[math.nan]), dict(dim=2, scale=math.inf), dict(dim=2, inv_freq=[1.0], scaling="linear")):
        with pytest.raises(ValueError):
            ta.Rotary(device="cpu", **kw)


def test_binding_refuses_host_tensors(ta):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    r = ta.Rotary(64, device="cpu")
    w = torch.ones(64)
    for call in (lambda: ta.rotary_fwd(x, x, i, r), lambda: ta.rotary_bwd(x, x, i, r),
                 lambda: ta.qk_norm_rotary_fwd(x, x, w, w, i, r), lambda: ta.qk_norm_rotary_bwd(x, x, x, x, w, w, i, r),
                 lambda: ta.cache_assign(i[None], i, i, i, i[:1], 4, 3), lambda: ta.packed_plan(i, 3, 2, 2),
                 lambda: ta.attn_packed_fwd(x, x, x, None), lambda: ta.attn_packed_bwd(x, x, x, x, x, x, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="KVCache"):
        ta.rotary_append(None, x, x, x, i, i, r)
    with pytest.raises(ValueError, match="neither"):
        ta.rotary_fwd(None, None, i, r)
