"""Operators around attention over prompts and pages as they are used in
training and serving, with the plain form of each one: sizes, inputs, one pass,
and the result in 64 bits.

  assign   cache_assign: page tables, slots, positions and token offsets of a
           step from the requests' lengths
  rotary   rotary_fwd / rotary_bwd: rotary positions of queries and keys
  norm     qk_norm_rotary_fwd / qk_norm_rotary_bwd: a norm of each head's
           queries and keys, then the rotation
  append   rotary_append: (norm and) rotation of a step's queries and keys, the
           keys and values written to their slots of a paged cache
  attn     attn_packed_fwd / attn_packed_bwd: attention of sequences packed one
           behind the other, shared key heads

Packed tokens are [tokens, heads, D]; sequence b has rows cu[b] .. cu[b + 1] - 1,
rows behind the last sequence belong to nobody.
"""
import math
import random

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_MIN_SCALE = 2.0 ** -60
_QMAX = 448.0
_EPS = 1e-6


# ------------------------------------------------------------------ cases
def _assign(name=None, *, B, kv, new, page, ended=0.0, idle=0.0, short=False):
    c = dict(op="assign", B=B, kv=kv, new=new, page=page, ended=ended, idle=idle, short=short)
    if name:
        c["name"] = name
    return c


def _rot(op, name=None, *, tokens, Hq, Hkv, D, rot, dtype, dir="fwd", layout="packed", interleaved=False, scaling="none",
         far=8192, cache="none", page=16, norm=False, skip=False):
    c = dict(op=op, tokens=tokens, Hq=Hq, Hkv=Hkv, D=D, rot=rot, dtype=dtype, dir=dir, layout=layout,
             interleaved=interleaved, scaling=scaling, far=far, cache=cache, page=page, norm=norm, skip=skip)
    if name:
        c["name"] = name
    return c


def _attn(name=None, *, B, N, Hq, Hkv, D, dtype, dir="fwd", least=1, causal=True, other=False, fused=False, pad=0):
    c = dict(op="attn", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, dir=dir, least=least, causal=causal, other=other,
             fused=fused, pad=pad)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # every step of a server: one token more for each conversation, most of them in the page they have
        _assign("assign_step", B=64, kv=8192, new=1, page=16),
        # a burst of prompts among running, idle and ended requests
        _assign("assign_prompts", B=512, kv=2048, new=4096, page=32, ended=0.2, idle=0.2),
        # a step's tokens at far positions of a long context, half of each head rotated
        _rot("rotary", "rotary_step_far", tokens=64, Hq=32, Hkv=8, D=128, rot=64, dtype="f16", interleaved=True,
             scaling="yarn", far=1000003),
        # gradients through the rotation, [batch, heads, tokens, D] tensors of a training step
        _rot("rotary", "rotary_train_bwd", tokens=8192, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16", dir="bwd",
             layout="heads"),
        # a prompt batch's projections, one tensor for queries, keys and values
        _rot("norm", "norm_prompt", tokens=16383, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16", layout="fused",
             scaling="linear", far=16383, norm=True),
        # the same in training: gradients of projections and of the two weights
        _rot("norm", "norm_train_bwd", tokens=8192, Hq=32, Hkv=4, D=64, rot=64, dtype="f16", dir="bwd", norm=True),
        # a step of generation: one token each for a batch, into 8-bit pages
        _rot("append", "append_step_e4m3", tokens=64, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16", layout="fused",
             cache="e4m3", norm=True, far=8192),
        # a prompt batch into 16-bit pages, some rows of it padding
        _rot("append", "append_prompt_bf16", tokens=8191, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16", layout="fused",
             cache="bf16", page=64, far=32768, scaling="ntk", skip=True),
        # a batch of short requests
        _attn("attn_short", B=64, N=250, Hq=32, Hkv=4, D=64, dtype="f16", fused=True, pad=13),
        # long prompts beside a short one
        _attn("attn_long", B=3, N=16384, Hq=32, Hkv=8, D=128, dtype="bf16", fused=True),
        # training on short documents packed into one row, a key head for each query head
        _attn("attn_short_bwd", B=24, N=700, Hq=16, Hkv=16, D=64, dtype="f16", dir="bwd"),
        # training on long documents
        _attn("attn_long_bwd", B=3, N=8192, Hq=32, Hkv=8, D=128, dtype="bf16", dir="bwd", least=2000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["assign", "rotary", "norm", "append", "attn", "attn", "attn"])
    if op == "assign":
        B = _log(rng, 1, 512)
        return _assign(B=B, kv=_log(rng, 1, 4096), new=rng.choice([1, _log(rng, 1, 4096)]),
                       page=rng.choice([8, 16, 24, 32, 64]), ended=rng.choice([0.0, 0.2]), idle=rng.choice([0.0, 0.3]),
                       short=rng.random() < 0.3)
    D = rng.choice([16, 32, 64, 64, 128, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    dtype = rng.choice(["bf16", "f16"])
    if op != "attn":
        rot = rng.choice([D, D, D // 2])
        tokens = _log(rng, 1, min(16383, (1 << 25) // (Hkv * G * D)))
        cache = "none"
        if op == "append":
            cache = rng.choice([dtype, "e4m3"])
        return _rot(op, tokens=tokens, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot, dtype=dtype,
                    dir="fwd" if op == "append" else rng.choice(["fwd", "bwd"]),
                    layout=rng.choice(["packed", "heads", "fused"]), interleaved=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), far=rng.choice([4096, 131072, 2000003]),
                    cache=cache, page=rng.choice([8, 16, 24, 64]),
                    norm=op == "norm" or (op == "append" and rng.random() < 0.5),
                    skip=op == "append" and rng.random() < 0.5)
    B = _log(rng, 1, 48)
    # pairs of a query and a key at most a quarter of those of the largest listed case
    cap = int(math.sqrt((1 << 35) / (B * Hkv * G * D)))
    N = _log(rng, 1, max(1, min(8192, cap)))
    return _attn(B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=dtype, dir=rng.choice(["fwd", "bwd"]),
                 causal=rng.random() < 0.75, other=rng.random() < 0.25, fused=rng.random() < 0.5,
                 pad=rng.choice([0, 0, 5]))


# ----------------------------------------------------------------- sizes
def _requests(c):
    """Tokens held, tokens to add (-1: the request has ended) and the pages that are free."""
    r = random.Random(c["B"] * 7919 + c["kv"] * 31 + c["new"])
    kv, new = [], []
    for _ in range(c["B"]):
        x = r.random()
        kv.append(r.randint(0, c["kv"]) if c["new"] > 1 else r.randint((c["kv"] + 1) // 2, c["kv"]))
        new.append(-1 if x < c["ended"] else 0 if x < c["ended"] + c["idle"] else r.randint((c["new"] + 3) // 4, c["new"]))
    page = c["page"]
    need = sum(-(-(k + n) // page) - -(-k // page) for k, n in zip(kv, new) if n > 0)
    back = sum(-(-k // page) for k, n in zip(kv, new) if n < 0)
    count = need // 2 if c["short"] else max(0, need - back) + 7
    total = sum(n for n in new if n > 0)
    total = max(1, total * 3 // 4 if c["short"] and c["B"] % 2 else total + (3 if c["B"] % 3 == 0 else 0))
    return kv, new, count, total


def _lens(c):
    """Queries and keys of each sequence."""
    r = random.Random(c["B"] * 1000003 + c["N"] * 101)
    q = [c["N"]] + [r.randint(min(c["least"], c["N"]), c["N"]) for _ in range(c["B"] - 1)]
    if c["least"] == 1 and c["B"] > 2:
        q[1] = 1
    k = list(q)
    if c["other"]:  # keys of another length: longer (a prefix), shorter, none
        k = [r.choice([n, n + r.randint(0, c["N"]), r.randint(0, n)]) for n in q]
    return q, k


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _inv_freq(c):
    """Angles per position of the rotated pairs, float64, and the factor of the rotated values."""
    rot, base = c["rot"], 10000.0
    i = np.arange(0, rot, 2, dtype=np.float64)
    f = base ** (-i / rot)
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "ntk":
        return (base * 8.0 ** (rot / (rot - 2.0))) ** (-i / rot) if rot > 2 else f, 1.0
    if c["scaling"] == "yarn":
        factor, first, fast, slow = 16.0, 4096.0, 32.0, 1.0
        at = [rot * math.log(first / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (fast, slow)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _batch(c):
    """Batch rows and tokens of each of a [batch, heads, tokens, D] tensor."""
    if c["layout"] != "heads":
        return 1, c["tokens"]
    for b in (4, 2):
        if c["tokens"] % b == 0:
            return b, c["tokens"] // b
    return 1, c["tokens"]


# ---------------------------------------------------------------- inputs
def _randn(gen, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * gain).to(_T[dtype])


def _qkv(gen, c, tokens, ktokens=None):
    """Queries, keys and values [tokens, heads, D]: tensors of their own, or parts of one projection."""
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c.get("fused") or c.get("layout") == "fused":
        if ktokens is None or ktokens == tokens:
            x = _randn(gen, (tokens, Hq + 2 * Hkv, D), c["dtype"])
            return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    n = tokens if ktokens is None else ktokens
    return (_randn(gen, (tokens, Hq, D), c["dtype"]), _randn(gen, (n, Hkv, D), c["dtype"]),
            _randn(gen, (n, Hkv, D), c["dtype"]))


def _tokens_first(c, x):
    """[tokens, heads, D] as the case's tensors are laid out."""
    if c["layout"] != "heads":
        return x
    b, t = _batch(c)
    return x.reshape(b, t, x.shape[1], x.shape[2]).transpose(1, 2).contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "assign":
        kv, new, count, total = _requests(c)
        page = c["page"]
        held = [-(-k // page) for k in kv]
        width = max(1, max(-(-(k + max(n, 0)) // page) for k, n in zip(kv, new)))
        num = sum(held) + count + sum(h for h, n in zip(held, new) if n < 0) + 3
        order = torch.randperm(num, generator=gen, device="cuda").to(torch.int32).cpu()
        table = torch.full((c["B"], width), -1, dtype=torch.int32)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        free = torch.full((num,), -1, dtype=torch.int32)
        free[:count] = order[at:at + count]
        s.update(pages=table.cuda(), free=free.cuda(), total=total)
        for n, x in (("kv", kv), ("new", new), ("count", [count])):
            s[n] = torch.tensor(x, dtype=torch.int32).cuda()
        return s
    if c["op"] == "attn":
        ql, kl = _lens(c)
        cq, ck = _offsets(ql), _offsets(kl)
        n, m = cq[-1] + c["pad"], ck[-1] + c["pad"]
        s["cu_q"], s["cu_k"] = cq, ck
        s["q"], s["k"], s["v"] = _qkv(gen, c, n, m)
        s["o"] = torch.zeros((n, c["Hq"], c["D"]), device="cuda", dtype=_T[c["dtype"]])
        s["lse"] = torch.zeros((n, c["Hq"]), device="cuda", dtype=torch.float32)
        if c["dir"] == "bwd":
            _run_attn_fwd(s)
            s["do"] = _randn(gen, (n, c["Hq"], c["D"]), c["dtype"])
            for g, of in (("dq", "q"), ("dk", "k"), ("dv", "v")):
                s[g] = torch.zeros(s[of].shape, device="cuda", dtype=_T[c["dtype"]])
        if own:
            import tiled_attention_tcgen05_gb300 as ta
            dq = torch.tensor(cq, dtype=torch.int32).cuda()
            dk = torch.tensor(ck, dtype=torch.int32).cuda() if c["other"] else None
            s["plan"] = ta.packed_plan(dq, n, c["Hq"], c["Hkv"], causal=c["causal"], cu_seqlens_k=dk, total_k=m)
            if c["dir"] == "bwd":
                s["ws"] = torch.empty(max(16, ta.attn_packed_bwd_workspace_bytes(n, c["Hq"])), device="cuda",
                                      dtype=torch.uint8)
        return s
    n, D = c["tokens"], c["D"]
    q, k, v = _qkv(gen, c, n)
    s["q"], s["k"], s["v"] = _tokens_first(c, q), _tokens_first(c, k), v
    b, t = _batch(c)
    pos = torch.randint(0, c["far"], (b, t), generator=gen, device="cuda", dtype=torch.int32)
    if t > 1:  # sequences at consecutive positions, the last token a far one
        pos = (pos[:, :1] + torch.arange(t, device="cuda", dtype=torch.int32)) % c["far"]
        pos[:, -1] = c["far"] - 1
    s["pos"] = pos if c["layout"] == "heads" else pos[0]
    f, scale = _inv_freq(c)
    s["freq"], s["scale"] = torch.from_numpy(f).cuda(), scale
    s["wq"] = s["wk"] = None
    if c["norm"]:
        s["wq"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(_T[c["dtype"]])
        s["wk"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(_T[c["dtype"]])
    if c["dir"] == "bwd":
        s["dyq"] = _tokens_first(c, _randn(gen, (n, c["Hq"], D), c["dtype"]))
        s["dyk"] = _tokens_first(c, _randn(gen, (n, c["Hkv"], D), c["dtype"]))
    if c["op"] == "append":
        page, Hkv = c["page"], c["Hkv"]
        P = -(-n // page) + 2
        s["ck"] = torch.zeros((P, Hkv, page, D), device="cuda", dtype=_T[c["cache"]])
        s["cv"] = torch.zeros_like(s["ck"])
        s["ks"] = s["vs"] = None
        if c["cache"] == "e4m3":
            s["ks"], s["vs"] = (torch.zeros((P, Hkv, page), device="cuda") for _ in range(2))
        slots = torch.randperm(P, generator=gen, device="cuda")[:, None] * page + torch.arange(page, device="cuda")
        slots = slots.reshape(-1)[:n].to(torch.int32)
        if c["skip"]:
            slots[torch.rand(n, generator=gen, device="cuda") < 0.05] = -1
        s["slots"] = slots.reshape(b, t) if c["layout"] == "heads" else slots
        s["v"] = _tokens_first(c, v)
    if own:
        import tiled_attention_tcgen05_gb300 as ta
        kw = {"none": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=8.0),
              "yarn": dict(scaling="yarn", factor=16.0, first_len=4096)}[c["scaling"]]
        s["rotary"] = ta.Rotary(c["rot"], interleaved=c["interleaved"], **kw)
        if c["op"] == "append":
            s["cache"] = ta.KVCache(s["ck"], s["cv"], s["ks"], s["vs"])
    return s


# ------------------------------------------------------------ plain forms
def _run_assign(s):
    c, page = s["case"], s["case"]["page"]
    kv, new, count, total = s["kv"].long(), s["new"].long(), s["count"].long(), s["total"]
    pages, free, width = s["pages"], s["free"], s["pages"].shape[1]
    held = (kv + page - 1) // page
    ended = new < 0
    add = new.clamp_min(0)
    # pages of ended requests go on top of the free ones
    col = torch.arange(width, device="cuda")[None]
    back = ended[:, None] & (col < held[:, None])
    ids = pages[back]
    free[count + torch.arange(ids.numel(), device="cuda")] = ids
    top = count + ids.numel()
    need = torch.where(ended, torch.zeros_like(kv), (kv + add + page - 1) // page - held)
    upto = torch.cumsum(need, 0)
    ok = ((need == 0) | (upto <= top)) & ((add == 0) | (torch.cumsum(add, 0) <= total))
    q = torch.where(ok, add, torch.zeros_like(add))
    need = torch.where(ok, need, torch.zeros_like(need))
    upto = torch.cumsum(need, 0)
    mine = (col >= held[:, None]) & (col < (held + need)[:, None])
    b, j = torch.nonzero(mine, as_tuple=True)
    pages[b, j] = free[top - 1 - ((upto - need - held)[b] + j)]
    out = torch.where(ended, torch.zeros_like(kv), kv + q)
    cu = torch.cat([torch.zeros_like(q[:1]), torch.cumsum(q, 0)])
    rows = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    real = b < c["B"]
    b = b.clamp_max(c["B"] - 1)
    p = kv[b] + rows - cu[b]
    col = (p // page).clamp(0, width - 1)
    slot = pages[b, col].long() * page + p % page
    pos = torch.where(real, p, torch.zeros_like(p))
    slot = torch.where(real, slot, torch.full_like(slot, -1))
    return [pages, free] + [x.to(torch.int32) for x in (out, q, cu, pos, slot, top - upto[-1:])]


def _angles(s):
    """cos and sin [..., tokens, 1, pairs] of the tokens' positions (packed) or [batch, 1, tokens, pairs]."""
    a = s["pos"].double()[..., None] * s["freq"]
    a = a.unsqueeze(1)
    return (torch.cos(a) * s["scale"]).float(), (torch.sin(a) * s["scale"]).float()


def _turn(s, x, back=False):
    """fp32 x with the first rot elements of its rows rotated (back: by the negative angle)."""
    c = s["case"]
    cos, sin = _angles(s)
    if back:
        sin = -sin
    rot = c["rot"]
    y = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _normed(x, w):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    return x * r * w.float()


def _rotated(s, name, w):
    x = s[name].float()
    return _turn(s, x if w is None else _normed(x, w))


def _run_rot(s):
    c, dt = s["case"], _T[s["case"]["dtype"]]
    if c["dir"] == "fwd":
        return [_rotated(s, "q", s["wq"]).to(dt), _rotated(s, "k", s["wk"]).to(dt)]
    out, grads = [], []
    for x, dy, w in (("q", "dyq", s["wq"]), ("k", "dyk", s["wk"])):
        g = _turn(s, s[dy].float(), back=True)
        if w is not None:
            x = s[x].float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
            x = x * r
            grads.append((g * x).reshape(-1, c["D"]).sum(0) if c["layout"] != "heads" else (g * x).sum((0, 1, 2)))
            g = g * w.float()
            g = r * (g - x * (g * x).mean(-1, keepdim=True))
        out.append(g.to(dt))
    return out + grads


def _rows_of(s, x):
    """[batch, heads, tokens, D] or [tokens, heads, D] -> [tokens, heads, D]."""
    return x if x.dim() == 3 else x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])


def _run_append(s):
    c = s["case"]
    q = _rotated(s, "q", s["wq"]).to(_T[c["dtype"]])
    slots = s["slots"].reshape(-1).long()
    t = torch.nonzero(slots >= 0)[:, 0]
    pg, row = slots[t] // c["page"], slots[t] % c["page"]
    for x, dst, scl in ((_rotated(s, "k", s["wk"]), "ck", "ks"), (s["v"].float(), "cv", "vs")):
        x = _rows_of(s, x)[t]
        if c["cache"] == "e4m3":
            amax = x.abs().amax(-1)
            scale = torch.clamp_min(amax / torch.full_like(amax, _QMAX), _MIN_SCALE)
            s[scl][pg, :, row] = scale
            x = x * (1.0 / scale)[..., None]
        s[dst][pg, :, row] = x.to(s[dst].dtype)
    return [q] + [s[n] for n in ("ck", "cv", "ks", "vs") if s[n] is not None]


def _heads_at_once(c, nq, nk):
    """Key heads whose scores are worked on together."""
    each = max(1, nq * nk * (c["Hq"] // c["Hkv"]))
    return max(1, min(c["Hkv"], (1 << 29) // each))


def _each(s):
    """Sequences in pieces of their key heads: rows of queries and keys, key heads h0 .. h1 - 1, hidden pairs."""
    c = s["case"]
    for b in range(c["B"]):
        q0, q1, k0, k1 = s["cu_q"][b], s["cu_q"][b + 1], s["cu_k"][b], s["cu_k"][b + 1]
        if q0 == q1:
            continue
        nq, nk = q1 - q0, k1 - k0
        hide = None
        if c["causal"]:
            i = torch.arange(nq, device="cuda")[:, None] + nk - nq
            hide = torch.arange(nk, device="cuda")[None] > i
        step = _heads_at_once(c, nq, nk)
        for h0 in range(0, c["Hkv"], step):
            yield q0, q1, k0, k1, h0, min(c["Hkv"], h0 + step), hide


def _by_head(c, x, h0, h1):
    """Query rows [n, Hq, D] of key heads h0 .. h1 - 1 -> [h1 - h0, G, n, D] fp32."""
    G = c["Hq"] // c["Hkv"]
    return x[:, h0 * G:h1 * G].float().reshape(x.shape[0], h1 - h0, G, -1).permute(1, 2, 0, 3)


def _run_attn_fwd(s):
    c = s["case"]
    G, o, lse = c["Hq"] // c["Hkv"], s["o"], s["lse"]
    for q0, q1, k0, k1, h0, h1, hide in _each(s):
        x = _by_head(c, s["q"][q0:q1], h0, h1)
        k = s["k"][k0:k1, h0:h1].float().permute(1, 0, 2)[:, None]
        v = s["v"][k0:k1, h0:h1].float().permute(1, 0, 2)[:, None]
        if k0 == k1:
            o[q0:q1, h0 * G:h1 * G] = 0
            lse[q0:q1, h0 * G:h1 * G] = -math.inf
            continue
        a = (x @ k.transpose(-1, -2)) * c["D"] ** -0.5
        if hide is not None:
            a = torch.where(hide, torch.full((), -math.inf, device="cuda"), a)
        m = a.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(a - m)
        l = p.sum(-1, keepdim=True)
        y = torch.where(l > 0, (p @ v) / l, torch.zeros_like(x))
        n = q1 - q0
        o[q0:q1, h0 * G:h1 * G] = y.permute(2, 0, 1, 3).reshape(n, -1, c["D"]).to(o.dtype)
        lse[q0:q1, h0 * G:h1 * G] = (m + torch.log(l))[..., 0].permute(2, 0, 1).reshape(n, -1)
    return [o, lse]


def _run_attn_bwd(s):
    c = s["case"]
    G, D, scale = c["Hq"] // c["Hkv"], c["D"], c["D"] ** -0.5
    for q0, q1, k0, k1, h0, h1, hide in _each(s):
        if k0 == k1:
            s["dq"][q0:q1, h0 * G:h1 * G] = 0
            continue
        x, o, do = (_by_head(c, s[n][q0:q1], h0, h1) for n in ("q", "o", "do"))
        L = _by_head(c, s["lse"][q0:q1, :, None], h0, h1)
        k = s["k"][k0:k1, h0:h1].float().permute(1, 0, 2)[:, None]
        v = s["v"][k0:k1, h0:h1].float().permute(1, 0, 2)[:, None]
        p = torch.exp((x @ k.transpose(-1, -2)) * scale - torch.where(L == -math.inf, torch.zeros_like(L), L))
        if hide is not None:
            p = torch.where(hide, torch.zeros((), device="cuda"), p)
        dv = (p.transpose(-1, -2) @ do).sum(1)
        ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        del p
        dk = (ds.transpose(-1, -2) @ x).sum(1) * scale
        dq = (ds @ k) * scale
        del ds
        s["dq"][q0:q1, h0 * G:h1 * G] = dq.permute(2, 0, 1, 3).reshape(q1 - q0, -1, D).to(s["dq"].dtype)
        s["dk"][k0:k1, h0:h1] = dk.transpose(0, 1).to(s["dk"].dtype)
        s["dv"][k0:k1, h0:h1] = dv.transpose(0, 1).to(s["dv"].dtype)
    return [s["dq"], s["dk"], s["dv"]]


def run(state):
    s, c = state, state["case"]
    op, bwd = c["op"], c.get("dir") == "bwd"
    if not own:
        if op == "attn":
            return _run_attn_bwd(s) if bwd else _run_attn_fwd(s)
        return {"assign": _run_assign, "rotary": _run_rot, "norm": _run_rot, "append": _run_append}[op](s)
    import tiled_attention_tcgen05_gb300 as ta
    if op == "assign":
        r = ta.cache_assign(s["pages"], s["kv"], s["new"], s["free"], s["count"], c["page"], s["total"])
        return [s["pages"], s["free"], r.kv_lens, r.q_lens, r.cu_seqlens, r.positions, r.slots, r.free_count]
    if op == "rotary":
        if bwd:
            return list(ta.rotary_bwd(s["dyq"], s["dyk"], s["pos"], s["rotary"]))
        return list(ta.rotary_fwd(s["q"], s["k"], s["pos"], s["rotary"]))
    if op == "norm":
        if bwd:
            return list(ta.qk_norm_rotary_bwd(s["dyq"], s["dyk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["rotary"],
                                              eps=_EPS))
        return list(ta.qk_norm_rotary_fwd(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["rotary"], eps=_EPS))
    if op == "append":
        q = ta.rotary_append(s["cache"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["rotary"], q_weight=s["wq"],
                             k_weight=s["wk"], eps=_EPS)
        return [q] + [s[n] for n in ("ck", "cv", "ks", "vs") if s[n] is not None]
    if bwd:
        return list(ta.attn_packed_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["plan"], dq=s["dq"],
                                       dk=s["dk"], dv=s["dv"], ws=s["ws"]))
    return list(ta.attn_packed_fwd(s["q"], s["k"], s["v"], s["plan"], o=s["o"], lse=s["lse"]))


def work(case):
    c = case
    if c["op"] == "assign":
        kv, new, _, total = _requests(c)
        page = c["page"]
        moved = sum(-(-k // page) if n < 0 else -(-(k + n) // page) - -(-k // page) for k, n in zip(kv, new))
        # per request: two lengths in, two out and an offset; a page read once and written once; a position and a slot
        return {"bytes": 20 * c["B"] + 8 * moved + 8 * total, "flops": 0}
    if c["op"] == "attn":
        ql, kl = _lens(c)
        pairs = 0
        for n, m in zip(ql, kl):
            if c["causal"]:  # query i sees the keys up to i + m - n
                lo = max(0, n - m)
                pairs += (n - lo) * (lo + m - n) + (n - lo) * (n - lo + 1) // 2
            else:
                pairs += n * m
        q, k = sum(ql) * c["Hq"], sum(kl) * c["Hkv"]
        if c["dir"] == "fwd":
            return {"bytes": (2 * q + 2 * k) * c["D"] * 2 + 4 * q, "flops": 4 * c["Hq"] * c["D"] * pairs}
        return {"bytes": (4 * q + 4 * k) * c["D"] * 2 + 4 * q, "flops": 10 * c["Hq"] * c["D"] * pairs}
    n, row = c["tokens"], c["D"] * 2
    heads = c["Hq"] + c["Hkv"]
    if c["op"] == "append":
        cached = row if c["cache"] != "e4m3" else c["D"] + 4
        return {"bytes": n * (2 * c["Hq"] * row + 2 * c["Hkv"] * (row + cached) + 8), "flops": n * heads * c["D"] * 8}
    streams = 3 if c["dir"] == "bwd" and c["norm"] else 2
    return {"bytes": n * (streams * heads * row + 4), "flops": n * heads * c["D"] * (8 if c["norm"] else 4)}


# ------------------------------------------------------- results in 64 bits
def _exact_assign(s):
    c, page = s["case"], s["case"]["page"]
    pages, free = s["pages"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    kv, new, count = s["kv"].tolist(), s["new"].tolist(), int(s["count"])
    stack = free[:count].tolist()
    for b, n in enumerate(new):
        if n < 0:
            stack += pages[b, :-(-kv[b] // page)].tolist()
    free[:len(stack)] = stack
    asked = tokens = 0
    out, lens, pos, slot = [], [], [], []
    size = len(stack)
    for b, n in enumerate(new):
        if n < 0:
            out.append(0)
            lens.append(0)
            continue
        h, want = -(-kv[b] // page), -(-(kv[b] + n) // page)
        asked += want - h
        tokens += n
        if (want > h and asked > size) or (n and tokens > s["total"]):
            out.append(kv[b])
            lens.append(0)
            continue
        for j in range(h, want):
            pages[b, j] = stack.pop()
        p = np.arange(kv[b], kv[b] + n)
        pos.append(p)
        slot.append(pages[b, p // page].astype(np.int64) * page + p % page)
        out.append(kv[b] + n)
        lens.append(n)
    rest = s["total"] - sum(lens)
    pos = np.concatenate(pos + [np.zeros(rest, dtype=np.int64)])
    slot = np.concatenate(slot + [np.full(rest, -1, dtype=np.int64)])
    res = [pages, free, out, lens, _offsets(lens), pos, slot, [len(stack)]]
    return [torch.from_numpy(np.asarray(x).astype(np.int32)).cuda() for x in res]


def _complex_turn(s, x, sign=1.0):
    """Rows x (float64) rotated as complex numbers."""
    c = s["case"]
    rot = c["rot"]
    f = torch.from_numpy(_inv_freq(c)[0]).cuda()
    a = (s["pos"].double()[..., None] * f).unsqueeze(1)
    z = torch.polar(torch.full_like(a, s["scale"]), sign * a)
    y = x.clone()
    if c["interleaved"]:
        w = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * z
        y[..., :rot] = torch.view_as_real(w).reshape(*x.shape[:-1], rot)
    else:
        w = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    return y


def _exact_rot(s):
    c = s["case"]
    D = c["D"]

    def forward(name, w):
        x = s[name].double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + _EPS) * w.double()
        return _complex_turn(s, x)

    if c["op"] != "append" and c["dir"] == "fwd":
        return [forward("q", s["wq"]), forward("k", s["wk"])]
    if c["op"] != "append":
        out, grads = [], []
        for n, dy, w in (("q", "dyq", s["wq"]), ("k", "dyk", s["wk"])):
            g = _complex_turn(s, s[dy].double(), -1.0)
            if w is None:
                out.append(g)
                continue
            x = s[n].double()
            z = torch.sqrt(x.square().sum(-1, keepdim=True) / D + _EPS)
            gw = g * w.double()
            # d/dx of x / z(x): the direction along x shrinks
            out.append(gw / z - x * (gw * x).sum(-1, keepdim=True) / (D * z ** 3))
            each = g * (x / z)
            grads.append(each.sum(tuple(range(each.dim() - 1))))
        return out + grads
    q = forward("q", s["wq"])
    slots = s["slots"].reshape(-1).tolist()
    t = torch.tensor([i for i, x in enumerate(slots) if x >= 0], dtype=torch.long).cuda()
    at = torch.tensor([x for x in slots if x >= 0], dtype=torch.long).cuda()
    pg, row = torch.div(at, c["page"], rounding_mode="floor"), torch.remainder(at, c["page"])
    res, scales = [], []
    for x, dst, scl in ((forward("k", s["wk"]), "ck", "ks"), (s["v"].double(), "cv", "vs")):
        x = _rows_of(s, x)[t]
        y = s[dst].double()
        if c["cache"] == "e4m3":
            sc = (x.abs().amax(-1) / _QMAX).clamp_min(_MIN_SCALE)
            z = s[scl].double()
            z[pg, :, row] = sc
            scales.append(z)
            x = x / sc[..., None]
        y[pg, :, row] = x
        res.append(y)
    return [q] + res + scales


def _exact_attn(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    fwd = c["dir"] == "fwd"
    out = {n: s[n].double() for n in (("o", "lse") if fwd else ("dq", "dk", "dv"))}
    for b in range(c["B"]):
        q0, q1, k0, k1 = s["cu_q"][b], s["cu_q"][b + 1], s["cu_k"][b], s["cu_k"][b + 1]
        if fwd:
            out["o"][q0:q1] = 0
            out["lse"][q0:q1] = -math.inf
        if q0 == q1 or k0 == k1:
            continue
        seen = torch.ones((q1 - q0, k1 - k0), device="cuda", dtype=torch.bool)
        if c["causal"]:
            seen = torch.tril(seen, (k1 - k0) - (q1 - q0))
        for h in range(Hq):
            j = h * Hkv // Hq
            q, k, v = s["q"][q0:q1, h].double(), s["k"][k0:k1, j].double(), s["v"][k0:k1, j].double()
            a = (q @ k.T / math.sqrt(D)).masked_fill_(~seen, -math.inf)
            if fwd:
                L = torch.logsumexp(a, -1)
                p = torch.exp(a - torch.where(L == -math.inf, torch.zeros_like(L), L)[:, None])
                out["o"][q0:q1, h], out["lse"][q0:q1, h] = p @ v, L
                continue
            L = s["lse"][q0:q1, h].double()
            p = torch.exp(a - torch.where(L == -math.inf, torch.zeros_like(L), L)[:, None])
            o, do = s["o"][q0:q1, h].double(), s["do"][q0:q1, h].double()
            ds = p * (do @ v.T - (o * do).sum(-1)[:, None]) / math.sqrt(D)
            out["dq"][q0:q1, h] = ds @ k
            out["dk"][k0:k1, j] += ds.T @ q
            out["dv"][k0:k1, j] += p.T @ do
    return list(out.values())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "assign":
        return _exact_assign(s)
    return _exact_attn(s) if case["op"] == "attn" else _exact_rot(s)
