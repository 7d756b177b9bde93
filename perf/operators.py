"""The key/value cache operators as they are used in generation, with the
plain form of each one: sizes, inputs, one pass, and the result in 64 bits.

  append  cache_append: new tokens' keys and values quantised into cache pages
  read    cache_read: a batch's pages gathered and dequantised
  keep    cache_keep: the accepted tokens of a draft moved together
  attn    attn_cache_fwd: attention of new tokens (one token, a tree of
          drafted tokens, a prompt's chunk) over the cached keys

The cache is k, v [pages, Hkv, page, D] with, for 8-bit types, one fp32 scale
per (token, head).  Position n of sequence b is row n % page of page
pages[b, n // page]; kv_lens counts a sequence's tokens with the new ones,
q_lens the new ones.
"""
import math
import random

import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_SIZE = {"bf16": 2, "f16": 2, "e4m3": 1, "int8": 1}
_QMAX = {"e4m3": 448.0, "int8": 127.0}
_MIN_SCALE = 2.0 ** -60


def _case(op, name=None, *, B, Hq=0, Hkv, D, T, N, page, dtype, cache, ragged=False, tree=False, strided=False):
    c = dict(op=op, B=B, Hq=Hq or Hkv, Hkv=Hkv, D=D, T=T, N=N, page=page, dtype=dtype, cache=cache, ragged=ragged,
             tree=tree, strided=strided)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # every step of generation writes one token a sequence: a latency-bound call
        _case("append", "append_step_e4m3", B=64, Hkv=8, D=128, T=1, N=4096, page=16, dtype="bf16", cache="e4m3",
              ragged=True, strided=True),
        # prompts of a batch written at once, projections' layout, odd lengths
        _case("append", "append_prompt_int8", B=4, Hkv=16, D=128, T=8191, N=8192, page=32, dtype="bf16", cache="int8",
              ragged=True, strided=True),
        # a sequence's cache read back for a pass over whole tensors
        _case("read", "read_one_int8", B=1, Hkv=32, D=64, T=1, N=1000, page=16, dtype="f16", cache="int8"),
        # a batch read back, e.g. to move it to another device
        _case("read", "read_batch_e4m3", B=16, Hkv=8, D=128, T=1, N=8192, page=64, dtype="bf16", cache="e4m3",
              ragged=True),
        # the accepted path of a small draft after one verification step
        _case("keep", "keep_one_bf16", B=1, Hkv=8, D=128, T=16, N=2048, page=16, dtype="bf16", cache="bf16",
              tree=True),
        # the same for a busy server's batch
        _case("keep", "keep_batch_e4m3", B=256, Hkv=8, D=128, T=64, N=1024, page=32, dtype="bf16", cache="e4m3",
              ragged=True, tree=True),
        # one user, one token, a short conversation: latency
        _case("attn", "step_one_bf16", B=1, Hq=32, Hkv=8, D=128, T=1, N=1024, page=16, dtype="bf16", cache="bf16"),
        # a batch of conversations of different lengths, one token each
        _case("attn", "step_batch_bf16", B=64, Hq=32, Hkv=8, D=128, T=1, N=8192, page=16, dtype="bf16", cache="bf16",
              ragged=True, strided=True),
        # few long documents over an 8-bit cache, one token each
        _case("attn", "step_long_e4m3", B=3, Hq=32, Hkv=4, D=128, T=1, N=131071, page=64, dtype="bf16", cache="e4m3"),
        # a draft's tree verified in one pass, keys for every query head
        _case("attn", "tree_int8", B=16, Hq=16, Hkv=16, D=64, T=48, N=4096, page=32, dtype="f16", cache="int8",
              ragged=True, tree=True, strided=True),
        # large trees with shared key heads
        _case("attn", "tree_shared_bf16", B=8, Hq=32, Hkv=4, D=128, T=64, N=8192, page=64, dtype="bf16", cache="bf16",
              ragged=True, tree=True),
        # a chunk of a long prompt over what is cached already
        _case("attn", "chunk_bf16", B=1, Hq=32, Hkv=8, D=128, T=2048, N=16384, page=64, dtype="bf16", cache="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "keep", "attn", "attn", "attn"])
    D = rng.choice([16, 32, 64, 64, 128, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    cache = rng.choice([dtype, "e4m3", "int8"])
    ragged, strided = rng.random() < 0.6, rng.random() < 0.5
    B = _log(rng, 1, 64)
    kw = dict(Hkv=Hkv, D=D, page=page, dtype=dtype, cache=cache, ragged=ragged, strided=strided)
    if op in ("append", "read"):
        N = _log(rng, 1, min(8192, max(1, (1 << 26) // (B * Hkv * D))))
        T = 1 if op == "read" else rng.choice([1, _log(rng, 1, N)])
        return _case(op, B=B, T=T, N=N, **kw)
    if op == "keep":
        T = _log(rng, 1, 64)
        return _case(op, B=B, T=T, N=T + _log(rng, 1, 2048), tree=True, **kw)
    G = rng.choice([1, 2, 3, 4, 7, 8])
    tree = rng.random() < 0.5
    T = _log(rng, 1, 96) if tree else rng.choice([1, 1, _log(rng, 1, 1024)])
    cost = B * Hkv * D * (1 + T * G // 64)
    N = T + _log(rng, 1, min(65536, max(1, (1 << 28) // cost)))
    return _case(op, B=B, Hq=Hkv * G, T=T, N=N, tree=tree, **kw)


def _lens(c):
    """Tokens a sequence holds (with the new ones) and new ones, per sequence."""
    if not c["ragged"]:
        return [c["N"]] * c["B"], [c["T"]] * c["B"]
    r = random.Random(c["B"] * 1000003 + c["N"] * 101 + c["T"])
    q = [c["T"]] + [r.randint((c["T"] + 1) // 2, c["T"]) for _ in range(c["B"] - 1)]
    n = [c["N"]] + [max(q[b], r.randint((c["N"] + 3) // 4, c["N"])) for b in range(1, c["B"])]
    return n, q


def _paths(c, q_lens):
    """Accepted tokens of each draft, ascending: a prefix, then tokens behind
    the accepted path's end (so that a second pass finds what the first did)."""
    r = random.Random(c["B"] * 7 + c["T"])
    out = []
    for q in q_lens:
        n = r.randint(1, q) if q < 4 else r.randint(q // 4, q // 2)
        head = r.randint(0, n)
        head = n if q - n < n - head else head
        out.append(list(range(head)) + sorted(r.sample(range(n, q), n - head)))
    return out


def _quant(x, cache):
    """Codes and scales of rows x [..., D]."""
    amax = x.float().abs().amax(-1)
    # a tensor as the divisor: by a number, torch multiplies with its rounded reciprocal
    scale = torch.clamp_min(amax / torch.full_like(amax, _QMAX[cache]), _MIN_SCALE)
    scale = torch.where(torch.isfinite(amax), scale, torch.full_like(scale, math.nan))
    inv = torch.where(torch.isfinite(amax), 1.0 / scale, torch.zeros_like(scale))[..., None]
    if cache == "int8":
        y = torch.round(x.double() * inv.double())
    else:
        y = x.float() * inv
    y = torch.where(torch.isfinite(amax)[..., None], y, torch.zeros_like(y))
    return y.to(_T[cache]), scale


def _view(gen, B, H, T, D, dtype, strided):
    """[B, H, T, D] values, contiguous or as a projection lays them out."""
    x = torch.randn((B, T, H, D) if strided else (B, H, T, D), generator=gen, device="cuda", dtype=torch.float32)
    x = x.to(_T[dtype])
    return x.transpose(1, 2) if strided else x


def _random_cache(gen, shape, cache, like):
    """Pages of cached rows: unit normals, some heads' channels larger, rows of different size."""
    P, H, page, D = shape
    gain = 1.0 + 3.0 * (torch.rand((H, 1, D), generator=gen, device="cuda") > 0.97)
    out, scale = torch.empty(shape, device="cuda", dtype=_T[cache]), None
    if cache in _QMAX:
        scale = torch.empty(shape[:3], device="cuda", dtype=torch.float32)
    step = max(1, (1 << 27) // (H * page * D))
    for p in range(0, P, step):
        n = min(step, P - p)
        x = torch.randn((n, H, page, D), generator=gen, device="cuda") * gain
        x *= torch.exp(0.25 * torch.randn((n, H, page, 1), generator=gen, device="cuda"))
        if scale is None:
            out[p:p + n] = x.to(_T[cache])
        else:
            x = x.to(_T[like])
            amax = x.float().abs().amax(-1)
            s = torch.clamp_min(amax / _QMAX[cache], _MIN_SCALE)
            y = x.float() / s[..., None]
            out[p:p + n] = (torch.round(y) if cache == "int8" else y).clamp(-_QMAX[cache], _QMAX[cache]).to(_T[cache])
            scale[p:p + n] = s
    return out, scale


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, T, D, Hkv, page = c["B"], c["T"], c["D"], c["Hkv"], c["page"]
    kv, ql = _lens(c)
    need = [(n + page - 1) // page for n in kv]
    P = sum(need) + 1
    order = torch.randperm(P, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s = {"case": c, "pages": table.cuda(), "kv_lens": torch.tensor(kv, dtype=torch.int32).cuda(),
         "q_lens": torch.tensor(ql, dtype=torch.int32).cuda()}
    shape = (P, Hkv, page, D)
    s["k"], s["ks"] = _random_cache(gen, shape, c["cache"], c["dtype"])
    s["v"], s["vs"] = _random_cache(gen, shape, c["cache"], c["dtype"])
    if c["op"] == "append":
        s["nk"] = _view(gen, B, Hkv, T, D, c["dtype"], c["strided"])
        s["nv"] = _view(gen, B, Hkv, T, D, c["dtype"], c["strided"])
    if c["op"] == "keep":
        paths = _paths(c, ql)
        keep = torch.zeros((B, T), dtype=torch.int32)
        for b, p in enumerate(paths):
            keep[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        s["keep"], s["keep_lens"] = keep.cuda(), torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
    if c["op"] == "attn":
        s["q"] = _view(gen, B, c["Hq"], T, D, c["dtype"], c["strided"])
        s["tree"] = None
        if c["tree"]:
            # each drafted token's parent is one of the tokens before it
            r = random.Random(seed)
            tree = torch.zeros((B, T, T), dtype=torch.bool)
            for b in range(B):
                for i in range(T):
                    if i and r.random() > 0.1:
                        tree[b, i] = tree[b, r.randrange(max(0, i - 8), i)]
                    tree[b, i, i] = True
            s["tree"] = tree.cuda()
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((B, c["Hq"], T), device="cuda", dtype=torch.float32)
    if own:
        import tiled_attention_tcgen05_gb300 as ta
        s["cache"] = ta.KVCache(s["k"], s["v"], s["ks"], s["vs"])
        if c["op"] == "attn":
            n = ta.attn_cache_workspace_bytes(B, c["Hq"], Hkv, T, table.shape[1] * page, D, s["q"].dtype, s["k"].dtype)
            s["ws"] = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
    return s


def _slots(s, pos):
    """Page and row of positions pos [B, n] (only those that exist are used)."""
    page = s["case"]["page"]
    col = (pos // page).clamp(0, s["pages"].shape[1] - 1)
    return torch.gather(s["pages"].long(), 1, col), pos % page


def _run_append(s):
    c = s["case"]
    T = c["T"]
    t = torch.arange(T, device="cuda")[None]
    ql, kv = s["q_lens"].long()[:, None], s["kv_lens"].long()[:, None]
    b, i = torch.nonzero(t < ql, as_tuple=True)
    pg, row = _slots(s, kv - ql + t)
    pg, row = pg[b, i], row[b, i]
    for x, dst, scl in ((s["nk"], "k", "ks"), (s["nv"], "v", "vs")):
        x = x.transpose(1, 2)[b, i]  # [tokens, Hkv, D]
        if c["cache"] in _QMAX:
            code, scale = _quant(x, c["cache"])
            s[dst][pg, :, row] = code
            s[scl][pg, :, row] = scale
        else:
            s[dst][pg, :, row] = x
    return _cache_out(s)


def _cache_out(s):
    return [s[n] for n in ("k", "v", "ks", "vs") if s[n] is not None]


def _rows(s, name, scale, b, n):
    """Cached rows of sequence b's first n positions as [Hkv, n, D] fp32."""
    page = s["case"]["page"]
    ids = s["pages"][b, :(n + page - 1) // page].long()
    x = s[name][ids].float()
    if s[scale] is not None:
        x = x * s[scale][ids][..., None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _run_read(s):
    c = s["case"]
    out = []
    for name, scale in (("k", "ks"), ("v", "vs")):
        y = torch.zeros((c["B"], c["Hkv"], c["N"], c["D"]), device="cuda", dtype=_T[c["dtype"]])
        for b, n in enumerate(_lens(c)[0]):
            y[b, :, :n] = _rows(s, name, scale, b, n).to(y.dtype)
        out.append(y)
    return out


def _run_keep(s):
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")[None]
    first = (s["kv_lens"] - s["q_lens"]).long()[:, None]
    b, i = torch.nonzero(t < s["keep_lens"][:, None], as_tuple=True)
    spg, srow = _slots(s, first + s["keep"].long())
    dpg, drow = _slots(s, first + t)
    for name in ("k", "v", "ks", "vs"):
        if s[name] is not None:
            s[name][dpg[b, i], :, drow[b, i]] = s[name][spg[b, i], :, srow[b, i]]
    return _cache_out(s) + [(first[:, 0] + s["keep_lens"]).to(torch.int32)]


def _run_attn(s):
    c = s["case"]
    T, G = c["T"], c["Hq"] // c["Hkv"]
    kv, ql = _lens(c)
    o, lse = s["o"], s["lse"]
    for b in range(c["B"]):
        n, q = kv[b], ql[b]
        k, v = _rows(s, "k", "ks", b, n), _rows(s, "v", "vs", b, n)
        seen = torch.ones((q, n), device="cuda", dtype=torch.bool)
        new = torch.ones((q, q), device="cuda", dtype=torch.bool).tril() if s["tree"] is None else s["tree"][b, :q, :q]
        seen[:, n - q:] = new
        for h in range(c["Hkv"]):
            x = s["q"][b, h * G:(h + 1) * G, :q].float()  # [G, q, D]
            a = (x @ k[h].T) * c["D"] ** -0.5
            a = torch.where(seen, a, torch.full_like(a, -math.inf))
            m = a.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = torch.exp(a - m)
            l = p.sum(-1, keepdim=True)
            y = torch.where(l > 0, (p @ v[h]) / l, torch.zeros_like(x))
            o[b, h * G:(h + 1) * G, :q] = y.to(o.dtype)
            lse[b, h * G:(h + 1) * G, :q] = (m + torch.log(l))[..., 0]
    return [o, lse]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _run_append, "read": _run_read, "keep": _run_keep, "attn": _run_attn}[op](s)
    import tiled_attention_tcgen05_gb300 as ta
    if op == "append":
        ta.cache_append(s["cache"], s["nk"], s["nv"], s["pages"], s["kv_lens"], s["q_lens"])
        return _cache_out(s)
    if op == "read":
        return list(ta.cache_read(s["cache"], s["pages"], s["kv_lens"], s["case"]["N"], dtype=_T[s["case"]["dtype"]]))
    if op == "keep":
        lens = ta.cache_keep(s["cache"], s["pages"], s["kv_lens"], s["q_lens"], s["keep"], s["keep_lens"])
        return _cache_out(s) + [lens]
    return list(ta.attn_cache_fwd(s["q"], s["cache"], s["pages"], s["kv_lens"], s["q_lens"], tree=s["tree"], o=s["o"],
                                  lse=s["lse"], ws=s["ws"]))


def work(case):
    c = case
    kv, ql = _lens(c)
    row = c["D"] * _SIZE[c["cache"]] + (4 if c["cache"] in _QMAX else 0)  # a cached row with its scale
    if c["op"] == "append":
        n = 2 * c["Hkv"] * sum(ql)
        return {"bytes": n * (c["D"] * _SIZE[c["dtype"]] + row), "flops": n * 2 * c["D"]}
    if c["op"] == "read":
        n = 2 * c["Hkv"]
        return {"bytes": n * (sum(kv) * row + c["B"] * c["N"] * c["D"] * _SIZE[c["dtype"]]),
                "flops": n * sum(kv) * c["D"]}
    if c["op"] == "keep":
        n = sum(len(p) for p in _paths(c, ql))
        return {"bytes": 2 * 2 * c["Hkv"] * n * row, "flops": 0}
    pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(kv, ql))
    new = sum(ql) * c["Hq"]
    return {"bytes": 2 * c["Hkv"] * sum(kv) * row + new * (2 * c["D"] * _SIZE[c["dtype"]] + 4),
            "flops": 4 * c["Hq"] * c["D"] * pairs}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, row by row of the
    page table on the host's indices."""
    c = case
    s = prepare(c, seed)
    kv, ql = _lens(c)
    page, Hkv, D = c["page"], c["Hkv"], c["D"]
    table = s["pages"].cpu().tolist()

    def slots(b, first, n):
        at = [(table[b][p // page], p % page) for p in range(first, first + n)]
        ids, rows = zip(*at) if at else ((), ())
        return torch.tensor(ids, dtype=torch.long).cuda(), torch.tensor(rows, dtype=torch.long).cuda()

    def whole(x):
        return None if x is None else (x.double() if x.dtype != torch.int8 else x.clone())

    def cached(name, b, n):  # [n, Hkv, D]
        ids, rows = slots(b, 0, n)
        x = s[name][ids, :, rows].double()
        sc = s[name + "s"]
        return x if sc is None else x * sc[ids, :, rows].double()[..., None]

    if c["op"] == "append":
        out = {n: whole(s[n]) for n in ("k", "v", "ks", "vs")}
        for b in range(c["B"]):
            ids, rows = slots(b, kv[b] - ql[b], ql[b])
            for src, dst in (("nk", "k"), ("nv", "v")):
                x = s[src][b, :, :ql[b]].transpose(0, 1).double()
                if c["cache"] in _QMAX:
                    sc = (x.abs().amax(-1) / _QMAX[c["cache"]]).clamp_min(_MIN_SCALE)
                    out[dst + "s"][ids, :, rows] = sc
                    # the codes are those of the stored scale, one 32-bit number
                    inv = (1.0 / sc.float()).double()
                    x = x * inv[..., None]
                    x = torch.round(x).to(torch.int8) if c["cache"] == "int8" else x
                out[dst][ids, :, rows] = x
        return [out[n] for n in ("k", "v", "ks", "vs") if out[n] is not None]
    if c["op"] == "read":
        res = []
        for name in ("k", "v"):
            y = torch.zeros((c["B"], Hkv, c["N"], D), device="cuda", dtype=torch.float64)
            for b in range(c["B"]):
                y[b, :, :kv[b]] = cached(name, b, kv[b]).transpose(0, 1)
            res.append(y)
        return res
    if c["op"] == "keep":
        names = [n for n in ("k", "v", "ks", "vs") if s[n] is not None]
        out = {n: whole(s[n]) for n in names}
        paths = _paths(c, ql)
        for b, path in enumerate(paths):
            first = kv[b] - ql[b]
            for i, j in enumerate(path):
                dst, src = first + i, first + j
                for n in names:
                    out[n][table[b][dst // page], :, dst % page] = whole(
                        s[n][table[b][src // page], :, src % page])
        lens = [kv[b] - ql[b] + len(paths[b]) for b in range(c["B"])]
        return [out[n] for n in names] + [torch.tensor(lens, dtype=torch.int32).cuda()]
    o = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(s["lse"].shape, device="cuda", dtype=torch.float64)
    tree = None if s["tree"] is None else s["tree"].cpu()
    for b in range(c["B"]):
        n, nq = kv[b], ql[b]
        k, v = cached("k", b, n), cached("v", b, n)
        hidden = torch.zeros((nq, n), dtype=torch.bool)
        for i in range(nq):
            if tree is None:
                hidden[i, n - nq + i + 1:] = True
            else:
                hidden[i, n - nq:] = ~tree[b, i, :nq]
        hidden = hidden.cuda()
        for h in range(c["Hq"]):
            j = h * Hkv // c["Hq"]
            a = (s["q"][b, h, :nq].double() @ k[:, j].T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            L = torch.logsumexp(a, -1)
            some = L > -math.inf
            p = torch.exp(a - torch.where(some, L, torch.zeros_like(L))[:, None])
            o[b, h, :nq] = p @ v[:, j]
            lse[b, h, :nq] = L
    return [o, lse]
