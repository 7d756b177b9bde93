"""Helpers of the key/value cache tests: caches with pages in random order
whose unused rows hold NaN, and the bounds of attn_cache_fwd's roundings."""
from __future__ import annotations

import random

import numpy as np
import torch

import oracle
from _parity import ROUND_U, to_np

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def values(seed, shape, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(TORCH[dtype])


def page_table(rng, need, spare=2):
    """A table [B, max + 1] of distinct pages in random order, -1 behind each
    sequence's own, and the number of pages."""
    P = sum(need) + spare
    ids = list(range(P))
    rng.shuffle(ids)
    t = torch.full((len(need), max(need, default=0) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    return t, P


class Setup:
    """A cache filled by the oracle's quantisation with kv_lens tokens a
    sequence; rows that no sequence owns hold NaN (codes and scales)."""

    def __init__(self, ta, kv_lens, Hkv, page, D, dtype, cache, seed, gain=1.0, device="cuda"):
        self.ta, self.kv, self.Hkv, self.page, self.D = ta, list(kv_lens), Hkv, page, D
        self.dtype, self.kind = dtype, cache
        rng = random.Random(seed)
        self.table, P = page_table(rng, [(n + page - 1) // page for n in self.kv])
        ct = TORCH[cache]
        shape = (P, Hkv, page, D)
        nan = 0x7F if cache in ("e4m3", "int8") else None
        self.cpu, self.scale, self.rows = {}, {}, {}
        for i, name in enumerate("kv"):
            if nan is None:
                t = torch.full(shape, float("nan"), dtype=ct)
                s = None
            else:
                t = torch.full(shape, nan, dtype=torch.uint8).view(ct)
                s = torch.full(shape[:3], float("nan"))
            rows = []  # what each sequence's rows stand for, fp64 [Hkv, N, D]
            for b, n in enumerate(self.kv):
                x = values(seed * 101 + 2 * b + i, (Hkv, n, D), dtype, gain)
                x = x * torch.exp(0.5 * values(seed * 77 + b, (Hkv, n, 1), "bf16").float()).to(x.dtype)
                if s is None:
                    code, sc = x, None
                    rows.append(x.double().numpy())
                else:
                    c, sc = oracle.cache_quantise(x, cache)
                    rows.append(c * sc.astype(np.float64)[..., None])
                    code = torch.from_numpy(c).float().to(ct)
                for p in range(n):
                    pg, r = oracle.cache_slot(self.table[b], page, p)
                    t.view(torch.uint8)[pg, :, r] = code.contiguous().view(torch.uint8).reshape(Hkv, n, -1)[:, p]
                    if s is not None:
                        s[pg, :, r] = torch.from_numpy(sc)[:, p]
            self.cpu[name], self.scale[name], self.rows[name] = t, s, rows
        self.cache = ta.KVCache(*(self.cpu[n].to(device) for n in "kv"),
                                *(None if self.scale[n] is None else self.scale[n].to(device) for n in "kv"))
        self.pages = self.table.to(device)
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32, device=device)


def int32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def random_tree(rng, T, loose=0.1):
    """Ancestors-and-self of a random draft (some tokens start a new root)."""
    t = np.zeros((T, T), dtype=bool)
    for i in range(T):
        if i and rng.random() > loose:
            t[i] = t[rng.randrange(i)]
        t[i, i] = True
    return t


def attention_reference(q, k, v, tree, kind, dtype, vscale_rows=None, sm_scale=None, rows=None):
    """Oracle O, L of one (sequence, key head) and the bounds |error| of O and L.
    rows: query rows per key head of the call (longer sequences' among them).

    With u the unit roundoffs (output type; the weights' type: dt for 16-bit
    caches, fp16 for 8-bit ones) and P the exact weights:
      * a score is a sum of D products in fp32, in any order and with
        truncating adds: e_ij <= s D 2^-23 sum_d |q k|; scaling it and forming
        the exponent rounds it twice more (2^-23 |S|); bf16 queries over an 8-bit
        cache are rounded to 2^-25 of their row's largest: s 2^-25 max|q| sum|k|.
        A weight is off by that and the exponential's 2^-22; numerator and sum
        both: O moves by 2 e (P |V|) and L by e;
      * rounding the weights: u_w (P |V|), and in fp16 below 2^-14 half a step of
        2^-24 of the row's largest P * scale (the reference of the exponent):
        2^-25 max_j(P_ij sv_j) sum_j |code_j|;
      * the product with V and the sum l: N fp32 adds, N 2^-23 (P |V|) each, and
        a few roundings of the joins: (N + 64) 2^-22 together;
      * the result's rounding u |O|;
      * with more than 32 rows 8-bit values may be multiplied out to fp16 (each
        rounded to 2^-11, or half a step of 2^-24 of the largest scale, which is
        at most max|v| / 127): 2^-11 (P |V|) + 2^-25 max|v| / 127 in O; the weights'
        half steps then count 2^-25 max_j P_ij sum_j |v_j|.
    """
    O, L = oracle.cache_attention(q, k, v, tree, sm_scale)
    qn, kn, vn = (np.asarray(x, dtype=np.float64) for x in (to_np(q), k, v))
    G, T, D = qn.shape
    N = kn.shape[0]
    s = oracle.default_scale(D, sm_scale)
    keep = np.ones((T, N), dtype=bool)
    keep[:, N - T:] = np.tril(np.ones((T, T), dtype=bool)) if tree is None else tree
    u_o = ROUND_U[dtype]
    u_w = ROUND_U[dtype] if kind in ("f16", "bf16") else 2.0 ** -11
    bO, bL = np.zeros_like(O), np.zeros_like(L)
    for g in range(G):
        S = s * (qn[g] @ kn.T)
        e = s * D * 2.0 ** -23 * (np.abs(qn[g]) @ np.abs(kn).T) + 2.0 ** -22 * np.abs(S) + 2.0 ** -22
        if kind not in ("f16", "bf16"):
            e += s * 2.0 ** -24 * np.abs(qn[g]).max(1, keepdims=True) * np.abs(kn).sum(1)[None]
        wide = kind not in ("f16", "bf16") and (rows or G * T) > 32
        e = np.where(keep, e, 0.0).max(1)
        P = np.where(keep, np.exp(np.where(keep, S, -np.inf) - np.where(np.isfinite(L[g]), L[g], 0.0)[:, None]), 0.0)
        PV = P @ np.abs(vn)
        bO[g] = (2 * e[:, None] + u_w + (N + 64) * 2.0 ** -22) * PV + u_o * np.abs(O[g])
        if vscale_rows is not None:
            code = np.abs(vn) / vscale_rows[:, None]
            bO[g] += 2.0 ** -25 * (P * vscale_rows[None]).max(1)[:, None] * code.sum(0)[None]
        if wide and N:
            bO[g] += 2.0 ** -11 * PV + 2.0 ** -25 * np.abs(vn).max() / 127
            bO[g] += 2.0 ** -25 * P.max(1)[:, None] * np.abs(vn).sum(0)[None]
        bL[g] = e + (N + 64) * 2.0 ** -22 + 2.0 ** -22 * np.where(np.isfinite(L[g]), np.abs(L[g]), 0.0)
    return O, L, bO, bL


def check(name, got, ref, bound):
    g = to_np(got) if hasattr(got, "detach") else np.asarray(got)
    assert g.shape == ref.shape, f"{name}: shape {g.shape} vs {ref.shape}"
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(g)), f"{name}: non-finite entries differ"
    assert np.array_equal(g[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), f"{name}: infinities differ"
    if fin.any():
        over = np.abs(g - ref)[fin] - np.broadcast_to(bound, ref.shape)[fin]
        assert over.max() <= 0, f"{name}: past its bound by {over.max():.3e} (error {np.abs(g - ref)[fin].max():.3e})"
