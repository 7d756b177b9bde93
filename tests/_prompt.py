"""Helpers of the tests of rotary positions, page assignment and packed
attention: inputs, and the bounds of the kernels' roundings."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from _parity import ROUND_U, to_np

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
# half a step of the smallest numbers of the type
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def values(seed, shape, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(TORCH[dtype])


def ints(x, device="cuda"):
    return torch.tensor(list(x), dtype=torch.int32, device=device)


def offsets(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def within(name, got, ref, bound):
    """|got - ref| <= bound element by element; infinities and NaN must match."""
    g = to_np(got) if hasattr(got, "detach") else np.asarray(got, dtype=np.float64)
    ref = np.asarray(ref, dtype=np.float64)
    assert g.shape == ref.shape, f"{name}: shape {g.shape} vs {ref.shape}"
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(g)), f"{name}: non-finite entries differ"
    assert np.array_equal(np.isnan(ref), np.isnan(g)), f"{name}: NaN differ"
    inf = ~fin & ~np.isnan(ref)
    assert np.array_equal(g[inf], ref[inf]), f"{name}: infinities differ"
    if fin.any():
        err = np.abs(g[fin] - ref[fin])
        over = (err - np.broadcast_to(bound, ref.shape)[fin]).max()
        assert over <= 0, f"{name}: past its bound by {over:.3e} (largest error {err.max():.3e})"


# ------------------------------------------------------------------ rotary
def partner(x, rot, interleaved):
    """|the other element of each element's pair|, 0 in the part that passes through."""
    p = np.zeros_like(x)
    n = rot // 2
    if interleaved:
        p[..., 0:rot:2], p[..., 1:rot:2] = x[..., 1:rot:2], x[..., 0:rot:2]
    else:
        p[..., :n], p[..., n:rot] = x[..., n:rot], x[..., :n]
    return np.abs(p)


def rotary_bound(h, ref, rot, interleaved, scale, dtype, D, norm):
    """Of an fp32 computation of the rotated rows h (normed ones), rounded once.

    An angle is the exact fraction of a turn but for its conversion to fp32, half a
    step of 2^-25 of half a turn: pi 2^-25; sinpi and cospi add an ulp or two, the
    factor's product one, the two products and the sum two: together below 2^-21 of
    scale (|h_j| + |h_l|).  A norm's row: D squares summed in fp32 in any order, D 2^-24
    relative in the sum (half of that in its root), rsqrt 2^-22 and three
    products: (D + 16) 2^-24."""
    rel = 2.0 ** -21 + ((D + 16) * 2.0 ** -24 if norm else 0.0)
    size = np.abs(h) * max(abs(scale), 1.0) + partner(h, rot, interleaved) * abs(scale)
    return rel * size + ROUND_U[dtype] * np.abs(ref) + TINY[dtype]


# --------------------------------------------------------- packed attention
def packed_bounds(q, k, v, cu_q, cu_k, causal, dtype, O, L, do=None, sm_scale=None):
    """Bounds |error| of attn_packed_fwd's O and L, and with do of attn_packed_bwd's
    dQ, dK, dV, from the roundings the kernels make (u: the type's unit):

      * a score, D products summed in fp32 in any order: s D 2^-23 |q| |k|; the
        exponent's product and sum 2^-22 |S| + 2^-22, exponential 2^-22: e per row;
      * O: numerator and sum off by e each, weights rounded (u, and half of the type's
        smallest step where they are tiny), N fp32 adds of the product and the sum, the
        rescaling and the reciprocal (N + 64) 2^-22, the result's rounding;
      * backward: P off by e and L's rounding, and rounded (u); dP D 2^-23 |dO| |V|;
        delta from the rounded O (u) and D fp32 adds; dS rounded (u); each sum of R terms
        in fp32 R 2^-22; the result's rounding."""
    qn, kn, vn = (to_np(x) for x in (q, k, v))
    u, tiny, D, G = ROUND_U[dtype], TINY[dtype], q.shape[2], q.shape[1] // k.shape[1]
    s = oracle.default_scale(D, sm_scale)
    bO, bL = u * np.abs(O) + tiny, np.zeros_like(L)
    out = [np.zeros_like(qn), np.zeros_like(kn), np.zeros_like(vn)]
    if do is not None:
        don = to_np(do)
    for b in range(len(cu_q) - 1):
        a, t = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        M, N = a.stop - a.start, t.stop - t.start
        if not M or not N:
            continue
        keep = oracle.allowed_mask(M, N, causal)
        for h in range(q.shape[1]):
            x, y, z = qn[a, h], kn[t, h // G], vn[t, h // G]
            S = s * (x @ y.T)
            e = s * D * 2.0 ** -23 * (np.abs(x) @ np.abs(y).T) + 2.0 ** -22 * np.abs(S) + 2.0 ** -21
            e = np.where(keep, e, 0.0)
            er = e.max(1)
            Lr = np.where(np.isfinite(L[a, h]), L[a, h], 0.0)
            P = np.where(keep, np.exp(np.where(keep, S, -np.inf) - Lr[:, None]), 0.0)
            PV = P @ np.abs(z)
            bO[a, h] += (2 * er[:, None] + u + (N + 64) * 2.0 ** -22) * PV + tiny * np.abs(z).sum(0)[None]
            bL[a, h] = er + (N + 64) * 2.0 ** -22 + 2.0 ** -22 * np.abs(Lr)
            if do is None:
                continue
            g, o = don[a, h], O[a, h]
            eP = P * (e + 2.0 ** -22 * np.abs(Lr)[:, None] + 2.0 ** -20)
            GV, GO = np.abs(g) @ np.abs(z).T, (np.abs(g) * np.abs(o)).sum(1)[:, None]
            dP = np.abs(g @ z.T - (g * o).sum(1)[:, None])
            dS = P * dP
            edP = D * 2.0 ** -23 * (GV + GO) + (u + D * 2.0 ** -23) * GO
            edS = eP * (dP + edP) + P * edP
            edS = np.where(keep, edS * (1 + u) + u * dS + 2.0 ** -22 * dS + tiny, 0.0)
            eP = np.where(keep, eP * (1 + u) + u * P + tiny, 0.0)
            out[0][a, h] += s * (edS @ np.abs(y) + N * 2.0 ** -22 * ((dS + edS) @ np.abs(y)))
            R = M * G
            out[1][t, h // G] += s * (edS.T @ np.abs(x) + R * 2.0 ** -22 * ((dS + edS).T @ np.abs(x)))
            out[2][t, h // G] += eP.T @ np.abs(g) + R * 2.0 ** -22 * ((P + eP).T @ np.abs(g))
    return (bO, bL) if do is None else (bO, bL, *out)


def packed_case(q, k, v, cu_q, cu_k, causal, dtype, do=None, sm_scale=None):
    """Oracle results and bounds, in the order O, L (, dQ, dK, dV)."""
    ref = oracle.packed_attention(q, k, v, cu_q, cu_k, causal, sm_scale, do)
    bounds = packed_bounds(q, k, v, cu_q, cu_k, causal, dtype, ref[0], ref[1], do, sm_scale)
    if do is not None:  # the results' own rounding
        bounds = bounds[:2] + tuple(b + ROUND_U[dtype] * np.abs(r) + TINY[dtype] for b, r in zip(bounds[2:], ref[2:]))
    return ref, bounds
