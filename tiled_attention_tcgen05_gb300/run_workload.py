"""Runs the library's entry points on one of the synthetic workloads for a
number of steps: the command line used for profiling (ncu) and timing runs.

  python -m tiled_attention_tcgen05_gb300.run_workload --workload 3 --steps 2 --warmup 1

Workloads (synth_inputs.WORKLOADS): 1 fwd+bwd fp16 B1 H2 S128 D64 non-causal;
2 fwd+bwd bf16 causal B4 H16 S2048 D128; 3 fwd+bwd bf16 causal B1 H32 S8192
D128; 4 JVP forward (with tL) and the backward of the JVP, fp16 B2 H8 S1024
D64 (--causal 0/1); 5 piecewise fwd+bwd bf16 causal B2 H16 S4096 D64 w=512.
--shape B,H,S,D replaces the workload's sizes; --op merge / --op fp8 / --op cache
runs the merge (forward and backward), the e5m2 forward or a generation step
over a key/value cache (append, attention; --cache its type, --tokens new
tokens a sequence) instead; --kv-split sets
the key split of the one-query-tile forward.  Prints the mean milliseconds per
step.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import synth_inputs as si  # noqa: E402
import tiled_attention_tcgen05_gb300 as ta  # noqa: E402


def make_cache_step(shape=None, cache="bf16", tokens=1):
    """A generation step of B conversations of up to S tokens (from S / 4 on),
    H query heads over H / 4 key heads, pages of 16: the new tokens' keys and
    values appended, and their attention over the cache."""
    B, H, S, D = shape if shape is not None else (64, 32, 8192, 128)
    ct = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[cache]
    Hkv, page = max(1, H // 4), 16
    lens = [S - (S * 3 // 4) * b // B for b in range(B)]
    need = (S + page - 1) // page
    c = ta.kv_cache(B * need, Hkv, page, D, ct)
    pages = torch.randperm(B * need, generator=torch.Generator().manual_seed(si.seed_for(8, 0))).int().view(B, need).cuda()
    kv_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    fill = max(1, (1 << 26) // (Hkv * S * D))
    for b in range(0, B, fill):  # the conversations so far
        n = min(fill, B - b)
        k, v = (torch.randn(n, Hkv, S, D, device="cuda").bfloat16() for _ in range(2))
        ta.cache_append(c, k, v, pages[b:b + n], torch.full((n,), S, dtype=torch.int32, device="cuda"))
    q = si.randn((B, H, tokens, D), "bf16", si.seed_for(8, 1)).cuda()
    k, v = (si.randn((B, Hkv, tokens, D), "bf16", si.seed_for(8, i)).cuda() for i in (2, 3))
    ws = torch.empty(ta.attn_cache_workspace_bytes(B, H, Hkv, tokens, S, D, torch.bfloat16, ct), device="cuda",
                     dtype=torch.uint8)

    def step():
        ta.cache_append(c, k, v, pages, kv_lens)
        ta.attn_cache_fwd(q, c, pages, kv_lens, ws=ws)
    return step


def make_op_step(op: str, shape=None):
    """Steps of the entry points that are not a fwd+bwd workload, on the
    benchmark's shape (B1 H32 S8192 D128) unless `shape` is given:
    merge (attn_merge_fwd + attn_merge_bwd, bf16) and fp8 (attn_fwd_fp8,
    e5m2, causal)."""
    B, H, S, D = shape if shape is not None else (1, 32, 8192, 128)
    if op == "merge":
        o1, o2, do = (si.randn((B, H, S, D), "bf16", si.seed_for(6, i)).cuda() for i in range(3))
        l1, l2 = (si.randn((B, H, S), "f32", si.seed_for(6, 3 + i)).cuda() * 3 for i in range(2))

        def step():
            ta.merge_fwd(o1, l1, o2, l2)
            ta.merge_bwd(o1, l1, o2, l2, do)
        return step
    if op == "fp8":
        q = si.randn((B, H, S, D), "e5m2", si.seed_for(7, 0)).cuda()
        k = si.randn((B, H, S, D), "e5m2", si.seed_for(7, 1)).cuda()
        vt = si.randn((B, H, D, S), "e5m2", si.seed_for(7, 2)).cuda()
        return lambda: ta.attn_fwd_fp8(q, k, vt, True)
    raise ValueError(f"unknown op {op}")


def make_step(wid: int, causal_override=None, shape=None):
    w = si.WORKLOADS[wid]
    B, H, M, N, D, dt = w["B"], w["H"], w["M"], w["N"], w["D"], w["dtype"]
    causal = w["causal"] if causal_override is None else bool(causal_override)
    if shape is not None:
        B, H, M, D = shape
        N = M
    if w["mode"] == "jvp":
        names = ("q", "k", "v", "tq", "tk", "tv", "do", "dto")
    elif w["mode"] == "piecewise":
        names = ("q1", "k1", "q2", "k2", "v", "do")
    else:
        names = ("q", "k", "v", "do")
    x = {n: t.cuda() for n, t in si.attention_inputs(B, H, M, N, D, dt, wid, names=names).items()}
    if w["mode"] == "jvp":
        def jvp_step():
            o, lse, to, tlse = ta.attn_fwd_jvp(*(x[n] for n in names[:6]), causal=bool(causal), with_tlse=True)
            ta.attn_bwd_jvp(*(x[n] for n in names[:6]), o, lse, to, tlse, x["do"], x["dto"], causal=bool(causal))
        return jvp_step
    if w["mode"] == "piecewise":
        def step():
            o, lse = ta.piecewise_fwd(x["q1"], x["k1"], x["q2"], x["k2"], x["v"], w["w"], causal)
            ta.piecewise_bwd(x["q1"], x["k1"], x["q2"], x["k2"], x["v"], o, lse, x["do"], w["w"], causal)
        return step

    def step():
        o, lse = ta.attn_fwd(x["q"], x["k"], x["v"], causal)
        ta.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], causal)
    return step


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", type=int, default=3)
    ap.add_argument("--steps", type=int, default=2)
    ap.add_argument("--warmup", type=int, default=1)
    ap.add_argument("--causal", type=int, default=None)
    ap.add_argument("--shape", type=str, default=None, help="B,H,S,D instead of the workload's own (M = N = S)")
    ap.add_argument("--op", type=str, default=None, choices=["merge", "fp8", "cache"],
                    help="time attn_merge_fwd/bwd, attn_fwd_fp8 or a step over a key/value cache instead of a workload")
    ap.add_argument("--cache", type=str, default="bf16", choices=["bf16", "e4m3", "int8"], help="cache type of --op cache")
    ap.add_argument("--tokens", type=int, default=1, help="new tokens a sequence of --op cache")
    ap.add_argument("--kv-split", type=str, default="auto", choices=["auto", "never", "always"],
                    help="key split of the one-query-tile forward (JVP, D = 128 piecewise)")
    a = ap.parse_args()
    ta.load()
    ta.set_fwd_kv_split(a.kv_split)
    shape = tuple(int(x) for x in a.shape.split(",")) if a.shape else None
    if a.op == "cache":
        step = make_cache_step(shape, a.cache, a.tokens)
    else:
        step = make_op_step(a.op, shape) if a.op else make_step(a.workload, a.causal, shape)
    for _ in range(a.warmup):
        step()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(a.steps):
        step()
    e1.record()
    status = ta.sync_status()
    name = f"op {a.op}" if a.op else f"workload {a.workload}"
    print(f"{name}: {e0.elapsed_time(e1) / max(1, a.steps):.3f} ms/step, status {status}")
    return 0 if status == "TA_OK" else 1


if __name__ == "__main__":
    sys.exit(main())
