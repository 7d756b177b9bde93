"""The workspace that attention over a cache asks for (no GPU)."""
import torch


def test_sequences_without_tokens_need_what_others_need():
    from tiled_attention_tcgen05_gb300 import build
    path = build.build()
    import tiled_attention_tcgen05_gb300 as ta
    ta.load(path)
    for D in (16, 128):
        for T in (1, 40):
            for ct in (torch.bfloat16, torch.int8):
                n = [ta.attn_cache_workspace_bytes(2, 8, 2, T, N, D, torch.bfloat16, ct) for N in (0, 1, 10 ** 6)]
                assert n[0] > 0 and n[0] == n[1] == n[2]
    assert ta.attn_cache_workspace_bytes(2, 8, 2, 1, -1, 64) == 0
