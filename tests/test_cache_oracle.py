"""Pins of the oracle's key/value cache functions (no GPU)."""
import numpy as np
import pytest
import torch

import oracle


def test_e4m3_grid_is_torchs():
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_grid(), codes)


@pytest.mark.parametrize("kind,dtype", [("e4m3", torch.bfloat16), ("e4m3", torch.float16), ("int8", torch.bfloat16)])
def test_quantise_error_and_extremes(kind, dtype):
    x = (torch.randn(200, 64, generator=torch.Generator().manual_seed(3)) * torch.logspace(-6, 3, 200)[:, None]).to(dtype)
    code, scale = oracle.cache_quantise(x, kind)
    xs = x.double().numpy()
    back = code * scale.astype(np.float64)[:, None]
    q = oracle.CACHE_QMAX[kind]
    assert np.abs(code).max() == q  # every row's largest element takes the largest code
    assert np.array_equal(np.abs(code).max(1), np.full(200, q))
    # half a step: of the integers, or of e4m3 (2^-4 relative, 2^-10 absolute below 2^-6)
    step = 0.5 if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(xs) / scale[:, None], 2.0 ** -10)
    assert (np.abs(back - xs) <= (step * (1 + 1e-6) + q * 2.0 ** -23) * scale[:, None]).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_quantise_zero_tiny_and_non_finite_rows(kind):
    x = np.zeros((4, 8))
    x[1] = 2.0 ** -100
    x[2, 3] = np.inf
    x[3, 1] = np.nan
    code, scale = oracle.cache_quantise(x, kind)
    assert (code == 0).all()
    assert scale[0] == scale[1] == 2.0 ** -60 and np.isnan(scale[2:]).all()


def test_e4m3_codes_match_torch_rounding():
    y = torch.linspace(-448, 448, 40001)
    x = torch.cat([y, torch.tensor([448.0])])[None]
    code, scale = oracle.cache_quantise(x, "e4m3")
    assert scale[0] == 1.0
    assert np.array_equal(code, x.to(torch.float8_e4m3fn).double().numpy())


def test_chain_is_causal_attention():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 5, 16)), rng.standard_normal((19, 16)), rng.standard_normal((19, 16))
    O, L = oracle.cache_attention(q, k, v)
    for g in range(2):
        Oc, Lc = oracle.attention_fwd(q[g], k, v, True)
        assert np.allclose(O[g], Oc, atol=1e-12) and np.allclose(L[g], Lc, atol=1e-12)


def test_tree_rows_are_attention_over_their_own_keys():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((1, 4, 8)), rng.standard_normal((10, 8)), rng.standard_normal((10, 8))
    tree = np.array([[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [0, 0, 0, 0]], dtype=bool)
    O, L = oracle.cache_attention(q, k, v, tree)
    for i in range(4):
        own = list(range(6)) + [6 + j for j in range(4) if tree[i, j]]
        Oi, Li = oracle.attention_fwd(q[0, i:i + 1], k[own], v[own], False)
        assert np.allclose(O[0, i], Oi[0], atol=1e-12) and np.allclose(L[0, i], Li[0], atol=1e-12)


def test_row_that_sees_nothing_and_hidden_nan():
    q, k, v = np.ones((1, 2, 8)), np.ones((2, 8)), np.ones((2, 8))
    k[1] = v[1] = np.nan
    O, L = oracle.cache_attention(q, k, v, np.array([[1, 0], [0, 0]], dtype=bool))
    assert np.array_equal(O[0], [[1] * 8, [0] * 8]) and L[0, 1] == -np.inf and np.isfinite(L[0, 0])
