"""Pins of the oracle's rotary positions, head norms, page assignment and packed
attention: closed forms, finite differences, invariants."""
import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_closed_form_and_inverse(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 10))
    f, pos, scale = np.array([1.0, 0.3, 0.01]), np.array([0, 1, 7, 100, -3]), 1.5
    y = oracle.rotary(x, pos, f, interleaved, scale)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    for i in range(3):
        j, l = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
        c, s = np.cos(pos * f[i])[:, None], np.sin(pos * f[i])[:, None]
        assert np.allclose(y[..., j], scale * (x[..., j] * c - x[..., l] * s), atol=1e-14)
        assert np.allclose(y[..., l], scale * (x[..., l] * c + x[..., j] * s), atol=1e-14)
    back = oracle.rotary(y, pos, f, interleaved, 1 / scale, back=True)
    assert np.allclose(back, x, atol=1e-14)


def test_rotary_products_depend_on_distances_only():
    rng = np.random.default_rng(2)
    q, k, f = rng.standard_normal((1, 8)), rng.standard_normal((1, 8)), 10000.0 ** (-np.arange(4) / 4)
    a = oracle.rotary(q, [105], f) @ oracle.rotary(k, [100], f).T
    b = oracle.rotary(q, [5], f) @ oracle.rotary(k, [0], f).T
    assert np.allclose(a, b, atol=1e-12)


def test_head_norm_backward_by_differences():
    rng = np.random.default_rng(3)
    x, w, g = rng.standard_normal((4, 6)), rng.standard_normal(6), rng.standard_normal((4, 6))
    eps, h = 1e-3, 1e-6
    dx, dw = oracle.head_norm_bwd(x, w, eps, g)
    loss = lambda x, w: (g * oracle.head_norm(x, w, eps)).sum()
    for i in range(4):
        for j in range(6):
            d = np.zeros_like(x)
            d[i, j] = h
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[i, j]) < 1e-8
    for j in range(6):
        d = np.zeros(6)
        d[j] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[j]) < 1e-8
    assert np.allclose((oracle.head_norm(x, np.ones(6), 0.0) ** 2).mean(1), 1.0)


def test_assign_pages_small_case_by_hand():
    # page 4; request 0 grows into a new page, 1 ends, 2 fits its page, 3 is new
    pages = [[5, -1, -1], [6, 7, -1], [8, -1, -1], [-1, -1, -1]]
    out = oracle.assign_pages(pages, [4, 5, 2, 0], [1, -1, 2, 6], [0, 1, -1, -1, -1], 2, 4, 12)
    table, free, kv, q, cu, pos, slots, count = out
    assert free[:4] == [0, 1, 6, 7]
    assert table == [[5, 7, -1], [6, 7, -1], [8, -1, -1], [6, 1, -1]] and count == 1
    assert kv == [5, 0, 4, 6] and q == [1, 0, 2, 6] and cu == [0, 1, 1, 3, 9]
    assert pos == [4, 2, 3, 0, 1, 2, 3, 4, 5, 0, 0, 0]
    assert slots == [28, 34, 35, 24, 25, 26, 27, 4, 5, -1, -1, -1]


def test_assign_pages_short_of_pages_and_rows():
    # one free page: request 0 takes it, 1 goes without, 2 needs none
    out = oracle.assign_pages([[0, -1], [1, -1], [2, -1]], [4, 4, 1], [1, 1, 1], [9], 1, 4, 8)
    assert out[2:5] == ([5, 4, 2], [1, 0, 1], [0, 1, 1, 2]) and out[7] == 0
    # two rows: the third request's token has none left
    out = oracle.assign_pages([[0], [1], [2]], [1, 1, 1], [1, 1, 1], [], 0, 4, 2)
    assert out[3] == [1, 1, 0]


def test_packed_attention_is_each_sequence_alone():
    rng = np.random.default_rng(4)
    q, k, v, do = (rng.standard_normal((9, h, 5)) for h in (4, 2, 2, 4))
    O, L, dq, dk, dv = oracle.packed_attention(q, k, v, [1, 4, 4, 8], [0, 5, 6, 9], True, do=do)
    assert not O[0].any() and not O[8].any() and not dk[5].any()
    for a, t in ((slice(1, 4), slice(0, 5)), (slice(4, 8), slice(6, 9))):
        for h in range(4):
            o, l = oracle.attention_fwd(q[a, h], k[t, h // 2], v[t, h // 2], True)
            assert np.allclose(O[a, h], o) and np.array_equal(np.isfinite(L[a, h]), np.isfinite(l))
    # gradients by differences
    h = 1e-6
    loss = lambda q, k, v: (do * oracle.packed_attention(q, k, v, [1, 4, 4, 8], [0, 5, 6, 9], True)[0]).sum()
    for x, g, at in ((0, dq, (2, 3, 1)), (0, dq, (7, 0, 4)), (1, dk, (3, 1, 2)), (2, dv, (7, 0, 0)), (1, dk, (6, 0, 3))):
        lo, hi = [q.copy(), k.copy(), v.copy()], [q.copy(), k.copy(), v.copy()]
        lo[x][at] -= h
        hi[x][at] += h
        assert abs((loss(*hi) - loss(*lo)) / (2 * h) - g[at]) < 1e-7
