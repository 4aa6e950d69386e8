"""Pins of the oracle of window attention, the rotating store and rotary positions with several axes (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import serving as S
from oracle import window as W


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_the_mask_by_hand():
    assert W.visible(4, 6, 2, 1).astype(int).tolist() == [[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0],
                                                          [1, 0, 0, 0, 1, 1]]
    assert W.visible(3, 3, 1, 0).tolist() == np.eye(3, dtype=bool).tolist()
    assert not W.visible(5, 2, 9, 9)[:3].any()                       # negative positions see nothing
    assert W.visible(2, 4, 1, 9).tolist() == np.tril(np.ones((4, 4), bool))[2:].tolist()


def test_a_window_as_long_as_the_text_is_causal_attention():
    q, k, v = rnd(1, 9, 4, 8), rnd(2, 9, 2, 8), rnd(3, 9, 2, 8)
    for window, sink in ((9, 0), (100, 3), (1, 9)):
        O, L, _ = W.window_attn(q, k, v, [0, 9], window, sink)
        Of, Lf = oracle.full_attention(q, k, v, True)
        assert np.allclose(O, Of, atol=1e-12) and np.allclose(L, Lf, atol=1e-12)


def test_a_row_sees_its_window_and_the_first_tokens():
    q, k, v = rnd(1, 30, 2, 8), rnd(2, 30, 1, 8), rnd(3, 30, 1, 8)
    O, L, _ = W.window_attn(q, k, v, [0, 30], 5, 2)
    for p, h in ((0, 0), (3, 1), (6, 0), (29, 1)):
        ids = [x for x in range(p + 1) if x > p - 5 or x < 2]
        s = k[ids, 0] @ q[p, h] / np.sqrt(8)
        assert np.allclose(O[p, h], np.exp(s - s.max()) @ v[ids, 0] / np.exp(s - s.max()).sum())
        assert np.isclose(L[p, h], np.log(np.exp(s).sum()))


@pytest.mark.parametrize("window,sink", [(3, 0), (4, 2), (100, 0)])
def test_the_gradient_against_differences(window, sink):
    qsl = [1, 8, 8, 13]
    q, k, v, do = rnd(1, 14, 4, 6), rnd(2, 14, 2, 6), rnd(3, 14, 2, 6), rnd(4, 14, 4, 6)
    grads, _ = W.window_attn_grad(do, q, k, v, qsl, window, sink, 0.7)

    def loss(*x):
        return np.nansum(W.window_attn(*x, qsl, window, sink, 0.7)[0] * do)

    for i, g in enumerate(grads):
        assert np.isnan(g[[0, 13]]).all() and not np.isnan(g[1:13]).any()
        for seed in range(5):
            u = rnd(10 + seed, *g.shape)
            u[[0, 13]] = 0
            hi, lo = [q, k, v], [q, k, v]
            hi[i], lo[i] = hi[i] + 1e-5 * u, lo[i] - 1e-5 * u
            assert np.isclose((loss(*hi) - loss(*lo)) / 2e-5, np.nansum(g * u), rtol=1e-6, atol=1e-8)


def test_the_gradient_of_parts_of_the_keys_adds_up():
    """With O and LSE of all keys, the gradients over the window's tokens and over the first tokens are those of both."""
    q, k, v, do = rnd(1, 14, 4, 6), rnd(2, 14, 2, 6), rnd(3, 14, 2, 6), rnd(4, 14, 4, 6)
    qsl = [0, 14]
    O, L, _ = W.window_attn(q, k, v, qsl, 5, 3)
    both, _ = W.window_attn_grad(do, q, k, v, qsl, 5, 3)
    again, _ = W.window_attn_grad(do, q, k, v, qsl, 5, 3, o=O, lse=L)
    assert all(np.allclose(a, b, atol=1e-12) for a, b in zip(both, again))
    near, _ = W.window_attn_grad(do, q, k, v, qsl, 5, 0, o=O, lse=L)
    far, _ = W.window_attn_grad(do, q, k, v, qsl, 1, 3, o=O, lse=L)
    # first tokens that are in the window too, and each token itself, are counted twice: take them out
    twice = [np.zeros_like(x) for x in both]
    for p in range(14):
        for x in {y for y in range(max(0, p - 4), p + 1) if y < 3 or y == p}:
            for h in range(4):
                pr = np.exp(q[p, h] @ k[x, h // 2] / np.sqrt(6) - L[p, h])
                ds = pr * (do[p, h] @ (v[x, h // 2] - O[p, h])) / np.sqrt(6)
                twice[0][p, h] += ds * k[x, h // 2]
                twice[1][x, h // 2] += ds * q[p, h]
                twice[2][x, h // 2] += pr * do[p, h]
    for a, b, c, d in zip(near, far, twice, both):
        assert np.allclose(a + b - c, d, atol=1e-10)


def test_over_the_cache_as_on_packed_rows():
    ctx, n, bs, I, pcp, dcp = [20, 7, 0, 3], [5, 7, 0, 6], 4, 2, 1, 2
    qsl = np.concatenate([[0], np.cumsum(n)])
    q, kc, vc = rnd(1, 18, 4, 8), rnd(2, 2, 9, 2, 4, 8), rnd(3, 2, 9, 2, 4, 8)
    table = np.array([[7, 1, 4], [0, -1, -1], [-1, -1, -1], [3, -1, -1]])
    full = S.chunk_attn(q, kc, vc, table, qsl, ctx, bs, I, pcp, dcp)
    got = W.cp_window_attn(q, kc, vc, table, qsl, ctx, 50, 0, bs, I, pcp, dcp)
    assert all(np.allclose(a, b, atol=1e-12) for a, b in zip(full, got))
    assert (got[0][12:15] == 0).all() and np.isneginf(got[1][12:15]).all()
    # blocks out of sight are not looked at
    far = table.copy()
    far[0, 1] = 10 ** 6                                  # tokens 8 .. 15
    a, b = (W.cp_window_attn(q[:1], kc, vc, t, [0, 1], [20], 4, 8, bs, I, pcp, dcp)[0] for t in (table, far))
    assert np.array_equal(a, b)


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_axes(style):
    x, f = rnd(1, 5, 3, 20), np.array([1.0, 0.3, 0.2, 0.05, 0.01, 0.5])
    pos = np.array([3, 9, 100, 0, 7])
    one = S.rope_apply(x, pos, f, 1.3, style)
    for axis in ([0] * 6, [0, 1, 2, 0, 1, 2], [2, 2, 1, 1, 0, 0]):
        assert np.allclose(W.rope_apply_axes(x, [pos, pos, pos], f, axis, 1.3, style), one, atol=1e-12)
    three = np.stack([pos, pos * 2, pos + 1])
    y = W.rope_apply_axes(x, three, f, [0, 0, 1, 1, 2, 2], 1.0, style)
    for i, a in enumerate([0, 0, 1, 1, 2, 2]):
        e = (i, i + 6) if style == "half" else (2 * i, 2 * i + 1)
        z = (x[:, :, e[0]] + 1j * x[:, :, e[1]]) * np.exp(1j * three[a] * f[i])[:, None]
        assert np.allclose(y[:, :, e[0]], z.real) and np.allclose(y[:, :, e[1]], z.imag)
    assert np.array_equal(y[:, :, 12:], x[:, :, 12:])
    # the backward direction is the transpose
    dy = rnd(2, 5, 3, 20)
    dx = W.rope_apply_axes(dy, three, f, [0, 0, 1, 1, 2, 2], 1.3, style, True)
    assert np.isclose((W.rope_apply_axes(x, three, f, [0, 0, 1, 1, 2, 2], 1.3, style) * dy).sum(), (x * dx).sum())


def test_the_store_is_the_slot_mapping_and_the_scatter():
    ctx, n, bs, I, pcp, dcp = [20, 7, 3], [5, 7, 1], 4, 2, 1, 2
    qsl = np.concatenate([[0], np.cumsum(n)])
    table = np.array([[7, 1, 4], [0, -1, -1], [3, -1, -1]])
    k, v, kc, vc = rnd(1, 13, 2, 8), rnd(2, 13, 2, 8), rnd(3, 2, 9, 2, 4, 8), rnd(4, 2, 9, 2, 4, 8)
    place = np.array([x for _, _, x in W.append_rows(qsl, ctx)])
    assert place.tolist() == [15, 16, 17, 18, 19, 0, 1, 2, 3, 4, 5, 6, 2]
    slot = oracle.cp_slot_mapping(qsl, place, table, bs, I, pcp, dcp)
    a, b = W.cp_rope_append(k, v, kc, vc, table, qsl, ctx, bs, I, pcp, dcp)
    k2, v2 = kc.copy(), vc.copy()
    oracle.cp_kv_scatter(k, v, slot, k2, v2, bs)
    assert np.array_equal(a, k2) and np.array_equal(b, v2)
