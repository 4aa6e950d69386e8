"""Attention with a sliding window and first tokens that stay visible, on packed
sequences with its gradient and over the sharded paged cache; the store of new
tokens with their rotation; rotary positions with several axes.  Test
infrastructure only.

The mask is the definition: the query at position p sees the tokens x <= p with
x > p - window or x < n_sink.  The gradient is that of
O = softmax(scale Q K^T) V, written out with explicit matrices.  Sources of the
cache's layout and of the rotary form: as ``oracle.serving``.

Parity status: pinned (a window as long as the text against plain causal
attention, the gradient against differences, the store against the slot mapping
and scatter, equal axes against one axis).
"""

from __future__ import annotations

import numpy as np

from .attention import _as64
from .kvcache import cp_token_location
from .serving import rope_apply


def visible(n, ctx, window, n_sink):
    """[n, ctx]: which tokens the last n positions of a text of ctx tokens see."""
    p = (int(ctx) - int(n) + np.arange(n))[:, None]
    x = np.arange(int(ctx))[None, :]
    return (x <= p) & ((x > p - window) | (x < n_sink))


def attend(q, k, v, seen, scale=None):
    """O [n, Hq, d], LSE [n, Hq], the same average of |V|, and the weights P [n, Hq, ctx] (0 / -inf where nothing is seen).
    Values that a row does not see are not used, whatever they are."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    s = np.einsum("nhd,khd->nhk", q, np.repeat(k, G, axis=1)) * (scale or 1.0 / np.sqrt(d))
    s = np.where(seen[:, None, :], s, -np.inf)
    m = s.max(axis=2, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, :, None])
    l = e.sum(axis=2)
    p = e / np.where(l > 0, l, 1.0)[:, :, None]
    v = np.repeat(np.where(seen.any(axis=0)[:, None, None], v, 0.0), G, axis=1)
    return (np.einsum("nhk,khd->nhd", p, v), np.where(l > 0, m + np.log(np.where(l > 0, l, 1.0)), -np.inf),
            np.einsum("nhk,khd->nhd", p, np.abs(v)), p)


def window_attn(q, k, v, qsl, window, n_sink=0, scale=None):
    """(O, LSE, A) of packed sequences, A the average of |V|; rows of no sequence NaN."""
    q, k, v = _as64(q), _as64(k), _as64(v)
    T, Hq, d = q.shape
    O, A, L = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    for r in range(len(qsl) - 1):
        a, b = int(qsl[r]), int(qsl[r + 1])
        O[a:b], L[a:b], A[a:b], _ = attend(q[a:b], k[a:b], v[a:b], visible(b - a, b - a, window, n_sink), scale)
    return O, L, A


def window_attn_grad(do, q, k, v, qsl, window, n_sink=0, scale=None, o=None, lse=None):
    """(dQ, dK, dV) and, of each, a bound of the error that it may have where P and dS are rounded to bf16 (2^-8),
    delta is formed from an O rounded to bf16 and all else is fp32 (2^-11 of what is summed); rows of no sequence NaN.
    o and lse: those of more keys than these (then P = e^{s - lse} sums to less than 1)."""
    do, q, k, v = _as64(do), _as64(q), _as64(k), _as64(v)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    G, scale = Hq // Hkv, scale or 1.0 / np.sqrt(d)
    r8, r11 = 2.0 ** -8, 2.0 ** -11
    out = [np.full(x.shape, np.nan) for x in (q, k, v, q, k, v)]
    for r in range(len(qsl) - 1):
        a, b = int(qsl[r]), int(qsl[r + 1])
        seen = visible(b - a, b - a, window, n_sink)
        Q, D, K, V = q[a:b], do[a:b], np.repeat(k[a:b], G, axis=1), np.repeat(v[a:b], G, axis=1)
        O, L, _, P = attend(Q, k[a:b], v[a:b], seen, scale)
        if lse is not None:
            O, P = _as64(o)[a:b], P * np.exp(L - _as64(lse)[a:b])[:, :, None]
        dP = np.einsum("nhd,khd->nhk", D, V)
        aP = np.einsum("nhd,khd->nhk", np.abs(D), np.abs(V))
        delta, ad = (D * O).sum(2)[:, :, None], (np.abs(D) * np.abs(O)).sum(2)[:, :, None]
        dS = P * (dP - delta)
        E = r8 * np.abs(dS) + P * (r8 * ad + r11 * (aP + ad))
        fold = lambda x: x.reshape(b - a, Hkv, G, d).sum(axis=2)  # noqa: E731
        rows = [np.einsum("nhk,khd->nhd", dS, K) * scale, fold(np.einsum("nhk,nhd->khd", dS, Q)) * scale,
                fold(np.einsum("nhk,nhd->khd", P, D)),
                np.einsum("nhk,khd->nhd", E, np.abs(K)) * scale, fold(np.einsum("nhk,nhd->khd", E, np.abs(Q))) * scale,
                fold(np.einsum("nhk,nhd->khd", P, np.abs(D))) * (r8 + r11)]
        for y, x in zip(out, rows):
            y[a:b] = x
    return out[:3], out[3:]


def cp_window_attn(q, k_cache, v_cache, block_table, qsl, ctx_lens, window, n_sink, bs, I, pcp, dcp, scale=None):
    """(O, LSE, A) of the last n_r tokens of each request over the sharded paged cache; only tokens that some query of
    the request sees are looked up.  Rows of no request NaN."""
    q, kc, vc = _as64(q), _as64(k_cache), _as64(v_cache)
    T, Hq, d = q.shape
    O, A, L = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    for r, ctx in enumerate(ctx_lens):
        a, b, ctx = int(qsl[r]), int(qsl[r + 1]), int(ctx)
        seen = visible(b - a, ctx, window, n_sink)
        k, v = np.zeros((ctx, kc.shape[2], d)), np.zeros((ctx, kc.shape[2], d))
        for x in np.nonzero(seen.any(axis=0))[0]:
            vb, dev, off = cp_token_location(int(x), bs, I, pcp, dcp)
            k[x], v[x] = kc[dev, block_table[r][vb], :, off], vc[dev, block_table[r][vb], :, off]
        O[a:b], L[a:b], A[a:b], _ = attend(q[a:b], k, v, seen, scale)
    return O, L, A


def rope_apply_axes(x, positions, inv_freq, axis, mscale=1.0, style="half", backward=False):
    """Pair i turned by positions[axis[i]] * inv_freq[i]: one axis after another, each with the others' frequencies 0
    and the factor mscale once."""
    y = _as64(x)
    f, axis = np.asarray(inv_freq, dtype=np.float64), np.asarray(axis)
    for a in range(len(positions)):
        y = rope_apply(y, positions[a], np.where(axis == a, f, 0.0), 1.0, style, backward)
    rot = 2 * len(f)
    y[..., :rot] = y[..., :rot] * mscale
    return y


def append_rows(qsl, ctx_lens):
    """(token, request, place in its context) of every token of a request."""
    for r, ctx in enumerate(ctx_lens):
        for t in range(int(qsl[r]), int(qsl[r + 1])):
            yield t, r, int(ctx) - (int(qsl[r + 1]) - t)


def cp_rope_append(k, v, k_cache, v_cache, block_table, qsl, ctx_lens, bs, I, pcp, dcp):
    """The caches after the rows k (turned already) and v [T, Hkv, d] have been stored."""
    kc, vc = _as64(k_cache).copy(), _as64(v_cache).copy()
    k, v = _as64(k), _as64(v)
    for t, r, x in append_rows(qsl, ctx_lens):
        vb, dev, off = cp_token_location(x, bs, I, pcp, dcp)
        kc[dev, block_table[r][vb], :, off], vc[dev, block_table[r][vb], :, off] = k[t], v[t]
    return kc, vc


__all__ = ["visible", "attend", "window_attn", "window_attn_grad", "cp_window_attn", "rope_apply_axes", "append_rows",
           "cp_rope_append"]
