"""Serving operators around the sharded paged cache: attention of a chunk of
new tokens, the attention weight of cached tokens, eviction by it, and rotary
positions in their general form.  Test infrastructure only.

Sources: vLLM-Ascend developer guide "Context Parallel (CP)" (chunked prefill,
section "Block table"); guijiagi.com tag page "Ring Attention", article on the
evolution of long-context techniques (rotary form; table of extrapolation
methods).  The eviction rule is the definition stated in ``evict``.

Parity status: pinned (chunk attention against plain attention over the tokens
and against the one-token decode, weights against explicit softmax matrices,
eviction against hand-worked examples, rotations against complex products and
differences).
"""

from __future__ import annotations

import numpy as np

from .attention import _as64
from .kvcache import cp_token_location


def token_rows(cache, table_row, tokens, bs, I, pcp, dcp):
    """Rows [len(tokens), Hkv, ...] of some tokens of one request."""
    out = np.zeros((len(tokens),) + (cache.shape[2],) + cache.shape[4:], dtype=np.float64)
    for i, x in enumerate(tokens):
        vb, dev, off = cp_token_location(int(x), bs, I, pcp, dcp)
        out[i] = cache[dev, table_row[vb], :, off]
    return out


def _softmax_rows(q, k, seen, scale):
    """exp(scores - max) [n, Hq, N], its sum and the max of the visible scores."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    s = np.einsum("nhd,khd->nhk", q, np.repeat(k, G, axis=1)) * (scale or 1.0 / np.sqrt(d))
    s = np.where(seen[:, None, :], s, -np.inf)
    m = s.max(axis=2, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, :, None])
    return e, e.sum(axis=2), m


def chunk_attn(q, k_cache, v_cache, block_table, qsl, ctx_lens, bs, I, pcp, dcp, causal=True, scale=None):
    """Per request r: queries q[qsl[r]:qsl[r+1]] are its last tokens; each sees the cached tokens
    x < ctx_lens[r] (causal: x <= its own position).  Returns (O, LSE, A) over all rows, A the same
    average of |V| (for error bounds); rows of no request are NaN, rows that see nothing 0 / -inf."""
    q, kc, vc = _as64(q), _as64(k_cache), _as64(v_cache)
    T, Hq, d = q.shape
    O, A, L = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    G = Hq // kc.shape[2]
    for r, ctx in enumerate(ctx_lens):
        a, b = int(qsl[r]), int(qsl[r + 1])
        n, ctx = b - a, int(ctx)
        k = token_rows(kc, block_table[r], range(ctx), bs, I, pcp, dcp)
        v = np.repeat(token_rows(vc, block_table[r], range(ctx), bs, I, pcp, dcp), G, axis=1)
        pos = ctx - n + np.arange(n)
        seen = np.arange(ctx)[None, :] <= pos[:, None] if causal else np.ones((n, ctx), dtype=bool)
        e, l, m = _softmax_rows(q[a:b], k, seen, scale)
        ls = np.where(l > 0, l, 1.0)
        O[a:b] = np.einsum("nhk,khd->nhd", e, v) / ls[:, :, None]
        A[a:b] = np.einsum("nhk,khd->nhd", e, np.abs(v)) / ls[:, :, None]
        L[a:b] = np.where(l > 0, m + np.log(ls), -np.inf)
    return O, L, A


def attn_weights(q, lse, k_cache, block_table, qsl, ctx_lens, bs, I, pcp, dcp, w_in=None, causal=True, scale=None):
    """w[dev, block, g, slot] of every token x < ctx_lens[r]: (old ? w_in : 0) + sum of e^{s - lse} over
    the queries and heads of g that see x; NaN in every other slot."""
    q, kc, lse = _as64(q), _as64(k_cache), _as64(lse)
    W, NB, Hkv, _, d = kc.shape
    Hq = q.shape[1]
    out = np.full(kc.shape[:4], np.nan)
    for r, ctx in enumerate(ctx_lens):
        a, b = int(qsl[r]), int(qsl[r + 1])
        n, ctx = b - a, int(ctx)
        k = np.repeat(token_rows(kc, block_table[r], range(ctx), bs, I, pcp, dcp), Hq // Hkv, axis=1)
        s = np.einsum("nhd,khd->nhk", q[a:b], k) * (scale or 1.0 / np.sqrt(d))
        for x in range(ctx):
            vb, dev, off = cp_token_location(x, bs, I, pcp, dcp)
            old = not causal or x < ctx - n
            w = _as64(w_in[dev, block_table[r][vb], :, off]) if (w_in is not None and old) else np.zeros(Hkv)
            for i in range(n):
                if causal and x > ctx - n + i:
                    continue
                live = np.isfinite(lse[a + i])
                p = np.where(live, np.exp(s[i, :, x] - np.where(live, lse[a + i], 0.0)), 0.0)
                w = w + p.reshape(Hkv, -1).sum(axis=1)
            out[dev, block_table[r][vb], :, off] = w
    return out


def evict_choice(w, keep, n_sink, n_recent):
    """Positions that one K/V head keeps of a context with weights w [N], ascending: all of them when
    N <= keep; else the first n_sink, the last n_recent and the heaviest others (of equal weights the
    earlier one; NaN lightest)."""
    N = len(w)
    if N <= keep:
        return list(range(N))
    mid = range(n_sink, N - n_recent)
    value = lambda x: -np.inf if np.isnan(w[x]) else float(w[x])  # noqa: E731
    nan = lambda x: bool(np.isnan(w[x]))  # noqa: E731
    best = sorted(mid, key=lambda x: (nan(x), -value(x), x))[:keep - n_sink - n_recent]
    return sorted(list(range(n_sink)) + best + list(range(N - n_recent, N)))


def evict(k_cache, v_cache, weights, block_table, ctx_lens, keep, bs, I, pcp, dcp, n_sink=0, n_recent=0,
          dst_block_table=None):
    """(kept [R, Hkv, keep], new_lens [R], k_cache, v_cache, weights) after the eviction."""
    k, v, w = (np.array(t, copy=True) for t in (k_cache, v_cache, weights))
    R, Hkv = len(ctx_lens), k.shape[2]
    kept = np.full((R, Hkv, keep), -1, dtype=np.int64)
    new = np.minimum(np.asarray(ctx_lens), keep)
    dst = block_table if dst_block_table is None else dst_block_table
    for r in range(R):
        at = [cp_token_location(x, bs, I, pcp, dcp) for x in range(int(ctx_lens[r]))]
        for g in range(Hkv):
            ids = evict_choice([weights[dev, block_table[r][vb], g, off] for vb, dev, off in at], keep, n_sink, n_recent)
            kept[r, g, :len(ids)] = ids
            for j, x in enumerate(ids):
                vb, dev, off = at[x]
                vb2, dev2, off2 = at[j]
                for new_t, old_t in ((k, k_cache), (v, v_cache), (w, weights)):
                    new_t[dev2, dst[r][vb2], g, off2] = old_t[dev, block_table[r][vb], g, off]
    return kept, new, k, v, w


def evict_by_sort(weights, block_table, ctx_lens, keep, bs, I, pcp, dcp, n_sink=0, n_recent=0, dst_block_table=None):
    """The same choice by sorting whole rows, for long contexts: (kept [R, Hkv, keep], moves), where moves lists, per
    request and head, (device, block, slot) arrays of the tokens' old places and of their new ones."""
    w = np.asarray(weights, dtype=np.float64)
    R, Hkv = len(ctx_lens), w.shape[2]
    table = np.asarray(block_table, dtype=np.int64)
    dst = table if dst_block_table is None else np.asarray(dst_block_table, dtype=np.int64)
    V = bs * pcp * dcp

    def at(row, x):
        lbi = x % V // I
        return lbi % (pcp * dcp), row[x // V], lbi // (pcp * dcp) * I + x % V % I

    kept, moves = np.full((R, Hkv, keep), -1, dtype=np.int64), []
    for r in range(R):
        N = int(ctx_lens[r])
        pos = np.arange(N)
        dev, blk, off = at(table[r], pos)
        for g in range(Hkv):
            ids = pos
            if N > keep:
                mid = pos[n_sink:N - n_recent]
                val = w[dev, blk, g, off][mid]
                nan = np.isnan(val)
                order = np.lexsort((mid, -np.where(nan, 0.0, val), nan))[:keep - n_sink - n_recent]
                ids = np.concatenate([pos[:n_sink], np.sort(mid[order]), pos[N - n_recent:]])
            kept[r, g, :len(ids)] = ids
            moves.append((r, g, (dev[ids], blk[ids], off[ids]), at(dst[r], np.arange(len(ids)))))
    return kept, moves


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, trained_len=32768.0):
    """(inv_freq [rot/2], mscale): theta_i = base^(-2i/rot) and its changes for longer contexts."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        turns = trained_len * f / (2 * np.pi)
        g = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return (1 - g) * f / factor + g * f, 0.1 * np.log(factor) + 1.0
    return f, 1.0


def rope_apply(x, positions, inv_freq, mscale=1.0, style="half", backward=False, idx=None):
    """Pairs of the first 2*len(inv_freq) components as complex numbers, times mscale * e^{+-i m f}; the
    rest copied.  positions per OUTPUT row; out[r] from x[idx[r]] (zero rows where idx[r] < 0)."""
    x = _as64(x)
    if idx is not None:
        idx = np.asarray(idx)
        x = np.where((idx >= 0)[:, None, None], x[np.maximum(idx, 0)], 0.0)
    half = len(inv_freq)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None, :]
    turn = mscale * np.exp((-1j if backward else 1j) * a)[:, None, :]
    u, v = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = (x[:, :, u] + 1j * x[:, :, v]) * turn
    y = x.copy()
    y[:, :, u], y[:, :, v] = z.real, z.imag
    return y


__all__ = ["token_rows", "chunk_attn", "attn_weights", "evict_choice", "evict", "evict_by_sort", "rope_frequencies", "rope_apply"]
