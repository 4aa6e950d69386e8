"""Pins of the float64 oracle of the serving operators (CPU), and the host-side parts and refusals of the
library's entry points for them (validation happens before any CUDA call)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S


@pytest.fixture(scope="module")
def ra():
    from context_long_sequence_ring_gb300 import build, ringattn
    if not os.path.exists(build.LIB):
        build.build()
    yield ringattn
    ringattn.rope_frequencies(64)      # leaves no error text behind


def _cache(seed, ctx, Hkv, d, bs, I, pcp, dcp):
    """Random tokens of several requests and the paged caches that hold them (NaN elsewhere)."""
    rng = np.random.default_rng(seed)
    V = bs * pcp * dcp
    nvb = [-(-x // V) for x in ctx]
    table = np.full((len(ctx), max(nvb) + 1), -1)
    ids = rng.permutation(sum(nvb) + 2)
    k = np.full((pcp * dcp, sum(nvb) + 2, Hkv, bs, d), np.nan)
    v = k.copy()
    toks, at = [], 0
    for r, x in enumerate(ctx):
        table[r, :nvb[r]] = ids[at:at + nvb[r]]
        at += nvb[r]
        kt, vt = rng.standard_normal((2, x, Hkv, d))
        for t in range(x):
            vb, dev, off = oracle.cp_token_location(t, bs, I, pcp, dcp)
            k[dev, table[r, vb], :, off], v[dev, table[r, vb], :, off] = kt[t], vt[t]
        toks.append((kt, vt))
    return k, v, table, toks


@pytest.mark.parametrize("bs,I,pcp,dcp", [(4, 2, 1, 1), (4, 2, 2, 2), (6, 1, 1, 3)])
def test_chunk_equals_attention_over_the_tokens(bs, I, pcp, dcp):
    ctx, n, Hq, Hkv, d = [1, 19, 7, 30], [1, 5, 0, 30], 4, 2, 8
    k, v, table, toks = _cache(1, ctx, Hkv, d, bs, I, pcp, dcp)
    qsl = np.concatenate([[1], 1 + np.cumsum(n)])
    q = np.random.default_rng(2).standard_normal((qsl[-1] + 2, Hq, d))
    O, L, A = S.chunk_attn(q, k, v, table, qsl, ctx, bs, I, pcp, dcp)
    for r in range(4):
        rows = slice(qsl[r], qsl[r + 1])
        if n[r]:
            o, l = oracle.attention_rows(q[rows], np.arange(ctx[r] - n[r], ctx[r]), *toks[r], True, None)
            assert np.abs(O[rows] - o).max() < 1e-12 and np.abs(L[rows] - l).max() < 1e-12
    assert np.isnan(O[0]).all() and np.isnan(L[-2:]).all()
    assert (A[1:-2] >= np.abs(O[1:-2]) - 1e-12).all()
    # one token per request is the decode
    one = S.chunk_attn(q[:4], k, v, table, np.arange(5), ctx, bs, I, pcp, dcp)
    o, l = oracle.cp_decode(q[:4], np.nan_to_num(k), np.nan_to_num(v), np.maximum(table, 0), ctx, bs, I, pcp, dcp, 2)
    assert np.abs(one[0] - o).max() < 1e-12 and np.abs(one[1] - l).max() < 1e-12


def test_chunk_rows_that_see_nothing():
    k, v, table, _ = _cache(3, [2, 3], 1, 4, 4, 2, 1, 1)
    q = np.ones((9, 2, 4))
    O, L, _ = S.chunk_attn(q, k, v, table, [0, 5, 9], [2, 0], 4, 2, 1, 1)
    assert (O[:3] == 0).all() and np.isneginf(L[:3]).all() and np.isfinite(L[3:5]).all()
    assert (O[5:] == 0).all() and np.isneginf(L[5:]).all()
    O, L, _ = S.chunk_attn(q, k, v, table, [0, 5, 9], [2, 0], 4, 2, 1, 1, causal=False)
    assert np.isfinite(L[:5]).all() and np.abs(L[0] - L[4]).max() == 0


def test_weights_are_softmax_columns():
    ctx, n, Hq, Hkv, d, bs, I, pcp, dcp = [11, 6], [4, 2], 4, 2, 8, 4, 2, 1, 2
    k, v, table, toks = _cache(4, ctx, Hkv, d, bs, I, pcp, dcp)
    q = np.random.default_rng(5).standard_normal((6, Hq, d))
    _, L, _ = S.chunk_attn(q, k, v, table, [0, 4, 6], ctx, bs, I, pcp, dcp)
    w_in = np.random.default_rng(6).random(k.shape[:4])
    w = S.attn_weights(q, L, k, table, [0, 4, 6], ctx, bs, I, pcp, dcp, w_in=w_in)
    w0 = S.attn_weights(q, L, k, table, [0, 4, 6], ctx, bs, I, pcp, dcp)
    got = S.token_rows(w0[..., None], table[0], range(11), bs, I, pcp, dcp)[..., 0]
    want = np.zeros((11, Hkv))
    for i in range(4):
        for h in range(Hq):
            e = np.exp(toks[0][0][:8 + i, h // 2] @ q[i, h] / np.sqrt(d))
            want[:8 + i, h // 2] += e / e.sum()
    assert np.abs(got - want).max() < 1e-12
    assert abs(np.nansum(w0) - 6 * Hq) < 1e-10                   # every row's weights sum to 1
    old = S.token_rows((w - w0)[..., None], table[0], range(11), bs, I, pcp, dcp)[..., 0]
    assert np.abs(old[:7] - S.token_rows(w_in[..., None], table[0], range(7), bs, I, pcp, dcp)[..., 0]).max() < 1e-12
    assert (old[7:] == 0).all()                                  # the chunk's own tokens start from 0
    L[0] = -np.inf
    assert abs(np.nansum(S.attn_weights(q, L, k, table, [0, 4, 6], ctx, bs, I, pcp, dcp)) - 5 * Hq) < 1e-10


def test_evict_hand_worked():
    nan = float("nan")
    assert S.evict_choice([1, 2, 3], 3, 0, 0) == [0, 1, 2]
    assert S.evict_choice([5, 1, 4, 4, 0, 9], 3, 0, 0) == [0, 2, 5]          # the earlier of the equal 4s
    assert S.evict_choice([5, 1, 4, 4, 0, 9], 3, 1, 1) == [0, 2, 5]
    assert S.evict_choice([0, 1, 4, 7, 0, 0], 3, 1, 1) == [0, 3, 5]
    assert S.evict_choice([0, 0, 0, 0], 2, 0, 0) == [0, 1]
    assert S.evict_choice([0.0, -0.0, 0.0, 0], 3, 0, 0) == [0, 1, 2]
    assert S.evict_choice([nan, -3.0, nan, 1], 2, 0, 0) == [1, 3]
    assert S.evict_choice([nan, nan, nan], 2, 0, 0) == [0, 1]
    assert S.evict_choice([9, 9, 1, 1], 2, 0, 2) == [2, 3]


@pytest.mark.parametrize("fresh", [False, True])
def test_evict_moves_tokens(fresh):
    ctx, bs, I, pcp, dcp = [9, 3], 4, 2, 1, 1
    k, v, table, toks = _cache(7, ctx, 2, 4, bs, I, pcp, dcp)
    w = np.random.default_rng(8).random(k.shape[:4])
    dst = np.array([[0, 1], [2, 3]]) if fresh else None
    if fresh:
        grow = lambda t: np.concatenate([np.full_like(t[:, :4], -7.0), t], axis=1)  # noqa: E731
        k, v, w, table = grow(k), grow(v), grow(w), np.where(table >= 0, table + 4, table)
    kept, new, k2, v2, w2 = S.evict(k, v, w, table, ctx, 5, bs, I, pcp, dcp, 1, 1, dst)
    assert new.tolist() == [5, 3] and (kept[1, :, 3:] == -1).all()
    to = table if dst is None else dst
    for r in range(2):
        out = S.token_rows(k2, to[r], range(new[r]), bs, I, pcp, dcp)
        for g in range(2):
            assert np.array_equal(out[:, g], toks[r][0][kept[r, g, :new[r]], g])
    if fresh:
        assert np.array_equal(k2[:, 4:], k[:, 4:], equal_nan=True) and (k2[0, 1, :, 2:] == -7).all()


def test_rope_forms():
    rng = np.random.default_rng(9)
    x = rng.standard_normal((5, 3, 12))
    pos = [0, 1, 77, 5000, 2 ** 24 - 1]
    f, m = S.rope_frequencies(12)
    assert np.abs(S.rope_apply(x, pos, f) - oracle.apply_rope(x, pos)).max() < 1e-7   # angles of 1.6e7 rad
    assert np.abs(S.rope_apply(x, pos[:4], f, idx=[1, -1, 0, 4])[1]).max() == 0
    # interleaved is half with the components reordered
    order = [0, 2, 4, 1, 3, 5]
    f6 = f[:3]
    y = S.rope_apply(x, pos, f6, 1.25, "interleaved")
    z = S.rope_apply(np.concatenate([x[..., order], x[..., 6:]], -1), pos, f6, 1.25, "half")
    assert np.abs(y[..., order] - z[..., :6]).max() < 1e-12 and np.array_equal(y[..., 6:], x[..., 6:])
    # the backward direction is the transpose: <dy, R x> = <R^T dy, x>, against differences
    dy = rng.standard_normal(x.shape)
    g = S.rope_apply(dy, pos, f6, 1.25, "interleaved", backward=True)
    for at in [(2, 1, 3), (3, 0, 0), (4, 2, 5), (1, 1, 8)]:
        e = np.zeros_like(x)
        e[at] = 1e-3
        diff = ((S.rope_apply(x + e, pos, f6, 1.25, "interleaved") - S.rope_apply(x - e, pos, f6, 1.25, "interleaved"))
                * dy).sum() / 2e-3
        assert abs(diff - g[at]) < 1e-9
    assert np.abs(S.rope_apply(S.rope_apply(x, pos, f), pos, f, backward=True) - x).max() < 1e-9


@pytest.mark.parametrize("rot", [2, 4, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 4.0), ("yarn", 16.0)])
def test_frequencies_of_the_library(ra, rot, scaling, factor):
    if scaling == "ntk" and rot == 2:
        with pytest.raises(ra.RingAttnError):
            ra.rope_frequencies(rot, 10000.0, scaling, factor)
        return
    f, m = ra.rope_frequencies(rot, 500000.0, scaling, factor, 8192)
    F, M = S.rope_frequencies(rot, 500000.0, scaling, factor, 8192)
    assert np.abs(f.numpy() / F - 1).max() < 1e-13 and abs(m - M) < 1e-14   # a few roundings of 2^-53 each
    if scaling == "ntk":
        assert f[0] == 1.0 and abs(f[-1] * factor / 500000.0 ** (-(rot - 2.0) / rot) - 1) < 1e-12
    if scaling == "yarn" and rot >= 64:                                     # fast ones kept, slow ones divided
        base = S.rope_frequencies(rot, 500000.0)[0]
        assert f[0] == 1.0 and abs(f[-1] * factor / base[-1] - 1) < 1e-13


def test_frequency_refusals(ra):
    for args in [(64, 1.0), (64, float("inf")), (63,), (0,), (258,), (64, 1e4, "linear", 0.5),
                 (64, 1e4, "yarn", 2.0, 0.0), (64, 1e4, "linear", float("nan"))]:
        with pytest.raises(ra.RingAttnError) as e:
            ra.rope_frequencies(*args)
        assert e.value.status == ra.RA_ERR_INVALID_ARG, args
    with pytest.raises(KeyError):
        ra.rope_frequencies(64, scaling="cubic")


P = ctypes.c_void_p(1 << 20)      # never dereferenced: validation fails first
INV, UNS = 1, 2


def test_rope_apply_refusals(ra):
    f = (ctypes.c_double * 128)(*([1.0] * 128))

    def run(**kw):
        a = dict(src=1 << 20, src_rows=8, srs=512, shs=64, dst=1 << 24, drs=512, dhs=64, rows=8, H=8, d=64, rot=64,
                 dt=1, style=0, idx=None, pos=P, f=f, m=1.0, b=0)
        a.update(kw)
        return ra.lib().ra_rope_apply(ctypes.c_void_p(a["src"]), a["src_rows"], a["srs"], a["shs"],
                                      ctypes.c_void_p(a["dst"]), a["drs"], a["dhs"], a["rows"], a["H"], a["d"], a["rot"],
                                      a["dt"], a["style"], a["idx"], a["pos"], a["f"], a["m"], a["b"], None)

    bad = (ctypes.c_double * 128)(*([7.0] * 128))
    nan = (ctypes.c_double * 128)(*([float("nan")] * 128))
    for kw in [dict(rot=63), dict(rot=0), dict(rot=66), dict(rot=258, d=512), dict(d=0), dict(d=1025), dict(H=0), dict(dt=2),
               dict(style=2), dict(rows=-1, src_rows=-1), dict(src_rows=9), dict(f=bad), dict(f=nan), dict(f=None),
               dict(m=float("inf")), dict(srs=-1), dict(dhs=32), dict(drs=0), dict(drs=500), dict(src=0), dict(pos=None),
               dict(src=(1 << 20) + 1), dict(dst=1 << 20, drs=513), dict(dst=(1 << 20) + 64),
               dict(idx=P, dst=1 << 20), dict(dst=(1 << 20) - 128)]:
        assert run(**kw) == INV and ra.last_error() != "", kw
    assert run(rows=0, src_rows=0, src=0) == 0


def test_chunk_attn_and_weights_refusals(ra):
    def args(kw):
        a = dict(q=P, k=P, v=P, bt=P, qsl=P, ctx=P, T=9, R=2, Hq=8, Hkv=4, d=128, bs=32, I=16, pcp=2, dcp=2, mv=4, nb=16,
                 c=1, s=0.0, o=P, dt=1, lse=P, ws=P, wsb=1 << 30, w=P)
        a.update(kw)
        return a

    def chunk(**kw):
        a = args(kw)
        return ra.lib().ra_cp_chunk_attn(*(a[x] for x in ("q", "k", "v", "bt", "qsl", "ctx", "T", "R", "Hq", "Hkv", "d", "bs",
                                                          "I", "pcp", "dcp", "mv", "nb", "c", "s", "o", "dt", "lse", "ws",
                                                          "wsb")), None)

    def weights(**kw):
        a = args(kw)
        return ra.lib().ra_cp_attn_weights(*(a[x] for x in ("q", "lse", "k", "bt", "qsl", "ctx", "T", "R", "Hq", "Hkv", "d",
                                                            "bs", "I", "pcp", "dcp", "mv", "nb", "c", "s")), None, a["w"], None)

    odd = ctypes.c_void_p((1 << 20) + 8)
    both = [(dict(R=0), INV), (dict(Hq=0), INV), (dict(Hq=6), INV), (dict(T=-1), INV), (dict(T=1 << 29), INV),
            (dict(bs=32, I=12), INV), (dict(d=96), UNS), (dict(Hq=4 * 65), UNS), (dict(bs=24, I=8), UNS), (dict(nb=0), INV),
            (dict(nb=1 << 31), INV), (dict(nb=1 << 27, Hkv=8), INV), (dict(mv=0), INV), (dict(pcp=0), INV),
            (dict(q=None), INV), (dict(k=None), INV), (dict(bt=None), INV), (dict(qsl=None), INV), (dict(ctx=None), INV),
            (dict(q=odd), INV), (dict(k=odd), INV)]
    for kw, st in both:
        assert chunk(**kw) == st and ra.last_error() != "", kw
        assert weights(**kw) == st and ra.last_error() != "", kw
    for kw in [dict(v=None), dict(v=odd), dict(o=None), dict(o=odd), dict(dt=7), dict(ws=None), dict(ws=odd), dict(wsb=8)]:
        assert chunk(**kw) == INV, kw
    assert "workspace" in ra.last_error()
    for kw in [dict(lse=None), dict(w=None), dict(w=ctypes.c_void_p((1 << 20) + 2))]:
        assert weights(**kw) == INV, kw
    assert chunk(T=0) == 0
    assert ra.cp_chunk_attn_workspace_size(8, 4, 128) >= 16
    n = ctypes.c_size_t(0)
    assert ra.lib().ra_cp_chunk_attn_workspace_size(0, 4, 128, ctypes.byref(n)) == INV


def test_evict_refusals(ra):
    def run(**kw):
        a = dict(k=P, v=ctypes.c_void_p(1 << 22), w=P, bt=P, dbt=None, ctx=P, R=2, Hkv=4, d=64, dt=1, bs=32, I=16, pcp=1,
                 dcp=2, mv=4, dmv=0, nb=16, keep=10, sink=2, rec=3, kept=P, new=ctypes.c_void_p(1 << 23))
        a.update(kw)
        return ra.lib().ra_cp_evict(*(a[x] for x in ("k", "v", "w", "bt", "dbt", "ctx", "R", "Hkv", "d", "dt", "bs", "I", "pcp",
                                                     "dcp", "mv", "dmv", "nb", "keep", "sink", "rec", "kept", "new")), None)

    for kw, st in [(dict(keep=0), INV), (dict(sink=-1), INV), (dict(rec=-1), INV), (dict(sink=8), INV), (dict(R=0), INV),
                   (dict(I=12), INV), (dict(dt=3), INV), (dict(d=0), INV), (dict(d=4), UNS), (dict(d=16384), UNS),
                   (dict(dbt=P), INV), (dict(k=None), INV), (dict(v=P), INV), (dict(w=None), INV), (dict(kept=None), INV),
                   (dict(new=P), INV), (dict(new=None), INV), (dict(k=ctypes.c_void_p((1 << 20) + 4)), INV),
                   (dict(sink=2 ** 31 - 1, rec=2 ** 31 - 1, keep=2 ** 31 - 1), INV), (dict(R=65536), INV), (dict(keep=2 ** 30 + 1), INV),
                   (dict(R=16384), INV), (dict(bs=2 ** 24, I=16), INV)]:
        assert run(**kw) == st and ra.last_error() != "", kw


def test_binding_refusals_without_a_device(ra):
    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        ra.rope_apply(x, torch.zeros(4, dtype=torch.int32), torch.ones(2, dtype=torch.float64))
    c = torch.zeros(1, 2, 1, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ra.cp_chunk_attn(c[0, :, 0, :2], c, c, i[None], i, i[:1], 16, 1, 1)
    with pytest.raises(ValueError):
        ra.cp_evict(c, c, torch.zeros(1, 2, 1, 16), i[None], i[:1], 4, 16, 1, 1)


@pytest.mark.parametrize("fresh", [False, True])
def test_evict_by_sort_is_the_same_choice(fresh):
    ctx, bs, I, pcp, dcp, keep = [29, 5, 40], 4, 2, 1, 2, 12
    k, v, table, _ = _cache(17, ctx, 2, 4, bs, I, pcp, dcp)
    w = np.floor(np.random.default_rng(18).random(k.shape[:4]) * 6)
    w[w == 5], w[w == 4], w[w == 3] = np.nan, -0.0, -1.0
    dst = None
    if fresh:
        grow = lambda t: np.concatenate([np.full_like(t[:, :6], -7.0), t], axis=1)  # noqa: E731
        k, v, w, table, dst = grow(k), grow(v), grow(w), np.where(table >= 0, table + 6, table), np.arange(6).reshape(3, 2)
    for sink, recent in ((0, 0), (1, 3), (12, 0)):
        want, _, k2, v2, w2 = S.evict(k, v, w, table, ctx, keep, bs, I, pcp, dcp, sink, recent, dst)
        kept, moves = S.evict_by_sort(w, table, ctx, keep, bs, I, pcp, dcp, sink, recent, dst)
        assert np.array_equal(kept, want)
        for old, new in ((k, k2), (v, v2), (w, w2)):
            got = old.copy()
            for _, g, src, to in moves:
                got[to[0], to[1], g, to[2]] = old[src[0], src[1], g, src[2]]
            assert np.array_equal(got, new, equal_nan=True)


def test_rope_apply_rows_past_32_bits_are_refused(ra):
    """A row of 2^31 components or more: the threads of a row would not fit in 32 bits."""
    f = (ctypes.c_double * 128)(*([1.0] * 128))
    for H, d, rows in [(1 << 25, 64, 1), (1 << 29, 128, 1), (1 << 30, 64, 3), ((1 << 31) - 1, 2, 1)]:
        st = ra.lib().ra_rope_apply(P, rows, 0, 0, ctypes.c_void_p(1 << 44), H * d, d, rows, H, d, 2, 1, 0, None, P, f, 1.0, 0,
                                    None)
        assert st == INV and "H*d" in ra.last_error(), (H, d)
