"""GPU parity of the serving operators (chunk attention over the paged cache, attention weights, eviction,
rotary positions) against the float64 oracle.

Tolerances.  Chunk attention: P is rounded to bf16 for the tensor cores (relative 2^-8 of each term, so of
A = sum p|v|/l), the output is rounded to its type (2^-8 or 2^-24 of |O|), and the scores, exps and sums are
fp32: a score is off by at most (d + 2) 2^-24 sum|q k| scale, about 130 * 2^-24 * 7.5 = 2^-14 for normal q, k,
each weight and the row sum by that factor, with ex2 and the running rescale well inside 2^-12 together.
So |O - O_ref| <= 2^-8 (A + |O|) + 2^-11 A, and |LSE - LSE_ref| <= 2^-12.
Weights: each term e^{s - lse} is off by 2^-14 (score) + |s - lse| 2^-23, sums of n fp32 terms by n 2^-24:
within 2^-12 of the value for the sizes here.
Rotations: the angle is off by 2^-23 turns (7.5e-7 rad), sin and cos by 2^-22 and products by three fp32
roundings: 1.2e-6 < 2^-19 of |a| + |b|, plus the output's rounding."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S
from tests._gpu import ra_lib, check_status

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]
DEV = torch.device("cuda")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ra():
    return ra_lib()


def paged(seed, ctx, Hkv, d, bs, I, pcp, dcp, dt=BF, poison=True, spare=2):
    """Paged caches with random tokens of several requests; every other slot NaN, table entries past the
    context -1.  Returns CPU tensors (k, v, table)."""
    g = torch.Generator().manual_seed(seed)
    W, V = pcp * dcp, bs * pcp * dcp
    nvb = [-(-int(x) // V) for x in ctx]
    nb = sum(nvb) + spare
    table = torch.full((len(ctx), max(nvb) + 1), -1, dtype=torch.int32)
    ids = torch.randperm(nb, generator=g).to(torch.int32)
    k = torch.randn((W, nb, Hkv, bs, d), generator=g).to(dt)
    v = torch.randn((W, nb, Hkv, bs, d), generator=g).to(dt)
    live = torch.zeros((W, nb, bs), dtype=torch.bool)
    at = 0
    for r, x in enumerate(ctx):
        table[r, :nvb[r]] = ids[at:at + nvb[r]]
        at += nvb[r]
        p = torch.arange(int(x))
        o = p % V
        lbi = o // I
        live[lbi % W, table[r, p // V].long(), lbi // W * I + o % I] = True
    if poison:
        dead = ~live[:, :, None, :, None]
        k.masked_fill_(dead, float("nan"))
        v.masked_fill_(dead, float("nan"))
    return k, v, table, ids[at:]


def batch(seed, n, Hq, d, before=0, after=0):
    qsl = torch.tensor(np.concatenate([[before], before + np.cumsum(n)]), dtype=torch.int32)
    g = torch.Generator().manual_seed(seed + 1000)
    return torch.randn((int(qsl[-1]) + after, Hq, d), generator=g).to(BF), qsl


def dev(*ts):
    return [t.to(DEV) for t in ts]


def assert_chunk(o, lse, ref, rows=None):
    O, L, A = (t if rows is None else t[rows] for t in ref)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(o - O)
    assert np.isfinite(o).all()
    assert (err <= 2.0 ** -8 * (A + np.abs(O)) + 2.0 ** -11 * A).all(), err.max()
    assert np.array_equal(np.isneginf(lse), np.isneginf(L)) and not np.isnan(lse).any()
    both = np.isfinite(L)
    assert (np.abs(lse[both] - L[both]) <= 2.0 ** -12).all(), np.abs(lse[both] - L[both]).max()


CHUNKS = [
    # ctx, n, Hq, Hkv, d, bs, I, pcp, dcp
    ([1], [1], 4, 2, 128, 128, 16, 1, 1),
    ([1, 2, 129, 127], [1, 1, 1, 1], 8, 1, 64, 16, 16, 1, 1),
    ([300, 5, 77], [3, 5, 1], 6, 2, 128, 32, 4, 2, 2),
    ([257, 0, 300, 128], [33, 0, 300, 128], 6, 2, 64, 64, 16, 1, 2),
    ([700], [260], 5, 5, 128, 128, 128, 2, 4),
    ([700], [517], 8, 2, 128, 48, 16, 1, 1),
    ([130, 500, 20], [130, 66, 20], 16, 1, 64, 16, 1, 1, 3),
    ([1500, 900], [2, 9], 64, 1, 128, 128, 16, 2, 4),
    ([200, 333], [130, 40], 9, 3, 64, 256, 32, 1, 1),
    ([1029, 64, 3], [4, 1, 2], 40, 8, 128, 80, 80, 1, 2),
    ([2100], [1], 32, 8, 128, 128, 16, 2, 4),
]
# few rows a tile, units of 16 and 32, every group size
FEW = [
    ([900, 40, 17], [1, 4, 16], 3, 3, 128, 16, 1, 1, 1),
    ([513, 260], [5, 3], 10, 2, 64, 32, 2, 2, 2),
    ([400, 1300, 31], [2, 1, 3], 16, 2, 128, 64, 16, 1, 2),
    ([700, 129], [1, 2], 32, 2, 64, 48, 48, 1, 1),
    ([1500], [4], 4, 1, 128, 128, 128, 1, 4),
    ([1600, 5], [1, 1], 34, 2, 128, 32, 8, 1, 1),
]


@pytest.mark.parametrize("case", CHUNKS + FEW, ids=lambda c: "%s-%s-h%d.%d-d%d-b%d.%d-w%d" % (c[0], c[1], c[2], c[3], c[4], c[5],
                                                                                  c[6], c[7] * c[8]))
@pytest.mark.parametrize("causal", [True, False])
def test_chunk_attn(ra, case, causal):
    ctx, n, Hq, Hkv, d, bs, I, pcp, dcp = case
    k, v, table, _ = paged(sum(ctx), ctx, Hkv, d, bs, I, pcp, dcp)
    q, qsl = batch(sum(ctx), n, Hq, d)
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, bs, I, pcp, dcp, causal)
    qd, kd, vd, td, sd, cd = dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32))
    o, lse = ra.cp_chunk_attn(qd, kd, vd, td, sd, cd, I, pcp, dcp, causal=causal)
    check_status(ra)
    assert_chunk(o, lse, ref)
    o32, lse32 = ra.cp_chunk_attn(qd, kd, vd, td, sd, cd, I, pcp, dcp, causal=causal, out_dtype=torch.float32)
    assert o32.dtype == torch.float32 and torch.equal(o32.to(BF), o) and torch.equal(lse32, lse)


@pytest.mark.parametrize("d,bs,Hq,Hkv", [(128, 32, 8, 2), (64, 16, 12, 3)])
def test_chunk_attn_many_requests_of_all_kinds(ra, d, bs, Hq, Hkv):
    """Several tiles to a CTA, one kind after another: single tokens, drafts, pieces of prompts, nothing."""
    rng = np.random.default_rng(d)
    n = rng.choice([0, 1, 1, 2, 4, 6, 20, 50, 90], size=330)
    ctx = np.maximum(n + rng.integers(-3, 70, size=330), 0)
    k, v, table, _ = paged(d, ctx.tolist(), Hkv, d, bs, 4, 1, 2)
    q, qsl = batch(d, n, Hq, d)
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, bs, 4, 1, 2)
    args = dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32))
    o, lse = ra.cp_chunk_attn(*args, 4, 1, 2)
    check_status(ra)
    assert_chunk(o, lse, ref)
    w = ra.cp_attn_weights(args[0], lse, args[1], *args[3:], 4, 1, 2)
    check_status(ra)
    want = S.attn_weights(q, lse.cpu(), k, table, qsl, ctx, bs, 4, 1, 2)
    assert_weights(w, want)


@pytest.mark.parametrize("d,bs,I,pcp", [(64, 16, 16, 1), (64, 64, 8, 2), (128, 32, 16, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunk_attn_long_parts(ra, d, bs, I, pcp, causal):
    """Enough keys that each CTA walks many tiles of several row tiles of both kinds, borders anywhere."""
    rng = np.random.default_rng(bs)
    n = rng.choice([1, 1, 3, 7, 70, 150], size=40)
    ctx = n + rng.integers(200, 1900, size=40)
    Hq, Hkv = 12, 4
    k, v, table, _ = paged(bs, ctx.tolist(), Hkv, d, bs, I, pcp, 1)
    q, qsl = batch(bs, n, Hq, d)
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, bs, I, pcp, 1, causal)
    o, lse = ra.cp_chunk_attn(*dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32)), I, pcp, 1, causal=causal)
    check_status(ra)
    assert_chunk(o, lse, ref)


def test_chunk_attn_nan_queries_and_keys_reach_only_who_sees_them(ra):
    ctx, n, Hq, Hkv, d = [300, 40, 70], [1, 9, 40], 4, 2, 128
    k, v, table, _ = paged(31, ctx, Hkv, d, 16, 16, 1, 1)
    q, qsl = batch(31, n, Hq, d)
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, 16, 16, 1, 1)
    q[1, 0] = float("nan")                       # one head of a query of request 1
    k[0, table[2, 4], 1, 5] = float("nan")       # token 69 of request 2: K/V head 1, seen by its last query alone
    o, lse = ra.cp_chunk_attn(*dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1)
    check_status(ra)
    bad = torch.zeros((50, Hq), dtype=torch.bool)
    bad[1, 0] = True
    bad[49, 2:] = True
    assert o.cpu()[bad].isnan().all() and lse.cpu()[bad].isnan().all()
    assert not o.cpu()[~bad].isnan().any()
    good = ~bad.numpy()
    O, L, A = ref
    err = np.abs(o.double().cpu().numpy() - O)
    assert (err[good] <= (2.0 ** -8 * (A + np.abs(O)) + 2.0 ** -11 * A)[good]).all()
    assert (np.abs(lse.double().cpu().numpy() - L)[good] <= 2.0 ** -12).all()


def test_chunk_attn_rows_that_see_nothing_and_rows_of_nobody(ra):
    ctx, n, Hq, Hkv, d = [3, 0, 40, 6], [7, 4, 2, 0], 4, 2, 128
    k, v, table, _ = paged(5, ctx, Hkv, d, 16, 16, 1, 1)
    q, qsl = batch(5, n, Hq, d, before=3, after=5)
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, 16, 16, 1, 1)
    o, lse = torch.full(q.shape, 7.0, dtype=BF, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
    ra.cp_chunk_attn(*dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1, o=o, lse=lse)
    check_status(ra)
    mine = slice(3, 3 + sum(n))
    assert_chunk(o[mine], lse[mine], ref, mine)
    rest = np.r_[0:3, 3 + sum(n):q.shape[0]]
    assert (o[rest] == 7).all() and (lse[rest] == 7).all()


def test_chunk_attn_scale_sharp_and_large_values(ra):
    ctx, n, Hq, Hkv, d = [600], [70], 4, 2, 64
    k, v, table, _ = paged(6, ctx, Hkv, d, 16, 4, 1, 2)
    q, qsl = batch(6, n, Hq, d)
    k[..., 0] *= 40      # scores of tens: a growing maximum, weights that underflow
    v = v * 100
    # scores off by (d + 2) 2^-24 sum|q k|: sum|q k| up to ~6 * 160 + 60, scale 0.3: weights off by 1.3e-3 each
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, 16, 4, 1, 2, True, 0.3)
    o, lse = ra.cp_chunk_attn(*dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32)), 4, 1, 2, scale=0.3)
    check_status(ra)
    O, L, A = ref
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * (A + np.abs(O)) + 2.6e-3 * A).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.6e-3).all()


def test_chunk_attn_shared_blocks_and_future_tokens(ra):
    """Two requests on one prefix block; V and K of tokens that a query does not see are finite but huge."""
    ctx, n, Hq, Hkv, d, bs = [40, 33], [20, 17], 4, 2, 64, 16
    k, v, table, _ = paged(7, ctx, Hkv, d, bs, 16, 1, 1)
    table[1, 0] = table[0, 0]
    last = table[0, 2]
    v[0, last, :, 7] = 3e38
    k[0, last, :, 7] = 50.0
    q, qsl = batch(7, n, Hq, d)
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, bs, 16, 1, 1)
    o, lse = ra.cp_chunk_attn(*dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1)
    check_status(ra)
    rows = np.r_[0:19, 20:37]        # all but the one query that sees token 39
    assert_chunk(o[rows], lse[rows], ref, rows)


def test_chunk_attn_matches_decode_and_segmented_prefill(ra):
    ctx, Hq, Hkv, d, bs, I, pcp, dcp = [900, 17, 2049], 16, 4, 128, 64, 16, 2, 2
    k, v, table, _ = paged(8, ctx, Hkv, d, bs, I, pcp, dcp, poison=False)
    q, qsl = batch(8, [1, 1, 1], Hq, d)
    kd, vd, td, cd = dev(k, v, table.clamp(min=0), torch.tensor(ctx, dtype=torch.int32))
    o, lse = ra.cp_chunk_attn(q.to(DEV), kd, vd, td, qsl.to(DEV), cd, I, pcp, dcp, out_dtype=torch.float32)
    o2, lse2 = ra.cp_decode(q.to(DEV), kd, vd, td, cd, I, pcp, dcp, out_dtype=torch.float32)
    check_status(ra)
    # each side is within the bound above of the exact value; A <= max|v| < 6
    assert (o - o2).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -11) * 6 and (lse - lse2).abs().max() <= 2.0 ** -11
    q, qsl = batch(9, [500], Hq, d)
    pos = torch.arange(2049, dtype=torch.int32, device=DEV)
    kt, vt = ra.cp_kv_gather(kd, vd, td[2:].contiguous(), torch.tensor([0, 2049], dtype=torch.int32, device=DEV), pos, I,
                             pcp, dcp)
    o, lse = ra.cp_chunk_attn(q.to(DEV), kd, vd, td[2:].contiguous(), qsl.to(DEV), cd[2:], I, pcp, dcp)
    o2, lse2 = ra.segmented_prefill_fwd(q.to(DEV), kt, vt, 2049 - 500, 1024)
    check_status(ra)
    assert (o.float() - o2.float()).abs().max() <= 2 * (2.0 ** -7 + 2.0 ** -11) * 6 and \
        (lse - lse2).abs().max() <= 2.0 ** -11


def test_chunk_attn_bad_tables_and_ranges_are_reported(ra):
    ctx, n, Hq, Hkv, d, bs = [40, 90, 33], [2, 3, 4], 4, 2, 64, 16
    k, v, table, _ = paged(10, ctx, Hkv, d, bs, 16, 1, 1)
    q, qsl = batch(10, n, Hq, d)
    keep = torch.ones(90, dtype=torch.bool)
    for bad in (-1, k.shape[1], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 2] = bad                       # tokens 32..47 of request 1 are left out
        o, lse = ra.cp_chunk_attn(*dev(q, k, v, t, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS
        ref = S.chunk_attn(q, k, v, table, qsl, ctx, bs, 16, 1, 1)
        rows = np.r_[0:2, 5:9]
        assert_chunk(o[rows], lse[rows], ref, rows)
        keep[32:48] = False
        kt = S.token_rows(k.double().numpy(), table[1].numpy(), range(90), bs, 16, 1, 1)
        vt = S.token_rows(v.double().numpy(), table[1].numpy(), range(90), bs, 16, 1, 1)
        for i in range(3):
            seen = np.nonzero(keep.numpy() & (np.arange(90) <= 87 + i))[0]
            Or, Lr = oracle.attention_rows(q[2 + i:3 + i], [len(seen)], kt[seen], vt[seen], False, None)
            Ar, _ = oracle.attention_rows(q[2 + i:3 + i], [len(seen)], kt[seen], np.abs(vt[seen]), False, None)
            assert_chunk(o[2 + i:3 + i], lse[2 + i:3 + i], (Or, Lr, Ar))
    # a context longer than the table is cut to it
    o, lse = ra.cp_chunk_attn(*dev(q, k, v, table[:, :6].contiguous(), qsl,
                                   torch.tensor([40, 90, 2 ** 31 - 1], dtype=torch.int32)), 16, 1, 1)
    assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS
    # query ranges that decrease or leave [0, T] are left out, the others are computed
    for qs in ([0, 2, 1, 9], [-1, 2, 5, 9], [0, 2, 5, 10]):
        o = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
        ra.cp_chunk_attn(*dev(q, k, v, table, torch.tensor(qs, dtype=torch.int32), torch.tensor(ctx, dtype=torch.int32)), 16,
                         1, 1, o=o)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS and torch.isfinite(o.float()).all()
    assert_chunk(o[:5], ra.cp_chunk_attn(*dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1)[1][:5],
                 S.chunk_attn(q, k, v, table, qsl, ctx, bs, 16, 1, 1), slice(0, 5))
    check_status(ra)


def test_chunk_attn_replayed_with_other_lengths(ra):
    """A captured call replayed with other lengths, tables and queries, next to another on its own workspace."""
    Hq, Hkv, d, bs, I, pcp, dcp = 8, 2, 128, 16, 16, 1, 2
    graphs = []
    for seed in (0, 1):
        st = dict(q=torch.zeros((40, Hq, d), dtype=BF, device=DEV), t=torch.zeros((3, 40), dtype=torch.int32, device=DEV),
                  s=torch.zeros(4, dtype=torch.int32, device=DEV), c=torch.zeros(3, dtype=torch.int32, device=DEV),
                  k=torch.zeros((2, 90, Hkv, bs, d), dtype=BF, device=DEV), v=torch.zeros((2, 90, Hkv, bs, d), dtype=BF, device=DEV))
        ws = torch.empty(ra.cp_chunk_attn_workspace_size(Hq, Hkv, d), dtype=torch.uint8, device=DEV)
        o, lse = torch.zeros((40, Hq, d), dtype=BF, device=DEV), torch.zeros((40, Hq), device=DEV)

        def call():
            ra.cp_chunk_attn(st["q"], st["k"], st["v"], st["t"], st["s"], st["c"], I, pcp, dcp, workspace=ws, o=o, lse=lse)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((st, o, lse, g, ws))     # the workspace lives as long as its graph
    for ctx, n in [([1000, 3, 64], [1, 1, 1]), ([700, 40, 1], [30, 9, 1]), ([5, 1200, 0], [5, 20, 0])]:
        refs = []
        for i, (st, o, lse, g, _) in enumerate(graphs):
            k, v, table, _ = paged(sum(ctx) + i, ctx, Hkv, d, bs, I, pcp, dcp)
            q, qsl = batch(sum(ctx) + i, n, Hq, d)
            refs.append(S.chunk_attn(q, k, v, table, qsl, ctx, bs, I, pcp, dcp))
            st["q"][:q.shape[0]] = q.to(DEV)
            st["k"][:, :k.shape[1]], st["v"][:, :k.shape[1]] = k.to(DEV), v.to(DEV)
            st["t"][:, :table.shape[1]] = table.to(DEV)
            st["s"].copy_(qsl)
            st["c"].copy_(torch.tensor(ctx, dtype=torch.int32))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][3].replay()
        with torch.cuda.stream(side):
            graphs[1][3].replay()
        torch.cuda.current_stream().wait_stream(side)
        check_status(ra)
        for (st, o, lse, _, _), ref in zip(graphs, refs):
            assert_chunk(o[:sum(n)], lse[:sum(n)], ref)


def test_chunk_attn_twice_is_bitwise_equal(ra):
    ctx, n, Hq, Hkv, d = [3000, 1, 800, 2000], [5, 1, 400, 1], 8, 2, 128
    k, v, table, _ = paged(11, ctx, Hkv, d, 128, 16, 1, 1)
    q, qsl = batch(11, n, Hq, d)
    args = dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32))
    a, b = (ra.cp_chunk_attn(*args, 16, 1, 1) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ref = S.chunk_attn(q, k, v, table, qsl, ctx, 128, 16, 1, 1)
    assert_chunk(*a, ref)


# ---------------------------------------------------------------------- weights

def assert_weights(got, ref):
    got = got.double().cpu().numpy()
    live = ~np.isnan(ref)
    assert (np.abs(got[live] - ref[live]) <= 2.0 ** -12 * ref[live] + 1e-9).all(), \
        (np.abs(got[live] - ref[live]) / (ref[live] + 1e-9)).max()
    return live


@pytest.mark.parametrize("case", CHUNKS[:-2] + [([1100], [700], 8, 2, 128, 128, 16, 1, 1)], ids=lambda c: "%s-%s" % (c[0], c[1]))
@pytest.mark.parametrize("mode", ["new", "add", "in place", "all see all"])
def test_attn_weights(ra, case, mode):
    ctx, n, Hq, Hkv, d, bs, I, pcp, dcp = case
    causal = mode != "all see all"
    k, v, table, _ = paged(sum(ctx), ctx, Hkv, d, bs, I, pcp, dcp)
    q, qsl = batch(sum(ctx), n, Hq, d, after=2)
    _, L, _ = S.chunk_attn(q, k, v, table, qsl, ctx, bs, I, pcp, dcp, causal)
    lse = torch.from_numpy(L).float()
    w_in = torch.rand(k.shape[:4]) * 3
    ref = S.attn_weights(q, lse, k, table, qsl, ctx, bs, I, pcp, dcp, None if mode == "new" else w_in.numpy(), causal)
    qd, ld, kd, td, sd, cd, wd = dev(q, lse, k, table, qsl, torch.tensor(ctx, dtype=torch.int32), w_in)
    out = wd if mode == "in place" else torch.full(w_in.shape, 7.0, device=DEV)
    got = ra.cp_attn_weights(qd, ld, kd, td, sd, cd, I, pcp, dcp, w_in=None if mode == "new" else wd, w_out=out, causal=causal)
    check_status(ra)
    live = assert_weights(got, ref)
    rest = got.cpu().numpy()[~live]
    assert (rest == (w_in.numpy()[~live] if mode == "in place" else 7.0)).all()
    if mode == "new":
        again = ra.cp_attn_weights(qd, ld, kd, td, sd, cd, I, pcp, dcp)
        assert torch.equal(again.cpu()[torch.from_numpy(live)], got.cpu()[torch.from_numpy(live)])
        assert (again.cpu().numpy()[~live] == 0).all()


def test_attn_weights_rows_without_lse_and_short_contexts(ra):
    ctx, n, Hq, Hkv, d, bs = [3, 0, 50], [7, 4, 9], 4, 2, 64, 16
    k, v, table, _ = paged(12, ctx, Hkv, d, bs, 16, 1, 1)
    q, qsl = batch(12, n, Hq, d)
    o, lse = ra.cp_chunk_attn(*dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1)
    lse[14] = -float("inf")
    ref = S.attn_weights(q, lse.cpu(), k, table, qsl, ctx, bs, 16, 1, 1)
    got = ra.cp_attn_weights(q.to(DEV), lse, *dev(k, table, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1)
    check_status(ra)
    assert_weights(got, ref)
    t = table.clone()
    t[2, 1] = 99
    got = ra.cp_attn_weights(q.to(DEV), lse, *dev(k, t, qsl, torch.tensor(ctx, dtype=torch.int32)), 16, 1, 1)
    assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS and not got.isnan().any()


# ---------------------------------------------------------------------- eviction

EVICTS = [
    # ctx, keep, sink, recent, Hkv, d, bs, I, pcp, dcp, dtype
    ([9], 5, 1, 1, 2, 64, 16, 4, 1, 1, BF),
    ([300, 20, 150, 0], 100, 4, 17, 3, 64, 16, 16, 1, 1, BF),
    ([1025, 2050], 512, 0, 0, 2, 128, 128, 16, 2, 4, BF),
    ([1500], 1499, 4, 100, 1, 64, 32, 1, 1, 2, torch.float32),
    ([4000, 3999], 1, 0, 0, 2, 8, 64, 64, 1, 1, BF),
    ([700, 650], 64, 20, 44, 2, 4, 16, 8, 1, 3, torch.float32),
    ([9000], 2500, 3, 500, 1, 128, 128, 16, 1, 1, BF),
    ([2049], 1024, 0, 1024, 2, 256, 48, 16, 1, 1, BF),
]


def _same(got, ref):
    bits = lambda t: t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)  # noqa: E731
    return torch.equal(bits(got.cpu()), bits(ref))


@pytest.mark.parametrize("case", EVICTS, ids=lambda c: "%s-to-%d.%d.%d-d%d" % (c[0], c[1], c[2], c[3], c[5]))
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("weights", ["spread", "ties", "odd"])
def test_evict(ra, case, fresh, weights):
    ctx, keep, sink, recent, Hkv, d, bs, I, pcp, dcp, dt = case
    V = bs * pcp * dcp
    more = -(-min(keep, max(ctx)) // V)
    k, v, table, spare = paged(keep, ctx, Hkv, d, bs, I, pcp, dcp, dt, spare=len(ctx) * more + 1)
    g = torch.Generator().manual_seed(keep)
    w = torch.rand(k.shape[:4], generator=g) * 4
    if weights == "ties":
        w = torch.floor(w * 2) / 2
    if weights == "odd":
        r = torch.rand(w.shape, generator=g)
        for hi, val in [(0.5, float("nan")), (0.4, -0.0), (0.3, 0.0), (0.2, -1.0), (0.1, float("inf")), (0.05, 1e-42),
                        (0.02, -float("inf"))]:
            w[r < hi] = val
    dst = spare[:len(ctx) * more].view(len(ctx), more) if fresh else None
    ref_k, ref_n, k2, v2, w2 = S.evict(*(t.view(torch.int16 if t.element_size() == 2 else torch.int32).numpy() for t in (k, v)),
                                       w.numpy(), table, ctx, keep, bs, I, pcp, dcp, sink, recent, dst)
    kd, vd, wd, td, cd = dev(k, v, w, table, torch.tensor(ctx, dtype=torch.int32))
    kept, new = ra.cp_evict(kd, vd, wd, td, cd, keep, I, pcp, dcp, n_sink=sink, n_recent=recent,
                            dst_block_table=None if dst is None else dst.to(DEV))
    check_status(ra)
    assert np.array_equal(kept.cpu().numpy(), ref_k) and np.array_equal(new.cpu().numpy(), ref_n)
    bits = lambda t: t.view(torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()  # noqa: E731
    assert np.array_equal(bits(kd), k2) and np.array_equal(bits(vd), v2)
    assert np.array_equal(bits(wd), w2.view(np.int32))


def test_evict_bad_tables_are_reported(ra):
    ctx, Hkv, d, bs = [70, 50], 2, 64, 16
    k, v, table, spare = paged(13, ctx, Hkv, d, bs, 16, 1, 1, spare=8)
    w = torch.rand(k.shape[:4])
    want = S.evict_choice(w.numpy()[0, table[1, :4].numpy()].transpose(0, 2, 1).reshape(-1, 2)[:50, 0], 20, 0, 0)
    for change in ("source", "length", "destination", "table"):
        t, dst, c = table.clone(), spare[:4].view(2, 2).clone(), list(ctx)
        if change == "source":
            t[0, 1] = 77
        if change == "length":
            c[0] = 1000
            t = t[:, :4].contiguous()
        if change == "destination":
            dst[0, 1] = -3
        if change == "table":
            dst = dst[:, :1].contiguous()
        kd, vd, wd = dev(k, v, w)
        kept, new = ra.cp_evict(kd, vd, wd, *dev(t, torch.tensor(c, dtype=torch.int32)), 20, 16, 1, 1,
                                dst_block_table=dst.to(DEV))
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS, change
        assert new.tolist() == [20, 20] and kept[1, 0].tolist() == want
        if change == "source":
            assert not ((kept[0] >= 16) & (kept[0] < 32)).any()      # 54 good tokens are enough


def test_evict_is_captured_and_replayed(ra):
    ctx, Hkv, d, bs, I = [900, 400], 2, 64, 16, 16
    k, v, table, spare = paged(14, ctx, Hkv, d, bs, I, 1, 1, spare=2 * 16)
    w = torch.rand(k.shape[:4])
    kd, vd, wd, td, cd, dd = dev(k, v, w, table, torch.tensor(ctx, dtype=torch.int32), spare[:32].view(2, 16))
    kept, new = torch.empty((2, Hkv, 250), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    call = lambda: ra.cp_evict(kd, vd, wd, td, cd, 250, I, 1, 1, n_sink=2, n_recent=9, dst_block_table=dd, kept=kept, new_lens=new)  # noqa
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (1, 2):
        w = torch.rand(k.shape[:4], generator=torch.Generator().manual_seed(seed))
        c = [900 - 100 * seed, 400]
        wd.copy_(w)
        cd.copy_(torch.tensor(c, dtype=torch.int32))
        g.replay()
        check_status(ra)
        ref, n, *_ = S.evict(k.float().numpy(), v.float().numpy(), w.numpy(), table, c, 250, bs, I, 1, 1, 2, 9, dd.cpu())
        assert np.array_equal(kept.cpu().numpy(), ref) and new.tolist() == n.tolist()


# ---------------------------------------------------------------------- rotary positions

def assert_rope(y, ref, x, rot, style, mscale, dt):
    y = y.double().cpu().numpy()
    x = np.abs(x.double().numpy())
    half = rot // 2
    size = np.zeros_like(x)
    u, v = (slice(0, half), slice(half, rot)) if style == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    size[..., u] = size[..., v] = x[..., u] + x[..., v]
    step = torch.finfo(dt).eps / 2
    tol = 2.0 ** -19 * abs(mscale) * size + step * np.abs(ref) + 1e-40
    tol[..., rot:] = 0
    assert (np.abs(y - ref) <= tol).all(), (np.abs(y - ref) - tol).max()


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("rows,H,d,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (7, 3, 64, 32), (33, 5, 80, 40), (129, 2, 256, 256),
                                          (3, 1, 1, 0), (65, 13, 96, 48), (5, 2, 1024, 16), (17, 4, 24, 6), (300, 8, 128, 64)])
@pytest.mark.parametrize("backward", [False, True])
def test_rope_apply(ra, style, dt, rows, H, d, rot, backward):
    x = torch.randn((rows, H, d), generator=torch.Generator().manual_seed(rows)).to(dt)
    pos = torch.randint(0, 2 ** 24, (rows,), generator=torch.Generator().manual_seed(d), dtype=torch.int32)
    pos[-1] = 2 ** 24 - 1
    if rot == 0:                       # nothing to turn is refused
        with pytest.raises(ra.RingAttnError):
            ra.rope_apply(x.to(DEV), pos.to(DEV), torch.empty(0, dtype=torch.float64), style=style)
        return
    f, m = ra.rope_frequencies(rot, 10000.0, "yarn", 4.0, 4096)
    ref = S.rope_apply(x, pos, f.numpy(), m, style, backward)
    y = ra.rope_apply(x.to(DEV), pos.to(DEV), f, m, style, backward=backward)
    check_status(ra)
    assert_rope(y, ref, x, rot, style, m, dt)
    z = x.to(DEV)
    assert ra.rope_apply(z, pos.to(DEV), f, m, style, backward=backward, out=z) is z and torch.equal(y, z)


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("view", ["fused", "heads first", "odd rows", "odd start", "padded heads", "broadcast"])
def test_rope_apply_strides(ra, style, dt, view):
    rows, H, d, rot = 37, 6, 64, 48
    g = torch.Generator().manual_seed(3)
    base = torch.randn(40 * 12 * 80, generator=g).to(dt)
    shape = {"fused": ((9 * d, d, 1), 2 * d), "heads first": ((d, rows * d, 1), 0), "odd rows": ((6 * d + 3, d, 1), 0),
             "odd start": ((6 * d, d, 1), 1), "padded heads": ((6 * 72, 72, 1), 8), "broadcast": ((d, 0, 1), 0)}[view]
    x = base.as_strided((rows, H, d), *shape)
    xd = base.to(DEV).as_strided((rows, H, d), *shape)
    pos = torch.arange(1000, 1000 + rows, dtype=torch.int32)
    f, _ = ra.rope_frequencies(rot)
    ref = S.rope_apply(x, pos, f.numpy(), 1.0, style)
    y = ra.rope_apply(xd, pos.to(DEV), f, style=style)
    check_status(ra)
    assert_rope(y, ref, x, rot, style, 1.0, dt)
    if view == "broadcast":
        with pytest.raises(ra.RingAttnError):
            ra.rope_apply(xd, pos.to(DEV), f, style=style, out=xd)
        return
    guard = torch.full((40 * 12 * 80,), 7.0, dtype=dt, device=DEV)
    out = guard.as_strided((rows, H, d), *shape)
    ra.rope_apply(xd, pos.to(DEV), f, style=style, out=out)
    assert torch.equal(out, y)
    out.fill_(7.0)
    assert (guard == 7).all()                                     # nothing outside the view was written
    ra.rope_apply(xd, pos.to(DEV), f, style=style, out=xd)      # in place, strided
    check_status(ra)
    assert torch.equal(xd, y)


def test_rope_apply_gather_gradient_and_errors(ra):
    rows, H, d, rot = 50, 3, 64, 64
    perm, restore = ra.zigzag_partition([rows], 4)
    g = torch.Generator().manual_seed(4)
    x = torch.randn((rows, H, d), generator=g)
    pos = torch.arange(rows, dtype=torch.int32, device=DEV)
    pz = torch.where(perm >= 0, pos[perm.clamp(min=0).long()], 0).to(torch.int32)
    f, _ = ra.rope_frequencies(rot)
    y = ra.rope_apply(x.to(DEV), pz, f, idx=perm, style="interleaved")
    check_status(ra)
    ref = S.rope_apply(x, pz.cpu(), f.numpy(), 1.0, "interleaved", idx=perm.cpu().numpy())
    xz = torch.where((perm >= 0).cpu()[:, None, None], x[perm.clamp(min=0).long().cpu()], 0)
    assert_rope(y, ref, xz, rot, "interleaved", 1.0, torch.float32)
    assert (y[perm < 0] == 0).all()
    # half layout: the same rows as the fused gather of the zigzag prologue, to rounding
    a, b = ra.rope_apply(x.to(DEV), pz, f, idx=perm), ra.rope_gather(x.to(DEV), pos, perm)
    assert (a - b).abs().max() <= 2 * 2.0 ** -19 * 2 * x.abs().max()
    # gradient of sum(dy * rope(x[perm])): back through the inverse permutation, against differences of the oracle
    dy = torch.randn(y.shape, generator=g)
    dx = ra.rope_apply(dy.to(DEV), pos, f, idx=restore, style="interleaved", backward=True).cpu()
    loss = lambda t: (S.rope_apply(t, pz.cpu(), f.numpy(), 1.0, "interleaved", idx=perm.cpu().numpy()) * dy.double().numpy()).sum()  # noqa
    for at in [(0, 0, 0), (49, 2, 63), (17, 1, 30)]:
        e = torch.zeros(x.shape, dtype=torch.float64)
        e[at] = 1e-3
        diff = (loss(x.double() + e) - loss(x.double() - e)) / 2e-3
        assert abs(diff - dx[at].item()) <= 2.0 ** -19 * 2 * float(dy.abs().max()) + 1e-9
    # bad rows and positions are reported
    idx = torch.tensor([0, 50, -1], dtype=torch.int32, device=DEV)
    y = ra.rope_apply(x.to(DEV), pos[:3].contiguous(), f, idx=idx)
    assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS and (y[1:] == 0).all()
    for bad in (-1, 2 ** 24):
        y = ra.rope_apply(x[:2].to(DEV), torch.tensor([0, bad], dtype=torch.int32, device=DEV), f)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS and torch.equal(y.cpu(), x[:2])
    assert ra.rope_apply(x[:0].to(DEV), pos[:0], f).shape == (0, H, d)
    check_status(ra)


# ---------------------------------------------------------------------- together

def test_serving_step_prompt_evict_decode(ra):
    """A prompt in two pieces, its weights, an eviction into fresh blocks, then a decoded token: as a server
    runs them, each step on the cache that the one before left."""
    Hq, Hkv, d, bs, I, pcp, dcp = 8, 2, 64, 16, 4, 1, 2
    L, cut, keep, V = 230, 150, 96, 32
    g = torch.Generator().manual_seed(21)
    qkv = torch.randn((L + 1, Hq + 2 * Hkv, d), generator=g).to(BF).to(DEV)
    f, m = ra.rope_frequencies(d, 10000.0, "linear", 4.0)
    pos = torch.arange(L + 1, dtype=torch.int32, device=DEV)
    rot = ra.rope_apply(qkv[:, :Hq + Hkv], pos, f, m, "interleaved")
    q, k, v = rot[:, :Hq].contiguous(), rot[:, Hq:].contiguous(), qkv[:, Hq + Hkv:].contiguous()
    kc = torch.full((2, 20, Hkv, bs, d), float("nan"), dtype=BF, device=DEV)
    vc, w = kc.clone(), torch.full((2, 20, Hkv, bs), float("nan"), device=DEV)
    table = torch.randperm(20, generator=g)[:8].to(torch.int32).view(1, 8).to(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    def append(a, b, tab, at):
        slot = ra.cp_slot_mapping(i32(0, b - a), torch.arange(at, at + b - a, dtype=torch.int32, device=DEV), tab, bs, I, pcp, dcp)
        ra.cp_kv_scatter(k[a:b].contiguous(), v[a:b].contiguous(), slot, kc, vc)

    for a, b in ((0, cut), (cut, L)):
        append(a, b, table, a)
        o, lse = ra.cp_chunk_attn(q[a:b].contiguous(), kc, vc, table, i32(0, b - a), i32(b), I, pcp, dcp)
        ra.cp_attn_weights(q[a:b].contiguous(), lse, kc, table, i32(0, b - a), i32(b), I, pcp, dcp, w_in=w, w_out=w)
        check_status(ra)
        kn, vn, tn = kc.double().cpu().numpy(), vc.double().cpu().numpy(), table.cpu().numpy()
        assert_chunk(o, lse, S.chunk_attn(q[a:b], kn, vn, tn, [0, b - a], [b], bs, I, pcp, dcp))
    total = S.token_rows(w.double().cpu().numpy()[..., None], tn[0], range(L), bs, I, pcp, dcp)[..., 0]
    # every query's weights of a head sum to 1, to within the bound of one weight
    assert abs(total.sum() - L * Hq) <= 2.0 ** -12 * L * Hq
    fresh = torch.tensor([[x for x in range(20) if x not in table.cpu().tolist()[0]][:4]], dtype=torch.int32, device=DEV)
    kept, new = ra.cp_evict(kc, vc, w, table, i32(L), keep, I, pcp, dcp, n_sink=4, n_recent=32, dst_block_table=fresh)
    check_status(ra)
    assert new.tolist() == [keep] and all(kept[0, h].tolist() == S.evict_choice(total[:, h], keep, 4, 32) for h in range(Hkv))
    append(L, L + 1, fresh, keep)
    o, lse = ra.cp_chunk_attn(q[L:].contiguous(), kc, vc, fresh, i32(0, 1), i32(keep + 1), I, pcp, dcp)
    o2, _ = ra.cp_decode(q[L:].contiguous(), kc, vc, fresh, i32(keep + 1), I, pcp, dcp)
    check_status(ra)
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    for h in range(Hq):
        ids = kept[0, h // 4].tolist() + [L]
        s = kn[ids, h // 4] @ q[L, h].double().cpu().numpy() / 8
        p = np.exp(s - s.max())
        p /= p.sum()
        want, A = p @ vn[ids, h // 4], p @ np.abs(vn[ids, h // 4])
        for got in (o, o2):
            err = np.abs(got[0, h].double().cpu().numpy() - want)
            assert (err <= 2.0 ** -8 * (A + np.abs(want)) + 2.0 ** -11 * A).all()
    # the in-place form gives the same packed context
    kept2, _ = ra.cp_evict(kc, vc, w, table, i32(L), keep, I, pcp, dcp, n_sink=4, n_recent=32)
    check_status(ra)
    assert torch.equal(kept2, kept)
    a = S.token_rows(kc.double().cpu().numpy(), table.cpu().numpy()[0], range(keep), bs, I, pcp, dcp)
    b = S.token_rows(kc.double().cpu().numpy(), fresh.cpu().numpy()[0], range(keep), bs, I, pcp, dcp)
    assert np.array_equal(a, b)


def test_calls_on_a_side_stream(ra):
    """Each operator runs on the current stream: after a delay there, the inputs written before it are seen."""
    ctx, n, Hq, Hkv, d = [300], [20], 4, 2, 64
    k, v, table, _ = paged(15, ctx, Hkv, d, 16, 16, 1, 1)
    q, qsl = batch(15, n, Hq, d)
    kd, vd, td, sd, cd = dev(k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32))
    src = q.to(DEV)
    o0, l0 = ra.cp_chunk_attn(src, kd, vd, td, sd, cd, 16, 1, 1)
    w0 = ra.cp_attn_weights(src, l0, kd, td, sd, cd, 16, 1, 1)
    f, _ = ra.rope_frequencies(d)
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    r0 = ra.rope_apply(src, pos, f)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.zeros_like(src)
        torch.cuda._sleep(20_000_000)
        late.copy_(src)
        o1, l1 = ra.cp_chunk_attn(late, kd, vd, td, sd, cd, 16, 1, 1)
        w1 = ra.cp_attn_weights(late, l1, kd, td, sd, cd, 16, 1, 1)
        r1 = ra.rope_apply(late, pos, f)
    s.synchronize()
    check_status(ra)
    assert torch.equal(o0, o1) and torch.equal(l0, l1) and torch.equal(w0, w1) and torch.equal(r0, r1)


def test_calls_on_two_streams_at_once(ra):
    """Two streams, a workspace each: every operator gives what it gives alone, however the calls overlap."""
    ctx, n, Hq, Hkv, d = [3000, 700, 41], [1, 90, 5], 8, 2, 128
    sets = []
    for seed in (31, 32):
        k, v, table, _ = paged(seed, ctx, Hkv, d, 32, 16, 2, 1)
        q, qsl = batch(seed, n, Hq, d)
        sets.append(dev(q, k, v, table, qsl, torch.tensor(ctx, dtype=torch.int32), torch.rand(k.shape[:4])))
    f, _ = ra.rope_frequencies(d)
    pos = torch.arange(sum(n), dtype=torch.int32, device=DEV)

    def step(q, k, v, t, s, c, w):
        o, lse = ra.cp_chunk_attn(q, k, v, t, s, c, 16, 2, 1)
        new = ra.cp_attn_weights(q, lse, k, t, s, c, 16, 2, 1)
        k2, v2, w2 = k.clone(), v.clone(), w.clone()
        kept, lens = ra.cp_evict(k2, v2, w2, t, c, 256, 16, 2, 1, n_sink=3, n_recent=50)
        return [o, lse, new, ra.rope_apply(q, pos, f), kept, lens, k2.view(torch.int16), v2.view(torch.int16), w2]

    alone = [step(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, x in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(step(*x))
        torch.cuda.synchronize()
        check_status(ra)
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_caches_past_32_bit_offsets(ra):
    """The same tokens at the far end of a cache of more than 2^31 elements: the same results to the bit."""
    ctx, n, Hq, Hkv, d, bs, NB = [1500, 260], [3, 70], 16, 8, 128, 128, 17000
    k, v, table, spare = paged(33, ctx, Hkv, d, bs, 16, 1, 1, spare=6)
    q, qsl = batch(33, n, Hq, d)
    w = torch.rand(k.shape[:4])
    dst = spare[:6].view(2, 3)
    far = lambda t: torch.where(t >= 0, NB - 1 - t, t).to(torch.int32)  # noqa: E731
    small = dev(k, v, w)
    big = [torch.empty((1, NB) + tuple(t.shape[2:]), dtype=t.dtype, device=DEV) for t in small]
    assert big[0].numel() > 2 ** 31
    at = far(torch.arange(k.shape[1])).long().to(DEV)
    for b, t in zip(big, small):
        b[:, at] = t
    qd, sd, cd = dev(q, qsl, torch.tensor(ctx, dtype=torch.int32))
    out = []
    for (kc, vc, wc), tab, to in ((small, table, dst), (big, far(table), far(dst))):
        td = tab.to(DEV)
        o, lse = ra.cp_chunk_attn(qd, kc, vc, td, sd, cd, 16, 1, 1)
        ra.cp_attn_weights(qd, lse, kc, td, sd, cd, 16, 1, 1, w_in=wc, w_out=wc)
        kept, lens = ra.cp_evict(kc, vc, wc, td, cd, 300, 16, 1, 1, n_sink=2, n_recent=20, dst_block_table=to.to(DEV))
        check_status(ra)
        out.append([o, lse, kept, lens])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    for b, t in zip(big, small):
        a, c = b[:, at], t
        if a.dtype == BF:
            a, c = a.view(torch.int16), c.view(torch.int16)
        assert torch.equal(a, c)


def test_rope_apply_more_threads_than_a_launch(ra):
    """2^31 - 1 rows of one word each, in place: two launches, element offsets past 32 bits."""
    rows, d, m = 2 ** 31 - 1, 4, 400
    g = torch.Generator().manual_seed(34)
    x = torch.zeros((rows, 1, d), dtype=BF, device=DEV)
    pos = torch.zeros(rows, dtype=torch.int32, device=DEV)
    f, _ = ra.rope_frequencies(d)
    parts = []
    for a in (0, 2 ** 30, rows - m):
        xs, ps = dev(torch.randn((m, 1, d), generator=g).to(BF), torch.randint(0, 100000, (m,), generator=g).to(torch.int32))
        x[a:a + m], pos[a:a + m] = xs, ps
        parts.append((a, ra.rope_apply(xs, ps, f, style="interleaved")))
    ra.rope_apply(x, pos, f, style="interleaved", out=x)
    check_status(ra)
    for a, want in parts:
        assert torch.equal(x[a:a + m], want)
    assert not x[m:2 ** 30].any()


# ---------------------------------------------------------------------- failure detection

CHILD = r"""
import json, sys, torch
sys.path.insert(0, sys.argv[1])
from context_long_sequence_ring_gb300 import ringattn as ra
dev = torch.device("cuda:0")
g = torch.Generator().manual_seed(3)
rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
out = {}
for d in (64, 128):
    k, v, table = rnd(1, 40, 2, 64, d), rnd(1, 40, 2, 64, d), torch.arange(40, dtype=torch.int32, device=dev).view(2, 20)
    for name, n in (("single", 1), ("prompt", 300)):
        q, qsl, ctx = rnd(2 * n, 8, d), i32(0, n, 2 * n), i32(1200, 1000)
        lse = torch.zeros((2 * n, 8), device=dev)
        ra.cp_chunk_attn(q, k, v, table, qsl, ctx, 16, 1, 1)
        st = ra.device_status()
        out["chunk %s %d" % (name, d)] = [int(st), ra.last_error() if st else ""]
        ra.cp_attn_weights(q, lse, k, table, qsl, ctx, 16, 1, 1)
        st = ra.device_status()
        out["weights %s %d" % (name, d)] = [int(st), ra.last_error() if st else ""]
# the context still works: a kernel without waits gives the exact result
src = torch.arange(64 * 8, dtype=torch.float32, device=dev).view(64, 8)
idx = torch.randperm(64, generator=g).to(torch.int32).to(dev)
out["gather_ok"] = bool(torch.equal(ra.gather_rows(src, idx).cpu(), src.cpu()[idx.long().cpu()]))
out["final_status"] = int(ra.device_status())
print(json.dumps(out))
"""


def test_timeouts_are_reported_and_the_context_survives():
    """As for the other tensor-core kernels: with a wait limit of 64 cycles the first wait that is not satisfied at once
    expires; the kernel records it, lets its copies and products land, frees tensor memory and returns."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, root], env=dict(os.environ, RA_WAIT_LIMIT_CYCLES="64"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    res = json.loads(r.stdout.strip().splitlines()[-1])
    from context_long_sequence_ring_gb300 import ringattn
    for name, (st, msg) in ((n, x) for n, x in res.items() if isinstance(x, list)):
        assert st == ringattn.RA_ERR_TIMEOUT, (name, st, msg)
        assert ("chunk attention" if "chunk" in name else "attention weights") in msg, (name, msg)
    assert len(res) == 10 and res["gather_ok"] and res["final_status"] == 0
