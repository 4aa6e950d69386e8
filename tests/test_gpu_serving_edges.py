"""Edges of the serving operators: queries whose LSE is not a number or that are marked as seeing nothing, evictions of
every cluster size and past the keys that shared memory holds, ranges that are left out, and batches whose work is
counted in coarser units.  Tolerances as in the parity tests of the same operators."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from tests._gpu import ra_lib, check_status
from tests.test_gpu_serving import BF, DEV, _same, assert_chunk, assert_weights, batch, dev, paged

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module")
def ra():
    return ra_lib()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


# ---------------------------------------------------------------------- weights

# ctx, n, Hq, Hkv, d, bs, I, W: query tiles that stay in shared memory, that pass by, one token, a few
WEIGHTS = [
    ([300], [40], 8, 2, 128, 32, 16, 2),
    ([700], [517], 8, 2, 128, 48, 16, 1),
    ([257, 300], [33, 300], 6, 2, 64, 64, 16, 2),
    ([900, 77], [1, 3], 8, 2, 64, 16, 16, 1),
]


def weights_inputs(case):
    ctx, n, Hq, Hkv, d, bs, I, W = case
    k, v, table, _ = paged(sum(ctx), ctx, Hkv, d, bs, I, W, 1)
    q, qsl = batch(sum(ctx), n, Hq, d)
    _, L, _ = S.chunk_attn(q, k, v, table, qsl, ctx, bs, I, W, 1)
    return q, torch.from_numpy(L).float(), k, table, qsl


def run_weights(ra, case, q, lse, k, table, qsl, causal=True):
    got = ra.cp_attn_weights(*dev(q, lse, k, table, qsl, i32(*case[0])), case[6], case[7], 1, causal=causal)
    check_status(ra)
    return got


@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: "%s-%s-d%d" % (c[0], c[1], c[4]))
def test_weights_of_a_nan_lse_reach_only_the_tokens_it_sees(ra, case):
    ctx, n, Hq, Hkv, d, bs, I, W = case
    q, lse, k, table, qsl = weights_inputs(case)
    for r in range(len(ctx)):
        for i in {0, n[r] // 2, n[r] - 1}:
            bad = lse.clone()
            bad[int(qsl[r]) + i, 1] = float("nan")           # head 1, of K/V head 0
            left = lse.clone()
            left[int(qsl[r]) + i, 1] = -float("inf")
            want = S.attn_weights(q, left, k, table, qsl, ctx, bs, I, W, 1)
            got = run_weights(ra, case, q, bad, k, table, qsl).double().cpu().numpy()
            x = np.arange(ctx[r] - n[r] + i + 1)             # the tokens that this query sees
            lbi = x % (bs * W) // I
            seen = np.zeros(want.shape, dtype=bool)
            seen[lbi % W, table[r].numpy()[x // (bs * W)], 0, lbi // W * I + x % (bs * W) % I] = True
            assert np.isnan(got[seen]).all()
            assert not np.isnan(got[~seen]).any()
            want[seen] = np.nan                              # left out of the comparison
            assert_weights(torch.from_numpy(got), want)


@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: "%s-%s-d%d" % (c[0], c[1], c[4]))
@pytest.mark.parametrize("causal", [True, False])
def test_weights_of_queries_marked_as_seeing_nothing(ra, case, causal):
    """An LSE of -inf (or +inf: e^-inf) leaves a query out whatever its row holds, e.g. padding that was never written."""
    ctx, n, Hq, Hkv, d, bs, I, W = case
    q, lse, k, table, qsl = weights_inputs(case)
    ends = [int(qsl[r + 1]) - 1 for r in range(len(ctx))]
    for mark in (-float("inf"), float("inf")):
        left, qs, ref = lse.clone(), q.clone(), lse.clone()
        for row, junk in zip([0, q.shape[0] // 2] + ends, (float("nan"), float("inf"), float("nan"), 3e38)):
            left[row], ref[row], qs[row] = mark, -float("inf"), junk
        want = S.attn_weights(q, ref, k, table, qsl, ctx, bs, I, W, 1, causal=causal)
        assert_weights(run_weights(ra, case, qs, left, k, table, qsl, causal), want)


def test_weights_replayed_with_other_lengths(ra):
    """A captured call replayed with other lengths: query tiles that stay, that pass by, single tokens, none."""
    Hq, Hkv, d, bs, I, W = 8, 2, 128, 16, 16, 2
    q, lse = torch.zeros((520, Hq, d), dtype=BF, device=DEV), torch.zeros((520, Hq), device=DEV)
    k, w = torch.zeros((W, 90, Hkv, bs, d), dtype=BF, device=DEV), torch.zeros((W, 90, Hkv, bs), device=DEV)
    t, s, c = (torch.zeros(x, dtype=torch.int32, device=DEV) for x in ((3, 40), 4, 3))
    call = lambda: ra.cp_attn_weights(q, lse, k, t, s, c, I, W, 1, w_in=w, w_out=w)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for ctx, n in [([1000, 3, 64], [1, 1, 1]), ([700, 40, 1], [500, 9, 1]), ([5, 1200, 0], [0, 20, 0]), ([300, 40, 64], [64, 0, 5])]:
        kc, _, table, _ = paged(sum(ctx), ctx, Hkv, d, bs, I, W, 1)
        qc, qsl = batch(sum(ctx), n, Hq, d)
        _, L, _ = S.chunk_attn(qc, kc, kc, table, qsl, ctx, bs, I, W, 1)
        L = torch.from_numpy(L).float()
        old = torch.rand(w.shape)
        q[:qc.shape[0]], lse[:qc.shape[0]], k[:, :kc.shape[1]] = qc.to(DEV), L.to(DEV), kc.to(DEV)
        t[:, :table.shape[1]] = table.to(DEV)
        s.copy_(qsl)
        c.copy_(i32(*ctx))
        w.copy_(old)
        graph.replay()
        check_status(ra)
        want = S.attn_weights(qc, L, kc, table, qsl, ctx, bs, I, W, 1, w_in=old[:, :kc.shape[1]].numpy())
        live = assert_weights(w[:, :kc.shape[1]], want)
        assert torch.equal(w.cpu()[:, :kc.shape[1]][torch.from_numpy(~live)], old[:, :kc.shape[1]][torch.from_numpy(~live)])


# ---------------------------------------------------------------------- chunk attention

def test_chunk_attn_work_in_coarser_units(ra):
    """A long piece with two tokens to a row tile among single tokens: the sum of its costs is past 2^30, so parts are
    cut, and joined, in coarser units.  Sampled rows against 64 bits; a wide block table changes nothing."""
    Hq, Hkv, d, bs, n = 512, 8, 64, 64, 20000
    g = torch.Generator(device=DEV).manual_seed(41)
    ctx = [3000, 20000] + [700 + 97 * i for i in range(30)]
    new = [1, n] + [1] * 30
    nvb = [-(-x // bs) for x in ctx]
    NB = sum(nvb)
    k, v = (torch.randn((1, NB, Hkv, bs, d), generator=g, device=DEV).to(BF) for _ in range(2))
    table = torch.full((32, 1 << 14), -1, dtype=torch.int32)
    ids = torch.randperm(NB, generator=torch.Generator().manual_seed(42)).to(torch.int32)
    at = 0
    for r, x in enumerate(nvb):
        table[r, :x] = ids[at:at + x]
        at += x
    qsl = i32(*np.concatenate([[0], np.cumsum(new)]).tolist())
    q = torch.randn((int(qsl[-1]), Hq, d), generator=g, device=DEV).to(BF)
    args = [*dev(table[:, :max(nvb)].contiguous(), qsl, i32(*ctx)), bs, 1, 1]
    o, lse = ra.cp_chunk_attn(q, k, v, *args)
    check_status(ra)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    rng = np.random.default_rng(43)
    for r in range(32):
        kt, vt = (t[0, table[r, :nvb[r]].long().to(DEV)].permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :ctx[r]].double()
                  for t in (k, v))
        for i in (rng.integers(0, n, 40).tolist() + [0, n - 1] if new[r] > 1 else [0]):
            row, see = int(qsl[r]) + i, ctx[r] - new[r] + i + 1
            s = torch.matmul(q[row].double().view(Hkv, -1, d), kt[:, :see].transpose(1, 2)) * d ** -0.5
            p = torch.softmax(s, -1)
            ref = [torch.matmul(p, vt[:, :see]), torch.logsumexp(s, -1), torch.matmul(p, vt[:, :see].abs())]
            assert_chunk(o[row], lse[row], [t.reshape(Hq, *t.shape[2:]).cpu().numpy() for t in ref])
    o2, lse2 = ra.cp_chunk_attn(q, k, v, table.to(DEV), *args[1:])
    check_status(ra)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---------------------------------------------------------------------- eviction

# ctx, width of the table in tokens (0: as needed), keep, sink, recent, Hkv, d, bs, I, pcp, dcp: clusters of 8, 4, 2 and 1,
# keys in shared memory whole, cut off (24576 to a CTA), or cut off by the table alone
LONG = {
    "8, past the keys": ([200001, 70], 0, 5000, 4, 1000, 1, 8, 64, 16, 1, 1),
    "4": ([900 + 37 * r for r in range(5)], 0, 300, 2, 50, 8, 8, 32, 4, 1, 2),
    "4, past the keys": ([100003, 5, 300, 99, 1001], 0, 777, 0, 0, 8, 8, 128, 16, 2, 1),
    "2": ([600 + 41 * r for r in range(10)], 0, 256, 4, 100, 8, 8, 16, 2, 1, 1),
    "1": ([31 * r for r in range(20)], 0, 128, 1, 7, 8, 8, 16, 16, 1, 1),
    "1, past the keys": ([30001] + [47 * r for r in range(1, 20)], 0, 600, 3, 64, 8, 8, 64, 1, 1, 1),
    "1, a wide table": ([800 - 31 * r for r in range(20)], 50000, 100, 4, 16, 8, 8, 64, 16, 1, 1),
}


@pytest.mark.parametrize("name", LONG)
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("weights", ["spread", "ties", "odd"])
def test_evict_with_clusters_of_every_size(ra, name, fresh, weights):
    ctx, wide, keep, sink, recent, Hkv, d, bs, I, pcp, dcp = LONG[name]
    R, V = len(ctx), bs * pcp * dcp
    more = -(-min(keep, max(ctx)) // V)
    k, v, table, spare = paged(keep, ctx, Hkv, d, bs, I, pcp, dcp, spare=R * more + 1)
    if wide:
        table = torch.nn.functional.pad(table, (0, wide // V - table.shape[1]), value=-1)
    g = torch.Generator().manual_seed(keep)
    w = torch.rand(k.shape[:4], generator=g) * 4
    if weights == "ties":
        w = torch.floor(w * 2) / 2
    if weights == "odd":
        r = torch.rand(w.shape, generator=g)
        for hi, val in [(0.999, float("nan")), (0.95, -0.0), (0.9, 0.0), (0.6, -1.0), (0.05, float("inf")), (0.04, 1e-42),
                        (0.02, -float("inf"))]:
            w[r < hi] = val
    dst = spare[:R * more].view(R, more) if fresh else None
    ref, moves = S.evict_by_sort(w.numpy(), table, ctx, keep, bs, I, pcp, dcp, sink, recent, dst)
    kd, vd, wd = dev(k, v, w)
    kept, new = ra.cp_evict(kd, vd, wd, *dev(table, i32(*ctx)), keep, I, pcp, dcp, n_sink=sink, n_recent=recent,
                            dst_block_table=None if dst is None else dst.to(DEV))
    check_status(ra)
    assert np.array_equal(kept.cpu().numpy(), ref) and new.tolist() == [min(x, keep) for x in ctx]
    for got, t, bits in ((kd, k, torch.int16), (vd, v, torch.int16), (wd, w, torch.int32)):
        old = t.view(bits)
        want = old.clone()
        for _, h, src, to in moves:
            want[to[0], to[1], h, to[2]] = old[src[0], src[1], h, src[2]]
        assert _same(got, want)


# ---------------------------------------------------------------------- ranges that are left out

def test_requests_with_bad_query_ranges_are_left_out_and_the_others_computed(ra):
    ctx, Hq, Hkv, d, bs = [40, 90, 33], 4, 2, 64, 16
    k, v, table, _ = paged(51, ctx, Hkv, d, bs, 16, 1, 1)
    q, _ = batch(51, [9], Hq, d)
    w_in = torch.rand(k.shape[:4])
    for qsl, good in [([-1, 2, 5, 9], [1, 2]), ([0, 2, 5, 10], [0, 1]), ([4, 6, 0, 4], [0, 2]), ([7, 3, 9, 2 ** 31 - 1], [1]),
                      ([-2 ** 31, -1, 3, 5], [2])]:
        args = dev(k, v, table, i32(*qsl), i32(*ctx))
        o = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
        lse = torch.full(q.shape[:2], 7.0, device=DEV)
        ra.cp_chunk_attn(q.to(DEV), *args, 16, 1, 1, o=o, lse=lse)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS, qsl
        w = ra.cp_attn_weights(q.to(DEV), lse, args[0], *args[2:], 16, 1, 1, w_in=w_in.to(DEV))
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS, qsl
        rest = np.ones(9, dtype=bool)
        for r in range(3):
            if r in good:
                a, b = qsl[r], qsl[r + 1]
                one = (q[a:b], k, v, table[r:r + 1], [0, b - a], ctx[r:r + 1], bs, 16, 1, 1)
                assert_chunk(o[a:b], lse[a:b], S.chunk_attn(*one))
                rest[a:b] = False
                want = S.attn_weights(one[0], lse[a:b].cpu(), k, *one[3:], w_in=w_in.numpy())
            else:      # its tokens keep what they had
                want = S.attn_weights(q[:0], lse[:0].cpu(), k, table[r:r + 1], [0, 0], ctx[r:r + 1], bs, 16, 1, 1, w_in=w_in.numpy())
            assert_weights(w, want)
        assert (o[torch.from_numpy(rest)] == 7).all()
        assert (lse[torch.from_numpy(rest)] == 7).all()


def test_a_context_past_the_table_is_cut_to_it(ra):
    """All tokens of the table are seen (the queries' positions are past them); the other requests are untouched."""
    Hq, Hkv, d, bs = 4, 2, 64, 16
    ctx, n = [40, 96, 33], [2, 3, 4]
    k, v, table, _ = paged(52, ctx, Hkv, d, bs, 16, 1, 1)
    table = table[:, :6].contiguous()                     # 96 tokens
    q, qsl = batch(52, n, Hq, d)
    for long in (97 + 3, 5000, 2 ** 31 - 1):
        args = dev(k, v, table, qsl, i32(40, long, 33))
        o, lse = ra.cp_chunk_attn(q.to(DEV), *args, 16, 1, 1)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS
        rows = np.r_[0:2, 5:9]
        assert_chunk(o[rows], lse[rows], S.chunk_attn(q, k, v, table, qsl, ctx, bs, 16, 1, 1), rows)
        ref = S.chunk_attn(q[2:5], k, v, table[1:2], [0, 3], [96], bs, 16, 1, 1, causal=False)
        assert_chunk(o[2:5], lse[2:5], ref)
