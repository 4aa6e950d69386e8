"""GPU parity of attention with a sliding window and first tokens that stay visible, over the sharded paged cache and on
packed sequences with its gradient, against the float64 oracle.

Tolerances.  Forward: those of the chunk attention (tests/test_gpu_serving.py), whose arithmetic it is.
Backward: P and dS are rounded to bf16 (2^-8 of each term), delta is formed from an O rounded to bf16 (2^-8 sum |dO||O|)
in fp32, and scores, exps and sums are fp32 (a score is off by at most 2^-14, a weight by that factor: 2^-11 of what is
summed covers them together).  The oracle forms the sums of these bounds over the visible pairs; the outputs'
rounding adds half a step, 2^-8 (bf16) or 2^-24 (fp32) of the value."""
import numpy as np
import pytest
import torch

from oracle import window as O
from oracle.serving import token_rows
from tests._gpu import ra_lib, check_status
from tests.test_gpu_serving import BF, DEV, CHUNKS, assert_chunk, batch, dev, paged

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]
FAR = 2 ** 31 - 1


@pytest.fixture(scope="module")
def ra():
    return ra_lib()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


# ---------------------------------------------------------------------- over the paged cache

def run_paged(ra, q, k, v, table, qsl, ctx, window, sink, I, pcp, dcp, **kw):
    o, lse = ra.cp_window_attn(*dev(q, k, v, table, qsl, i32(*ctx)), window, I, pcp, dcp, n_sink=sink, **kw)
    check_status(ra)
    return o, lse


MASKS = [(1, 0), (1, 3), (17, 4), (64, 0), (128, 1), (200, 130), (FAR, 0), (40, FAR)]


@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "%s-%s-h%d.%d-d%d-b%d.%d-w%d" % (c[0], c[1], c[2], c[3], c[4], c[5],
                                                                                 c[6], c[7] * c[8]))
@pytest.mark.parametrize("window,sink", MASKS)
def test_paged(ra, case, window, sink):
    ctx, n, Hq, Hkv, d, bs, I, pcp, dcp = case
    k, v, table, _ = paged(sum(ctx), ctx, Hkv, d, bs, I, pcp, dcp)
    q, qsl = batch(sum(ctx), n, Hq, d)
    ref = O.cp_window_attn(q, k, v, table, qsl, ctx, window, sink, bs, I, pcp, dcp)
    o, lse = run_paged(ra, q, k, v, table, qsl, ctx, window, sink, I, pcp, dcp)
    assert_chunk(o, lse, ref)
    o32, lse32 = run_paged(ra, q, k, v, table, qsl, ctx, window, sink, I, pcp, dcp, out_dtype=torch.float32)
    assert o32.dtype == torch.float32 and torch.equal(o32.to(BF), o) and torch.equal(lse32, lse)


def drop_unseen(k, v, table, ctx, n, window, sink, V, junk):
    """Table entries of blocks that no query sees become junk, and what other blocks hold there NaN."""
    t = table.clone()
    for r, x in enumerate(ctx):
        seen = O.visible(n[r], x, window, sink).any(axis=0)
        for vb in range(-(-x // V)):
            if not seen[vb * V:(vb + 1) * V].any():
                t[r, vb] = junk
                k[:, table[r, vb]] = float("nan")
                v[:, table[r, vb]] = float("nan")
    return t


@pytest.mark.parametrize("d,bs,I,pcp,window,sink", [(128, 16, 4, 1, 100, 4), (64, 32, 16, 2, 33, 0), (64, 16, 16, 1, 1, 1),
                                                    (128, 128, 16, 1, 150, 2)])
@pytest.mark.parametrize("junk", [-1, 10 ** 9, -2 ** 31, "another"])
def test_paged_blocks_out_of_sight_may_be_gone(ra, d, bs, I, pcp, window, sink, junk):
    ctx, n, Hq, Hkv = [1300, 700, 260], [1, 70, 200], 8, 2
    k, v, table, spare = paged(3, ctx, Hkv, d, bs, I, pcp, 1)
    q, qsl = batch(3, n, Hq, d)
    t = drop_unseen(k, v, table, ctx, n, window, sink, bs * pcp, int(spare[0]) if junk == "another" else junk)
    k[:, spare[0]] = v[:, spare[0]] = float("nan")
    assert (t != table).any()
    ref = O.cp_window_attn(q, k, v, table, qsl, ctx, window, sink, bs, I, pcp, 1)
    o, lse = run_paged(ra, q, k, v, t, qsl, ctx, window, sink, I, pcp, 1)
    assert_chunk(o, lse, ref)


def test_paged_many_requests_of_all_kinds(ra):
    for d, bs, Hq, Hkv, window, sink in [(128, 32, 8, 2, 50, 2), (64, 16, 12, 3, 20, 0)]:
        rng = np.random.default_rng(d)
        n = rng.choice([0, 1, 1, 2, 4, 6, 20, 50, 90], size=330)
        ctx = np.maximum(n + rng.integers(-3, 120, size=330), 0).tolist()
        k, v, table, _ = paged(d, ctx, Hkv, d, bs, 4, 1, 2)
        q, qsl = batch(d, n, Hq, d)
        ref = O.cp_window_attn(q, k, v, table, qsl, ctx, window, sink, bs, 4, 1, 2)
        assert_chunk(*run_paged(ra, q, k, v, table, qsl, ctx, window, sink, 4, 1, 2), ref)


@pytest.mark.parametrize("d,bs,I,pcp", [(64, 16, 16, 1), (64, 64, 8, 2), (128, 32, 16, 2)])
@pytest.mark.parametrize("window,sink", [(400, 4), (700, 0), (130, 200)])
def test_paged_long_parts(ra, d, bs, I, pcp, window, sink):
    """Enough keys that each CTA walks many tiles of several row tiles of both kinds, borders anywhere."""
    rng = np.random.default_rng(bs)
    n = rng.choice([1, 1, 3, 7, 70, 150], size=40)
    ctx = (n + rng.integers(200, 1900, size=40)).tolist()
    Hq, Hkv = 12, 4
    k, v, table, _ = paged(bs, ctx, Hkv, d, bs, I, pcp, 1)
    q, qsl = batch(bs, n, Hq, d)
    ref = O.cp_window_attn(q, k, v, table, qsl, ctx, window, sink, bs, I, pcp, 1)
    assert_chunk(*run_paged(ra, q, k, v, table, qsl, ctx, window, sink, I, pcp, 1), ref)


def test_paged_rows_that_see_nothing_and_rows_of_nobody(ra):
    ctx, n, Hq, Hkv, d = [3, 0, 40, 6], [7, 4, 2, 0], 4, 2, 128
    k, v, table, _ = paged(5, ctx, Hkv, d, 16, 16, 1, 1)
    q, qsl = batch(5, n, Hq, d, before=3, after=5)
    ref = O.cp_window_attn(q, k, v, table, qsl, ctx, 2, 1, 16, 16, 1, 1)
    o, lse = torch.full(q.shape, 7.0, dtype=BF, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
    run_paged(ra, q, k, v, table, qsl, ctx, 2, 1, 16, 1, 1, o=o, lse=lse)
    mine = slice(3, 3 + sum(n))
    assert_chunk(o[mine], lse[mine], ref, mine)
    rest = np.r_[0:3, 3 + sum(n):q.shape[0]]
    assert (o[rest] == 7).all() and (lse[rest] == 7).all()


def test_paged_nan_queries_and_keys_reach_only_who_sees_them(ra):
    ctx, n, Hq, Hkv, d, window, sink = [300, 70], [9, 40], 4, 2, 128, 20, 3
    k, v, table, _ = paged(31, ctx, Hkv, d, 16, 16, 1, 1)
    q, qsl = batch(31, n, Hq, d)
    ref = O.cp_window_attn(q, k, v, table, qsl, ctx, window, sink, 16, 16, 1, 1)
    q[1, 0] = float("nan")
    k[0, table[1, 3], 1, 2] = float("nan")       # token 50 of request 1, K/V head 1: seen by positions 50 .. 69
    o, lse = run_paged(ra, q, k, v, table, qsl, ctx, window, sink, 16, 1, 1)
    bad = torch.zeros((49, Hq), dtype=torch.bool)
    bad[1, 0] = True
    bad[9 + 20:9 + 40, 2:] = True
    assert o.cpu()[bad].isnan().all() and lse.cpu()[bad].isnan().all()
    good = ~bad.numpy()
    err = np.abs(o.double().cpu().numpy() - ref[0])
    assert (err[good] <= (2.0 ** -8 * (ref[2] + np.abs(ref[0])) + 2.0 ** -11 * ref[2])[good]).all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1])[good] <= 2.0 ** -12).all()


def test_paged_bad_blocks_and_ranges_are_reported(ra):
    ctx, n, Hq, Hkv, d, bs, window, sink = [40, 90, 33], [2, 3, 4], 4, 2, 64, 16, 30, 2
    k, v, table, _ = paged(10, ctx, Hkv, d, bs, 16, 1, 1)
    q, qsl = batch(10, n, Hq, d)
    ref = O.cp_window_attn(q, k, v, table, qsl, ctx, window, sink, bs, 16, 1, 1)
    for bad in (-1, k.shape[1], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 4] = bad                       # tokens 64 .. 79 of request 1 are left out
        o, lse = ra.cp_window_attn(*dev(q, k, v, t, qsl, i32(*ctx)), window, 16, 1, 1, n_sink=sink)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS
        rows = np.r_[0:2, 5:9]
        assert_chunk(o[rows], lse[rows], ref, rows)
        seen = O.visible(3, 90, window, sink)
        seen[:, 64:80] = False
        kt, vt = (token_rows(x.double().numpy(), table[1].numpy(), range(90), bs, 16, 1, 1) for x in (k, v))
        Or, Lr, Ar, _ = O.attend(q[2:5].double().numpy(), kt, vt, seen)
        assert_chunk(o[2:5], lse[2:5], (Or, Lr, Ar))
    for qs in ([0, 2, 1, 9], [-1, 2, 5, 9], [0, 2, 5, 10]):
        o = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
        ra.cp_window_attn(*dev(q, k, v, table, i32(*qs), i32(*ctx)), window, 16, 1, 1, n_sink=sink, o=o)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS and torch.isfinite(o.float()).all()
    # a context longer than its table is cut to it
    ra.cp_window_attn(*dev(q, k, v, table[:, :6].contiguous(), qsl, i32(40, 90, 2 ** 31 - 1)), window, 16, 1, 1)
    assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS
    check_status(ra)


def test_paged_window_of_everything_is_chunk_attention_and_calls_repeat(ra):
    ctx, n, Hq, Hkv, d = [3000, 1, 800, 2000], [5, 1, 400, 1], 8, 2, 128
    k, v, table, _ = paged(11, ctx, Hkv, d, 128, 16, 1, 1)
    q, qsl = batch(11, n, Hq, d)
    args = dev(q, k, v, table, qsl, i32(*ctx))
    ref = ra.cp_chunk_attn(*args, 16, 1, 1)
    for _ in range(2):
        got = ra.cp_window_attn(*args, FAR, 16, 1, 1)
        check_status(ra)
        # each within its bound of the exact value (A <= max |v| < 6)
        assert (got[0].float() - ref[0].float()).abs().max() <= 2 * (2.0 ** -7 + 2.0 ** -11) * 6
        assert (got[1] - ref[1]).abs().max() <= 2.0 ** -11
    twice = [ra.cp_window_attn(*args, 333, 16, 1, 1, n_sink=4) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*twice))


def test_paged_replayed_with_other_lengths_beside_another_stream(ra):
    """One captured call for any lengths, next to another graph on its own workspace."""
    Hq, Hkv, d, bs, I, window, sink, R, T = 8, 2, 64, 16, 4, 70, 3, 3, 320
    graphs = []
    for i in range(2):
        k, v, _, _ = paged(20 + i, [800, 800, 800], Hkv, d, bs, I, 1, 2, poison=False)
        table = torch.randperm(k.shape[1], generator=torch.Generator().manual_seed(i)).to(torch.int32)[:75].view(3, 25)
        q = torch.randn((T, Hq, d), generator=torch.Generator().manual_seed(30 + i)).to(BF)
        qd, kd, vd, td = dev(q, k, v, table)
        s, c = (torch.zeros(m, dtype=torch.int32, device=DEV) for m in (R + 1, R))
        ws = torch.empty(ra.cp_window_attn_workspace_size(Hq, Hkv, d), dtype=torch.uint8, device=DEV)
        o, lse = torch.zeros((T, Hq, d), dtype=BF, device=DEV), torch.zeros((T, Hq), device=DEV)

        def call():
            ra.cp_window_attn(qd, kd, vd, td, s, c, window, I, 1, 2, n_sink=sink, workspace=ws, o=o, lse=lse)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((q, k, v, table, s, c, o, lse, g, (qd, kd, vd, td, ws)))
    for n, ctx in (([1, 1, 1], [800, 3, 412]), ([300, 0, 20], [700, 0, 800]), ([0, 0, 0], [5, 5, 5]), ([7, 160, 1], [7, 161, 800])):
        qsl = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
        for x in graphs:
            x[4].copy_(qsl)
            x[5].copy_(i32(*ctx))
            x[6].fill_(7.0)
            x[7].fill_(7.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][8].replay()
        with torch.cuda.stream(side):
            graphs[1][8].replay()
        torch.cuda.current_stream().wait_stream(side)
        check_status(ra)
        m = sum(n)
        for q, k, v, table, s, c, o, lse, _, _ in graphs:
            if m:
                assert_chunk(o[:m], lse[:m], O.cp_window_attn(q[:m], k, v, table, qsl, ctx, window, sink, bs, I, 1, 2))
            assert (o[m:] == 7).all() and (lse[m:] == 7).all()


def test_paged_past_32_bit_offsets(ra):
    """Blocks at the far end of caches of more than 2^31 elements."""
    NB, Hq, Hkv, d, bs, ctx, n, window, sink = 17000, 16, 8, 128, 128, [300, 200], [130, 1], 90, 4
    k, v, table, _ = paged(40, ctx, Hkv, d, bs, 16, 1, 1, poison=False)
    q, qsl = batch(40, n, Hq, d)
    ref = O.cp_window_attn(q, k, v, table, qsl, ctx, window, sink, bs, 16, 1, 1)
    far = NB - k.shape[1]
    kc, vc = (torch.zeros((1, NB, Hkv, bs, d), dtype=BF, device=DEV) for _ in range(2))
    kc[:, far:], vc[:, far:] = k.to(DEV), v.to(DEV)
    o, lse = ra.cp_window_attn(*dev(q), kc, vc, *dev(torch.where(table < 0, table, table + far), qsl, i32(*ctx)), window, 16, 1, 1,
                               n_sink=sink)
    check_status(ra)
    assert_chunk(o, lse, ref)


# ---------------------------------------------------------------------- packed sequences

# lengths, Hq, Hkv, d, window, sink
PACKED = [
    ([1], 4, 2, 128, 1, 0),
    ([1, 2, 129, 127], 8, 1, 64, 5, 2),
    ([300, 5, 77], 6, 2, 128, 64, 4),
    ([257, 0, 300, 128], 6, 2, 64, 130, 1),
    ([700], 5, 5, 128, 100, 130),
    ([517], 8, 2, 128, FAR, 0),
    ([130, 500, 20], 16, 1, 64, 33, 300),
    ([1029, 64, 3], 40, 8, 128, 300, 4),
    ([900], 64, 1, 128, 128, 16),
    ([400, 131], 3, 3, 128, 1, 1),
    ([256, 384], 4, 4, 64, 128, 0),
    ([385], 7, 1, 128, 127, 0),
    ([640, 1, 1, 1], 9, 3, 64, 129, 128),
    ([333], 2, 2, 64, 40, FAR),
    ([1500], 4, 2, 64, 700, 0),
    ([1111], 12, 4, 128, 1024, 129),
]


def packed(seed, n, Hq, Hkv, d, before=0, after=0):
    """q, k, v as parts of one projection's rows, do, and the sequences' borders."""
    g = torch.Generator().manual_seed(seed)
    qsl = torch.tensor(np.concatenate([[before], before + np.cumsum(n)]), dtype=torch.int32)
    T = int(qsl[-1]) + after
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(BF)
    return x, torch.randn((T, Hq, d), generator=g).to(BF), qsl


def parts(x, Hq, Hkv):
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def assert_grads(got, ref, rows=None):
    for name, x, want, bound in zip(("dq", "dk", "dv"), got, *ref):
        half = 2.0 ** -8 if x.dtype == BF else 2.0 ** -24
        x = x.double().cpu().numpy()
        if rows is not None:
            x, want, bound = x[rows], want[rows], bound[rows]
        live = ~np.isnan(want)
        assert np.isfinite(x[live]).all(), name
        over = np.abs(x - want)[live] - (bound + half * np.abs(want))[live]
        # a sum of n terms in fp32: n 2^-24 of its size, far inside the bound but where that is next to 0
        assert over.max(initial=0.0) <= 2.0 ** -20, (name, over.max())


@pytest.mark.parametrize("case", PACKED, ids=lambda c: "%s-h%d.%d-d%d-w%d.%d" % c)
def test_packed(ra, case):
    n, Hq, Hkv, d, window, sink = case
    x, do, qsl = packed(sum(n), n, Hq, Hkv, d)
    q, k, v = parts(x, Hq, Hkv)
    ref = O.window_attn(q, k, v, qsl, window, sink)
    xd, dd, sd = dev(x, do, qsl)
    qd, kd, vd = parts(xd, Hq, Hkv)
    o, lse = ra.window_attn_fwd(qd, kd, vd, sd, window, n_sink=sink)
    check_status(ra)
    assert_chunk(o, lse, ref)
    o32, lse32 = ra.window_attn_fwd(qd, kd, vd, sd, window, n_sink=sink, out_dtype=torch.float32)
    assert torch.equal(o32.to(BF), o) and torch.equal(lse32, lse)
    grads = O.window_attn_grad(do, q, k, v, qsl, window, sink)
    # from the exact O and LSE, rounded once: the bound counts that
    oe, le = torch.from_numpy(ref[0]).to(BF).to(DEV), torch.from_numpy(ref[1]).float().to(DEV)
    for dt in (BF, torch.float32):
        got = ra.window_attn_bwd(dd, qd, kd, vd, oe, le, sd, window, n_sink=sink, out_dtype=dt)
        check_status(ra)
        assert all(g.dtype == dt for g in got)
        assert_grads(got, grads)
    # into parts of one gradient
    dx = torch.full(x.shape, 7.0, dtype=BF, device=DEV)
    a = parts(dx, Hq, Hkv)
    b = ra.window_attn_bwd(dd, qd, kd, vd, oe, le, sd, window, n_sink=sink, dq=a[0], dk=a[1], dv=a[2])
    c = ra.window_attn_bwd(dd, *(t.contiguous() for t in (qd, kd, vd)), oe, le, sd, window, n_sink=sink)
    check_status(ra)
    assert all(torch.equal(s, t) for s, t in zip(b, c))


def test_packed_many_sequences(ra):
    """More sequences than a block of the list building holds, empty ones among them; several rounds of key tiles, and first
    tokens that long sequences see from afar."""
    rng = np.random.default_rng(8)
    n = rng.choice([0, 0, 1, 1, 2, 5, 40, 130], size=1500)
    n[[3, 700, 1100, 1499]] = [600, 450, 513, 700]
    Hq, Hkv, d, window, sink = 4, 2, 64, 100, 3
    x, do, qsl = packed(8, n, Hq, Hkv, d)
    q, k, v = parts(x, Hq, Hkv)
    ref = O.window_attn(q, k, v, qsl, window, sink)
    xd, dd, sd = dev(x, do, qsl)
    o, lse = ra.window_attn_fwd(*parts(xd, Hq, Hkv), sd, window, n_sink=sink)
    check_status(ra)
    assert_chunk(o, lse, ref)
    oe, le = torch.from_numpy(ref[0]).to(BF).to(DEV), torch.from_numpy(ref[1]).float().to(DEV)
    got = ra.window_attn_bwd(dd, *parts(xd, Hq, Hkv), oe, le, sd, window, n_sink=sink)
    check_status(ra)
    assert_grads(got, O.window_attn_grad(do, q, k, v, qsl, window, sink))


def test_packed_rows_of_nobody_and_ranges(ra):
    n, Hq, Hkv, d, window, sink = [100, 0, 150], 4, 2, 128, 60, 2
    x, do, qsl = packed(1, n, Hq, Hkv, d, before=5, after=9)
    x[:5] = do[:5] = float("nan")              # rows of nobody hold anything
    x[-9:] = do[-9:] = float("nan")
    q, k, v = parts(x, Hq, Hkv)
    ref = O.window_attn(q, k, v, qsl, window, sink)
    grads = O.window_attn_grad(do, q, k, v, qsl, window, sink)
    xd, dd, sd = dev(x, do, qsl)
    qd, kd, vd = parts(xd, Hq, Hkv)
    T = x.shape[0]
    o, lse = torch.full((T, Hq, d), 7.0, dtype=BF, device=DEV), torch.full((T, Hq), 7.0, device=DEV)
    ra.window_attn_fwd(qd, kd, vd, sd, window, n_sink=sink, o=o, lse=lse)
    dx = torch.full(x.shape, 7.0, dtype=BF, device=DEV)
    dq, dk, dv = parts(dx, Hq, Hkv)
    ra.window_attn_bwd(dd, qd, kd, vd, o, lse, sd, window, n_sink=sink, dq=dq, dk=dk, dv=dv)
    check_status(ra)
    mine, rest = slice(5, T - 9), np.r_[0:5, T - 9:T]
    assert_chunk(o[mine], lse[mine], ref, mine)
    assert (o[rest] == 7).all() and (lse[rest] == 7).all() and (dx[rest] == 7).all()
    oe, le = torch.from_numpy(ref[0]).to(BF).to(DEV), torch.from_numpy(ref[1]).float().to(DEV)
    got = ra.window_attn_bwd(dd, qd, kd, vd, oe, le, sd, window, n_sink=sink)
    assert_grads(got, grads, mine)
    # sequences whose range decreases or leaves [0, T] are left out, the others are computed
    for qs, good in (([5, 105, 90, 255], slice(5, 90)), ([-1, 105, 105, 255], slice(105, 255)), ([5, 105, 105, T + 1], slice(5, 105))):
        o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
        ra.window_attn_fwd(qd, kd, vd, i32(*qs).to(DEV), window, n_sink=sink, o=o2, lse=lse2)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS
        assert_chunk(o2[good], lse2[good], ref, good)
        dx2 = torch.full_like(dx, 7.0)
        a = parts(dx2, Hq, Hkv)
        ra.window_attn_bwd(dd, qd, kd, vd, oe, le, i32(*qs).to(DEV), window, n_sink=sink, dq=a[0], dk=a[1], dv=a[2])
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS
        assert_grads(a, grads, good)
    check_status(ra)


def test_packed_neighbours_with_nan_and_infinities_do_not_reach_a_sequence(ra):
    """Sequences that end inside a tile, between neighbours full of NaN and infinities: the same bits as without them."""
    n, Hq, Hkv, d = [90, 130, 200], 6, 2, 128
    x, do, qsl = packed(2, n, Hq, Hkv, d)
    mine = slice(90, 220)
    out = []
    for junk in (None, float("nan"), float("inf")):
        y, e = x.clone(), do.clone()
        if junk is not None:
            y[:90] = y[220:] = e[:90] = e[220:] = junk
        yd, ed, sd = dev(y, e, qsl)
        q, k, v = parts(yd, Hq, Hkv)
        o, lse = ra.window_attn_fwd(q, k, v, sd, 50, n_sink=3)
        out.append([t[mine] for t in (o, lse, *ra.window_attn_bwd(ed, q, k, v, o, lse, sd, 50, n_sink=3))])
        check_status(ra)
    assert all(torch.isfinite(t).all() for t in out[0])
    for got in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], got))


def test_packed_gradient_of_rows_without_weight(ra):
    """A row whose LSE is +inf has no weight: no gradient of its own, none in what it sees."""
    n, Hq, Hkv, d = [300], 4, 2, 64
    x, do, qsl = packed(3, n, Hq, Hkv, d)
    xd, dd, sd = dev(x, do, qsl)
    q, k, v = parts(xd, Hq, Hkv)
    o, lse = ra.window_attn_fwd(q, k, v, sd, 70, n_sink=2)
    lse[40, 1] = lse[200] = float("inf")
    dq, dk, dv = ra.window_attn_bwd(dd, q, k, v, o, lse, sd, 70, n_sink=2, out_dtype=torch.float32)
    check_status(ra)
    assert (dq[40, 1] == 0).all() and (dq[200] == 0).all() and dq[40, 0].any()
    d2 = dd.clone()
    d2[40, 1] = d2[200] = 0                    # no gradient there instead: the same dV
    _, lse2 = ra.window_attn_fwd(q, k, v, sd, 70, n_sink=2)
    dv2 = ra.window_attn_bwd(d2, q, k, v, o, lse2, sd, 70, n_sink=2, out_dtype=torch.float32)[2]
    assert torch.equal(dv, dv2)


@pytest.mark.parametrize("n,window,sink", [([300, 41], 60, 3), ([700], 600, 0)])
def test_packed_gradient_of_a_part_of_the_keys(ra, n, window, sink):
    """o and lse of a softmax over more keys than these (as on one of several devices): what these keys contribute."""
    Hq, Hkv, d = 6, 2, 128
    x, do, qsl = packed(8, n, Hq, Hkv, d)
    q, k, v = parts(x, Hq, Hkv)
    g = torch.Generator().manual_seed(9)
    T = sum(n)
    ref = O.window_attn(q, k, v, qsl, window, sink)
    more = torch.rand((T, Hq), generator=g, dtype=torch.float64) * 3        # how much the other keys add to the LSE
    more[::5] = 1e-6                                                       # next to nothing, for some rows
    lse = (torch.from_numpy(ref[1]) + more).float()
    w = torch.exp(-more)[..., None]
    o = (torch.from_numpy(ref[0]) * w + torch.randn((T, Hq, d), generator=g, dtype=torch.float64) * (1 - w)).to(BF)
    want, bound = O.window_attn_grad(do, q, k, v, qsl, window, sink, o=o, lse=lse)
    xd, dd, sd, od, ld = dev(x, do, qsl, o, lse)
    got = ra.window_attn_bwd(dd, *parts(xd, Hq, Hkv), od, ld, sd, window, n_sink=sink)
    check_status(ra)
    assert_grads(got, (want, bound))


def test_packed_scale_sharp_and_large_values(ra):
    n, Hq, Hkv, d, window, sink, scale = [600], 4, 2, 64, 150, 4, 0.3
    x, do, qsl = packed(6, n, Hq, Hkv, d)
    x[:, Hq:Hq + Hkv, 0] *= 40      # scores of tens: a growing maximum, weights that underflow
    x[:, Hq + Hkv:] *= 100
    q, k, v = parts(x, Hq, Hkv)
    # scores off by (d + 2) 2^-24 sum|q k|: sum|q k| up to ~6 * 160 + 60, scale 0.3: weights off by 1.3e-3 each
    ref = O.window_attn(q, k, v, qsl, window, sink, scale)
    xd, dd, sd = dev(x, do, qsl)
    qd, kd, vd = parts(xd, Hq, Hkv)
    o, lse = ra.window_attn_fwd(qd, kd, vd, sd, window, n_sink=sink, scale=scale)
    check_status(ra)
    assert (np.abs(o.double().cpu().numpy() - ref[0]) <= 2.0 ** -8 * (ref[2] + np.abs(ref[0])) + 2.6e-3 * ref[2]).all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= 2.6e-3).all()
    want, bound = O.window_attn_grad(do, q, k, v, qsl, window, sink, scale)
    oe, le = torch.from_numpy(ref[0]).to(BF).to(DEV), torch.from_numpy(ref[1]).float().to(DEV)
    got = ra.window_attn_bwd(dd, qd, kd, vd, oe, le, sd, window, n_sink=sink, scale=scale)
    check_status(ra)
    # bound holds 2^-11 (4.9e-4) of what is summed for the weights' own error: here it is 1.3e-3 + 4.9e-4, at most 4 times
    assert_grads(got, (want, [4 * b for b in bound]))


@pytest.mark.parametrize("Hq,Hkv,d,window", [(4, 2, 128, 64), (6, 2, 64, 3), (1, 1, 64, 8)])
def test_packed_gradient_of_short_rows_is_exact(ra, Hq, Hkv, d, window):
    """Rows of 2 to 8 keys, whose delta is summed from P and dP: o's rounding to bf16 (up to 2^-8 of the delta, 0.003 of
    dQ's norm with 2 keys) does not reach dQ.  What is left is the arithmetic of fp32 and dS in two parts of bf16: a weight
    off by 2^-11 at most, and with it dQ's norm."""
    n = [2, 3, 4, 5, 8, 2, 7, 6] * 20
    x, do, qsl = packed(d, n, Hq, Hkv, d)
    q, k, v = parts(x, Hq, Hkv)
    ref = O.window_attn(q, k, v, qsl, window, 0)
    dq, _, _ = O.window_attn_grad(do, q, k, v, qsl, window, 0)[0]
    xd, dd, sd = dev(x, do, qsl)
    oe, le = torch.from_numpy(ref[0]).to(BF).to(DEV), torch.from_numpy(ref[1]).float().to(DEV)
    got = ra.window_attn_bwd(dd, *parts(xd, Hq, Hkv), oe, le, sd, window, out_dtype=torch.float32)[0].double().cpu().numpy()
    check_status(ra)
    assert np.linalg.norm(got - dq) <= 2.0 ** -11 * np.linalg.norm(dq)


def test_packed_gradient_against_differences(ra):
    """Directional differences of the oracle's forward pass, in 64 bits, against the kernels' gradients."""
    n, Hq, Hkv, d, window, sink = [150, 40], 4, 2, 64, 45, 3
    x, do, qsl = packed(7, n, Hq, Hkv, d)
    ts = [t.double().numpy() for t in parts(x, Hq, Hkv)]
    want, bound = O.window_attn_grad(do, *ts, qsl, window, sink)
    xd, dd, sd = dev(x, do, qsl)
    q, k, v = parts(xd, Hq, Hkv)
    ref = O.window_attn(*ts, qsl, window, sink)
    oe, le = torch.from_numpy(ref[0]).to(BF).to(DEV), torch.from_numpy(ref[1]).float().to(DEV)
    got = ra.window_attn_bwd(dd, q, k, v, oe, le, sd, window, n_sink=sink, out_dtype=torch.float32)
    check_status(ra)
    for i in range(3):
        for seed in range(3):
            u = np.random.default_rng(seed).standard_normal(ts[i].shape)
            hi, lo = list(ts), list(ts)
            hi[i], lo[i] = ts[i] + 1e-5 * u, ts[i] - 1e-5 * u
            f = [(O.window_attn(*y, qsl, window, sink)[0] * do.double().numpy()).sum() for y in (hi, lo)]
            g = (got[i].double().cpu().numpy() * u).sum()
            assert abs((f[0] - f[1]) / 2e-5 - g) <= (bound[i] * np.abs(u)).sum() + 1e-6


def test_packed_replayed_with_other_lengths_beside_another_stream(ra):
    """Forward and backward captured together and replayed with other lengths, next to another graph on its own workspace."""
    Hq, Hkv, d, T, window, sink = 6, 2, 128, 700, 150, 4
    graphs = []
    for _ in range(2):
        x, dx = torch.zeros((T, Hq + 2 * Hkv, d), dtype=BF, device=DEV), torch.zeros((T, Hq + 2 * Hkv, d), dtype=BF, device=DEV)
        do, s = torch.zeros((T, Hq, d), dtype=BF, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
        ws = torch.empty(ra.window_attn_workspace_size(T, 3, Hq, Hkv, d), dtype=torch.uint8, device=DEV)
        o, lse = torch.zeros((T, Hq, d), dtype=BF, device=DEV), torch.zeros((T, Hq), device=DEV)

        def call():
            q, k, v = parts(x, Hq, Hkv)
            dq, dk, dv = parts(dx, Hq, Hkv)
            ra.window_attn_fwd(q, k, v, s, window, n_sink=sink, workspace=ws, o=o, lse=lse)
            ra.window_attn_bwd(do, q, k, v, o, lse, s, window, n_sink=sink, workspace=ws, dq=dq, dk=dk, dv=dv)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((x, dx, do, s, o, lse, g, ws))
    for n in ([300, 0, 400], [1, 130, 7], [0, 0, 0], [699, 1, 0]):
        refs = []
        for i, (x, dx, do, s, o, lse, g, _) in enumerate(graphs):
            xh, dh, qsl = packed(sum(n) + i, n, Hq, Hkv, d, after=T - sum(n))
            x.copy_(xh)
            do.copy_(dh)
            s.copy_(qsl)
            for t in (dx, o, lse):
                t.fill_(7.0)
            refs.append((O.window_attn(*parts(xh, Hq, Hkv), qsl, window, sink), xh, dh, qsl))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][6].replay()
        with torch.cuda.stream(side):
            graphs[1][6].replay()
        torch.cuda.current_stream().wait_stream(side)
        check_status(ra)
        for (x, dx, do, s, o, lse, _, _), (ref, xh, dh, qsl) in zip(graphs, refs):
            m = sum(n)
            if m:
                assert_chunk(o[:m], lse[:m], ref, slice(0, m))
                # the same as a call of its own
                again = ra.window_attn_bwd(do, *parts(x, Hq, Hkv), o, lse, s, window, n_sink=sink)
                check_status(ra)
                assert all(torch.equal(a[:m], b[:m]) for a, b in zip(parts(dx, Hq, Hkv), again))
            assert (o[m:] == 7).all() and (lse[m:] == 7).all() and (dx[m:] == 7).all()


def test_packed_is_the_paged_form_of_a_whole_prompt(ra):
    ctx, Hq, Hkv, d, bs, window, sink = [700, 333], 8, 2, 128, 32, 90, 4
    k, v, table, _ = paged(12, ctx, Hkv, d, bs, 16, 1, 2, poison=False)
    q, qsl = batch(12, ctx, Hq, d)
    kd, vd, td, sd, cd = dev(k, v, table.clamp(min=0), qsl, i32(*ctx))
    pos = torch.cat([torch.arange(c, dtype=torch.int32) for c in ctx]).to(DEV)
    kt, vt = ra.cp_kv_gather(kd, vd, td, sd, pos, 16, 1, 2)
    a = ra.window_attn_fwd(q.to(DEV), kt, vt, sd, window, n_sink=sink, out_dtype=torch.float32)
    b = ra.cp_window_attn(q.to(DEV), kd, vd, td, sd, cd, window, 16, 1, 2, n_sink=sink, out_dtype=torch.float32)
    check_status(ra)
    assert (a[0] - b[0]).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -11) * 6 and (a[1] - b[1]).abs().max() <= 2.0 ** -11


def test_packed_no_tokens(ra):
    e = lambda h: torch.zeros((0, h, 64), dtype=BF, device=DEV)  # noqa: E731
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    o, lse = ra.window_attn_fwd(e(4), e(2), e(2), s, 5)
    dq, dk, dv = ra.window_attn_bwd(e(4), e(4), e(2), e(2), o, lse, s, 5)
    assert o.shape == (0, 4, 64) and dq.shape == (0, 4, 64) and dk.shape == dv.shape == (0, 2, 64)
    check_status(ra)
