"""Edges of the serving operators: queries whose LSE is not a number or that are marked as seeing nothing, evictions of
every cluster size and past the keys that shared memory holds, ranges that are left out, and batches whose work is
counted in coarser units.  Tolerances as in the parity tests of the same operators."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from tests._gpu import ra_lib, check_status
from tests.test_gpu_serving import BF, DEV, assert_chunk, assert_weights, batch, dev, paged

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
