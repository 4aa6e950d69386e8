"""Limits of the attention kernels' waits are for a tile's time, however long the work between a warp's waits is: calls
under a limit of a few tiles give what calls without one give, to the bit, and report nothing.  A wait that expires ends
its kernel with an error status; no fault or endless wait is involved."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys, torch
sys.path.insert(0, sys.argv[1])
from context_long_sequence_ring_gb300 import ringattn as ra
dev = torch.device("cuda:0")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
status, res = [], []
g = torch.Generator().manual_seed(3)
rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)
def call(f):
    res.append([x.cpu() for x in f()])
    status.append([int(ra.device_status()), ra.last_error()])
def gradient(d, *lens):
    T, s = sum(lens), i32(*[sum(lens[:i]) for i in range(len(lens) + 1)])
    x, do = rnd(T, 48, d), rnd(T, 32, d)
    q, k, v = x[:, :32], x[:, 32:40], x[:, 40:]
    o, lse = rnd(T, 32, d), torch.full((T, 32), 9.0, device=dev)
    call(lambda: ra.window_attn_bwd(do, q, k, v, o, lse, s, 1 << 30))
def packed(d, *lens):
    T, s = sum(lens), i32(*[sum(lens[:i]) for i in range(len(lens) + 1)])
    x = rnd(T, 48, d)
    call(lambda: ra.window_attn_fwd(x[:, :32], x[:, 32:40], x[:, 40:], s, 1 << 30))
def paged(d, n, ctx, window):
    nb = -(-ctx // 128)
    q, k, v = rnd(n, 32, d), rnd(1, nb, 8, 128, d), rnd(1, nb, 8, 128, d)
    a = q, k, v, torch.arange(nb, dtype=torch.int32, device=dev).view(1, nb), i32(0, n), i32(ctx)
    call((lambda: ra.cp_window_attn(*a, window, 16, 1, 1, n_sink=4)) if window else (lambda: ra.cp_chunk_attn(*a, 16, 1, 1)))
def weights(d, n, ctx):
    nb = -(-ctx // 128)
    q, k, lse = rnd(n, 32, d), rnd(1, nb, 8, 128, d), torch.full((n, 32), 9.0, device=dev)
    table = torch.arange(nb, dtype=torch.int32, device=dev).view(1, nb)
    call(lambda: (ra.cp_attn_weights(q, lse, k, table, i32(0, n), i32(ctx), 16, 1, 1),))
for what, *a in json.loads(sys.argv[2]):
    globals()[what](*a)
if sys.argv[3] == "save":
    torch.save(res, sys.argv[4])
    same = None
else:
    same = all(torch.equal(x, y) for a, b in zip(res, torch.load(sys.argv[4])) for x, y in zip(a, b))
print(json.dumps([status, same]))
"""


def run(limit, work, *args):
    env = dict(os.environ)
    env.pop("RA_WAIT_LIMIT_CYCLES", None)
    if limit:
        env["RA_WAIT_LIMIT_CYCLES"] = str(limit)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, json.dumps(work), *args], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return json.loads(r.stdout.strip().splitlines()[-1])


def check(limit, work, tmp_path):
    path = str(tmp_path / "results.pt")
    status, _ = run(None, work, "save", path)
    assert all(st == 0 for st, _ in status), status
    status, same = run(limit, work, "compare", path)
    assert all(st == 0 for st, _ in status), status
    assert same


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [(16383,), (16321,), (8191, 5001, 130, 1, 3001)], ids=str)
def test_gradient_whose_last_tiles_alone_pass_a_sequences_end(d, lens, tmp_path):
    """The warp that zeroes rows past a sequence's end has its first tile after nearly all of the dQ kernel, which takes some
    10^6 cycles; no tile takes 2 * 10^5."""
    check(200000, [["gradient", d, *lens]], tmp_path)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("work", [["packed", 16383], ["packed", 9001, 40, 9003], ["paged", 8003, 16321, 12000],
                                  ["paged", 8003, 16321, 0]], ids=str)
def test_forward_of_items_of_many_tiles(d, work, tmp_path):
    """Items are announced four ahead, so that one is waited for while another is worked off, some 100 tiles and 2 * 10^5
    cycles; the warp that zeroes rows waits past several.  No tile takes 10^5 cycles."""
    check(100000, [[work[0], d, *work[1:]]], tmp_path)


@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_items_of_many_query_tiles(d, tmp_path):
    """As above, a pair of key tiles past 128 query tiles at a time."""
    check(100000, [["weights", d, 4096, 65500]], tmp_path)
