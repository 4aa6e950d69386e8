"""The way out of the serving kernels on the tensor cores when a wait expires at any point of their work: with limits
from the first load's latency up to a few row tiles', some waits pass and a later one expires, in any role.  Each call
must then either have finished, with the results of an unlimited call, or report the timeout; products, copies and
stores to tensor memory in flight land first, and the context stays usable.  No fault or endless wait is involved."""
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
res, status = {}, {}
for d in (64, 128):
    g = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)
    k, v, table = rnd(1, 320, 2, 64, d), rnd(1, 320, 2, 64, d), torch.arange(320, dtype=torch.int32, device=dev).view(2, 160)
    for name, n in (("single", 1), ("draft", 5), ("prompt", 300)):
        q, qsl, ctx = rnd(2 * n, 8, d), i32(0, n, 2 * n), i32(10200, 9001)
        for i in range(4):
            o, lse = ra.cp_chunk_attn(q, k, v, table, qsl, ctx, 16, 1, 1)
            status["chunk %s %d %d" % (name, d, i)] = [int(ra.device_status()), ra.last_error()]
            res["chunk %s %d %d" % (name, d, i)] = [o.cpu(), lse.cpu()]
        lse = torch.full((2 * n, 8), 9.0, device=dev)
        for i in range(4):
            w = ra.cp_attn_weights(q, lse, k, table, qsl, ctx, 16, 1, 1)
            status["weights %s %d %d" % (name, d, i)] = [int(ra.device_status()), ra.last_error()]
            res["weights %s %d %d" % (name, d, i)] = [w.cpu()]
src = torch.arange(64 * 8, dtype=torch.float32, device=dev).view(64, 8)
idx = torch.randperm(64, generator=g).to(torch.int32).to(dev)
ok = bool(torch.equal(ra.gather_rows(src, idx).cpu(), src.cpu()[idx.long().cpu()])) and ra.device_status() == 0
if len(sys.argv) == 3:
    torch.save(res, sys.argv[2])
    same = {}
else:
    want = torch.load(sys.argv[3])
    same = {x: all(torch.equal(a, b) for a, b in zip(res[x], want[x])) for x in res}
print(json.dumps([status, same, ok]))
"""


def run(limit, *args):
    env = dict(os.environ)
    env.pop("RA_WAIT_LIMIT_CYCLES", None)
    if limit:
        env["RA_WAIT_LIMIT_CYCLES"] = str(limit)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *args], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.fixture(scope="module")
def unlimited(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("limits") / "results.pt")
    status, _, ok = run(None, path)
    assert ok and all(st == 0 for st, _ in status.values())
    return path


@pytest.mark.parametrize("limit", [900, 2500, 6000, 20000])
def test_waits_that_expire_midway(unlimited, limit):
    from context_long_sequence_ring_gb300 import ringattn
    status, same, ok = run(limit, "compare", unlimited)
    assert ok
    for name, (st, msg) in status.items():
        assert st in (0, ringattn.RA_ERR_TIMEOUT), (name, st, msg)
        if st == 0:
            assert same[name], name
        else:
            assert ("chunk attention" if "chunk" in name else "attention weights") in msg, (name, msg)
