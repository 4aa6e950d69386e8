"""The way out of the window attention's kernels, forward and backward, when a wait expires: at the first wait that is not
satisfied at once, and at any point of their work.  Each call must either have finished, with the results of an
unlimited call, or report the timeout; products, copies and stores to tensor memory in flight land first, and the context
stays usable.  No fault or endless wait is involved."""
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
def call(name, f):
    for i in range(3):
        out = f()
        status["%s %d" % (name, i)] = [int(ra.device_status()), ra.last_error()]
        res["%s %d" % (name, i)] = [x.cpu() for x in out]
for d in (64, 128):
    g = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)
    k, v, table = rnd(1, 320, 2, 64, d), rnd(1, 320, 2, 64, d), torch.arange(320, dtype=torch.int32, device=dev).view(2, 160)
    for name, n in (("single", 1), ("prompt", 300)):
        q, qsl, ctx = rnd(2 * n, 8, d), i32(0, n, 2 * n), i32(10200, 9001)
        call("paged %s %d" % (name, d), lambda: ra.cp_window_attn(q, k, v, table, qsl, ctx, 3000, 16, 1, 1, n_sink=4))
    T = 2500
    x, do, s = rnd(T, 12, d), rnd(T, 8, d), i32(0, 1900, T)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    call("packed %d" % d, lambda: ra.window_attn_fwd(q, k, v, s, 700, n_sink=4))
    o, lse = rnd(T, 8, d), torch.full((T, 8), 9.0, device=dev)
    call("gradient %d" % d, lambda: ra.window_attn_bwd(do, q, k, v, o, lse, s, 700, n_sink=4))
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


@pytest.mark.parametrize("limit", [64, 900, 2500, 6000, 20000])
def test_waits_that_expire(unlimited, limit):
    from context_long_sequence_ring_gb300 import ringattn
    status, same, ok = run(limit, "compare", unlimited)
    assert ok
    for name, (st, msg) in status.items():
        assert st in (0, ringattn.RA_ERR_TIMEOUT), (name, st, msg)
        if limit == 64:
            assert st == ringattn.RA_ERR_TIMEOUT, (name, st, msg)
        if st == 0:
            assert same[name], name
        else:
            assert ("window attention gradient" if "gradient" in name else "window attention") in msg, (name, msg)


LONG = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
from context_long_sequence_ring_gb300 import ringattn as ra
dev = torch.device("cuda:0")
T = 16384
g = torch.Generator().manual_seed(1)
x, do = (torch.randn(T, h, 64, generator=g).to(torch.bfloat16).to(dev) for h in (48, 32))
s = torch.tensor([0, T], dtype=torch.int32, device=dev)
q, k, v = x[:, :32], x[:, 32:40], x[:, 40:]
o, lse = torch.zeros(T, 32, 64, dtype=torch.bfloat16, device=dev), torch.full((T, 32), 9.0, device=dev)
ra.window_attn_bwd(do, q, k, v, o, lse, s, 1 << 30)
print(ra.device_status(), ra.last_error())
"""


def test_a_limit_is_for_a_tile_and_not_for_an_item():
    """A key tile of the first tokens meets 512 query tiles, some 10^6 cycles; no wait for one of them takes 2 * 10^5."""
    env = dict(os.environ, RA_WAIT_LIMIT_CYCLES="200000")
    r = subprocess.run([sys.executable, "-c", LONG, ROOT], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.split()[0] == "0", r.stdout
