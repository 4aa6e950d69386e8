"""Calls by threads that have made no CUDA call before, one after another, and a process's first calls by several threads at the
same time, each with its stream, outputs and workspace."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = r"""
import sys, threading, torch
sys.path.insert(0, sys.argv[1])
from context_long_sequence_ring_gb300 import ringattn as ra
d, dev = 64, torch.device("cuda:0")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
g = torch.Generator().manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)
q, k, v, s, lse = rnd(40, 2, d), rnd(40, 1, d), rnd(40, 1, d), i32(0, 40), torch.full((40, 2), 5.0, device=dev)
kc, vc, table, ctx = rnd(1, 3, 1, 16, d), rnd(1, 3, 1, 16, d), i32(0, 1, 2).view(1, 3), i32(40)
Q, K, V = rnd(256, 2, d), rnd(256, 1, d), rnd(256, 1, d)
calls = {
    "forward": lambda w, o: ra.window_attn_fwd(q, k, v, s, 30, workspace=w, o=o[0], lse=o[1]),
    "gradient": lambda w, o: ra.window_attn_bwd(q, q, k, v, q, lse, s, 30, workspace=w, dq=o[0], dk=o[2], dv=o[3]),
    "window": lambda w, o: ra.cp_window_attn(q, kc, vc, table, s, ctx, 30, 16, 1, 1, workspace=w, o=o[0], lse=o[1]),
    "chunk": lambda w, o: ra.cp_chunk_attn(q, kc, vc, table, s, ctx, 16, 1, 1, workspace=w, o=o[0], lse=o[1]),
    "weights": lambda w, o: (ra.cp_attn_weights(q, lse, kc, table, s, ctx, 16, 1, 1, w_out=o[4]),),
    "prefill": lambda w, o: ra.ring_attn_fwd(Q, K, V, True, 1, o=o[5], lse=o[6]),
}
def space():
    f32 = dict(dtype=torch.float32, device=dev)
    like = torch.zeros_like
    return torch.empty(64 << 20, dtype=torch.uint8, device=dev), (like(q), torch.zeros((40, 2), **f32), like(k), like(v),
                                                                  torch.zeros((1, 3, 1, 16), **f32), like(Q),
                                                                  torch.zeros((256, 2), **f32))
def collect(results, i, f, w, o):
    try:
        results[i] = f(w, o)
    except Exception as e:
        results[i] = str(e)
def same(name, results, want):
    torch.cuda.synchronize()
    for r in results:
        assert not isinstance(r, str), (name, r)
        assert all(torch.equal(a, b) for a, b in zip(r, want)), name
    assert ra.device_status() == 0, ra.last_error()
"""

FRESH = SETUP + r"""
w, o = space()
torch.cuda.synchronize()
for name, f in calls.items():
    results = [None]
    t = threading.Thread(target=collect, args=(results, 0, f, w, o))
    t.start(); t.join(); torch.cuda.synchronize()
    results = [x if isinstance(x, str) else [y.clone() for y in x] for x in results]
    same(name, results, f(w, o))
"""

TOGETHER = SETUP + r"""
N = 12
streams, spaces, last = [torch.cuda.Stream() for _ in range(N)], [space() for _ in range(N)], space()
torch.cuda.synchronize()
for name, f in calls.items():
    gate, results = threading.Barrier(N), [None] * N
    def work(i):
        with torch.cuda.stream(streams[i]):
            torch.cuda.current_stream().synchronize()      # this thread has its context
            gate.wait()
            collect(results, i, f, *spaces[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
    for t in threads: t.start()
    for t in threads: t.join()
    torch.cuda.synchronize()
    results = [x if isinstance(x, str) else [y.clone() for y in x] for x in results]
    same(name, results, f(*last))
"""


def run(child):
    r = subprocess.run([sys.executable, "-c", child, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_thread_that_has_no_context():
    run(FRESH)


@pytest.mark.parametrize("process", range(4))
def test_several_threads_at_once(process):
    """What a library looks up once must be there for all of them."""
    run(TOGETHER)
