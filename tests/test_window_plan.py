"""The window attention's work division on the host: the arithmetic that the kernel runs (ra_chunk_plan.cuh), walked over
every part of a batch.  Each tile of each item has to be taken exactly once, and no part may do much more than its share."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_long_sequence_ring_gb300", "csrc")

# Reads "d G Hkv window n_sink R", then "n ctx" of each request; prints the parts' largest work over the even share and
# whether all tiles were taken once.  An item's tiles are cut out of its row of 32-token units: those of first tokens that end
# before its window, and those from the first that its first row sees to the last that its last row sees.
HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#include "ra_chunk_plan.cuh"
struct Request { WindowItems it; int n, L; long long pos0; };
int main() {
  int d, G, Hkv, window, n_sink, R;
  while (scanf("%d %d %d %d %d %d", &d, &G, &Hkv, &window, &n_sink, &R) == 6) {
    const Rates rt = rates_of(d);
    const int tpt = 128 / G;
    std::vector<Request> q(R);
    uint64_t sum = 0;
    uint32_t items = 0;
    for (auto& x : q) {
      scanf("%d %d", &x.n, &x.L);
      x.pos0 = static_cast<long long>(x.L) - x.n;
      x.it.set(rt, x.n, x.n > tpt ? (x.n + 2 * tpt - 1) / (2 * tpt) : (x.n > 0), tpt, x.pos0, x.L, window, n_sink);
      sum += Hkv * x.it.upto(x.it.items);
      items += Hkv * x.it.items;
    }
    Plan p;
    p.scale(sum);
    auto scaled = [&] {
      uint64_t t = 0;
      for (auto& x : q) t += static_cast<uint64_t>(Hkv) * p.prefix(x.it, x.it.items);
      return t;
    };
    bool ok = scaled() < (1ull << 32);
    p.divide(static_cast<uint32_t>(scaled()), rt);
    if (p.try_pieces(items, rt)) p.use_pieces(static_cast<uint32_t>(scaled()));
    std::vector<double> work(kCtas, 0.0);
    uint64_t at = 0;
    double all = 0;
    for (auto& x : q)
      for (int g = 0; g < Hkv; ++g)
        for (int k = 0; k < x.it.items; ++k) {
          const long long per = (x.it.pair ? 2 : 1) * tpt;
          const long long first = x.pos0 + k * per, end = std::min<long long>(x.pos0 + std::min<long long>((k + 1) * per, x.n), x.L);
          const long long from = std::max(0ll, first + 1 - window) / 32;
          const long long units = std::max(0ll, (end + 31) / 32 - from) + std::min((n_sink + 31ll) / 32, from);
          const int nt = static_cast<int>((units + 3) / 4);
          const uint32_t c = p.cost(x.it, k);
          if (c <= p.over(x.it)) ok = false;
          int next = 0;
          int c0 = static_cast<int>(at / p.share);
          for (int i = c0 > 0 ? c0 - 1 : 0; i < kCtas && p.lo(i) < at + c; ++i) {
            int t0, t1;
            if (p.lo(i + 1) <= at) continue;
            cut(p.lo(i), p.lo(i + 1), static_cast<uint32_t>(at), p.over(x.it), c, nt, t0, t1);
            if (t1 <= t0) continue;
            if (t0 != next) ok = false;
            next = t1;
            work[i] += (t1 - t0) * 128.0 * (x.it.pair ? kPairCost : rt.f_split) + x.it.start;
          }
          if (next != nt) ok = false;
          all += nt * 128.0 * (x.it.pair ? kPairCost : rt.f_split) + x.it.start;
          at += c;
        }
    if (p.piece <= 0.f && at != p.total) ok = false;
    double most = 0;
    for (double w : work) most = w > most ? w : most;
    printf("%.4f %d\n", most / (all / kCtas), ok ? 1 : 0);
  }
}
"""


@pytest.fixture(scope="module")
def divide(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "a host compiler is required"
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(HARNESS)
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wno-unknown-pragmas", "-I", CSRC, "-o", str(at / "plan"), str(at / "plan.cpp")],
                   check=True)

    def run(d, G, Hkv, window, n_sink, requests):
        text = "%d %d %d %d %d %d\n" % (d, G, Hkv, window, n_sink, len(requests)) + "".join("%d %d\n" % x for x in requests)
        out = subprocess.run([str(at / "plan")], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert out[1] == "1", "a tile was lost or taken twice"
        return float(out[0])

    return run


# A part of 16384 tokens and more is at least 13 items of 6 tiles (and 4 for their start and end): a tile and a start more or
# less at either end are within 15 % of it (2 of 13 items).
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(4, 8), (8, 8), (16, 8)])
@pytest.mark.parametrize("n,ctx", [(16384, 16384), (32768, 131072), (262144, 262144)])
@pytest.mark.parametrize("window,n_sink", [(512, 4), (4096, 0), (4096, 1000), (1 << 30, 0)])
def test_a_long_piece_is_divided_evenly(divide, d, G, Hkv, n, ctx, window, n_sink):
    worst = divide(d, G, Hkv, window, n_sink, [(n, ctx)])
    assert worst <= 1.15, worst


def test_every_tile_is_taken_once(divide):
    """Random batches: windows of one token and longer than any context, first tokens past the window's start, empty
    requests and contexts shorter than their queries."""
    rng = random.Random(6)
    for _ in range(200):
        G, Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16, 40, 64]), rng.choice([1, 2, 8])
        reqs = []
        for _ in range(rng.choice([1, 2, 7, 33, 200])):
            ctx = int(2 ** rng.uniform(0, rng.choice([8, 14, 20, 26])))
            n = rng.choice([0, 1, 1, rng.randint(1, 8), int(2 ** rng.uniform(0, 13))])
            reqs.append((n, ctx))
        window = rng.choice([1, 2, 100, 128, 1000, 4096, 1 << 20, 1 << 30])
        n_sink = rng.choice([0, 1, 4, 31, 32, 500, 1 << 20, 1 << 30])
        divide(rng.choice([64, 128]), G, Hkv, window, n_sink, reqs)
