"""The chunk attention's work division on the host: the arithmetic that the kernel runs (ra_chunk_plan.cuh), walked over
every part of a batch.  Each tile of each item has to be taken exactly once, and no part may do much more than its share."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_long_sequence_ring_gb300", "csrc")

# Reads "d G Hkv causal R", then "n ctx" of each request; prints parts' largest work over the even share, the shift
# and whether all tiles were taken once.  Work: keys of the tiles at a key's cost, and the start and end of an item.
HARNESS = r"""
#include <cstdio>
#include <vector>
#include "ra_chunk_plan.cuh"
struct Request { Items it; int n, L; long long pos0; };
int main() {
  int d, G, Hkv, causal, R;
  while (scanf("%d %d %d %d %d", &d, &G, &Hkv, &causal, &R) == 5) {
    const Rates rt = rates_of(d);
    const int tpt = 128 / G;
    std::vector<Request> q(R);
    uint64_t sum = 0;
    uint32_t items = 0;
    for (auto& x : q) {
      scanf("%d %d", &x.n, &x.L);
      x.pos0 = static_cast<long long>(x.L) - x.n;
      x.it.set(rt, x.n, x.n > tpt ? (x.n + 2 * tpt - 1) / (2 * tpt) : (x.n > 0), tpt, x.pos0, x.L, causal != 0);
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
    if (p.shift == 0) ok = ok && scaled() == sum + items;
    p.divide(static_cast<uint32_t>(scaled()), rt);
    if (p.try_pieces(items, rt)) p.use_pieces(static_cast<uint32_t>(scaled()));
    std::vector<double> work(kCtas, 0.0);
    uint64_t at = 0;
    double all = 0;
    for (auto& x : q)
      for (int g = 0; g < Hkv; ++g)
        for (int k = 0; k < x.it.items; ++k) {
          const int per = (x.it.pair ? 2 : 1) * tpt;
          const int last = (k + 1) * per < x.n ? (k + 1) * per : x.n;
          long long see = causal ? x.pos0 + last : x.L;
          if (see < 0) see = 0;
          if (see > x.L) see = x.L;
          const int nt = static_cast<int>((see + 127) / 128);
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
            const double w = (t1 - t0) * 128.0 * (x.it.pair ? kPairCost : rt.f_split) + x.it.start;
            work[i] += w;
          }
          if (next != nt) ok = false;
          all += nt * 128.0 * (x.it.pair ? kPairCost : rt.f_split) + x.it.start;
          at += c;
        }
    if (p.piece <= 0.f && at != p.total) ok = false;
    double most = 0;
    for (double w : work) most = w > most ? w : most;
    printf("%.4f %d %d\n", most / (all / kCtas), p.shift, ok ? 1 : 0);
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

    def run(d, G, Hkv, causal, requests):
        text = "%d %d %d %d %d\n" % (d, G, Hkv, causal, len(requests)) + "".join("%d %d\n" % x for x in requests)
        out = subprocess.run([str(at / "plan")], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert out[2] == "1", "a tile was lost or taken twice"
        return float(out[0]), int(out[1])

    return run


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(8, 8), (4, 8), (16, 8), (64, 1), (1, 8), (16, 1)])
@pytest.mark.parametrize("n,ctx", [(16384, 16384), (65536, 65536), (131072, 131072), (262144, 262144), (65536, 1048576),
                                   (32768, 131072)])
def test_a_long_piece_is_divided_evenly(divide, d, G, Hkv, n, ctx):
    for causal in (1, 0):
        worst, shift = divide(d, G, Hkv, causal, [(n, ctx)])
        # whole tiles, and an item more or less: within a tenth of the share
        assert worst <= 1.1, (worst, shift)


@pytest.mark.parametrize("G,Hkv,prompt,singles,limit", [
    (16, 8, [(16384, 16384)], 255, 1.1), (16, 8, [(2048, 2048)] * 8, 56, 1.1), (8, 8, [(65536, 65536)], 64, 1.1),
    (16, 8, [(65536, 65536)], 255, 1.1)])
def test_a_prompt_among_single_tokens_is_divided_evenly(divide, G, Hkv, prompt, singles, limit):
    worst, shift = divide(128, G, Hkv, 1, prompt + [(1, 4096)] * singles)
    assert worst <= limit, (worst, shift)


def test_sums_past_the_unit_are_shifted(divide):
    assert divide(128, 4, 8, 1, [(4096, 32768)])[1] == 0
    assert divide(128, 8, 8, 1, [(65536, 65536)])[1] > 0
    assert divide(128, 8, 8, 0, [(262144, 1 << 24)] * 4)[1] > 8


def test_every_tile_is_taken_once(divide):
    """Random batches from one token to billions of keys, empty requests and contexts shorter than their queries."""
    rng = random.Random(5)
    for _ in range(150):
        G, Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16, 40, 64]), rng.choice([1, 2, 8])
        reqs = []
        for _ in range(rng.choice([1, 2, 7, 33, 200])):
            ctx = int(2 ** rng.uniform(0, rng.choice([8, 14, 20, 26])))
            n = rng.choice([0, 1, 1, rng.randint(1, 8), int(2 ** rng.uniform(0, 13))])
            reqs.append((n, ctx))
        divide(rng.choice([64, 128]), G, Hkv, rng.choice([0, 1]), reqs)
