"""How a cluster's producers end after a wait that ran out (csrc/cluster_drain.cuh), on the host: the header's own step is run
against a model of the barriers.  Every CTA of a pair, or of two pairs that multicast to each other, has asked for a number of
fills of its own; the copies land in any order, before, between and after the steps.  Each barrier's phase has to end, and no
sooner than the last copy that was asked for has landed."""
import pathlib
import shutil
import subprocess

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "transformer_fwd_bwd_gb300" / "csrc"

MODEL = r"""
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>
#include "cluster_drain.cuh"
using xt::gemm::DrainStep;
using xt::gemm::drain_step;

struct Bar {  // an mbarrier: arrivals and bytes that its phase still lacks
  int count, pending, phase = 0;
  long tx = 0;
  explicit Bar(int c) : count(c), pending(c) {}
  void check() { if (pending == 0 && tx == 0) { ++phase; pending = count; } }
  void arrive() { --pending; check(); }
  void expect(long b) { tx += b; arrive(); }
  void land(long b) { tx -= b; check(); }
};
struct Copy { int fill; long bytes; };
std::mt19937 rng(1);
int draw(int lo, int hi) { return lo + int(rng() % unsigned(hi - lo + 1)); }

// CTA `self`'s barriers, one for each of the last fills; old: only its own fills are waited for.  Returns false where a phase
// ended early, never ended, or (old) a copy was left behind.
template <int CL>
bool drains(int self, const int (&issued)[CL], const uint32_t (&bytes)[CL], int base, int relayed, bool relay, bool old) {
  int most = *std::max_element(issued, issued + CL);
  bool good = true;
  for (int f = most - 1; f >= base; --f) {
    Bar bar(relay ? 2 : 1);
    uint32_t want = 0;
    for (uint32_t b : bytes) want += b;
    std::vector<Copy> copies;
    for (int c = 0; c < CL; ++c)
      if (issued[c] > f && bytes[c]) copies.push_back({f, long(bytes[c])});
    std::shuffle(copies.begin(), copies.end(), rng);
    size_t early = copies.empty() ? 0 : size_t(draw(0, int(copies.size()))), next = 0;
    const bool announced = issued[self] > f;
    const size_t before = size_t(draw(0, int(early)));
    while (next < before) bar.land(copies[next++].bytes);  // before the announcement
    if (announced) bar.expect(want);
    if (relay && relayed > f) bar.arrive();
    while (next < early) bar.land(copies[next++].bytes);
    if (old) {
      if (!announced && !copies.empty()) good = false;      // nobody waits for them
      if (announced) {
        while (next < copies.size()) bar.land(copies[next++].bytes);
        if (bar.phase != 1) good = false;
      }
      continue;
    }
    const DrainStep d = drain_step<CL>(f, issued, self, bytes);
    if (d.wait != !copies.empty()) good = false;
    if (!d.wait) continue;
    if (d.complete) bar.land(d.complete);
    if (d.expect) bar.expect(d.expect);
    if (relay && relayed <= f) bar.arrive();
    while (next < copies.size()) {
      if (bar.phase != 0) good = false;
      bar.land(copies[next++].bytes);
    }
    if (bar.phase != 1 || bar.tx != 0) good = false;
  }
  return good;
}

int main(int argc, char**) {
  const bool old = argc > 1;
  int bad = 0;
  for (int i = 0; i < 200000; ++i) {
    const int stages = draw(2, 8), base = draw(0, 20);
    {  // a pair: the even CTA's barriers count both CTAs' stages
      const int n[2] = {base + draw(0, stages), base + draw(0, stages)};
      const uint32_t b[2] = {65536, 65536};
      bad += !drains<2>(0, n, b, base, 0, false, old);
    }
    {  // two pairs: B's rows come in halves from both, the odd CTA's stages are passed on to the even one
      int n[4];
      for (int& v : n) v = base + draw(0, stages);
      for (int self = 0; self < 4; ++self) {
        const int rank = self & 1, pair = self >> 1;
        uint32_t b[4];
        for (int c = 0; c < 4; ++c) b[c] = (rank == 0 && (c >> 1) == pair ? 32768u : 0u) + ((c & 1) == rank ? 16384u : 0u);
        const int relayed = base + draw(0, std::max(0, std::min(n[1], n[3]) - base));
        bad += !drains<4>(self, n, b, base, relayed, rank == 0, old);
      }
    }
  }
  std::printf("%d\n", bad);
  return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("drain")
    (d / "model.cpp").write_text(MODEL)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", str(CSRC), "-o", str(d / "model"), str(d / "model.cpp")], check=True)
    return str(d / "model")


def test_every_copy_is_waited_for_and_every_phase_ends(model):
    assert int(subprocess.run([model], capture_output=True, text=True, check=True).stdout) == 0


def test_the_model_sees_copies_that_only_their_own_cta_asked_for(model):
    """Waiting for the own fills alone: copies of a CTA that went further are left, announced bytes never come."""
    assert int(subprocess.run([model, "own"], capture_output=True, text=True, check=True).stdout) > 0
