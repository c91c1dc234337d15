"""The turns of accumulators in the experts' products on CTA pairs, run on the CPU
with the kernel's own arithmetic (csrc/fp8_experts_turns.h): releases that the odd
CTA sends to the even one's barriers take as long as they like, and none may be
under way when the pair's last barrier opens."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MODEL = r"""
#include <stdio.h>
#include <stdlib.h>
#include <functional>
#include <random>
#include <vector>
#include "fp8_experts_turns.h"
using namespace fp8q::experts;

// Barriers count phases; a parity wait for phase t passes where the phase of that
// parity that ended last is not the one before t: asked two phases early, it would.
struct Barrier {
  int need, got = 0;
  unsigned phase = 0;
  void arrive() { if (++got == need) got = 0, ++phase; }
  bool passes(unsigned t) const { return (phase & 1u) != (t & 1u); }   // as the hardware sees it
  bool fits(unsigned t) const { return phase == t || phase == t + 1; }
};

template <int ACC, int TEAMS, bool SETTLE>
bool run(unsigned tiles, unsigned seed, bool lazy) {
  constexpr int WARPS = 2, FULL = ACC * TEAMS;
  std::mt19937 rng(seed);
  std::vector<Barrier> full[2], empty(ACC, Barrier{2 * WARPS});
  for (auto &f : full) f.assign(FULL, Barrier{1});
  std::vector<int> flight;   // accumulators whose remote release is under way
  // the issuing warp, as a list of steps; each says whether it could be taken
  unsigned issued = 0;
  std::vector<std::pair<unsigned, unsigned>> last;
  bool listed = false;
  const auto issue = [&]() -> bool {
    if (issued < tiles) {
      const unsigned a = accumulator_of<ACC>(issued), t = turn_of<ACC>(issued);
      if (t > 0 && !empty[a].fits(t - 1)) printf("early wait\n"), exit(2);
      if (t > 0 && !empty[a].passes(t - 1)) return false;
      for (auto &f : full) f[issued % FULL].arrive();
      ++issued;
      return true;
    }
    if (!listed) {
      listed = true;
      if (SETTLE)
        settle<ACC>(tiles, [&](uint32_t a, uint32_t t) { last.push_back({a, t}); return true; });
      return true;
    }
    if (last.empty()) return false;
    const auto [a, t] = last.back();
    if (!empty[a].fits(t)) printf("early wait\n"), exit(2);
    if (!empty[a].passes(t)) return false;
    last.pop_back();
    return true;
  };
  struct Warp { int cta; unsigned j; };
  std::vector<Warp> warps;
  for (int c = 0; c < 2; ++c)
    for (int t = 0; t < TEAMS; ++t)
      for (int w = 0; w < WARPS; ++w) warps.push_back({c, (unsigned)t});
  const auto drain = [&](Warp &w) -> bool {
    if (w.j >= tiles) return false;
    const Barrier &f = full[w.cta][w.j % FULL];
    const unsigned t = w.j / FULL;
    if (!f.fits(t)) printf("early wait\n"), exit(2);
    if (!f.passes(t)) return false;
    const unsigned a = accumulator_of<ACC>(w.j);
    if (w.cta == 0) empty[a].arrive(); else flight.push_back((int)a);
    w.j += TEAMS;
    return true;
  };
  const auto land = [&] {
    if (flight.empty()) return false;
    const size_t k = rng() % flight.size();
    empty[flight[k]].arrive();
    flight.erase(flight.begin() + (long)k);
    return true;
  };
  while (true) {
    bool all = issued == tiles && listed && last.empty();
    for (auto &w : warps) all = all && w.j >= tiles;
    if (all) return flight.empty();   // the pair's last barrier opens
    bool moved = false;
    const size_t n = warps.size() + 1, from = rng() % n;
    for (size_t i = 0; i < n && !moved; ++i) {
      const size_t k = (from + i) % n;
      moved = k == warps.size() ? issue() : drain(warps[k]);
    }
    if ((!moved || (!lazy && rng() % 4 == 0)) && land()) moved = true;
    if (!moved) printf("stuck\n"), exit(3);
  }
}

template <int ACC, int TEAMS, bool SETTLE>
int left_behind() {
  int bad = 0;
  for (unsigned tiles = 0; tiles < 14; ++tiles)
    for (unsigned seed = 0; seed < 40; ++seed)
      for (int lazy = 0; lazy < 2; ++lazy) bad += !run<ACC, TEAMS, SETTLE>(tiles, seed, lazy != 0);
  return bad;
}

int main() {
  printf("%d %d %d\n", left_behind<1, 1, true>(), left_behind<3, 2, true>(), left_behind<2, 1, true>());
  printf("%d %d\n", left_behind<1, 1, false>(), left_behind<3, 2, false>());
  return 0;
}
"""


@pytest.fixture(scope="module")
def ran(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    src, exe = d / "turns.cpp", d / "turns"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I",
                    os.path.join(ROOT, "scaled_quantize_fp8_warp_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    return [list(map(int, line.split())) for line in r.stdout.splitlines()]


def test_no_release_is_under_way_at_the_end(ran):
    assert ran[0] == [0, 0, 0]


def test_the_model_sees_releases_nobody_waits_for(ran):
    """Without the issuing warp's last waits, which a relaxed barrier does not stand in for."""
    assert all(n > 0 for n in ran[1])
