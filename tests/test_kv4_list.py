"""How attention over the 4-bit KV cache cuts its list of steps and where the parts of a cut item meet, on the CPU: the
kernels' own arithmetic (csrc/kv4_list.cuh, compiled for the host), walked through by CTAs that arrive in any order."""
import ctypes
import os
import random
import subprocess

import pytest

from fp8_w8a8_quantized_amax_b200 import build as fbuild

WALK = r"""
#include <map>
#include <utility>
#include <vector>
#include "kv4_list.cuh"
using namespace fp8q::kv4;

namespace {
struct Cut { int item, part; };
struct Cta {
  std::vector<Cut> cuts;                  // its parts of cut items, in order
  size_t at = 0;
  bool arrived = false;                   // the last to arrive: its store of zero and its join come next
  few::Meeting meet = {};
};
}  // namespace

// 0; 1: two meetings with one counter; 2: a join of a part that is not there; 3: an item that is not joined; 4: a counter
// that is not zero at the end; 5: a counter outside the header.  `lone` plants a mistake: a group of one part counts at
// its CTA's counter of the first level, as the others do.
extern "C" int walk(const int64_t* steps, int items, int ctas, int lone, unsigned seed) {
  int64_t total = 0;
  for (int i = 0; i < items; ++i) total += steps[i] + few::kOver;
  const Range range = {total / ctas, total % ctas};
  std::vector<Cta> all(ctas);
  std::vector<few::Joins> joins(items);
  std::vector<std::vector<int>> have(items);                    // parts that the result in a part's place holds
  std::map<int, std::pair<int, int>> meetings;                  // counter -> (item, level and first part)
  auto first = [&](int i, int cta) {
    few::Meeting m = joins[i].first(cta);
    const int from = (cta - joins[i].c0) / few::kJoin * few::kJoin;
    if (lone && m.final && joins[i].parts > few::kJoin) m = {from, 1, 1, joins[i].c0 + from, false};
    return m;
  };
  int64_t s = 0;
  int open = 0, shared = 0;
  for (int i = 0; i < items; ++i) {
    const int64_t i0 = s + few::kOver, i1 = i0 + steps[i];
    s = i1;
    const int c0 = range.owner(i0), c1 = range.owner(i1 - 1);
    joins[i] = {c0, c1 - c0 + 1};
    if (c0 == c1) continue;
    ++open;
    have[i].assign(c1 - c0 + 1, 0);
    for (int c = c0; c <= c1; ++c) {
      if (range.begin(c) >= i1 || range.begin(c + 1) <= i0) return 2;
      all[c].cuts.push_back({i, c - c0});
      few::Meeting m[2] = {first(i, c), joins[i].second()};
      for (int l = 0; l < (m[0].final ? 1 : 2); ++l) {
        if (m[l].counter < 0 || m[l].counter >= 2 * kMaxCtas) return 5;
        const std::pair<int, int> id = {i, m[l].final ? -1 : m[l].from};
        const auto was = meetings.emplace(m[l].counter, id).first->second;
        if (was != id) shared = 1;
      }
    }
  }
  if (shared && !lone) return 1;
  std::vector<int> count(2 * kMaxCtas, 0), busy;
  for (int c = 0; c < ctas; ++c)
    if (!all[c].cuts.empty()) busy.push_back(c);
  unsigned long long rng = seed * 2862933555777941757ull + 3037000493ull;
  while (!busy.empty()) {                                       // any CTA that has something left goes one step further
    rng = rng * 6364136223846793005ull + 1442695040888963407ull;
    const size_t pick = (rng >> 33) % busy.size();
    const int c = busy[pick];
    Cta& x = all[c];
    const Cut cut = x.cuts[x.at];
    bool next = false;
    if (!x.arrived) {
      if (have[cut.item][cut.part] == 0) {
        have[cut.item][cut.part] = 1;
        x.meet = first(cut.item, c);
      }
      if (count[x.meet.counter]++ == x.meet.n - 1) x.arrived = true;
      else next = true;
    } else {
      x.arrived = false;
      count[x.meet.counter] = 0;
      int sum = 0;
      for (int k = 0; k < x.meet.n; ++k) {
        const int there = have[cut.item][x.meet.from + k * x.meet.stride];
        if (there == 0) return 2;
        sum += there;
      }
      if (x.meet.final) {
        if (sum != joins[cut.item].parts) return 2;
        --open;
        next = true;
      } else {
        have[cut.item][x.meet.from] = sum;
        x.meet = joins[cut.item].second();
      }
    }
    if (next && ++x.at == x.cuts.size()) {
      busy[pick] = busy.back();
      busy.pop_back();
    }
  }
  if (open) return 3;
  for (int v : count)
    if (v) return 4;
  return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    at = tmp_path_factory.mktemp("kv4_list")
    src, so = at / "walk.cpp", at / "walk.so"
    src.write_text(WALK)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-x", "c++", str(src), "-I",
                    fbuild.CSRC, "-o", str(so)], check=True, capture_output=True, text=True)
    f = ctypes.CDLL(str(so)).walk
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_uint]

    def go(steps, ctas, lone=False, seed=1):
        a = (ctypes.c_int64 * len(steps))(*steps)
        return f(ctypes.addressof(a), len(steps), ctas, int(lone), seed)

    return go


def steps_of(lens, heads, tiles=1):
    """The items' steps of 128 keys: `heads` items (times the row tiles) a sequence."""
    return [max(1, (n + 127) // 128) for n in lens for _ in range(heads * tiles)]


# tokens of 8 key heads on 148 SMs with four CTAs each, but for the last two: equal contexts, and seven key heads
SHARED = [([91885, 182], 8, 592), ([32000, 1000, 16384, 100000], 8, 592), ([65536, 1000, 16000, 65536], 8, 592),
          ([16384] * 4, 8, 592), ([131072] * 5, 7, 592)]


@pytest.mark.parametrize("lens,heads,ctas", SHARED)
def test_a_group_of_one_part_meets_no_other_item(walk, lens, heads, ctas):
    steps = steps_of(lens, heads)
    for seed in range(200):
        assert walk(steps, ctas, seed=seed) == 0
    # what the walk is there to find: the lone part counted in its CTA, where the next item's first group counts
    assert any(walk(steps, ctas, lone=True, seed=seed) for seed in range(200))


def test_no_two_meetings_share_a_counter(walk):
    rng = random.Random(0)
    for i in range(3000):
        heads = rng.choice([1, 2, 3, 4, 7, 8, 8, 8, 18])
        lens = [int(2 ** rng.uniform(0, 17)) for _ in range(rng.randint(1, 16))]
        if rng.random() < 0.2:
            lens = [lens[0]] * len(lens)
        ctas = rng.choice([148, 132, 64, 7, 3]) * rng.choice([3, 4, 5])
        steps = steps_of(lens, heads, rng.choice([1, 1, 2, 5]))
        ctas = min(ctas, sum(steps) + len(steps), 1024)
        for seed in range(3):
            assert walk(steps, ctas, seed=3 * i + seed) == 0, (lens, heads, ctas)


def test_one_item_over_every_number_of_ctas(walk):
    for ctas in range(2, 1025):
        assert walk([5000], ctas, seed=ctas) == 0
