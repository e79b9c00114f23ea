"""The waits between the warps of the attention of drafted tokens over an e4m3 cache, on the host.

The roles of one thread block as they stand in csrc/fat_tree_kernel.cuh (producers of the codes and
their copies, two teams of converters for K and for V, the MMA issuer, two groups of softmax warps),
each a list of waits and arrivals on barriers that count phases; a wait ends where the barrier's
last completed phase has the parity asked for.  Which barrier the queries of an item complete, and
who waits for it, is csrc/fat_tree_sync.h.  Whatever order the roles run in, each late or early in
turn and in random orders, all of them come to their ends, and the keys are converted for the
queries of their own item.
"""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensorized_online_softmax_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "fat_tree_sync.h"
using namespace fat;

enum Kind { kWait, kArrive, kSet, kCheck };
struct Op { Kind kind; int at; unsigned parity; };  // at: a barrier, or (set, check) an item
struct Bar { int expected, pending; unsigned done; };

struct Block {
  std::vector<Bar> bars;
  std::vector<std::vector<Op>> roles;
  int bar(int arrivals) { bars.push_back({arrivals, arrivals, 0}); return (int)bars.size() - 1; }
  std::vector<int> ring(int n, int arrivals) {
    std::vector<int> r;
    for (int i = 0; i < n; ++i) r.push_back(bar(arrivals));
    return r;
  }
  std::vector<Op>& role() { roles.emplace_back(); return roles.back(); }
};
void wait(std::vector<Op>& r, int bar, unsigned parity) { r.push_back({kWait, bar, parity & 1u}); }
void arrive(std::vector<Op>& r, int bar) { r.push_back({kArrive, bar, 0}); }

// items: tiles of each.  rule 0: fat_tree_sync.h; 1: one barrier for the queries of all items, its
// phases waited for one by one (a rule that stops, to see that the walk would find it).
Block make(const std::vector<int>& items, int raw, int rule) {
  Block b;
  b.roles.reserve(64);
  std::vector<int> item_of;
  for (int j = 0; j < (int)items.size(); ++j)
    for (int x = 0; x < items[j]; ++x) item_of.push_back(j);
  const int N = (int)item_of.size(), kWarps = 2;  // (of a team)
  const auto issued = b.ring(raw, 1), raw_full = b.ring(raw, 1), raw_empty = b.ring(raw, kWarps);
  const auto k_full = b.ring(2, kWarps), k_empty = b.ring(2, 1), v_full = b.ring(2, kWarps),
             v_empty = b.ring(2, 1), s_full = b.ring(2, 1), p_full = b.ring(2, 1),
             pv = b.ring(2, 1), v_type = b.ring(4, 1);
  const auto q_full = b.ring(kTreeQueryBars, 2);
  const int sync = b.bar(2);
  auto q_bar = [&](int j) { return q_full[rule == 0 ? tree_query_bar(j) : 0]; };
  auto q_parity = [&](int j) { return rule == 0 ? tree_query_parity(j) : j & 1u; };
  for (int is_v = 0; is_v < 2; ++is_v) {
    auto& producer = b.role();
    auto& copies = b.role();
    for (int n = 0; n < N + 2; ++n) {  // (the last two: there is no more)
      const int slot = (2 * n + is_v) % raw, phase = (2 * n + is_v) / raw;
      wait(producer, raw_empty[slot], (phase & 1u) ^ 1u);
      arrive(producer, issued[slot]);
      wait(copies, issued[slot], phase);
      arrive(copies, raw_full[slot]);
    }
    for (int team = 0; team < 2; ++team)
      for (int w = 0; w < kWarps; ++w) {
        auto& r = b.role();
        int seen = 0;  // items, the tile's own counted
        int n = team;
        for (; n < N; n += 2) {
          const int slot = (2 * n + is_v) % raw, phase = (2 * n + is_v) / raw, j = item_of[n];
          wait(r, raw_full[slot], phase);
          if (!is_v) {
            if (rule == 0 && seen != j + 1) wait(r, q_bar(j), q_parity(j));
            if (rule == 1) for (int x = seen; x <= j; ++x) wait(r, q_bar(x), q_parity(x));
            seen = j + 1;
            r.push_back({kCheck, j, 0});
          } else if (w == 0) {
            arrive(r, v_type[n % 4]);
          }
          wait(r, (is_v ? v_empty : k_empty)[team], (n / 2 & 1u) ^ 1u);
          if (!is_v) r.push_back({kCheck, j, 0});
          arrive(r, (is_v ? v_full : k_full)[team]);
          arrive(r, raw_empty[slot]);
        }
        wait(r, raw_full[(2 * n + is_v) % raw], (2 * n + is_v) / raw);
      }
  }
  auto& issuer = b.role();
  {
    int k = 0, v = 0;
    unsigned p_phase[2] = {0, 0};
    auto scores = [&](int g) {
      wait(issuer, k_full[k % 2], k / 2);
      arrive(issuer, s_full[g]);
      arrive(issuer, k_empty[k++ % 2]);
    };
    for (int j = 0; j < (int)items.size(); ++j) {
      const int tiles = items[j];
      wait(issuer, q_bar(j), q_parity(j));
      issuer.push_back({kCheck, j, 0});
      scores(0);
      if (tiles > 1) scores(1);
      for (int u = 0; u < tiles; ++u) {
        const int g = u & 1;
        wait(issuer, v_full[v % 2], v / 2);
        wait(issuer, p_full[g], p_phase[g]++);
        arrive(issuer, pv[g]);
        arrive(issuer, v_empty[v++ % 2]);
        if (u + 2 < tiles) scores(g);
      }
    }
  }
  for (int g = 0; g < 2; ++g) {
    auto& r = b.role();
    unsigned syncs = 0, phase = 0;
    int tile = 0;
    auto all = [&]() { arrive(r, sync); wait(r, sync, syncs++); };
    all();
    for (int j = 0; j < (int)items.size(); ++j) {
      all();  // (the queries' magnitudes)
      if (g == 0) r.push_back({kSet, j, 0});
      arrive(r, q_bar(j));
      int mine = 0;
      for (int x = 0; x < items[j]; ++x, ++tile) {
        if ((x & 1) != g) continue;
        wait(r, s_full[g], phase);
        if (mine) wait(r, pv[g], phase ^ 1u);
        wait(r, v_type[tile % 4], tile / 4);
        wait(r, v_full[tile % 2], tile / 2);
        arrive(r, p_full[g]);
        ++phase, ++mine;
      }
      if (mine) wait(r, pv[g], phase ^ 1u);
      all();
      all();  // (the copies of a row)
      if (j + 1 < (int)items.size()) all();
    }
  }
  return b;
}

// Runs to the end or until nothing can run.  pick: which of the roles that can run is next.
template <typename F>
int run(Block b, F&& pick) {
  std::vector<size_t> at(b.roles.size(), 0);
  int type = -1;
  for (;;) {
    std::vector<int> can;
    bool all = true;
    for (int i = 0; i < (int)b.roles.size(); ++i) {
      if (at[i] == b.roles[i].size()) continue;
      all = false;
      const Op& o = b.roles[i][at[i]];
      if (o.kind != kWait || (b.bars[o.at].done & 1u) != o.parity) can.push_back(i);
    }
    if (all) return 0;
    if (can.empty()) return 1;  // stopped
    const int i = pick(can);
    const Op& o = b.roles[i][at[i]++];
    if (o.kind == kArrive) {
      Bar& x = b.bars[o.at];
      if (--x.pending == 0) x.pending = x.expected, ++x.done;
    } else if (o.kind == kSet) {
      type = o.at;
    } else if (o.kind == kCheck && type != o.at) {
      return 2;  // another item's queries
    }
  }
}

// stdin: rule raw, then lines of items: count tiles...; out: runs that stop, and that mix items up
int main() {
  int rule, raw, n, runs = 0, bad[3] = {0, 0, 0};
  if (std::scanf("%d %d", &rule, &raw) != 2) return 1;
  std::mt19937 rng(5);
  while (std::scanf("%d", &n) == 1) {
    std::vector<int> items(n);
    for (int& x : items) if (std::scanf("%d", &x) != 1) return 1;
    const Block b = make(items, raw, rule);
    const int R = (int)b.roles.size();
    auto any = [&](const std::vector<int>& can) { return can[rng() % can.size()]; };
    for (int a = 0; a < R; ++a)
      for (int c = a; c < R; ++c) {  // both only when nothing else can run
        ++runs, ++bad[run(b, [&](const std::vector<int>& can) {
          std::vector<int> others;
          for (int x : can) if (x != a && x != c) others.push_back(x);
          return any(others.empty() ? can : others);
        })];
        ++runs, ++bad[run(b, [&](const std::vector<int>& can) {  // both whenever they can
          for (int x : can) if (x == a || x == c) return x;
          return any(can);
        })];
      }
    for (int x = 0; x < 200; ++x) ++runs, ++bad[run(b, any)];
  }
  std::printf("%d %d %d\n", runs, bad[1], bad[2]);
  return 0;
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("sync")
    src, exe = d / "sync.cc", d / "sync"
    src.write_text(HARNESS)
    subprocess.run([cxx, "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def walk(rule, raw, lists):
        text = f"{rule} {raw}\n" + "\n".join(f"{len(x)} " + " ".join(map(str, x)) for x in lists)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=300)
        assert out.returncode == 0, out.stdout + out.stderr
        return tuple(map(int, out.stdout.split()))
    return walk


def item_lists(seed, count):
    rng = random.Random(seed)
    out = [[1] * 12, [2] * 6, [1, 2] * 5, [2, 1] * 5, [1, 1, 3] * 4, [3, 1, 1] * 4, [1], [2], [7]]
    return out + [[rng.choice([1, 1, 1, 2, 3, 4]) for _ in range(rng.randint(1, 14))]
                  for _ in range(count)]


@pytest.mark.parametrize("raw", [4, 12])
def test_every_role_ends_and_no_item_takes_another_ones_queries(harness, raw):
    runs, stopped, mixed = harness(0, raw, item_lists(raw, 6))
    assert runs > 1000 and stopped == 0 and mixed == 0


def test_the_walk_finds_a_rule_that_stops(harness):
    """One barrier whose phases a team steps through one by one: with items of one tile it stops,
    with longer ones it does not."""
    assert harness(1, 12, [[1] * 12])[1] > 0
    assert harness(1, 12, [[2] * 6, [3, 2, 4]])[1:] == (0, 0)


LAYOUTS = r"""
#include <cstdio>
#include "fat_tree_kernel.cuh"
using namespace fat;
using namespace fat::tree;
template <int D, int kType, int kNB>
int check() {
  using L = Layout<D, kType, kNB>;
  // in order, each behind the end of the one ahead of it
  const int at[] = {L::kQ, L::kK, L::kV, L::kRaw, L::kScales, L::kInfo, L::kBars, L::kMisc, L::kFin,
                    L::kStart, L::kBytes};
  const int size[] = {L::kQBufs * kNB * L::kTile, L::kKStages * L::kTile, L::kStages * L::kTile,
                      L::kRawStages * L::kRawTile, L::kRawStages * kTreeTile, L::kRawStages * 8,
                      8 * L::kNumBars, 96, 4 * kTreeBlockRows * 4,
                      static_cast<int>(sizeof(DecodePlace)), 0};
  for (int i = 0; i < 10; ++i)
    if (at[i] + size[i] > at[i + 1]) return 1;
  return L::kBytes > 227 * 1024;
}
int main() {
  int bad = check<64, kBf16, 1>() + check<64, kBf16, 2>() + check<64, kE4M3Bf16, 1>() +
            check<128, kBf16, 1>() + check<128, kBf16, 2>() + check<128, kE4M3Bf16, 1>();
  std::printf("%d\n", bad);
  return 0;
}
"""


def test_what_the_roles_share_lies_apart(tmp_path):
    """The place where a block's share starts, which a late role may read when others are at work,
    is nobody else's."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "layouts.cu", tmp_path / "layouts"
    src.write_text(LAYOUTS)
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", CSRC,
                    "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout == "0\n", out.stdout + out.stderr
