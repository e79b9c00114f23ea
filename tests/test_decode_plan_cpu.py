"""The decode kernel's division of work (csrc/fat_decode_plan.h), built for the host.

A copy of the kernel's walk, in plain loops, over many tables of lengths: every
tile of every item is taken by exactly one block; a block leaves at most one
unfinished item in each of its two parts; the items left to be joined are
exactly those that no block has whole, and the block and part numbers that the
join reads are the ones that were written, in order.
"""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensorized_online_softmax_gb300", "csrc")

HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <tuple>
#include <vector>
#include "fat_decode_plan.h"
using namespace fat;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

// stdin, repeated: copies blocks least entries len...
int main() {
  int copies, blocks, least, entries, cases = 0;
  while (std::scanf("%d %d %d %d", &copies, &blocks, &least, &entries) == 4) {
    std::vector<int> len(entries);
    for (int& n : len) if (std::scanf("%d", &n) != 1) return 1;
    long long total = 0;
    for (int n : len) total += static_cast<long long>(decode_tiles(n)) * copies;
    const long long share = decode_share(total, blocks, least);
    CHECK(share * blocks >= total && share >= least);
    typedef std::tuple<int, int> Item;
    std::map<Item, std::vector<int>> taken;            // tiles in the order of the blocks
    std::map<Item, std::vector<std::pair<int, int>>> left;   // (block, part) written
    std::map<Item, std::tuple<int, int, int>> joins;   // first block, its part, last block
    std::set<Item> whole;
    for (int b = 0; b < blocks; ++b) {
      const long long begin = b * share;
      if (begin >= total) continue;
      const long long end = std::min(total, begin + share);
      DecodePlace p{};
      long long before = 0;
      for (int e = 0; e < entries; ++e) {
        const long long n = static_cast<long long>(decode_tiles(len[e])) * copies;
        if (begin < before + n) { p = decode_place(e, begin - before, decode_tiles(len[e])); break; }
        before += n;
      }
      long long first = begin - p.tile;
      std::set<int> parts;
      const int count = static_cast<int>(end - begin);
      for (int i = 0; i < count; ++i) {
        CHECK(p.entry < entries && p.item < copies && p.tile < p.tiles);
        CHECK(p.tiles == decode_tiles(len[p.entry]));
        const Item item{p.entry, p.item};
        taken[item].push_back(p.tile);
        const bool done = p.tile == p.tiles - 1;
        if (done || i == count - 1) {
          if (done && first >= begin) {
            whole.insert(item);
          } else {
            const int part = decode_part(first, begin);
            CHECK(parts.insert(part).second);
            left[item].push_back({b, part});
            if (!done && first >= begin)
              joins[item] = {b, part, static_cast<int>((first + p.tiles - 1) / share)};
          }
          first = begin + i + 1;
        }
        if (i + 1 < count && decode_advance(p, copies)) p.tiles = decode_tiles(len[p.entry]);
      }
    }
    for (int e = 0; e < entries; ++e)
      for (int m = 0; m < copies; ++m) {
        const auto& t = taken[Item{e, m}];
        CHECK(static_cast<int>(t.size()) == decode_tiles(len[e]));
        for (int i = 0; i < static_cast<int>(t.size()); ++i) CHECK(t[i] == i);
        const bool w = whole.count(Item{e, m}) != 0;
        CHECK(w != (joins.count(Item{e, m}) != 0));
        if (w) { CHECK(left.count(Item{e, m}) == 0); continue; }
        const auto j = joins[Item{e, m}];
        const auto& l = left[Item{e, m}];
        CHECK(static_cast<int>(l.size()) == std::get<2>(j) - std::get<0>(j) + 1);
        for (int c = std::get<0>(j); c <= std::get<2>(j); ++c) {
          CHECK(c < blocks);
          CHECK(l[c - std::get<0>(j)].first == c);
          CHECK(l[c - std::get<0>(j)].second == (c == std::get<0>(j) ? std::get<1>(j) : 0));
        }
      }
    ++cases;
  }
  std::printf("ok %d\n", cases);
  return 0;
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cc", d / "plan"
    src.write_text(HARNESS)
    subprocess.run([cxx, "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return str(exe)


def test_every_tile_goes_to_one_block_and_every_part_is_joined(harness):
    rng = random.Random(5)
    cases = [(1, 1, 1, [0]), (8, 304, 2, [200]), (8, 304, 2, [131072]), (20, 304, 2, [0] * 13),
             (1, 304, 1, [5] * 700), (2, 512, 4, [2 ** 31 - 1, 0, 2 ** 20])]
    for _ in range(400):
        entries = rng.choice([1, 2, 3, 17, 129, 400])
        top = rng.choice([1, 64, 65, 300, 5000, 100000 // entries + 1])
        cases.append((rng.choice([1, 2, 3, 8, 24]), rng.choice([1, 2, 7, 64, 304, 512]),
                      rng.choice([1, 2, 4, 9]),
                      [rng.choice([0, 1, 63, 64, 65, rng.randint(0, top)]) for _ in range(entries)]))
    cases = [c for c in cases if sum(n // 64 + 1 for n in c[3]) * c[0] < 3_000_000]
    text = "\n".join(f"{c} {b} {l} {len(n)} " + " ".join(map(str, n)) for c, b, l, n in cases)
    out = subprocess.run([harness], input=text, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout == f"ok {len(cases)}\n", out.stdout + out.stderr
