"""The decode kernel's division of work (csrc/fat_decode_plan.h) at sizes where every tile cannot
be walked: where each block starts, where items end, and what is joined, from the formulas the
kernel uses; the 32-bit and 64-bit forms of the share agree; as many blocks as the workspace has
room for."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensorized_online_softmax_gb300", "csrc")

HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "fat_decode_plan.h"
using namespace fat;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

static int shares() {
  std::mt19937_64 rng(7);
  const int top = 0x7fffffff - kDecodeMaxBlocks;  // up to here the kernel divides in 32 bits
  std::vector<int> totals = {1, 2, 63, 64, 65, 639, 640, 641, top - 1, top};
  for (int i = 0; i < 20000; ++i) totals.push_back(1 + rng() % top);
  for (int total : totals)
    for (int blocks : {1, 2, 7, 151, 152, 304, 456, 608, 639, 640})
      for (int least : {1, 2, 9}) {
        const int s = decode_share(total, blocks, least);
        const long long wide = decode_share(static_cast<long long>(total), blocks, least);
        CHECK(s == wide && s >= least);
        CHECK(static_cast<long long>(s) * blocks >= total);
        CHECK(s == least || static_cast<long long>(s - 1) * blocks < total);
      }
  return 0;
}

static int places() {
  std::mt19937_64 rng(8);
  for (int i = 0; i < 20000; ++i) {
    const int tiles = 1 + rng() % (i % 2 ? 1 << 24 : 100);
    const int item = rng() % (i % 3 ? 0x7fffffff : 1000), tile = rng() % tiles;
    const long long offset = static_cast<long long>(item) * tiles + tile;
    const DecodePlace p = decode_place(5, offset, tiles);
    CHECK(p.entry == 5 && p.item == item && p.tile == tile && p.tiles == tiles);
  }
  // either side of where the division changes its width
  for (long long offset : {0x7ffffffell, 0x7fffffffll, 0x80000000ll, 0x80000001ll, 0x1ffffffffll})
    for (int tiles : {1 << 24, (1 << 24) - 1, 12345678, 7}) {
      if (offset / tiles > 0x7fffffff) continue;
      const DecodePlace p = decode_place(0, offset, tiles);
      CHECK(static_cast<long long>(p.item) * tiles + p.tile == offset && p.tile < tiles);
    }
  return 0;
}

// The items on the line one by one (not their tiles): which blocks have part of each.
static int line(int copies, int blocks, int least, const std::vector<int>& len) {
  std::vector<long long> before(len.size() + 1, 0);
  for (size_t e = 0; e < len.size(); ++e)
    before[e + 1] = before[e] + static_cast<long long>(decode_tiles(len[e])) * copies;
  const long long total = before.back(), share = decode_share(total, blocks, least);
  CHECK(share * blocks >= total);
  std::vector<int> unfinished(2 * blocks, 0);  // by block and part
  for (size_t e = 0; e < len.size(); ++e) {
    const long long tiles = decode_tiles(len[e]);
    for (int m = 0; m < copies; ++m) {
      const long long first = before[e] + m * tiles, end = first + tiles;
      const long long c0 = first / share, c1 = (end - 1) / share;
      CHECK(c1 < blocks);
      if (c0 == c1) continue;  // whole in one block
      for (long long c = c0; c <= c1; ++c) {
        const int part = decode_part(first, c * share);
        CHECK(part == (c == c0 ? (first == c0 * share ? 0 : 1) : 0));
        CHECK(++unfinished[2 * c + part] == 1);
      }
      // what the first block notes for the join: the item's first tile as it sees it
      CHECK((first + decode_tiles(len[e]) - 1) / share == c1);
    }
  }
  // where a block starts, as the kernel finds it
  for (int b = 0; b < blocks; ++b) {
    const long long begin = b * share;
    if (begin >= total) continue;
    const size_t e = std::upper_bound(before.begin(), before.end(), begin) - before.begin() - 1;
    const DecodePlace p = decode_place(static_cast<int>(e), begin - before[e], decode_tiles(len[e]));
    CHECK(p.item < copies && p.tile < p.tiles);
    CHECK(before[e] + static_cast<long long>(p.item) * p.tiles + p.tile == begin);
    // (a block counts its tiles in 32 bits)
    CHECK(blocks < 456 || std::min(total, begin + share) - begin <= 0x7fffffff);
    // to the end of its item and into the next one
    DecodePlace q = p;
    q.tile = q.tiles - 1;
    const bool entry = decode_advance(q, copies);
    CHECK(q.tile == 0 && entry == (p.item == copies - 1));
    CHECK(entry ? q.item == 0 && q.entry == p.entry + 1 : q.item == p.item + 1 && q.entry == p.entry);
  }
  return 0;
}

int main() {
  if (shares() || places()) return 1;
  const int most = 1 << 30;
  std::mt19937_64 rng(9);
  int cases = 0;
  for (int blocks : {1, 7, 456, 512, 513, 608, 639, 640})
    for (int least : {1, 2, 4}) {
      std::vector<std::vector<int>> lens = {{most, 0, 1 << 20}, {most}, std::vector<int>(64, most),
                                            std::vector<int>(700, 5), {0}, {64 * 640}, {64 * 641}};
      std::vector<int> ragged;
      for (int i = 0; i < 3000; ++i)
        ragged.push_back(static_cast<int>(rng() % (i % 7 ? 3000 : i % 2 ? 1 << 20 : most)));
      lens.push_back(ragged);
      for (const auto& n : lens)
        for (int copies : {1, 2, 8, 33}) {
          if (line(copies, blocks, least, n)) return 1;
          ++cases;
        }
    }
  std::printf("ok %d\n", cases);
  return 0;
}
"""


def test_large_divisions(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "plan.cc", tmp_path / "plan"
    src.write_text(HARNESS)
    subprocess.run([cxx, "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout == f"ok {8 * 3 * 8 * 4}\n", out.stdout + out.stderr
