"""The division of chunk attention's work, on the CPU: the closed form of what a sequence's
first tiles count for against the sum over them, and the walk of every worker over the
tiles of all KV heads, which has to meet each step of each tile once, and no others.

Sequences of any length, bounds below and above them, rows of nobody, and rows that q
does not have, in front (offsets below 0) and behind (offsets past its rows).
"""

import os
import subprocess

import pytest

build = pytest.importorskip("mqa_logits_amd.build")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "chunk_split.hpp"

struct Sizes { int max_ctx, tokens, tile_tokens, whole; };

std::mt19937_64 rng(1);
int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }

int fail(const char* what, const Sizes& p, int ctx, int64_t lo, int64_t hi, int64_t got, int64_t want) {
  printf("%s: ctx=%d rows [%lld, %lld) of %d, bound %d, tiles of %d: %lld, not %lld\n", what, ctx, (long long)lo,
         (long long)hi, p.tokens, p.max_ctx, p.tile_tokens, (long long)got, (long long)want);
  return 1;
}

int closed_form(int n) {
  for (int i = 0; i < n; ++i) {
    const int size = i % 4 == 0 ? 70000 : 5000;
    const int lo = (int)pick(-40, 60), hi = lo + (int)pick(0, i % 3 ? size : 600);
    const Sizes p{(int)pick(0, size), (int)pick(0, hi + 300), (int)pick(1, 256), 0};
    const int ctx = (int)pick(-30, size);
    mqa::ChunkSeq s;
    s.set(p, ctx, lo, hi);
    int64_t sum = 0;
    for (int k = 0; k <= s.tiles; ++k) {
      if (s.before(p, k) != sum) return fail("before", p, ctx, lo, hi, s.before(p, k), sum);
      if (k < s.tiles) sum += s.steps(p, k);
    }
    for (int t = 0; t < s.n; ++t) {          // row s.first + t, of those from lo on
      const int64_t from_end = hi - (s.first + t);
      const int64_t want = std::max<int64_t>(std::min<int64_t>({ctx - from_end + 1, ctx, p.max_ctx}), 0);
      if (s.seen(t) != want) return fail("seen", p, ctx, lo, hi, s.seen(t), want);
    }
  }
  return 0;
}

// A call's workers, as the kernel walks them.
int walk(const Sizes& p, int members, int most, int least, const std::vector<int>& ctx, const std::vector<int>& offsets) {
  const int batch = (int)ctx.size();
  std::vector<mqa::ChunkSeq> seqs(batch);
  std::vector<int64_t> starts(batch + 1, 0);
  for (int b = 0; b < batch; ++b) {
    seqs[b].set(p, ctx[b], offsets[b], offsets[b + 1]);
    starts[b + 1] = starts[b] + seqs[b].before(p, seqs[b].tiles);
  }
  const int64_t all = starts[batch];
  if (all == 0) return 0;
  mqa::ChunkBorders borders;
  borders.divide(all * members, most, least);
  std::map<std::tuple<int, int, int>, std::vector<std::pair<int64_t, int64_t>>> parts;
  for (int worker = 0; worker < borders.workers; ++worker) {
    int64_t at = borders.border(worker);
    const int64_t end = borders.border(worker + 1);
    if (at >= end) continue;
    if (borders.owner(at) != worker || borders.owner(end - 1) != worker) return printf("owner of worker %d\n", worker);
    int member = (int)(at / all), b = 0, tile = 0;
    const int64_t want = at - member * all;
    while (starts[b + 1] <= want) ++b;
    while (tile + 1 < seqs[b].tiles && starts[b] + seqs[b].before(p, tile + 1) <= want) ++tile;
    int64_t tile_begin = member * all + starts[b] + seqs[b].before(p, tile);
    while (at < end) {
      if (member >= members) return printf("worker %d is past the last KV head\n", worker);
      const int64_t tile_end = tile_begin + seqs[b].steps(p, tile);
      parts[{member, b, tile}].push_back({at - tile_begin, std::min(end, tile_end) - tile_begin});
      at = tile_begin = tile_end;
      if (++tile >= seqs[b].tiles && at < end) {
        tile = 0;
        do {
          if (++b == batch) {
            b = 0;
            ++member;
          }
        } while (seqs[b].tiles == 0);
      }
    }
  }
  size_t tiles = 0;
  for (int member = 0; member < members; ++member)
    for (int b = 0; b < batch; ++b)
      for (int tile = 0; tile < seqs[b].tiles; ++tile) {
        ++tiles;
        int64_t at = 0;
        for (const auto& part : parts[{member, b, tile}]) {
          if (part.first != at) return printf("KV head %d, sequence %d, tile %d: a part from %lld, not %lld\n", member, b, tile, (long long)part.first, (long long)at);
          at = part.second;
        }
        if (at != seqs[b].steps(p, tile)) return printf("KV head %d, sequence %d, tile %d: %lld steps\n", member, b, tile, (long long)at);
      }
  return parts.size() == tiles ? 0 : printf("tiles that are none\n");
}

int walks(int n) {
  for (int i = 0; i < n; ++i) {
    const int batch = (int)pick(1, i % 2 ? 3 : 20), size = i % 3 ? 3000 : 300;
    std::vector<int> ctx, offsets{(int)pick(-20, 20)};
    for (int b = 0; b < batch; ++b) {
      ctx.push_back((int)pick(-5, size));
      offsets.push_back(offsets.back() + (pick(0, 3) ? (int)pick(0, 300) : 0));
    }
    const int whole = i % 5 == 0;
    const Sizes p{(int)pick(1, size + 200), std::max(0, offsets.back() + (int)pick(-300, 30)), (int)pick(1, 256), whole};
    if (walk(p, (int)pick(1, 9), (int)pick(1, 256), whole ? 1 : 4, ctx, offsets)) return 1;
  }
  return 0;
}

int main(int argc, char** argv) {
  const std::string what = argv[1];
  if (what == "closed_form") return closed_form(20000);
  if (what == "walks") return walks(3000);
  // one sequence of 4000 tokens, 256 of them new, 130 rows of q: 8 KV heads, tiles of 256 tokens
  if (walk({4000, 130, 256, 0}, 8, 128, 4, {4000}, {0, 256})) return 1;
  // 2359 tokens, 219 new, 97 rows: 64 heads on 8
  return walk({2359, 97, 32, 0}, 8, 256, 4, {2359}, {0, 219}) != 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    folder = tmp_path_factory.mktemp("split")
    source, out = str(folder / "split.cpp"), str(folder / "split")
    with open(source, "w") as f:
        f.write(PROGRAM)
    subprocess.run([build.HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O2", "-std=c++17",
                    "-I", build.CSRC, source, "-o", out], check=True, capture_output=True)
    return out


@pytest.mark.parametrize("what", ["closed_form", "walks", "cut_rows"])
def test_division(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
