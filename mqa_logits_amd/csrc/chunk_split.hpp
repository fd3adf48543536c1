// How chunk attention's work is divided: what a tile of a sequence's rows counts for, what
// its first k tiles do in closed form, and where the workers' pieces begin.  Integers
// alone, for the kernel and for a host program that checks one against the other.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

namespace mqa {

constexpr int kChunkKeys = 64;               // of a step
// Steps that beginning and ending a tile takes as long as (about 7 us; a step 2).
constexpr int kChunkTileSteps = 4;

// A sequence of the call.  (P: ChunkParams, or what a check has of it)
struct ChunkSeq {
  int64_t base;            // keys before its first new token (may be negative)
  int cap;                 // keys that its last row in q sees: of the context, unless q ends before
  int first, n;            // its rows of q
  int tiles;

  // ctx tokens, the last of them rows [lo, hi) of q, as far as q has those.
  template <class P>
  __host__ __device__ __forceinline__ void set(const P& p, int ctx, int64_t lo, int64_t hi) {
    const int64_t from = std::min(std::max(lo, (int64_t)0), (int64_t)p.tokens);
    const int64_t to = std::min(std::max(hi, from), (int64_t)p.tokens);
    base = (int64_t)ctx - (hi - lo) + (from - lo);   // (rows cut off in front: keys that stay)
    first = (int)from;
    n = (int)(to - from);
    // (no tile sees more, the last one neither if rows of it are cut off: `before` and
    // `steps` count it alike)
    cap = (int)std::max(std::min({(int64_t)ctx, (int64_t)p.max_ctx, base + n}), (int64_t)0);
    tiles = (n + p.tile_tokens - 1) / p.tile_tokens;
  }
  // keys that its row t sees
  __host__ __device__ __forceinline__ int seen(int64_t t) const {
    return (int)std::min(std::max(base + 1 + t, (int64_t)0), (int64_t)cap);
  }
  template <class P>
  __host__ __device__ __forceinline__ int tile_seen(const P& p, int i) const {
    return seen(std::min((int64_t)(i + 1) * p.tile_tokens, (int64_t)n) - 1);
  }
  // What a tile counts for in the split: its steps, and kChunkTileSteps to begin and end it.
  template <class P>
  __host__ __device__ __forceinline__ int steps(const P& p, int i) const {
    return p.whole ? 1 : (tile_seen(p, i) + kChunkKeys - 1) / kChunkKeys + kChunkTileSteps;
  }
  // The same for its first k tiles: none while no keys are seen, then the sum of
  // floor((tile_tokens * i + c) / 64), then the cap's.
  template <class P>
  __host__ __device__ __forceinline__ int64_t before(const P& p, int k) const {
    if (p.whole) return k;
    const int a = p.tile_tokens;
    const int64_t full = cap - base;
    const int64_t none = base >= 0 ? 0 : -base / a;                 // tiles that see nothing
    const int64_t until = full <= a ? 0 : (full + a - 1) / a - 1;   // tiles below the cap
    const int64_t i1 = std::min(none, (int64_t)k), i2 = std::min(std::max(until, i1), (int64_t)k);
    int64_t sum = (int64_t)k * kChunkTileSteps + (k - i2) * (int64_t)((cap + kChunkKeys - 1) / kChunkKeys);
    const int64_t m = i2 - i1, turns = m / kChunkKeys;
    if (m > 0) {
      const int64_t c = base + (i1 + 1) * a + kChunkKeys - 1;
      const int d = a & -a & (kChunkKeys - 1) ? a & -a : kChunkKeys;          // gcd(a, 64)
      const int64_t turn = ((int64_t)(a - 1) * (kChunkKeys - 1) + d - 1) / 2 + c / d * d;
      sum += turns * turn + (int64_t)a * kChunkKeys * (turns * (turns - 1) / 2);
      const int r = (int)(m - turns * kChunkKeys);
      sum += (int64_t)r * a * turns;
      for (int i = 0; i < r; ++i) sum += (c + (int64_t)a * i) / kChunkKeys;
    }
    return sum;
  }
};

// Workers' equal pieces of the steps of all tiles, laid end to end.
struct ChunkBorders {
  int64_t each, more;      // steps of a piece; pieces that have one more, the first
  int workers;             // with a piece

  // at most `most`, of `least` steps at least if there are that many
  __host__ __device__ __forceinline__ void divide(int64_t steps, int most, int least) {
    workers = (int)std::min((int64_t)most, std::max(steps / least, (int64_t)1));
    each = steps / workers;
    more = steps - each * workers;
  }
  __host__ __device__ __forceinline__ int64_t border(int64_t j) const { return j * each + std::min(j, more); }
  __host__ __device__ __forceinline__ int owner(int64_t step) const {
    const int64_t head = more * (each + 1);
    return (int)(step < head ? step / (each + 1) : more + (step - head) / each);
  }
};

}  // namespace mqa
