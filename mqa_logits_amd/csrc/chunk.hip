// Softmax attention of chunks of new tokens over a paged cache held in MXFP4
// (gfx950), and the kernel that joins split contexts.
//
//   out[r, :] = sum_j p[r, j] v[j, :],  p[r, :] = softmax_j(scale <q[r, :], k[j, :]>)
//
// over the keys j that row r, a (token, head) pair, sees.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "launch.hpp"

namespace mqa {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kKeys = 64;                    // of a step
constexpr int kStage = 16384;                // keys whose places LDS holds at a time
constexpr uint32_t kLastScale = 252;         // bytes above could overflow fp32: they count as NaN
// Scale bytes (2^-22 .. 2^9) whose steps are worked on in fp16.  Every e2m1 value
// under 2^-23 .. 2^13 is exact there; large ones are left out for what the weights'
// own end costs, see kRoom.
constexpr uint32_t kHalfLow = 105, kHalfHigh = 136;
// The running maximum is set kRoom octaves below the largest score, and follows a
// new one only when that leaves a weight above 2^kMost (fp16 ends at 65504); most
// steps rescale nothing.  The largest weight is then between 2^kRoom and 2^kMost,
// and half a step of fp16's least subnormal is 2^-37 of it at most.  The
// unnormalised sums of n keys stay within n * 2^15 times the largest value.
constexpr float kRoom = 12.f, kMost = 15.f;
constexpr float kLowest = -0x1.fffffep127f;  // a maximum before any key (finite: no inf - inf)
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  return HALF ? pack_f16(a, b) : pack_bf16(a, b);
}

// Byte SEL of w: two e2m1 elements times the scale.
template <bool HALF, int SEL>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t w, float scale) {
  if constexpr (HALF)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, SEL));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}
template <bool HALF>
__device__ __forceinline__ u32x4 cvt_eight(uint32_t w, float scale) {
  return u32x4{cvt_pair<HALF, 0>(w, scale), cvt_pair<HALF, 1>(w, scale), cvt_pair<HALF, 2>(w, scale),
               cvt_pair<HALF, 3>(w, scale)};
}
// Nothing derived from x is kept in registers through a loop around this.
__device__ __forceinline__ int here_only(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

template <bool HALF>
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Work split
// ---------------------------------------------------------------------------

// Sequence b of the call.
struct Seq {
  int64_t base;            // keys before its first new token (may be negative)
  int cap;                 // keys of the context
  int first, n;            // its rows of q
  int tiles;
  // UNIFORM: b is the same in every lane, and everything stays in scalar registers.
  template <bool UNIFORM>
  __device__ __forceinline__ static Seq of(const ChunkParams& p, int b) {
    Seq s;
    const auto get = [](int x) { return UNIFORM ? __builtin_amdgcn_readfirstlane(x) : x; };
    int64_t lo, hi;
    if (p.offsets) {
      lo = get(p.offsets[b]);
      hi = get(p.offsets[b + 1]);
    } else {
      lo = (int64_t)b * p.next_n;
      hi = lo + p.next_n;
    }
    const int ctx = get(p.ctx[b]);
    s.cap = min(max(ctx, 0), p.max_ctx);
    const int64_t from = min(max(lo, (int64_t)0), (int64_t)p.tokens);
    const int64_t to = min(max(hi, from), (int64_t)p.tokens);
    s.base = (int64_t)ctx - (hi - lo) + (from - lo);   // (rows cut off in front: keys that stay)
    s.first = (int)from;
    s.n = (int)(to - from);
    s.tiles = (s.n + p.tile_tokens - 1) / p.tile_tokens;
    return s;
  }
  // keys that its row t sees
  __device__ __forceinline__ int seen(int64_t t) const {
    return (int)min(max(base + 1 + t, (int64_t)0), (int64_t)cap);
  }
  __device__ __forceinline__ int tile_seen(const ChunkParams& p, int i) const {
    return seen(min((int64_t)(i + 1) * p.tile_tokens, (int64_t)n) - 1);
  }
  __device__ __forceinline__ int steps(const ChunkParams& p, int i) const {
    return p.whole ? 1 : max((tile_seen(p, i) + kKeys - 1) / kKeys, 1);
  }
  // steps of its first k tiles: one each while a step is enough, then
  // sum of floor((tile_tokens * i + c) / 64), then the context's
  __device__ __forceinline__ int64_t before(const ChunkParams& p, int k) const {
    if (p.whole) return k;
    const int a = p.tile_tokens;
    const int64_t room = kKeys - base, full = cap - base;
    const int64_t few = room < a ? 0 : room / a;                    // tiles that see at most 64 keys
    const int64_t until = full <= a ? 0 : (full + a - 1) / a - 1;   // tiles below the cap
    const int64_t i1 = min(few, (int64_t)k), i2 = min(max(until, i1), (int64_t)k);
    int64_t sum = i1 + (k - i2) * (int64_t)max((cap + kKeys - 1) / kKeys, 1);
    const int64_t m = i2 - i1, turns = m / kKeys;
    if (m > 0) {
      const int64_t c = base + (i1 + 1) * a + kKeys - 1;
      const int d = a & -a & (kKeys - 1) ? a & -a : kKeys;          // gcd(a, 64)
      const int64_t turn = ((int64_t)(a - 1) * (kKeys - 1) + d - 1) / 2 + c / d * d;
      sum += turns * turn + (int64_t)a * kKeys * (turns * (turns - 1) / 2);
      const int r = (int)(m - turns * kKeys);
      sum += (int64_t)r * a * turns;
      for (int i = 0; i < r; ++i) sum += (c + (int64_t)a * i) / kKeys;
    }
    return sum;
  }
};

__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Steps of all sequences before b0 + tid's among 256 from b0 on, and of all of them.
__device__ __forceinline__ int64_t scan(int64_t mine, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t y = __shfl_up((long long)x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = x;
  __syncthreads();
  int64_t before = x - mine;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += sums[w];
    total += sums[w];
  }
  return before;
}

// A worker's piece of the steps of all members' sequences' tiles, laid end to end.
struct Piece {
  int64_t begin, end, each, more, at;
  int64_t tile_begin;      // where the tile at `at` begins
  int workers, member, b, tile;

  __device__ __forceinline__ int64_t border(int64_t j) const { return j * each + min(j, more); }
  __device__ __forceinline__ int owner(int64_t step) const {
    const int64_t head = more * (each + 1);
    return (int)(step < head ? step / (each + 1) : more + (step - head) / each);
  }

  __device__ __forceinline__ bool find(const ChunkParams& p, int worker, int64_t* sums, int64_t* found) {
    int64_t all = 0, part;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      const int i = b0 + threadIdx.x;
      int64_t mine = 0;
      if (i < p.batch) {
        const Seq s = Seq::of<false>(p, i);
        mine = s.before(p, s.tiles);
      }
      scan(mine, sums, part);
      all += part;
    }
    all = uniform(all);
    const int64_t steps = all * p.members;
    workers = (int)min((int64_t)p.workers, max(steps / p.least, (int64_t)1));
    each = steps / workers;
    more = steps - each * workers;
    begin = at = border(worker);
    end = border(worker + 1);
    if (worker >= workers || begin >= end) return false;
    member = (int)(begin / all);
    const int64_t want = begin - member * all;
    int64_t base = 0;
    for (int b0 = 0; base <= want; b0 += kThreads) {
      const int i = b0 + threadIdx.x;
      int64_t mine = 0;
      if (i < p.batch) {
        const Seq s = Seq::of<false>(p, i);
        mine = s.before(p, s.tiles);
      }
      const int64_t here = base + scan(mine, sums, part);
      if (here <= want && want < here + mine) {
        found[0] = i;
        found[1] = here;
      }
      base += part;
    }
    __syncthreads();
    b = (int)uniform(found[0]);
    const int64_t start = uniform(found[1]);
    // the tile: 64 places at a time
    const Seq s = Seq::of<true>(p, b);
    int lo = 0, n = s.tiles;
    while (n > 1) {
      const int span = (n + 63) / 64, i = (threadIdx.x & 63) * span;
      const bool yes = i < n && start + s.before(p, lo + i) <= want;
      const int last = 63 - __builtin_clzll(__ballot(yes));
      lo += last * span;
      n = min(span, n - last * span);
    }
    tile = __builtin_amdgcn_readfirstlane(lo);
    tile_begin = uniform(member * all + start + s.before(p, tile));
    return true;
  }
};

// ---------------------------------------------------------------------------
// A step of 64 keys in LDS
// ---------------------------------------------------------------------------

template <int D>
struct Stage {
  static constexpr int kKeyPitch = D * 2 + 16;       // bytes; free of bank conflicts
  static constexpr int kValPitch = kKeys * 2 + 16;
  static constexpr int kBytes = kKeys * kKeyPitch + D * kValPitch;
};

// What a thread loads of a step.  The first half of the workgroup takes D/8 bytes
// of codes of a key each and their scale; the second D/32 bytes of V's codes of four
// keys and their scales.
struct Raw {
  u32x4 codes;
  uint32_t scales[4];
};

template <int D>
struct Loader {
  const ChunkParams& p;
  const uint32_t* places;  // first block (of 32 elements) of every 16th key
  uint32_t key_blocks;     // blocks from one key of the pool to the next

  // key0: the step's first key, from the stage's; n: keys of the context from there on
  template <bool KEYS>
  __device__ __forceinline__ void load(Raw& r, int tid, int key0, int n) const {
    if constexpr (KEYS) {
      const int j = tid >> 2, c = tid & 3;
      const uint32_t block = places[(key0 + j) >> 4] + (j & 15) * key_blocks;
      const uint8_t* src = p.k + ((uint64_t)block << 4) + c * (D / 8);
      if constexpr (D == 128) {
        r.codes = *reinterpret_cast<const u32x4*>(src);
      } else {
        const u32x2 x = *reinterpret_cast<const u32x2*>(src);
        r.codes = u32x4{x[0], x[1], 0u, 0u};
      }
      const uint32_t s = p.k_sf[(uint64_t)block + c * (D / 4) / 32];
      r.scales[0] = j < n ? s : 127u;        // (any finite one where nothing is stored)
    } else {
      const int j = Values::key(tid), c = Values::column(tid);
      const uint32_t first = places[(key0 + j) >> 4] + (j & 15) * key_blocks;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t block = first + i * key_blocks;
        const uint8_t* src = p.v + ((uint64_t)block << 4) + c * (D / 32);
        r.codes[i] = D == 128 ? *reinterpret_cast<const uint32_t*>(src) : *reinterpret_cast<const uint16_t*>(src);
        const uint32_t s = p.v_sf[(uint64_t)block + c * (D / 16) / 32];
        r.scales[i] = j + i < n ? s : 127u;
      }
    }
  }

  // The second half's keys and columns: 16 lanes in a row write all banks.
  struct Values {
    __device__ __forceinline__ static int quad(int tid) { return (tid & 3) | (tid >> 6 & 3) << 2; }
    __device__ __forceinline__ static int key(int tid) { return quad(tid) * 4; }
    __device__ __forceinline__ static int column(int tid) { return tid >> 2 & 15; }
  };
};

// K as rows of D (KEYS), or V transposed, into a step's LDS.
template <int D, bool KEYS, bool HALF>
__device__ __forceinline__ void put(const Raw& r, int tid, char* lds) {
  if constexpr (KEYS) {
    const int c = tid & 3;
    char* dst = lds + (tid >> 2) * Stage<D>::kKeyPitch + c * (D / 2);
    const float s = scale_of(r.scales[0]);
    if constexpr (D == 128) {
      // half of the lanes the other way round: 8 in a row write all banks
      const int turn = c & 2;
      const u32x4 x = turn ? u32x4{r.codes[2], r.codes[3], r.codes[0], r.codes[1]} : r.codes;
      char* one = dst + turn * 16;
      char* two = dst + (turn ^ 2) * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(one + i * 16) = cvt_eight<HALF>(x[i], s);
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(two + i * 16) = cvt_eight<HALF>(x[i + 2], s);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(dst + i * 16) = cvt_eight<HALF>(r.codes[i], s);
    }
  } else {
    // element e of the thread's D/16 is row e % (D/32) * 32 + 2 c + e / (D/32); four
    // keys are one half of what a lane multiplies of 16
    const int quad = Loader<D>::Values::quad(tid), c = Loader<D>::Values::column(tid);
    char* dst = lds + kKeys * Stage<D>::kKeyPitch + 2 * c * Stage<D>::kValPitch + (quad >> 2) * 32 +
                (quad & 1) * 16 + (quad >> 1 & 1) * 8;
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = scale_of(r.scales[i]);
    const auto two = [&](auto sel) {
      constexpr int SEL = decltype(sel)::value;
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = cvt_pair<HALF, SEL>(r.codes[i], s[i]);
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        constexpr int kCols = D / 32;
        const int e = 2 * SEL + odd, at = e % kCols * 32 + e / kCols;
        const uint32_t pick = odd ? 0x07060302u : 0x05040100u;
        *reinterpret_cast<u32x2*>(dst + at * Stage<D>::kValPitch) =
            u32x2{__builtin_amdgcn_perm(x[1], x[0], pick), __builtin_amdgcn_perm(x[3], x[2], pick)};
      }
    };
    two(std::integral_constant<int, 0>{});
    two(std::integral_constant<int, 1>{});
    if constexpr (D == 128) {
      two(std::integral_constant<int, 2>{});
      two(std::integral_constant<int, 3>{});
    }
  }
}

// Some scale is outside what the fp16 (or, for bf16 queries, K's bf16) products take.
template <bool KEYS, bool F16>
__device__ __forceinline__ bool wide_scales(const Raw& r) {
  const auto wide = [](uint32_t s) { return s - kHalfLow > kHalfHigh - kHalfLow; };
  if constexpr (KEYS) return F16 ? wide(r.scales[0]) : r.scales[0] > kLastScale;
  return wide(r.scales[0]) || wide(r.scales[1]) || wide(r.scales[2]) || wide(r.scales[3]);
}

// ---------------------------------------------------------------------------
// A wave's 32 * QT rows
// ---------------------------------------------------------------------------

template <int D, int QT, bool F16>
struct Rows {
  static constexpr int kSteps = D / 16, kCols = D / 32;
  u32x4 q[QT][kSteps];     // row l % 32, elements 16 st + 8 (l / 32) ..
  f32x16 o[QT][kCols];     // row l % 32; element kCols * m + col, m = i % 4 + 8 (i / 4) + 4 (l / 32)
  float m[QT], l[QT];      // running maximum (log2), the lane's part of the sum of weights
  float r[QT];             // and of the sum of the rounded ones
  int seen[QT];
  uint32_t nan_blocks[QT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      m[t] = kLowest;
      l[t] = r[t] = 0.f;
      nan_blocks[t] = 0;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][c][i] = 0.f;
    }
  }

  // One step.  WIDE: some scale is outside fp16's range; LDS holds bf16.
  template <bool MASKED>
  __device__ __forceinline__ void step(const char* lds, int key0, float c2) {
    part<false, MASKED, 2>(lds, 0, key0, c2);
  }
  __device__ __forceinline__ void wide_step(const char* lds, int key0, float c2) {
#pragma nounroll
    for (int h = 0; h < 2; ++h) part<true, true, 1>(lds, h, key0, c2);
  }

  // H halves of 32 keys of it.
  template <bool WIDE, bool MASKED, int H>
  __device__ __forceinline__ void part(const char* lds, int first, int key0, float c2) {
    const int lane = WIDE || MASKED ? here_only(threadIdx.x & 63) : threadIdx.x & 63, half = lane >> 5;
    const char* keys = lds + (first * 32 + (lane & 31)) * Stage<D>::kKeyPitch + half * 16;
    const char* vals = lds + kKeys * Stage<D>::kKeyPitch + (lane & 31) * Stage<D>::kValPitch + half * 16 + first * 64;
    f32x16 s[QT][H];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][h][i] = 0.f;
    // A product must not overlap its operands.  The compiler was seen to let one
    // with a constant 0 to add to overlap them: the operands are used once more
    // behind it, or (here) the zeros are registers.
    if (WIDE) asm volatile("" : "+v"(s[0][0]));
    // operands are read kAhead products before their use
    constexpr int kAhead = 4;
    const auto key_operand = [&](int n) {
      return *reinterpret_cast<const u32x4*>(keys + n % H * 32 * Stage<D>::kKeyPitch + n / H * 32);
    };
    u32x4 a[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) a[n] = key_operand(n);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < H * kSteps; ++n) {
      const int st = n / H, h = n % H;
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        if constexpr (WIDE && F16) {
          // the query's two exact bf16 parts; an infinity stays in the first alone
          u32x4 hi, lo;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f16x2 x = __builtin_bit_cast(f16x2, here_only(q[t][st][i]));
            const float y = (float)x[0], z = (float)x[1];
            hi[i] = pack_bf16(y, z);
            const float ry = y - bf16_lo(hi[i]), rz = z - bf16_hi(hi[i]);
            lo[i] = pack_bf16(__builtin_isfinite(y) ? ry : 0.f, __builtin_isfinite(z) ? rz : 0.f);
          }
          s[t][h] = mma<false>(a[n % kAhead], hi, s[t][h]);
          s[t][h] = mma<false>(a[n % kAhead], lo, s[t][h]);
        } else {
          s[t][h] = mma<F16>(a[n % kAhead], q[t][st], s[t][h]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (n < H) asm volatile("" ::"v"(a[n % kAhead]));   // still its own behind the product
      if (n + kAhead < H * kSteps) a[n % kAhead] = key_operand(n + kAhead);
    }
    const auto value_operand = [&](int n) {
      return *reinterpret_cast<const u32x4*>(vals + n % kCols * 32 * Stage<D>::kValPitch + n / kCols * 32);
    };
#pragma unroll
    for (int n = 0; n < kAhead; ++n) a[n] = value_operand(n);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MASKED) {
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = key0 + (first + h) * 32 + (i & 3) + 8 * (i >> 2) + 4 * half;
            s[t][h][i] = key < seen[t] ? s[t][h][i] : -__builtin_inff();
          }
    }
    u32x4 w[QT][WIDE ? 2 : 1][2 * H];        // [high and low part][16 keys]
#pragma unroll
    for (int t = 0; t < QT; ++t) weights<WIDE, H>(s[t], t, c2, w[t]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 2 * H * kCols; ++n) {
      const int k = n / kCols, c = n % kCols;
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int x = 0; x < (WIDE ? 2 : 1); ++x) o[t][c] = mma<!WIDE>(a[n % kAhead], w[t][x][k], o[t][c]);
      if (n + kAhead < 2 * H * kCols) a[n % kAhead] = value_operand(n + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Weights relative to the running maximum m.
  template <bool WIDE, int H>
  __device__ __forceinline__ void weights(const f32x16 (&s)[H], int t, float c2, u32x4 (&w)[WIDE ? 2 : 1][2 * H]) {
    float best = s[0][0];
#pragma unroll
    for (int i = 1; i < 16 * H; ++i) best = fmaxf(best, s[i >> 4][i & 15]);
    if (__builtin_expect(__any(__builtin_fmaf(best, c2, -m[t]) > kMost), 0)) {
      asm volatile("");                      // rare: nothing of it belongs before the branch
      best = fmaxf(best, __shfl_xor(best, 32)) * c2;
      const float next = fmaxf(m[t], best - kRoom);
      const float f = __builtin_amdgcn_exp2f(m[t] - next);
      m[t] = next;
      l[t] *= f;
      r[t] *= f;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][c][i] *= f;
    }
    float x[16 * H];
#pragma unroll
    for (int i = 0; i < 16 * H; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 4][i & 15], c2, -m[t]));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16 * H; i += 4) sum += (x[i] + x[i + 1]) + (x[i + 2] + x[i + 3]);
    l[t] += sum;
    if (WIDE) r[t] += sum;
#pragma unroll
    for (int k = 0; k < 2 * H; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[8 * k + 2 * i], b = x[8 * k + 2 * i + 1];
        const uint32_t hi = pack<!WIDE>(a, b);
        w[0][k][i] = hi;
        if constexpr (WIDE)
          w[1][k][i] = pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
        else
          r[t] = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, hi), f16x2{(_Float16)1.f, (_Float16)1.f}, r[t], false);
      }
  }
};

// The steps of a stage, for a wave of the half that loads K (KEYS) or V.
template <bool KEYS, int D, int QT, bool F16, class InContext>
__device__ __forceinline__ void walk(const Loader<D>& loader, Rows<D, QT, F16>& rows,
                                     char (&stage)[2][Stage<D>::kBytes], int* flags, uint8_t (&nan_marks)[2][kKeys][4],
                                     int stage0, int steps, int least, const InContext& in_context, float c2) {
  const int tid = threadIdx.x & (kThreads / 2 - 1);
  constexpr bool kHalf = KEYS ? F16 : true;
  Raw raw;
  const auto store = [&](int i) {
    const int me = here_only(tid);
    if (wide_scales<KEYS, F16>(raw)) flags[i & 1] = i;
    put<D, KEYS, kHalf>(raw, me, stage[i & 1]);
  };
  const auto fetch = [&](int i) { loader.template load<KEYS>(raw, here_only(tid), i * kKeys, in_context(i)); };
  fetch(0);
  store(0);
  fetch(min(1, steps - 1));
  __syncthreads();
  // Steps whose keys all rows see, then those at the rows' own ends.  (Past the
  // last step, the last again is stored and never used.)
  const int clear = min(max(least - stage0, 0) / kKeys, steps);
  int i = 0;
  const auto narrow = [&] { return __builtin_amdgcn_readfirstlane(flags[i & 1]) != i; };
  const auto turn = [&] {
    store(i + 1);
    fetch(min(i + 2, steps - 1));
    ++i;
    __syncthreads();
  };
#pragma nounroll
  while (i < clear && narrow()) {
    rows.template step<false>(stage[i & 1], 0, c2);
    turn();
  }
#pragma nounroll
  while (i < steps && narrow()) {
    rows.template step<true>(stage[i & 1], stage0 + i * kKeys, c2);
    turn();
  }
  if (__builtin_expect(i == steps, 1)) return;
  // from a step with unusual scales on, in bf16, NaN scales apart
  loader.template load<KEYS>(raw, here_only(tid), i * kKeys, in_context(i));
#pragma nounroll
  for (; i < steps; ++i) {
    const int me = here_only(tid);
    if constexpr (KEYS) {
      if (raw.scales[0] > kLastScale) raw.scales[0] = 255;
    } else {
      const int c = Loader<D>::Values::column(me), b = c * (D / 16) / 32;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool bad = raw.scales[j] > kLastScale;
        if (c % (512 / D) == 0) nan_marks[i & 1][Loader<D>::Values::key(me) + j][b] = bad;
        raw.scales[j] = bad ? 0u : raw.scales[j];
      }
    }
    __syncthreads();                         // the stage's last use is over
    put<D, KEYS, false>(raw, me, stage[i & 1]);
    __syncthreads();
    loader.template load<KEYS>(raw, here_only(tid), min(i + 1, steps - 1) * kKeys, in_context(min(i + 1, steps - 1)));
    const int key0 = stage0 + i * kKeys;
    uint32_t marks = 0;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) marks |= (uint32_t)nan_marks[i & 1][me & 63][b] << b;
    if (__builtin_expect(__any(marks != 0), 0))
#pragma nounroll
      for (int j = 0; j < kKeys; ++j) {
        const uint32_t word = __shfl(marks, j);
#pragma unroll
        for (int t = 0; t < QT; ++t)
          if (key0 + j < rows.seen[t]) rows.nan_blocks[t] |= word;
      }
    rows.wide_step(stage[i & 1], key0, c2);
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2)
chunk_kernel(const ChunkParams p) {
  constexpr int QT = 1;
  __shared__ __attribute__((aligned(16))) char stage[2][Stage<D>::kBytes];
  __shared__ uint32_t places[kStage / 16];
  __shared__ uint8_t nan_marks[2][kKeys][4];
  __shared__ int flags[2];
  __shared__ int64_t sums[kWaves], found[2];

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // neighbouring workers, which read the same keys, on one XCD
  const int worker = (blockIdx.x & 7) * ((p.workers + 7) / 8) + (blockIdx.x >> 3);
  Piece piece;
  const bool any = worker < p.workers && piece.find(p, worker, sums, found);
  if (!any) {
    if (p.notes && tid == 0 && worker < p.workers) p.notes[worker].parts = 0;
    return;
  }

  Rows<D, QT, F16> rows;
  ChunkNote note{};
  while (piece.at < piece.end) {
    const Seq s = Seq::of<true>(p, piece.b);
    const int kv_head = piece.member / p.head_groups;
    const int head0 = kv_head * p.group + piece.member % p.head_groups * p.tile_heads;
    const int heads = min(p.tile_heads, (kv_head + 1) * p.group - head0);
    const int token0 = piece.tile * p.tile_tokens;                     // of the sequence
    const int tokens = min(p.tile_tokens, s.n - token0);
    const int n_rows = tokens * heads;
    const int tile_seen = s.tile_seen(p, piece.tile);
    const int64_t tile_end = piece.tile_begin + s.steps(p, piece.tile);
    const int begin = p.whole ? 0 : (int)(piece.at - piece.tile_begin) * kKeys;
    const int end = p.whole ? tile_seen
                            : (int)min((int64_t)tile_seen, (min(tile_end, piece.end) - piece.tile_begin) * kKeys);
    const int wave_row = wave * 32 * QT;
    const int least = s.seen(token0);        // keys that all rows see
    rows.clear();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      // lanes past the last row repeat it; their results are dropped
      const int r = min(wave_row + t * 32 + (lane & 31), n_rows - 1);
      const int at = r / heads;
      rows.seen[t] = s.seen(token0 + at);
      const uint16_t* src = p.q + (int64_t)(s.first + token0 + at) * p.q_stride + (head0 + r - at * heads) * D + half * 8;
#pragma unroll
      for (int st = 0; st < D / 16; ++st) {
        rows.q[t][st] = *reinterpret_cast<const u32x4*>(src + st * 16);
        if (p.negate) rows.q[t][st] ^= 0x80008000u;
      }
    }
    const int32_t* table = p.bt + (int64_t)piece.b * p.bt_stride;
    const uint32_t key_blocks = p.kv_heads * (D / 32);
    const Loader<D> loader{p, places, key_blocks};
    for (int stage0 = begin; stage0 < end; stage0 += kStage) {
      const int stage_end = min(end, stage0 + kStage), n = stage_end - stage0;
      const int steps = (n + kKeys - 1) / kKeys;
      __syncthreads();                       // the last use of `places` and the stages is over
      for (int i = tid; i < steps * (kKeys / 16); i += kThreads) {
        const int j = min(stage0 + i * 16, s.cap - 1);
        const int id = min(max(table[j >> p.bs_shift], 0), p.num_blocks - 1);
        const uint32_t slot = ((uint32_t)id << p.bs_shift) + (stage0 + i * 16 & (1 << p.bs_shift) - 1);
        places[i] = slot * key_blocks + kv_head * (D / 32);
      }
      if (tid < 2) flags[tid] = -1;
      __syncthreads();
      const auto in_context = [&](int i) { return s.cap - stage0 - i * kKeys; };
      if (wave < kWaves / 2)
        walk<true>(loader, rows, stage, flags, nan_marks, stage0, steps, least, in_context, p.c2);
      else
        walk<false>(loader, rows, stage, flags, nan_marks, stage0, steps, least, in_context, p.c2);
    }

    const bool first_part = piece.at == piece.tile_begin, last_part = tile_end <= piece.end;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const float m = rows.m[t], l = rows.l[t] + __shfl_xor(rows.l[t], 32);
      const float rounded = rows.r[t] + __shfl_xor(rows.r[t], 32);
      const int r = here_only(wave_row + t * 32 + (lane & 31));
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (rows.nan_blocks[t] >> ((i >> 2) * 8 * (D / 32) / 32) & 1) rows.o[t][c][i] = __builtin_nanf("");
      if (r >= n_rows) continue;
      constexpr int kCols = D / 32;
      if (first_part && last_part) {
        const int at = r / heads;
        const int64_t row = (int64_t)(s.first + token0 + at) * p.q_heads + head0 + (r - at * heads);
        const float inv = rounded == 0.f ? 0.f : 1.f / rounded;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          // 4 * kCols adjacent elements
          uint32_t x[2 * kCols];
#pragma unroll
          for (int i = 0; i < 2 * kCols; ++i) {
            const int e = 2 * i, f = 2 * i + 1;
            x[i] = pack<F16>(rows.o[t][e % kCols][4 * a + e / kCols] * inv, rows.o[t][f % kCols][4 * a + f / kCols] * inv);
          }
          u32x4* dst = reinterpret_cast<u32x4*>(p.out + row * D + (8 * a + 4 * half) * kCols);
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i) dst[i] = u32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
        }
        if (p.lse && half == 0) p.lse[row] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
      } else {
        const int64_t part = ((int64_t)worker * 2 + (first_part ? 1 : 0)) * p.tile_rows + r;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          f32x4* dst = reinterpret_cast<f32x4*>(p.part_o + part * D + (8 * a + 4 * half) * kCols);
#pragma unroll
          for (int i = 0; i < kCols; ++i) {
            f32x4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = rows.o[t][(4 * i + j) % kCols][4 * a + (4 * i + j) / kCols];
            dst[i] = x;
          }
        }
        if (half == 0) p.part_ml[part] = make_float4(m, l, rounded, 0.f);
      }
    }
    if (last_part && !first_part) {
      const int from = piece.owner(piece.tile_begin);
      note = ChunkNote{from, worker - from + 1, s.first + token0, head0, heads, n_rows};
    }
    piece.at = piece.tile_begin = tile_end;
    if (++piece.tile >= s.tiles && piece.at < piece.end) {
      piece.tile = 0;
      do {
        if (++piece.b == p.batch) {
          piece.b = 0;
          ++piece.member;
        }
      } while (Seq::of<true>(p, piece.b).tiles == 0);
    }
  }
  if (p.notes && tid == 0) p.notes[worker] = note;
}

// Joins the parts of the tiles that were cut; a tile's note is its last worker's.
// Part 0 is in slot 1 of the first worker, the others in slots 0 of those after it.
template <int D, bool F16>
__global__ void __launch_bounds__(256)
chunk_join_kernel(const ChunkParams p) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes;
  const ChunkNote note = p.notes[blockIdx.x];
  const int r = blockIdx.y * kRows + threadIdx.x / kLanes, i = threadIdx.x % kLanes;
  if (note.parts == 0 || r >= note.rows) return;
  float m = kLowest, l = 0.f, rounded = 0.f;
  f32x4 x{0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < note.parts; j0 += 4) {
    float4 ml[4];
    f32x4 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = min(j0 + u, note.parts - 1);
      const int64_t at = ((int64_t)(note.worker + j) * 2 + (j == 0)) * p.tile_rows + r;
      ml[u] = p.part_ml[at];
      y[u] = reinterpret_cast<const f32x4*>(p.part_o + at * D)[i];
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = fmaxf(top, ml[u].x);
    const float f = __builtin_amdgcn_exp2f(m - top);
    m = top;
    l *= f;
    rounded *= f;
    x *= f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j0 + u < note.parts) {
        const float g = __builtin_amdgcn_exp2f(ml[u].x - m);
        l += ml[u].y * g;
        rounded += ml[u].z * g;
        x += y[u] * g;
      }
    }
  }
  const int at = r / note.heads;
  const int64_t row = (int64_t)(note.token + at) * p.q_heads + note.head + (r - at * note.heads);
  const float inv = rounded == 0.f ? 0.f : 1.f / rounded;
  reinterpret_cast<u32x2*>(p.out + row * D)[i] = u32x2{pack<F16>(x[0] * inv, x[1] * inv), pack<F16>(x[2] * inv, x[3] * inv)};
  if (p.lse && i == 0) p.lse[row] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
}

template <int D, bool F16>
hipError_t launch(const ChunkParams& p, hipStream_t s) {
  chunk_kernel<D, F16><<<(uint32_t)((p.workers + 7) / 8 * 8), kThreads, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.notes) return e;
  constexpr int kRows = 256 / (D / 4);
  chunk_join_kernel<D, F16><<<dim3(p.workers, (p.tile_rows + kRows - 1) / kRows), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk(int d, int f16, const ChunkParams& p, hipStream_t s) {
  if (d == 128) return f16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return f16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

}  // namespace mqa
