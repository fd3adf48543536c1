// Softmax attention of chunks of new tokens over a paged cache held in MXFP4
// (gfx950), and the kernel that joins split contexts.
//
//   out[r, :] = sum_j p[r, j] v[j, :],  p[r, :] = softmax_j(scale <q[r, :], k[j, :]>)
//
// over the keys j that row r, a (token, head) pair, sees.
//
// One pass over the cache with a running maximum and sum.  A tile is 256 rows of a
// sequence and KV head, 32 to each of a workgroup's eight waves; a step is 64 keys,
// which four waves load, convert and store to LDS as K, the other four as V, while all
// multiply the steps before (K two steps ahead in a ring of three, V one in a ring of
// two; one barrier a step).  Both products are computed transposed, so that nothing
// leaves the registers between them:
//
//   S^T[key, row] = K Q^T   A = 32 keys x 16 of D, B = 16 of D x 32 rows
//   O^T[d, row]  += V^T P^T A = 32 of D x 16 keys, B = 16 keys x 32 rows
//
// The order of the contracted index is free as long as A and B agree, so a lane's scores
// are its operand of the second product as they stand, and V is stored with the keys
// in that order.  e2m1 under its scale is exact in bf16 and, for the scales that
// occur (2^-22 .. 2^9), in fp16: K takes q's type, V fp16, in which a weight keeps 2^-12
// with one product, where bf16 took two.  At a step with other scales, or with NaN ones,
// a workgroup leaves the loop for one in bf16 with the weights in two parts, up to the end
// of the stretch (16384 keys at most).  That one takes 1.7 times as long (64 sequences as
// below with such a scale in every block 1.93 ms, with one in the middle of each 1.56),
// with D = 64 and fp16 queries 2.6 times.  The sum that a result is divided by is that of
// the rounded weights.
//
// What bounds it: the matrix cores and the vector ALU, and beyond them power.  A step is 32
// products (1024 cycles) a wave, two waves a SIMD, and 32 exponentials, scalings, sums
// and roundings a lane.  On this chip both go on at the same time when they come from
// one wave in turn, so each half of a step (32 keys) is finished, weights and second
// product, between the products of the scores that follow it; the order is fixed
// by hand.  With everything in bf16 and one part after the other 4096 query tokens over
// 65536 keys took 13.1 ms.  They take 8.4 now, 1.02 PFLOP/s (6.7 ms on a cache of
// zeros: the rest is the clock, which goes down to 2.0 GHz under random data; matrix
// cores busy 48%); 64 sequences of 1024..32768 keys, 32 query tokens of 64 heads,
// 1.14 ms, 0.99 PFLOP/s.  Short prompts pay for tiles' beginnings and ends: 33 of
// 1..1900 tokens take 480 us, of which about 7 us a tile (16 a workgroup, of ten steps)
// are the latencies of its first loads and its last stores.
//
// Work is divided evenly: the steps of all tiles, and a few for what a tile costs
// besides, lie end to end, and each of 256 workers takes as many.  A tile that a border
// cuts is left in parts, that a second kernel joins (15 us for 256 of them).  A tile
// costs its steps whatever rows it has: single new tokens beside a long chunk are better
// left to paged_attention (63 sequences of 1024..32768 keys, 64 heads on one KV head: 142 us
// here, 78 there).
#include <hip/hip_runtime.h>

#include <cstddef>
#include <type_traits>

#include "chunk_split.hpp"
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
constexpr int kKeys = kChunkKeys;            // of a step
constexpr int kStage = 16384;                // keys whose places LDS holds at a time
constexpr int kTileSteps = kChunkTileSteps;  // that beginning and ending a tile counts for
constexpr uint32_t kLastScale = 252;         // bytes above could overflow fp32: they count as NaN
// Scale bytes (2^-22 .. 2^9) whose steps are worked on in fp16.  Every e2m1 value
// under 2^-23 .. 2^13 is exact there; large ones are left out for what the weights'
// own end costs, see kRoom.
constexpr uint32_t kHalfLow = 105, kHalfHigh = 136;
// The running maximum is set kRoom octaves below the largest score, and follows a
// new one when a lane's weights of a step come to more than kMost (so that none is
// beyond fp16): most steps rescale nothing, and no step looks for its largest score.
// The row's largest weight is then 2^kRoom at least, and half a step of fp16's least
// subnormal is 2^-33 of it at most.  The unnormalised sums of n keys stay within
// n * 2^16 times the largest value.
constexpr float kRoom = 8.f, kMost = 65000.f;
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
struct Seq : ChunkSeq {
  // UNIFORM: b is the same in every lane, and everything stays in scalar registers.
  template <bool UNIFORM>
  __device__ __forceinline__ static Seq of(const ChunkParams& p, int b) {
    const auto get = [](int x) { return UNIFORM ? __builtin_amdgcn_readfirstlane(x) : x; };
    int64_t lo, hi;
    if (p.offsets) {
      lo = get(p.offsets[b]);
      hi = get(p.offsets[b + 1]);
    } else {
      lo = (int64_t)b * p.next_n;
      hi = lo + p.next_n;
    }
    Seq s;
    s.set(p, get(p.ctx[b]), lo, hi);
    return s;
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
struct Piece : ChunkBorders {
  int64_t begin, end, at;
  int64_t tile_begin;      // where the tile at `at` begins
  int member, b, tile;

  // One tile for each worker: no need to find out which.
  __device__ __forceinline__ bool take(const ChunkParams& p, int worker) {
    const int row = worker / p.direct;
    tile = worker - row * p.direct;
    member = row / p.batch;
    b = row - member * p.batch;
    begin = at = tile_begin = 0;
    end = 1;
    return tile < Seq::of<true>(p, b).tiles;
  }

  __device__ __forceinline__ bool find(const ChunkParams& p, int worker, int64_t* sums, int64_t* found) {
    int64_t all = 0, part, mine = 0, before = 0;
    const auto weigh = [&](int i) {
      if (i >= p.batch) return (int64_t)0;
      const Seq s = Seq::of<false>(p, i);
      return s.before(p, s.tiles);
    };
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      mine = weigh(b0 + threadIdx.x);
      before = scan(mine, sums, part);
      all += part;
    }
    all = uniform(all);
    divide(all * p.members, p.workers, p.least);
    begin = at = border(worker);
    end = border(worker + 1);
    if (worker >= workers || begin >= end) return false;
    member = (int)(begin / all);
    const int64_t want = begin - member * all;
    int64_t base = 0;
    for (int b0 = 0; base <= want; b0 += kThreads) {
      // (up to 512 sequences: as they are)
      if (p.batch > kThreads) {
        mine = weigh(b0 + threadIdx.x);
        before = scan(mine, sums, part);
      }
      const int64_t here = base + before;
      if (here <= want && want < here + mine) {
        found[0] = b0 + threadIdx.x;
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
  static constexpr int kKeyBytes = kKeys * kKeyPitch, kValBytes = D * kValPitch;
  // K's products are a step ahead of V's, and start before other waves' last use
  // of the step before: three buffers of K, two of V.
  char k[3][kKeyBytes];
  char v[2][kValBytes];
  int flags[4][2];         // [step][V, K]: the piece's step, if it has unusual scales
  uint8_t nan_marks[2][kKeys][4];
};

// Global memory, and a wave-uniform address kept in scalar registers, so that
// the lanes' loads from it take a 32-bit offset each instead of a 64-bit sum.
typedef const __attribute__((address_space(1))) uint8_t* Bytes;
template <class T>
__device__ __forceinline__ T load_from(Bytes p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) T*>(p);
}
__device__ __forceinline__ Bytes scalar(Bytes p) {
  asm("" : "+s"(p));
  return p;
}

__device__ __forceinline__ uint32_t lanes(uint32_t offset) {
  asm("" : "+v"(offset));
  return offset;
}

// What a thread loads of a step.  The first half of the workgroup takes D/8 bytes
// of codes of a key each and their scale; the second D/32 bytes of V's codes of four
// keys and their scales.  A wave's keys are 16 in a row.
//
// Whole words are loaded, and what a thread needs of them is taken out when they
// have arrived: of narrower loads the compiler cut the upper bits off at once,
// and waited for them.
struct Raw {
  u32x4 codes;
  uint32_t scales[4];
  uint32_t first;          // block of the wave's 16 keys (wave-uniform)
};

// The second half's keys and columns: 16 lanes in a row write all banks.
__device__ __forceinline__ int value_quad(int tid) { return (tid & 3) | (tid >> 6 & 3) << 2; }
__device__ __forceinline__ int value_column(int tid) { return tid >> 2 & 15; }

template <int D, bool KEYS>
struct Loader {
  Bytes codes, scales;
  uint32_t code_at, scale_at;      // the lane's offsets from its 16 keys' first block
  uint32_t key_blocks;             // blocks (of 32 elements) from one key of the pool to the next

  __device__ __forceinline__ Loader(const ChunkParams& p, int tid)
      : codes((Bytes)(KEYS ? p.k : p.v)), scales((Bytes)(KEYS ? p.k_sf : p.v_sf)), key_blocks(p.kv_heads * (D / 32)) {
    const uint32_t key = KEYS ? tid >> 2 & 15 : (tid & 3) * 4, c = KEYS ? tid & 3 : value_column(tid);
    code_at = key * key_blocks * 16 + c * (KEYS ? D / 8 : D / 32);
    scale_at = key * key_blocks + c * (KEYS ? D / 4 : D / 16) / 32;
  }
  // (pools are whole words, the words of the heads' scales in it whatever the head)
  __device__ __forceinline__ void load(Raw& r, uint32_t first) const {
    r.first = first;
    const Bytes from = scalar(codes + ((uint64_t)first << 4));
    if constexpr (KEYS) {
      if constexpr (D == 128) {
        r.codes = load_from<u32x4>(from + lanes(code_at));
      } else {
        const u32x2 x = load_from<u32x2>(from + lanes(code_at));
        r.codes = u32x4{x[0], x[1], 0u, 0u};
      }
      r.scales[0] = load_from<uint32_t>(word_of(first));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Bytes at = scalar(from + i * key_blocks * 16);
        r.codes[i] = load_from<uint32_t>(at + lanes(code_at & ~3u));
        r.scales[i] = load_from<uint32_t>(word_of(first + i * key_blocks));
      }
    }
  }
  // Of what has arrived: the thread's codes lowest, its scale bytes alone.
  __device__ __forceinline__ void take(Raw& r) const {
    if constexpr (KEYS) {
      r.scales[0] = r.scales[0] >> byte_at(r.first) & 0xffu;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 64) r.codes[i] >>= (code_at & 2) * 8;
        r.scales[i] = r.scales[i] >> byte_at(r.first + i * key_blocks) & 0xffu;
      }
    }
  }
  // The word of the scales of block `first` + scale_at; where its byte is in it.  With
  // D = 128 a head's four scales are a word.
  __device__ __forceinline__ Bytes word_of(uint32_t first) const {
    if constexpr (D == 128) return scalar(scales + first) + lanes(scale_at & ~3u);
    return scalar(scales + (first & ~3u)) + lanes((first & 3u) + scale_at & ~3u);
  }
  __device__ __forceinline__ uint32_t byte_at(uint32_t first) const {
    return ((D == 128 ? 0 : first & 3u) + scale_at & 3u) * 8;
  }
};

// Where nothing is stored, behind the n keys of the context from the step's first
// on, the scales may be anything: they are read as finite.
template <bool KEYS>
__device__ __forceinline__ void check_context(Raw& r, int tid, int n) {
  if constexpr (KEYS) {
    r.scales[0] = (tid >> 2) < n ? r.scales[0] : 127u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.scales[i] = value_quad(tid) * 4 + i < n ? r.scales[i] : 127u;
  }
}

// K as rows of D (KEYS), or V transposed, into its LDS: part SEL of D/32.
template <int D, bool KEYS, bool HALF, int SEL>
__device__ __forceinline__ void put_part(const Raw& r, int tid, char* lds) {
  if constexpr (KEYS) {
    // (half of the lanes the other way round: 8 in a row write all banks)
    const int c = tid & 3, turn = D == 128 ? c & 2 : 0;
    char* dst = lds + (tid >> 2) * Stage<D>::kKeyPitch + c * (D / 2) + (SEL ^ turn) * 16;
    uint32_t word = r.codes[SEL];
    if constexpr (D == 128) word = turn ? r.codes[SEL ^ 2] : word;
    *reinterpret_cast<u32x4*>(dst) = cvt_eight<HALF>(word, scale_of(r.scales[0]));
  } else {
    // element e of the thread's D/16 is row e % (D/32) * 32 + 2 c + e / (D/32); four
    // keys are one half of what a lane multiplies of 16
    constexpr int kCols = D / 32;
    const int quad = value_quad(tid), c = value_column(tid);
    char* dst = lds + 2 * c * Stage<D>::kValPitch + (quad >> 2) * 32 +
                (quad & 1) * 16 + (quad >> 1 & 1) * 8;
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = r.codes[i];
      x[i] = cvt_pair<HALF, SEL>(word, scale_of(r.scales[i]));
    }
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const int e = 2 * SEL + odd, at = e % kCols * 32 + e / kCols;
      const uint32_t pick = odd ? 0x07060302u : 0x05040100u;
      *reinterpret_cast<u32x2*>(dst + at * Stage<D>::kValPitch) =
          u32x2{__builtin_amdgcn_perm(x[1], x[0], pick), __builtin_amdgcn_perm(x[3], x[2], pick)};
    }
  }
}

template <int D, bool KEYS, bool HALF>
__device__ __forceinline__ void put(const Raw& r, int tid, char* lds) {
  put_part<D, KEYS, HALF, 0>(r, tid, lds);
  put_part<D, KEYS, HALF, 1>(r, tid, lds);
  if constexpr (D == 128) {
    put_part<D, KEYS, HALF, 2>(r, tid, lds);
    put_part<D, KEYS, HALF, 3>(r, tid, lds);
  }
}

// Some scale is outside what the fp16 (or, for bf16 queries, K's bf16) products take.
template <bool KEYS, bool F16>
__device__ __forceinline__ bool wide_scales(const Raw& r) {
  static_assert(kHalfHigh - kHalfLow == 31, "32 scales: the offsets' bits can be joined");
  const auto off = [&](int i) { return r.scales[i] - kHalfLow; };
  if constexpr (KEYS) return F16 ? off(0) > 31 : r.scales[0] > kLastScale;
  return (off(0) | off(1) | off(2) | off(3)) > 31;
}

// ---------------------------------------------------------------------------
// A wave's 32 rows
// ---------------------------------------------------------------------------

template <int D, bool F16>
struct Rows {
  static constexpr int kSteps = D / 16, kCols = D / 32;
  static constexpr int kKeyOps = kSteps, kValOps = 2 * kCols;   // products of 32 keys
  static constexpr int kAhead = 4;           // operands are read that many products before their use
  u32x4 q[kSteps];         // row l % 32, elements 16 st + 8 (l / 32) ..
  f32x16 o[kCols];         // row l % 32; element kCols * m + col, m = i % 4 + 8 (i / 4) + 4 (l / 32)
  float m, l;              // running maximum (log2), the lane's part of the sum of weights
  float r;                 // and of the sum of the rounded ones
  int seen;
  uint32_t nan_blocks;

  __device__ __forceinline__ void clear() {
    m = kLowest;
    l = r = 0.f;
    nan_blocks = 0;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[c][i] = 0.f;
  }

  // Operands of half a step: 32 keys' rows of K, V's columns of them.
  // (at: the lane's first, as an offset into the stage that the compiler takes as it is)
  __device__ __forceinline__ static uint32_t key_at(uint32_t buffer, int lane) {
    return lanes(buffer + (lane & 31) * Stage<D>::kKeyPitch + (lane >> 5) * 16);
  }
  __device__ __forceinline__ static uint32_t value_at(uint32_t buffer, int lane) {
    return lanes(buffer + (lane & 31) * Stage<D>::kValPitch + (lane >> 5) * 16);
  }
  __device__ __forceinline__ static u32x4 key_operand(const char* lds, uint32_t at, int n) {
    return *reinterpret_cast<const u32x4*>(lds + at + n * 32);
  }
  __device__ __forceinline__ static u32x4 value_operand(const char* lds, uint32_t at, int n) {
    return *reinterpret_cast<const u32x4*>(lds + at + n % kCols * 32 * Stage<D>::kValPitch + n / kCols * 32);
  }
  // A product must not overlap its operands.  The compiler was seen to let one with
  // a constant 0 to add to overlap them: they are used once more behind it.
  __device__ __forceinline__ static void keep(u32x4 a, u32x4 b) { asm volatile("" ::"v"(a), "v"(b)); }

  // The scores of 32 keys: key i % 4 + 8 (i / 4) + 4 (l / 32) of row l % 32.
  __device__ __forceinline__ void multiply(f32x16& x, const char* lds, uint32_t keys, int lane) const {
    const uint32_t k = key_at(keys, lane);
    u32x4 a[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) a[n] = key_operand(lds, k, n);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < kKeyOps; ++n) {
      x = mma<F16>(a[n % kAhead], q[n], x);
      __builtin_amdgcn_sched_barrier(0);
      if (n == 0) keep(a[0], q[0]);
      if (n + kAhead < kKeyOps) a[n % kAhead] = key_operand(lds, k, n + kAhead);
    }
    // The compiler was seen to read a product's result right behind a branch,
    // before it is there; the products end here.
    asm volatile("s_nop 7\n\ts_nop 7" : "+v"(x));
  }

  // Keys that a row does not see leave its scores.
  __device__ __forceinline__ void mask(f32x16& x, int lane, int key0) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = key0 + (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5);
      x[i] = key < seen ? x[i] : -__builtin_inff();
    }
  }

  // The running maximum of rows with `over` in a lane follows their largest score
  // (others keep theirs: a row's result does not depend on its neighbours).
  __device__ __forceinline__ void settle(float best, bool over, float c2) {
    best = fmaxf(best, __shfl_xor(best, 32)) * c2;
    over |= (bool)__shfl_xor((int)over, 32);
    const float next = over ? fmaxf(m, best - kRoom) : m;
    const float f = __builtin_amdgcn_exp2f(m - next);
    m = next;
    l *= f;
    r *= f;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[c][i] *= f;
  }

  // Rounded weights of 32 keys, two in a word, with what the lane's come to.
  struct Weights {
    u32x4 w[2];
    float sum, rounded;
    __device__ __forceinline__ void clear() { sum = rounded = 0.f; }
    __device__ __forceinline__ void add(int pair, float x, float y) {
      const uint32_t word = pack_f16(x, y);
      w[pair / 4][pair % 4] = word;
      sum += x;
      sum += y;
      rounded = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, word), f16x2{(_Float16)1.f, (_Float16)1.f}, rounded, false);
    }
    // what has been added is there, not put off to where it is used
    __device__ __forceinline__ void settle(int pair) {
      uint32_t word = w[pair / 4][pair % 4];
      asm volatile("" : "+v"(word), "+v"(rounded));
      w[pair / 4][pair % 4] = word;
    }
  };
  __device__ __forceinline__ void form(const f32x16& x, Weights& w, float c2) const {
    w.clear();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w.add(i, __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * i], c2, -m)), __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * i + 1], c2, -m)));
  }
  // Weights that are too large are formed anew.
  __device__ __forceinline__ void check(f32x16& x, Weights& w, float c2) {
    if (__builtin_expect(__any(w.sum > kMost), 0)) {
      asm volatile("" : "+v"(x));            // (rare: nothing of it belongs before the branch)
      float best = x[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) best = fmaxf(best, x[i]);
      settle(best, w.sum > kMost, c2);
      form(x, w, c2);
    }
    l += w.sum;
    r += w.rounded;
  }

  // The weights of the 32 keys of scores x and their V, with the products of the next
  // 32 keys between the weights, and other work (0 .. kValOps - 1) between V's: the
  // matrix cores and the vector ALU work side by side.
  // a: the first operands of `keys`, and then of `then`.
  template <class Work>
  __device__ __forceinline__ void finish_and_multiply(f32x16& x, f32x16& next, u32x4 (&a)[kAhead], const char* lds, uint32_t values,
                                                      uint32_t keys, uint32_t then, int lane, float c2, const Work& work) {
    const uint32_t k = key_at(keys, lane), v = value_at(values, lane), after = key_at(then, lane);
    Weights w;
    w.clear();
#pragma unroll
    for (int i = 0; i < 16; ++i) next[i] = 0.f;
    __builtin_amdgcn_sched_barrier(0);
    // A pair of weights is scaled and shifted beside one product, its exponentials
    // are taken beside the next, and it is rounded beside the one after that.
    constexpr int kEach = 8 / kKeyOps;       // pairs beside a product
    float f[kEach][2], e[kEach][2];
#pragma unroll
    for (int n = 0; n < kKeyOps + 2; ++n) {
      if (n < kKeyOps) {
        next = mma<F16>(a[n % kAhead], q[n], next);
        __builtin_amdgcn_sched_barrier(0);
        if (n == 0) keep(a[0], q[0]);
        if (n + kAhead < kKeyOps)
          a[n % kAhead] = key_operand(lds, k, n + kAhead);
        else
          a[n % kAhead] = value_operand(lds, v, n + kAhead - kKeyOps);
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (n >= 2) {
          w.add((n - 2) * kEach + j, e[j][0], e[j][1]);
          w.settle((n - 2) * kEach + j);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (n >= 1 && n <= kKeyOps) e[j][y] = __builtin_amdgcn_exp2f(f[j][y]);
          if (n < kKeyOps) f[j][y] = __builtin_fmaf(x[2 * (n * kEach + j) + y], c2, -m);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    static_assert(kKeyOps % kAhead == 0 && kValOps % kAhead == 0, "operands follow each other in turn");
    check(x, w, c2);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < kValOps; ++n) {
      o[n % kCols] = mma<true>(a[n % kAhead], w.w[n / kCols], o[n % kCols]);
      __builtin_amdgcn_sched_barrier(0);
      if (n + kAhead < kValOps)
        a[n % kAhead] = value_operand(lds, v, n + kAhead);
      else
        a[n % kAhead] = key_operand(lds, after, n + kAhead - kValOps);
      work(n);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // A step with unusual scales: LDS holds bf16, weights are split into two parts,
  // and fp16 queries as well.
  __device__ __forceinline__ void wide_step(const char* lds, uint32_t keys, uint32_t values, int key0, float c2) {
#pragma nounroll
    for (int half_step = 0; half_step < 2; ++half_step) {
      const int lane = here_only(threadIdx.x & 63);
      const uint32_t k = key_at(keys + half_step * 32 * Stage<D>::kKeyPitch, lane), v = value_at(values + half_step * 64, lane);
      f32x16 s;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
      asm volatile("" : "+v"(s));            // (zeros in registers: see keep)
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x4 a = key_operand(lds, k, st);
        if constexpr (F16) {
          // two exact parts; an infinity stays in the first alone
          u32x4 hi, lo;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f16x2 x = __builtin_bit_cast(f16x2, here_only(q[st][i]));
            const float y = (float)x[0], z = (float)x[1];
            hi[i] = pack_bf16(y, z);
            const float ry = y - bf16_lo(hi[i]), rz = z - bf16_hi(hi[i]);
            lo[i] = pack_bf16(__builtin_isfinite(y) ? ry : 0.f, __builtin_isfinite(z) ? rz : 0.f);
          }
          s = mma<false>(a, hi, s);
          s = mma<false>(a, lo, s);
        } else {
          s = mma<false>(a, q[st], s);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      asm volatile("s_nop 7\n\ts_nop 7" : "+v"(s));
      float best = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = key0 + half_step * 32 + (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5);
        s[i] = key < seen ? s[i] : -__builtin_inff();
        best = fmaxf(best, s[i]);
      }
      const bool over = __builtin_fmaf(best, c2, -m) > kRoom;
      if (__any(over)) settle(best, over, c2);
      u32x4 w[2][2];                         // [16 keys][part]
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i], c2, -m));
        const float z = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + 1], c2, -m));
        const uint32_t hi = pack_bf16(y, z);
        w[i / 4][0][i % 4] = hi;
        w[i / 4][1][i % 4] = pack_bf16(y - bf16_lo(hi), z - bf16_hi(hi));
        l += y + z;
        r += y + z;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const u32x4 a = value_operand(lds, v, n * kCols + c);
#pragma unroll
          for (int part = 0; part < 2; ++part) o[c] = mma<false>(a, w[n][part], o[c]);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  }
};

// The steps of a stretch, for a wave of the half that loads K (KEYS) or V.  While 32
// keys' weights are formed and multiplied with V, the next ones' scores are
// computed; K is put into LDS two steps ahead, V one.
template <bool KEYS, int D, bool F16>
__device__ __forceinline__ void walk(const ChunkParams& p, Rows<D, F16>& rows, Stage<D>& stage, const uint32_t* places,
                                     int walked, int stage0, int steps, int least, int keys_left, bool negate) {
  constexpr int kHalfKeys = 32 * Stage<D>::kKeyPitch, kHalfVals = 64;   // bytes to a step's second half
  const int tid = threadIdx.x & (kThreads / 2 - 1);
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr bool kHalf = KEYS ? F16 : true;
  constexpr int kLead = KEYS ? 2 : 1;        // steps that this half is ahead
  const float c2 = p.c2;
  const Loader<D, KEYS> loader(p, tid);
  char* const lds = reinterpret_cast<char*>(&stage);
  Raw raw, ahead;                            // the step to store next, and the one after it
  // first blocks of the wave's keys, of 64 steps from `held` on, one in each lane
  uint32_t held_places = 0;
  int held = -64;
  const auto fetch = [&](Raw& r, int i) {
    i = min(i, steps - 1);                   // (past the last step, the last again)
    if (i >= held + 64) {
      held = i & ~63;
      held_places = places[min(held + lane, steps - 1) * 4 + wave];
    }
    loader.load(r, __builtin_amdgcn_readlane(held_places, i & 63));
  };
  const auto keys = [&](int i) { return (uint32_t)offsetof(Stage<D>, k) + i % 3 * Stage<D>::kKeyBytes; };
  const auto values = [&](int i) { return (uint32_t)offsetof(Stage<D>, v) + (i & 1) * Stage<D>::kValBytes; };
  const auto target = [&](int i) { return lds + (KEYS ? keys(i) : values(i)); };
  // step i is in r
  const auto check_step = [&](Raw& r, int i) {
    loader.take(r);
    if (keys_left - i * kKeys < kKeys) check_context<KEYS>(r, here_only(tid), keys_left - i * kKeys);
    if (__builtin_expect(__any(wide_scales<KEYS, F16>(r)), 0)) stage.flags[i & 3][KEYS] = walked + i;
  };
  // to the next step: it is marked two barriers ahead of its products
  const auto advance = [&](int i) {
    raw = ahead;
    check_step(raw, i + kLead + 1);
    fetch(ahead, i + kLead + 2);
  };
  const auto narrow = [&](int i) {
    const int v = __builtin_amdgcn_readfirstlane(stage.flags[i & 3][0]), k = __builtin_amdgcn_readfirstlane(stage.flags[i & 3][1]);
    return v != walked + i && k != walked + i;
  };

  fetch(raw, 0);
  fetch(ahead, 1);
  check_step(raw, 0);
  put<D, KEYS, kHalf>(raw, here_only(tid), target(0));
  if constexpr (KEYS) {
    advance(-2);
    put<D, KEYS, kHalf>(raw, here_only(tid), target(1));    // (a step that is not there: never used)
  }
  advance(-1);
  __syncthreads();
  f32x16 x, y;                               // scores of a step's halves
  // (where the queries are there anyway; not a selection, which would wait for them
  // where they are loaded)
  if (negate) {
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      asm volatile("" : "+v"(rows.q[st]));
      rows.q[st] ^= 0x80008000u;
    }
  }
  rows.multiply(x, lds, keys(0), lane);
  rows.mask(x, here_only(lane), stage0);
  const int clear = max(least - stage0, 0) / kKeys;      // steps that all rows see whole
  int i = 0;
  bool good = narrow(0);
  u32x4 a[Rows<D, F16>::kAhead];
#pragma unroll
  for (int n = 0; n < Rows<D, F16>::kAhead; ++n)
    a[n] = Rows<D, F16>::key_operand(lds, Rows<D, F16>::key_at(keys(0) + kHalfKeys, lane), n);
  // (the last step's second half is multiplied by keys of no step, for nothing)
#pragma nounroll
  for (; i < steps && good; ++i) {
    char* const into = target(i + kLead);
    const int next_v = stage.flags[i + 1 & 3][0], next_k = stage.flags[i + 1 & 3][1];
    rows.finish_and_multiply(x, y, a, lds, values(i), keys(i) + kHalfKeys, keys(i + 1), lane, c2, [&](int n) {
      if (n == 1) put_part<D, KEYS, kHalf, 0>(raw, tid, into);
      if constexpr (D == 128)
        if (n == 5) put_part<D, KEYS, kHalf, 1>(raw, tid, into);
    });
    if (__builtin_expect(i >= clear, 0)) rows.mask(y, here_only(lane), stage0 + i * kKeys + 32);
    rows.finish_and_multiply(y, x, a, lds, values(i) + kHalfVals, keys(i + 1), keys(i + 1) + kHalfKeys, lane, c2, [&](int n) {
      if (n == 1) put_part<D, KEYS, kHalf, D / 64>(raw, tid, into);
      if constexpr (D == 128)
        if (n == 5) put_part<D, KEYS, kHalf, 3>(raw, tid, into);
    });
    if (__builtin_expect(i + 1 >= clear, 0)) rows.mask(x, here_only(lane), stage0 + (i + 1) * kKeys);
    advance(i);
    good = __builtin_amdgcn_readfirstlane(next_v) != walked + i + 1 && __builtin_amdgcn_readfirstlane(next_k) != walked + i + 1;
    __syncthreads();
  }
  if (__builtin_expect(i == steps, 1)) return;
  // from a step with unusual scales on, in bf16, NaN scales apart
  held = -64;                                // (the loads were ahead, maybe in the next 64 steps)
  fetch(raw, i);
#pragma nounroll
  for (; i < steps; ++i) {
    const int me = here_only(tid);
    loader.take(raw);
    check_context<KEYS>(raw, me, keys_left - i * kKeys);
    if constexpr (KEYS) {
      if (raw.scales[0] > kLastScale) raw.scales[0] = 255;
    } else {
      const int c = value_column(me), b = c * (D / 16) / 32;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool bad = raw.scales[j] > kLastScale;
        if (c % (512 / D) == 0) stage.nan_marks[i & 1][value_quad(me) * 4 + j][b] = bad;
        raw.scales[j] = bad ? 0u : raw.scales[j];
      }
    }
    __syncthreads();                         // the stage's last use is over
    put<D, KEYS, false>(raw, me, target(i));
    __syncthreads();
    fetch(raw, i + 1);
    const int key0 = stage0 + i * kKeys;
    uint32_t marks = 0;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) marks |= (uint32_t)stage.nan_marks[i & 1][me & 63][b] << b;
    if (__builtin_expect(__any(marks != 0), 0))
#pragma nounroll
      for (int j = 0; j < kKeys; ++j) {
        const uint32_t word = __shfl(marks, j);
        if (key0 + j < rows.seen) rows.nan_blocks |= word;
      }
    rows.wide_step(lds, keys(i), values(i), key0, c2);
  }
  __syncthreads();                           // (as at the end of other steps)
}

// A worker's piece, for a wave of the half that loads K (KEYS) or V.
template <bool KEYS, int D, bool F16>
__device__ __forceinline__ void work(const ChunkParams& p, Piece piece, int worker, Stage<D>& stage, uint32_t* places) {
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Rows<D, F16> rows;
  ChunkNote note{};
  Seq s = Seq::of<true>(p, piece.b);
  // what `places` holds: keys [held_from, held_until) of a sequence and KV head
  int held_b = -1, held_head = -1, held_from = 0, held_until = 0;
  int walked = 0;                            // steps of this piece so far
  while (piece.at < piece.end) {
    const int kv_head = piece.member / p.head_groups;
    const int head0 = kv_head * p.group + piece.member % p.head_groups * p.tile_heads;
    const int heads = min(p.tile_heads, (kv_head + 1) * p.group - head0);
    const int token0 = piece.tile * p.tile_tokens;                     // of the sequence
    const int tokens = min(p.tile_tokens, s.n - token0);
    const int n_rows = tokens * heads;
    const int tile_seen = s.tile_seen(p, piece.tile);
    const int64_t tile_end = piece.tile_begin + s.steps(p, piece.tile);
    // steps [begin, end) of this part, past the kTileSteps that a tile begins with
    const auto step_at = [&](int64_t at) { return (int)max(at - piece.tile_begin - kTileSteps, (int64_t)0); };
    const int begin = p.whole ? 0 : step_at(piece.at) * kKeys;
    const int end = p.whole ? tile_seen : (int)min((int64_t)tile_seen, (int64_t)step_at(min(tile_end, piece.end)) * kKeys);
    const int wave_row = wave * 32;
    const int least = s.seen(token0);        // keys that all rows see
    rows.clear();
    {
      // lanes past the last row repeat it; their results are dropped
      const int r = min(wave_row + (lane & 31), n_rows - 1);
      const int at = r / heads;
      rows.seen = s.seen(token0 + at);
      const uint16_t* src = p.q + (int64_t)(s.first + token0 + at) * p.q_stride + (head0 + r - at * heads) * D + half * 8;
#pragma unroll
      for (int st = 0; st < D / 16; ++st) rows.q[st] = *reinterpret_cast<const u32x4*>(src + st * 16);
    }
    const int32_t* table = p.bt + (int64_t)piece.b * p.bt_stride;
    const uint32_t key_blocks = p.kv_heads * (D / 32);
    for (int stage0 = begin; stage0 < end;) {
      const int window = stage0 & -kStage, stage_end = min(end, window + kStage);
      const int steps = (stage_end - stage0 + kKeys - 1) / kKeys;
      // (every wave is past the last step's barrier: nothing reads `places` or the stage)
      if (held_b != piece.b || held_head != kv_head || held_from < window || held_from > stage0 || held_until < stage0) {
        held_b = piece.b;
        held_head = kv_head;
        held_from = held_until = stage0;
      }
      if (held_until < stage0 + steps * kKeys) {
        // (at once for the sequence's later tiles)
        const int until = max(stage0 + steps * kKeys, min(s.cap, window + kStage) & -kKeys);
        for (int key = held_until + tid * 16; key < until; key += kThreads * 16) {
          const int id = min(max(table[min(key, s.cap - 1) >> p.bs_shift], 0), p.num_blocks - 1);
          const uint32_t slot = ((uint32_t)id << p.bs_shift) + (key & (1 << p.bs_shift) - 1);
          places[(key - window) / 16] = slot * key_blocks + kv_head * (D / 32);
        }
        held_until = until;
        __syncthreads();
      }
      walk<KEYS>(p, rows, stage, places + (stage0 - window) / 16, walked, stage0, steps, least, s.cap - stage0,
                 p.negate && stage0 == begin);
      walked += steps + 4;
      stage0 = stage_end;
    }

    const bool first_part = piece.at == piece.tile_begin, last_part = tile_end <= piece.end;
    {
      const float m = rows.m, l = rows.l + __shfl_xor(rows.l, 32);
      const float rounded = rows.r + __shfl_xor(rows.r, 32);
      const int r = here_only(wave_row + (lane & 31));
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (rows.nan_blocks >> ((i >> 2) * 8 * (D / 32) / 32) & 1) rows.o[c][i] = __builtin_nanf("");
      constexpr int kCols = D / 32;
      if (r >= n_rows) {
      } else if (first_part && last_part) {
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
            x[i] = pack<F16>(rows.o[e % kCols][4 * a + e / kCols] * inv, rows.o[f % kCols][4 * a + f / kCols] * inv);
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
            for (int j = 0; j < 4; ++j) x[j] = rows.o[(4 * i + j) % kCols][4 * a + (4 * i + j) / kCols];
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
          // (no tile is behind the last KV head, even if lengths change during the call)
          if (++piece.member == p.members) piece.end = piece.at;
        }
        s = Seq::of<true>(p, piece.b);
      } while (s.tiles == 0 && piece.at < piece.end);
    }
  }
  if (p.notes && tid == 0) p.notes[worker] = note;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2)
chunk_kernel(const ChunkParams p) {
  __shared__ __attribute__((aligned(16))) Stage<D> stage;
  __shared__ uint32_t places[kStage / 16];
  __shared__ int64_t sums[kWaves], found[2];

  const int tid = threadIdx.x;
  // neighbouring workers, which read the same keys, on one XCD
  const int worker = (blockIdx.x & 7) * ((p.workers + 7) / 8) + (blockIdx.x >> 3);
  if (tid < 8) stage.flags[tid >> 1][tid & 1] = -1;
  Piece piece;
  const bool any = worker < p.workers && (p.direct ? piece.take(p, worker) : piece.find(p, worker, sums, found));
  if (!any) {
    if (p.notes && tid == 0 && worker < p.workers) p.notes[worker].parts = 0;
    return;
  }
  if (__builtin_amdgcn_readfirstlane(tid >> 6) < kWaves / 2)
    work<true, D, F16>(p, piece, worker, stage, places);
  else
    work<false, D, F16>(p, piece, worker, stage, places);
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
