// The attention weight that every cached token has gathered (gfx950):
//
//   out[b, j] = before[b, j] + sum_r exp(scale <q[r, :], k[j, :]> - lse[r])
//
// over the rows r, (token, head) pairs of sequence b, that see key j.
//
// lse is known, so there is no maximum and no second product: an exponential of a
// score with its row's shift, and a sum over rows.  A wave holds 64 keys in registers as
// the product's B operand and takes the rows past them as A, 32 at a time; a result
// register is then 16 rows of one key, and the sum over rows stays in the lane.
// Queries keep their type; e2m1 under its scale is exact in it (fp16: from 2^-22 to 2^9;
// other scales' blocks are multiplied in bf16, with the query in two exact parts).
// Scores, weights and sums are fp32.
//
// Few rows (weights_kernel): the cache's bytes, D/2 + D/32 for a key and KV head.
// 32 sequences of 1024..32768 keys, 8 KV heads of 8 rows: 81 us, 3.6 TB/s; waves wait
// for memory 56% of the time.  Two items ahead instead of one, eight heads beside each
// other, or whole lines handed over through LDS measured the same.
// Many rows (weights_wide_kernel): matrix cores and vector ALU.  A tile of 32 rows x 64 keys
// is 16 products (512 cycles) and, a lane, 32 exponentials, shifts and additions
// (about 600), formed between the products of the tile that follows; two tiles of two
// waves of a SIMD take 2450 cycles.  64 sequences of 1024..32768 keys, 256 rows: 82 us,
// 0.86 PFLOP/s; 2048 rows of each of 8 KV heads past 32768 keys: 138 us, 0.99.
//
// Workers, two workgroups for each CU, share the blocks of 64 keys evenly by what
// they cost (Share); with a workgroup for each piece of a sequence instead, of 512
// keys or of 256, a third of the chip idled in the last round (gqa: 95 us).
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

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kFewResident = 2;              // workgroups for each CU, few rows
constexpr int kKeys = 64;                    // of a block: a wave's at a time
constexpr uint32_t kLastScale = 252;         // bytes above count as NaN
constexpr uint32_t kHalfLow = 105, kHalfHigh = 136;   // scale bytes under which e2m1 is exact in fp16
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
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
// x, as the compiler does not know it: what is computed from it is computed where it
// is used, not ahead of all loops and kept (out of registers) until then.
__device__ __forceinline__ int fresh(int x) {
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

// Sequence b's rows and what they see.
struct Seq {
  int64_t base;            // keys before its first new token (may be negative)
  int cap;                 // keys of the context
  int first, n;            // its new tokens in q
  int blocks;              // of 64 keys

  template <bool UNIFORM>
  __device__ __forceinline__ static Seq of(const WeightParams& p, int b) {
    const auto load = [](const int32_t* x) { return UNIFORM ? __builtin_amdgcn_readfirstlane(*x) : *x; };
    int64_t lo = (int64_t)b * p.next_n, hi = lo + p.next_n;
    if (p.offsets) {
      lo = load(p.offsets + b);
      hi = load(p.offsets + b + 1);
    }
    const int ctx = load(p.ctx + b);
    Seq s;
    s.cap = min(max(ctx, 0), p.max_ctx);
    const int64_t from = min(max(lo, (int64_t)0), (int64_t)p.tokens);
    const int64_t to = min(max(hi, from), (int64_t)p.tokens);
    s.base = (int64_t)ctx - (hi - lo) + (from - lo);
    s.first = (int)from;
    s.n = (int)(to - from);
    s.blocks = (s.cap + kKeys - 1) / kKeys;
    return s;
  }
  __device__ __forceinline__ int seen(int t) const {
    return (int)min(max(base + 1 + t, (int64_t)0), (int64_t)cap);
  }
  // sum over i < k of max(64 i - a, 0)
  __device__ __forceinline__ static int64_t ramp(int64_t k, int64_t a) {
    const int64_t j = a < 0 ? 0 : (a >> 6) + 1, m = max(k - j, (int64_t)0);
    return kKeys * (m * (2 * j + m - 1) / 2) - a * m;
  }
  // What the first k blocks cost: a block costs `fixed`, and 1 for each row that
  // sees its first key (the token at base + i sees the keys up to itself); the first one
  // `start` more, which is what a worker pays that goes on to the sequence.
  __device__ __forceinline__ int64_t cost(const WeightParams& p, int64_t k) const {
    return (k > 0 ? p.start : 0) + k * (p.fixed + (int64_t)n * p.group) - p.group * (ramp(k, base) - ramp(k, base + n));
  }
};

__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)x));
}

// A worker's share of the blocks of all sequences, laid end to end and cut where they
// cost the same: those that begin within [begin, end).
struct Share {
  int64_t begin, end, at;  // at: where sequence b begins
  int b;                   // the sequence that `begin` lies in
  Seq first;

  // Every thread; false: nothing.
  __device__ __forceinline__ bool find(const WeightParams& p, int worker) {
    __shared__ int64_t sums[kWaves], found;
    __shared__ Seq found_seq;
    __shared__ int found_b;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t mine = 0, before = 0, part = 0, all = 0;
    Seq s;
    const auto scan = [&](int b0) {
      mine = 0;
      if (b0 + (int)threadIdx.x < p.batch) {
        s = Seq::of<false>(p, b0 + threadIdx.x);
        mine = s.cost(p, s.blocks);
      }
      int64_t x = mine;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int64_t y = __shfl_up((long long)x, off);
        if (lane >= off) x += y;
      }
      __syncthreads();
      if (lane == 63) sums[wave] = x;
      __syncthreads();
      before = x - mine;
      part = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sums[w];
        part += sums[w];
      }
    };
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      scan(b0);
      all += part;
    }
    all = uniform(all);
    // (64 bits divided by a word's worth only where they are needed)
    const int64_t each = all >> 32 ? all / p.workers : (int64_t)((uint32_t)all / (uint32_t)p.workers);
    const int64_t more = all - each * p.workers;
    begin = each * worker + min((int64_t)worker, more);
    end = begin + each + (worker < more);
    if (begin >= end) return false;
    int64_t base = 0;
    for (int b0 = 0; base <= begin; b0 += kThreads) {
      if (p.batch > kThreads) scan(b0);      // (up to 256 sequences: as they are)
      const int64_t here = base + before;
      if (here <= begin && begin < here + mine) {
        found_b = b0 + threadIdx.x;
        found = here;
        found_seq = s;
      }
      base += part;
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(found_b);
    at = uniform(found);
    first.base = uniform(found_seq.base);
    first.cap = __builtin_amdgcn_readfirstlane(found_seq.cap);
    first.first = __builtin_amdgcn_readfirstlane(found_seq.first);
    first.n = __builtin_amdgcn_readfirstlane(found_seq.n);
    first.blocks = __builtin_amdgcn_readfirstlane(found_seq.blocks);
    return true;
  }
  // The first of s's blocks that begins at or behind `want` (searched for: 64
  // candidates at a time).
  __device__ __forceinline__ int first_block(const WeightParams& p, const Seq& s, int64_t want) const {
    if (want <= at) return 0;
    int lo = 0, hi = s.blocks;
    // (as long as every row sees a block's first key: a division)
    const int64_t each = p.fixed + (int64_t)s.n * p.group;
    if (each >> 31 == 0 && (want - at) >> 31 == 0) {
      const uint32_t i = want - at <= p.start ? 1 : ((uint32_t)(want - at - p.start) - 1) / (uint32_t)each + 1;
      if (i < (uint32_t)hi && (int64_t)i * kKeys <= s.base) return (int)i;
    }
    while (lo < hi) {
      const int step = (hi - lo + 63) / 64, i = lo + (threadIdx.x & 63) * step;
      const int n = __popcll(__ballot(i < hi && at + s.cost(p, i) < want));
      if (n == 0) return lo;
      hi = min(lo + n * step, hi);
      lo += (n - 1) * step + 1;
    }
    return lo;
  }
  // For each sequence of worker's share: work(b, sequence, first block, last).
  template <class Work>
  __device__ __forceinline__ void each(const WeightParams& p, int worker, Work work) {
    int from, to;
    const bool one = p.apart > 0;            // `apart` blocks of one sequence
    if (one) {
      const int of = p.workers / p.batch;
      b = worker / of;
      first = Seq::of<true>(p, b);
      from = (worker - b * of) * p.apart;
      to = min(from + p.apart, first.blocks);
    } else if (!find(p, worker)) {
      return;
    }
    Seq s = first;
    while (true) {
      if (!one) {
        from = first_block(p, s, begin);
        to = first_block(p, s, end);
      }
      if (from < to) work(b, s, from, to);
      if (one) break;
      at += s.cost(p, s.blocks);
      if (++b >= p.batch || at >= end) break;
      s = Seq::of<true>(p, b);
    }
  }
};

// Columns behind the contexts: this worker's.
__device__ __forceinline__ void clear_columns(const WeightParams& p, int worker) {
  const int each = max(p.workers / p.batch, 1);   // workers of a sequence
  for (int b = worker / each; b < p.batch; b += p.workers / each) {
    const int cap = min(max(__builtin_amdgcn_readfirstlane(p.ctx[b]), 0), p.max_ctx);
    for (int64_t j = cap + worker % each * kThreads + (int64_t)threadIdx.x; j < p.max_ctx; j += each * kThreads)
      p.out[b * p.out_stride + j] = 0.f;
  }
}

// BEFORE: x lacks what the key had.
template <bool BEFORE = true>
__device__ __forceinline__ void give(const WeightParams& p, int split, int b, int key, float x) {
  if (p.part)
    p.part[((int64_t)split * p.batch + b) * p.max_ctx + key] = x;
  else
    p.out[b * p.out_stride + key] = BEFORE && p.before ? p.before[b * p.before_stride + key] + x : x;
}

// A wave has 64 keys of a sequence and KV head in registers, and goes through the
// head's rows, 32 at a time:
//
//   S[row, key] = Q K^T   A = 32 rows x 16 of D, B = 16 of D x 32 keys
//
// A lane's results are 16 rows of one key, so what the rows give to a key is
// added up in one register, and rows that a tile lacks cost no exponentials.
// The order of the contracted index is free: half l / 32 of the lanes carries the
// D/2 elements from l / 32 * D/2 on.
constexpr int kChunk = 256;                  // rows whose places LDS holds at a time, for a wave
constexpr int kSpan = 16;                    // blocks that a wave takes before their sums are written

struct __attribute__((aligned(16))) Places {
  int64_t at[kChunk];      // first element of a row's query
  float shift[kChunk];     // -lse, in octaves; -inf for a row that gives nothing
  int seen[kChunk];        // keys that it sees
};

template <int D, bool F16>
struct Wave {
  static constexpr int kSteps = D / 16, kHalves = kKeys / 32;

  struct RawKeys {
    u32x4 x[kHalves][D / 64];
    uint32_t s[kHalves];     // the word that holds the scales
    uint32_t at;             // D = 64: bit h, whether half h's are its upper two bytes
  };
  u32x4 k[kHalves][kSteps];
  float sum[kHalves];

  // row: (slot, head) of the lane's key of each half
  __device__ __forceinline__ static void fetch_keys(RawKeys& r, const WeightParams& p, const uint32_t (&row)[kHalves]) {
    const int half = fresh(threadIdx.x & 63) >> 5;
    r.at = 0;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const uint8_t* src = p.k + (uint64_t)row[h] * (D / 2) + half * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) r.x[h][i] = *reinterpret_cast<const u32x4*>(src + i * 16);
      // (whole words: a narrower load would be waited for where it is issued)
      const uint64_t at = (uint64_t)row[h] * (D / 32);
      r.s[h] = *reinterpret_cast<const uint32_t*>(p.k_sf + (at & ~(uint64_t)3));
      if (D == 64) r.at |= (row[h] & 1) << h;
    }
  }

  // Whether some scale needs the wide products (fp16 queries).
  __device__ __forceinline__ bool put_keys(const RawKeys& r, uint32_t sign) {
    bool wide = false;
    const int half = fresh(threadIdx.x & 63) >> 5;
    float s[kHalves][D / 64];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const uint32_t bytes = D == 128 ? r.s[h] >> (16 * half) : r.s[h] >> (16 * (r.at >> h & 1) + 8 * half);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t byte = bytes >> (8 * i) & 0xffu;
        wide |= byte - kHalfLow > kHalfHigh - kHalfLow;
        s[h][i] = scale_of(byte > kLastScale ? 255u : byte);
      }
    }
    wide = F16 && __any(wide);
    if (F16 && !wide)
      convert<true>(r, s, sign);
    else
      convert<false>(r, s, sign);
    return wide;
  }
  template <bool HALF>
  __device__ __forceinline__ void convert(const RawKeys& r, const float (&s)[kHalves][D / 64], uint32_t sign) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const uint32_t word = r.x[h][st / 4][st % 4];
        k[h][st] = cvt_eight<HALF>(word ^ sign, s[h][st / 4]);
      }
  }
  // The keys' sums over both halves' rows; lane: of key `lane`.
  __device__ __forceinline__ float take_sums() {
    const float a = sum[0] + __shfl_xor(sum[0], 32), b = sum[1] + __shfl_xor(sum[1], 32);
    sum[0] = sum[1] = 0.f;
    return (threadIdx.x & 63) < 32 ? a : b;
  }

  struct Tile { u32x4 q[kSteps]; };
  __device__ __forceinline__ static void fetch_tile(Tile& x, const WeightParams& p, const Places& places, int tile) {
    const int lane = threadIdx.x & 63;
    const uint16_t* src = p.q + places.at[tile * 32 + (lane & 31)] + (lane >> 5) * (D / 2);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) x.q[st] = *reinterpret_cast<const u32x4*>(src + st * 8);
  }

  // rows: that the tile has.  key0: the first of the keys (MASKED: some
  // row may not see all of them).
  template <bool WIDE, bool MASKED, class Places>
  __device__ __forceinline__ void add(const Tile& x, const Places& places, int tile, int rows, int key0, float c2) {
    const int lane = fresh(threadIdx.x & 63), half = lane >> 5;
    f32x4 shift[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) shift[a] = *reinterpret_cast<const f32x4*>(&places.shift[tile * 32 + 8 * a + 4 * half]);
    f32x16 s[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[h][i] = 0.f;
    // A product must not overlap its operands.  The compiler was seen to let one
    // with a constant 0 to add to overlap them: the zeros are registers, or the
    // operands are used once more behind it.
    if constexpr (WIDE) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h) asm volatile("" : "+v"(s[h]));
    }
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      if constexpr (WIDE) {
        // the query's two exact bf16 parts; an infinity stays in the first alone
        u32x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t word = x.q[st][i];   // (a cast of the element itself takes the first one's)
          const f16x2 y = __builtin_bit_cast(f16x2, word);
          const float a = (float)y[0], b = (float)y[1];
          hi[i] = pack_bf16(a, b);
          const float ra = a - bf16_lo(hi[i]), rb = b - bf16_hi(hi[i]);
          lo[i] = pack_bf16(__builtin_isfinite(a) ? ra : 0.f, __builtin_isfinite(b) ? rb : 0.f);
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          s[h] = mma<false>(hi, k[h][st], s[h]);
          s[h] = mma<false>(lo, k[h][st], s[h]);
        }
      } else {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) s[h] = mma<F16>(x.q[st], k[h][st], s[h]);
        if (st == 0) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int h = 0; h < kHalves; ++h) asm volatile("" ::"v"(x.q[0]), "v"(k[h][0]));
        }
      }
    }
    // (the compiler was seen to read a product's result too early behind a branch)
#pragma unroll
    for (int h = 0; h < kHalves; ++h) asm volatile("s_nop 7\n\ts_nop 7" : "+v"(s[h]));
    // registers 4 a .. 4 a + 3: rows 8 a + 4 half ..
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (8 * a >= rows) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][4 * a + i], c2, shift[a][i]));
          if constexpr (MASKED)
            sum[h] += key0 + h * 32 + (lane & 31) < places.seen[tile * 32 + 8 * a + 4 * half + i] ? w : 0.f;
          else
            sum[h] += w;
        }
      }
    }
  }
};

// A tile's scores whose weights are still to be formed.
template <int D, bool F16>
struct Pending {
  f32x16 s[kKeys / 32];
  const float* shifts;     // of the lane's rows, in LDS: row 8 a + i at 8 a + i
  __device__ __forceinline__ void clear(const float* none) {  // of rows that give nothing
    shifts = none;
#pragma unroll
    for (int h = 0; h < kKeys / 32; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[h][i] = 0.f;
  }
  __device__ __forceinline__ void form(Wave<D, F16>& w, float c2) const {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const f32x4 shift = *reinterpret_cast<const f32x4*>(shifts + 8 * a);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < kKeys / 32; ++h)
          w.sum[h] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][4 * a + i], c2, shift[i]));
    }
  }
  // The products of 32 rows in LDS (rows that give to every key, or zeros), with the
  // weights of the tile before formed between them: the matrix cores and the vector
  // ALU work side by side.
  __device__ __forceinline__ void multiply(Wave<D, F16>& w, const char* q, const float* own_shifts, const Pending& before, float c2) {
    constexpr int kSteps = D / 16, kHalves = kKeys / 32, kAhead = 4;
    u32x4 a[kAhead];
    f32x4 shift[4];
#pragma unroll
    for (int st = 0; st < kAhead; ++st) a[st] = *reinterpret_cast<const u32x4*>(q + st * 16);
    shift[0] = *reinterpret_cast<const f32x4*>(before.shifts);
    shifts = own_shifts;
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[h][i] = 0.f;
    __builtin_amdgcn_sched_barrier(0);
    // A weight is scaled and shifted beside one product, its exponential taken beside
    // the next and added beside the one after that, so that none waits for another.
    constexpr int kSlots = kSteps * kHalves, kEach = 16 / kSlots;
    float x[kHalves][kEach], y[kHalves][kEach];
#pragma unroll
    for (int n = 0; n < kSlots + 2; ++n) {
      if (n < kSlots) {
        const int st = n / kHalves, h = n % kHalves;
        s[h] = mma<F16>(a[st % kAhead], w.k[h][st], s[h]);
        __builtin_amdgcn_sched_barrier(0);
        if (st == 0) asm volatile("" ::"v"(a[0]), "v"(w.k[h][0]));   // (as in Wave::add)
        if (h == kHalves - 1 && st + kAhead < kSteps)
          a[st % kAhead] = *reinterpret_cast<const u32x4*>(q + (st + kAhead) * 16);
        const int i = n * kEach;
        if (i % 4 == 0 && i < 12) shift[i / 4 + 1] = *reinterpret_cast<const f32x4*>(before.shifts + 2 * i + 8);
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          if (n >= 2) w.sum[h] += y[h][e];
          if (n >= 1 && n <= kSlots) y[h][e] = __builtin_amdgcn_exp2f(x[h][e]);
          if (n < kSlots) {
            const int i = n * kEach + e;
            x[h][e] = __builtin_fmaf(before.s[h][i], c2, shift[i >> 2][i & 3]);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Pool slot of key j, whose block is `id`.
__device__ __forceinline__ uint32_t slot_of(const WeightParams& p, int id, int j) {
  return ((uint32_t)min(max(id, 0), p.num_blocks - 1) << p.bs_shift) + (j & (1 << p.bs_shift) - 1);
}

__device__ __forceinline__ uint32_t slot_at(const WeightParams& p, const int32_t* table, int j) {
  return slot_of(p, table[j >> p.bs_shift], j);
}

// Few rows.  Waves of a workgroup beside each other: on different KV heads (heads of them,
// so that whole rows of the cache are read at about the same time), then on every
// so manieth block of keys.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, kFewResident)
weights_kernel(const WeightParams p) {
  using W = Wave<D, F16>;
  constexpr int kHalves = kKeys / 32;
  __shared__ Places all_places[kWaves];
  __shared__ float all_sums[kWaves][kSpan * kKeys];
  __shared__ uint32_t all_slots[kWaves][kSpan * kKeys / 16];   // of every 16th key
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int beside = p.heads_beside, apart = kWaves / beside, first_head = wave % beside, mine = wave / beside;
  const uint32_t sign = p.negate ? 0x88888888u : 0u;
  Places& places = all_places[wave];
  float* const sums = all_sums[wave];
  uint32_t* const slots = all_slots[wave];
  Share share;
  share.each(p, blockIdx.x, [&](int b, const Seq& s, int from, int to) {
    const int32_t* table = p.bt + (int64_t)b * p.bt_stride;
    const int64_t rows_all = (int64_t)s.n * p.group;
    for (int b0 = from; b0 < to; b0 += kSpan * apart) {
      const int here = min(to - b0, kSpan * apart), blocks = (here - mine + apart - 1) / apart;
      const auto key_of = [&](int block) { return (b0 + mine + block * apart) * kKeys; };
      for (int i = lane; i < blocks * kKeys; i += 64) sums[i] = 0.f;
      if (lane < blocks * (kKeys / 16))
        slots[lane] = slot_at(p, table, min(key_of(lane / 4) + lane % 4 * 16, s.cap - 1) & ~15);
      __builtin_amdgcn_wave_barrier();
      const auto fetch = [&](typename W::RawKeys& raw, int block, int head) {
        uint32_t row[kHalves];
        const int key = fresh(lane) & 31;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const int i = block * kKeys + h * 32 + key;
          row[h] = (slots[i >> 4] + (i & 15)) * p.kv_heads + head;
        }
        W::fetch_keys(raw, p, row);
      };
      W w;
      typename W::RawKeys raw;
      typename W::Tile x;
      if (blocks > 0 && rows_all > 0) {
        fetch(raw, 0, first_head);
        for (int head = first_head; head < p.kv_heads; head += beside) {
          for (int64_t r0 = 0; r0 < rows_all; r0 += kChunk) {
            const int rows = (int)min(rows_all - r0, (int64_t)kChunk), tiles = (rows + 31) / 32;
            __builtin_amdgcn_wave_barrier();
            bool left_out = false;           // a row that gives nothing, whatever its scores
            for (int i = 0; i < tiles * 32; i += 64) {
              const int lane = fresh(tid) & 63, r = min(i + lane, rows - 1);
              const int t = (int)((r0 + r) / p.group);
              const int q_head = head * p.group + (int)(r0 + r - (int64_t)t * p.group);
              const int64_t token = s.first + t;
              const float lse = p.lse[token * (p.kv_heads * p.group) + q_head];
              const bool gives = i + lane < rows && lse != -__builtin_inff();
              left_out |= i + lane < rows && !gives;
              places.at[i + lane] = token * p.q_stride + q_head * D;
              places.shift[i + lane] = gives ? -lse * kLog2e : -__builtin_inff();
              places.seen[i + lane] = gives ? s.seen(t) : 0;
            }
            __builtin_amdgcn_wave_barrier();
            const bool some_left_out = __any(left_out);
            const int most = s.seen((int)((r0 + rows - 1) / p.group));
            W::fetch_tile(x, p, places, 0);
            for (int block = 0; block < blocks; ++block) {
              const int key0 = key_of(block);
              const bool wide = w.put_keys(raw, sign);
              // the next block, or the first of the next rows or the next head
              const bool again = block + 1 == blocks, more_rows = r0 + kChunk < rows_all;
              fetch(raw, again ? 0 : block + 1, again && !more_rows ? min(head + beside, p.kv_heads - 1) : head);
              if (most <= key0) continue;    // none of these rows sees it
              w.sum[0] = w.sum[1] = 0.f;
#pragma nounroll
              for (int t = 0; t < tiles; ++t) {
                if (tiles > 1) W::fetch_tile(x, p, places, t);
                const int n = min(rows - t * 32, 32);
                const bool masked = some_left_out || s.seen((int)((r0 + t * 32) / p.group)) < key0 + kKeys;
                if (F16 && wide)
                  w.template add<F16, true>(x, places, t, n, key0, p.c2);
                else if (masked)
                  w.template add<false, true>(x, places, t, n, key0, p.c2);
                else
                  w.template add<false, false>(x, places, t, n, key0, p.c2);
              }
              sums[block * kKeys + lane] += w.take_sums();
            }
          }
        }
      }
      // the heads beside each other
      __syncthreads();
      for (int i = tid; i < here * kKeys; i += kThreads) {
        const int key = b0 * kKeys + i, block = i / kKeys;
        if (key >= s.cap) break;
        float x = 0.f;
        for (int j = 0; j < beside; ++j)
          x += all_sums[block % apart * beside + j][block / apart * kKeys + i % kKeys];
        give(p, 0, b, key, x);
      }
      __syncthreads();
    }
  });
  clear_columns(p, blockIdx.x);
}

// Many rows: up to 256 lie in LDS, a part of one head's or all of a few heads'
// (a unit), and every wave passes its blocks of keys by them, without a barrier.
// What a span's keys gathered from one unit waits in LDS for the next.
// (The rows read by every wave from global memory, 16 bytes of each of 32 at a time, kept
// the address unit busy for most of the time; through LDS 64 at a time, past keys that
// stayed, a piece cost a barrier and the rows' places again, and a workgroup of 256
// keys was gone before it had paid for its beginning: 64 sequences of 256 rows took
// 110 us, 256 rows past 32768 keys 186.)
constexpr int kTiles = 8, kWideSpan = 32;

template <int D>
struct __attribute__((aligned(16))) Rows {
  static constexpr int kPitch = D * 2 + 16;  // bytes; free of bank conflicts
  char q[kTiles * 32 * kPitch];
  float shift[kTiles * 32];
  int seen[kTiles * 32];
  float sums[kWideSpan * kKeys];
  int left_out[kWaves];    // a row that gives nothing, whatever its scores
  float none[32];          // shifts of rows that give nothing
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2)
weights_wide_kernel(const WeightParams p) {
  using W = Wave<D, F16>;
  constexpr int kHalves = kKeys / 32, kPitch = Rows<D>::kPitch;
  __shared__ Rows<D> x;
  const int tid = threadIdx.x, lane = tid & 63, split = blockIdx.y;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t sign = p.negate ? 0x88888888u : 0u;
  const float* const none = x.none + 4 * (lane >> 5);
  if (tid < 32) x.none[tid] = -__builtin_inff();   // (read behind barriers)
  Share share;
  share.each(p, blockIdx.x, [&](int b, const Seq& s, int from, int to) {
    const int32_t* table = p.bt + (int64_t)b * p.bt_stride;
    const int rows = s.n * p.group;          // of a head
    const int tiles_all = (rows + 31) / 32, heads = max(min(kTiles / max(tiles_all, 1), p.kv_heads), 1);   // of a unit
    const int groups = (p.kv_heads + heads - 1) / heads, units = (tiles_all + kTiles - 1) / kTiles * groups;
    // (the sums of one unit need not wait for another's: all blocks at once)
    const int spans = units - split > p.splits ? (to - from + kWideSpan - 1) / kWideSpan : 1;
    for (int span = 0; span < spans; ++span) {
      const int b0 = from + (int)((int64_t)(to - from) * span / spans);
      const int here = from + (int)((int64_t)(to - from) * (span + 1) / spans) - b0, key_base = b0 * kKeys;
      if (split >= units) {
        for (int i = tid; i < here * kKeys && key_base + i < s.cap; i += kThreads) give(p, split, b, key_base + i, 0.f);
        continue;
      }
      W w;
      typename W::RawKeys raw;
      // Blocks are fetched in the order in which they are used, their entries of the
      // table a block earlier.
      int coming = wave;                     // block whose entries are on their way
      int entry[kHalves];
      uint32_t slot[kHalves];                // of the lane's keys of the block before it
      const auto look_up = [&] {
        const int key = (b0 + coming) * kKeys + (fresh(lane) & 31);
#pragma unroll
        for (int h = 0; h < kHalves; ++h) entry[h] = table[min(key + h * 32, s.cap - 1) >> p.bs_shift];
      };
      const auto next_block = [&] {
        const int key = (b0 + coming) * kKeys + (fresh(lane) & 31);
#pragma unroll
        for (int h = 0; h < kHalves; ++h) slot[h] = slot_of(p, entry[h], min(key + h * 32, s.cap - 1));
        coming = coming + kWaves < here ? coming + kWaves : wave;
        look_up();
      };
      const auto fetch = [&](int head) {
        uint32_t row[kHalves];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) row[h] = slot[h] * p.kv_heads + head;
        W::fetch_keys(raw, p, row);
      };
      if (wave < here) look_up();
      Pending<D, F16> pending[2];
      w.sum[0] = w.sum[1] = 0.f;
      for (int unit = split; unit < units; unit += p.splits) {
        const int part = unit / groups, head0 = (unit - part * groups) * heads;
        const int r0 = part * kTiles * 32, n = min(rows - r0, kTiles * 32), tiles = (n + 31) / 32;
        const int n_heads = min(heads, p.kv_heads - head0);
        const bool first_unit = unit == split, last_unit = unit + p.splits >= units;
        __syncthreads();                     // (the rows before are done with)
        {
          const int tid = fresh(threadIdx.x);
          // Quotients by products: of at most 7 by at most 8, and of less than 2^16
          // by a group of less than 2^16 (the factors too large by less than 1).
          const int t0 = r0 / p.group, of0 = r0 - t0 * p.group, per_tile = 63 / tiles + 1;
          const uint32_t per_group = 0xffffffffu / (uint32_t)p.group + 1;
          const auto place = [&](int i, int& head, int& t, int& of) {   // of the i-th row in LDS; is there one?
            head = (i / 32 * per_tile) >> 6;
            const int r = i - head * tiles * 32, q = p.group == 1 ? of0 + r : (int)__umulhi((uint32_t)(of0 + r), per_group);
            t = t0 + q;
            of = of0 + r - q * p.group;
            return head < n_heads && r < n;
          };
          int head, t, of;
          const bool is = place(tid, head, t, of);
          float lse = 0.f;
          if (is) lse = p.lse[(int64_t)(s.first + t) * (p.kv_heads * p.group) + (head0 + head) * p.group + of];
          const int seen = s.seen(t);
          // (rows that are none: zeros, whose weight is 0)
          constexpr int kPieces = D / 8, kPass = kThreads / kPieces, kLoads = kTiles * 32 / kPass;
          u32x4 piece[kLoads];
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            piece[j] = u32x4{0, 0, 0, 0};
            if (place(tid / kPieces + j * kPass, head, t, of))
              piece[j] = *reinterpret_cast<const u32x4*>(p.q + (s.first + t) * p.q_stride + ((head0 + head) * p.group + of) * D + tid % kPieces * 8);
          }
          if (first_unit && wave < here) {
            next_block();
            fetch(head0);
          }
#pragma unroll
          for (int j = 0; j < kLoads; ++j)
            *reinterpret_cast<u32x4*>(x.q + (tid / kPieces + j * kPass) * kPitch + tid % kPieces * 16) = piece[j];
          const bool gives = is && lse != -__builtin_inff();
          x.shift[tid] = gives ? -lse * kLog2e : -__builtin_inff();
          x.seen[tid] = gives ? seen : 0;
          const bool left_out = __any(is && !gives);
          if (lane == 0) x.left_out[wave] = left_out;
        }
        __syncthreads();
        const bool left_out = x.left_out[0] || x.left_out[1] || x.left_out[2] || x.left_out[3];
        const int clear_to = left_out ? 0 : s.seen(r0 / p.group);        // keys that every row sees
        const int most = s.seen((r0 + n - 1) / p.group);
        int owed = -1;                       // block whose last tile is pending
        float prior = 0.f;                   // what a block's keys had before
        const auto look = [&](int block) {
          const int key = key_base + block * kKeys + fresh(lane);
          if (p.before && !p.part && last_unit && key < s.cap) prior = p.before[b * p.before_stride + key];
        };
        const auto flush = [&](int block) {
          const int i = block * kKeys + fresh(lane);
          float y = w.take_sums();
          if (!first_unit) y += x.sums[i];
          if (!last_unit)
            x.sums[i] = y;
          else if (key_base + i < s.cap)
            give<false>(p, split, b, key_base + i, prior + y);
        };
        const auto drain = [&] {
          // (nothing of it belongs ahead of the branch, where multiply's own would follow it)
#pragma unroll
          for (int h = 0; h < kHalves; ++h) asm volatile("" : "+v"(pending[1].s[h]));
          pending[1].form(w, p.c2);
          if (owed >= 0) flush(owed);
          owed = -1;
        };
        pending[1].clear(none);
        for (int block = wave; block < here; block += kWaves) {
          const int key0 = key_base + block * kKeys;
          bool open = false;                 // the pending tile is this block's
          if (owed >= 0) look(owed);
          // The wave that got further gives way to the other one of its SIMD.  (Otherwise
          // the older one is served first, and the chip is half empty at the end.)
          if (block * 4 < here)
            __builtin_amdgcn_s_setprio(3);
          else if (block * 2 < here)
            __builtin_amdgcn_s_setprio(2);
          else if (block * 4 < here * 3)
            __builtin_amdgcn_s_setprio(1);
          else
            __builtin_amdgcn_s_setprio(0);
          for (int head = 0; head < n_heads; ++head) {
            const bool wide = w.put_keys(raw, sign);
            if (head + 1 < n_heads) {
              fetch(head0 + head + 1);
            } else if (block + kWaves < here || !last_unit) {
              next_block();
              fetch(block + kWaves < here ? head0 : (unit + p.splits) % groups * heads);
            }
            if (most <= key0) continue;
            const int tile0 = head * tiles;
            if (key0 + kKeys <= clear_to && !(F16 && wide)) {
              const int of = fresh(lane);
              const char* q = x.q + (tile0 * 32 + (of & 31)) * kPitch + (of >> 5) * D;
              const float* shifts = x.shift + tile0 * 32 + 4 * (of >> 5);
              for (int t = 0; t + 1 < tiles; t += 2) {
                pending[0].multiply(w, q, shifts, pending[1], p.c2);
                if (owed >= 0) flush(owed);
                owed = -1;
                pending[1].multiply(w, q + 32 * kPitch, shifts + 32, pending[0], p.c2);
                q += 64 * kPitch;
                shifts += 64;
              }
              if (tiles & 1) {
                pending[0].multiply(w, q, shifts, pending[1], p.c2);
                if (owed >= 0) flush(owed);
                owed = -1;
                pending[1] = pending[0];
              }
              open = true;
              continue;
            }
            drain();
            open = false;
            for (int t = 0; t < tiles; ++t) {
              const int of = fresh(lane);
              const char* q = x.q + ((tile0 + t) * 32 + (of & 31)) * kPitch + (of >> 5) * D;
              typename W::Tile tile;
#pragma unroll
              for (int st = 0; st < D / 16; ++st) tile.q[st] = *reinterpret_cast<const u32x4*>(q + st * 16);
              if (F16 && wide)
                w.template add<F16, true>(tile, x, tile0 + t, n - t * 32, key0, p.c2);
              else
                w.template add<false, true>(tile, x, tile0 + t, n - t * 32, key0, p.c2);
            }
            pending[1].clear(none);
          }
          if (open)
            owed = block;
          else {
            if (owed >= 0) {
              drain();
              pending[1].clear(none);
            }
            look(block);
            flush(block);
          }
        }
        if (owed >= 0) {
          look(owed);
          drain();
        }
      }
    }
  });
  if (!p.part) clear_columns(p, blockIdx.x);
}

// Adds the splits' sums, in their order.
__global__ void __launch_bounds__(64)
weights_join_kernel(const WeightParams p) {
  const int key = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
  if (key >= p.max_ctx) return;
  const int cap = min(max(p.ctx[b], 0), p.max_ctx);
  float x = 0.f;
  if (key < cap) {
    const float* part = p.part + (int64_t)b * p.max_ctx + key;
    const int64_t stride = (int64_t)p.batch * p.max_ctx;
    constexpr int kAhead = 16;
    for (int i = 0; i < p.splits; i += kAhead) {
      float y[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) y[j] = part[min(i + j, p.splits - 1) * stride];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) x += i + j < p.splits ? y[j] : 0.f;
    }
    if (p.before) x += p.before[b * p.before_stride + key];
  }
  p.out[b * p.out_stride + key] = x;
}

template <int D, bool F16>
hipError_t launch(const WeightParams& p, hipStream_t s) {
  if (p.wide)
    weights_wide_kernel<D, F16><<<dim3(p.workers, p.splits), kThreads, 0, s>>>(p);
  else
    weights_kernel<D, F16><<<p.workers, kThreads, 0, s>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.part) return e;
  weights_join_kernel<<<dim3((p.max_ctx + 63) / 64, p.batch), 64, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_weights(int d, int f16, const WeightParams& p, hipStream_t s) {
  if (d == 128) return f16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return f16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

}  // namespace mqa
