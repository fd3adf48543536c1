// The attention weight that every cached token has gathered (gfx950):
//
//   out[b, j] = before[b, j] + sum_r exp(scale <q[r, :], k[j, :]> - lse[r])
//
// over the rows r, (token, head) pairs of sequence b, that see key j.
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
  int first, n;            // its rows of q
  __device__ __forceinline__ Seq(const WeightParams& p, int b) {
    int64_t lo = (int64_t)b * p.next_n, hi = lo + p.next_n;
    if (p.offsets) {
      lo = __builtin_amdgcn_readfirstlane(p.offsets[b]);
      hi = __builtin_amdgcn_readfirstlane(p.offsets[b + 1]);
    }
    const int ctx = __builtin_amdgcn_readfirstlane(p.ctx[b]);
    cap = min(max(ctx, 0), p.max_ctx);
    const int64_t from = min(max(lo, (int64_t)0), (int64_t)p.tokens);
    const int64_t to = min(max(hi, from), (int64_t)p.tokens);
    base = (int64_t)ctx - (hi - lo) + (from - lo);
    first = (int)from;
    n = (int)(to - from);
  }
  __device__ __forceinline__ int seen(int t) const {
    return (int)min(max(base + 1 + t, (int64_t)0), (int64_t)cap);
  }
};

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
constexpr int kKeys = 64;                    // of a wave

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
    uint32_t s[kHalves];
  };
  u32x4 k[kHalves][kSteps];
  float sum[kHalves];

  // block: of the lane's key of each half
  __device__ __forceinline__ static void fetch_keys(RawKeys& r, const WeightParams& p, const uint32_t (&block)[kHalves]) {
    const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const uint8_t* src = p.k + ((uint64_t)block[h] << 4) + half * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) r.x[h][i] = *reinterpret_cast<const u32x4*>(src + i * 16);
      const uint8_t* sf = p.k_sf + (uint64_t)block[h] + half * (D / 64);
      r.s[h] = D == 128 ? *reinterpret_cast<const uint16_t*>(sf) : *sf;
    }
  }

  // Whether some scale needs the wide products (fp16 queries).
  __device__ __forceinline__ bool put_keys(const RawKeys& r) {
    bool wide = false;
    float s[kHalves][D / 64];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t byte = r.s[h] >> (8 * i) & 0xffu;
        wide |= byte - kHalfLow > kHalfHigh - kHalfLow;
        s[h][i] = scale_of(byte > kLastScale ? 255u : byte);
      }
    wide = F16 && __any(wide);
    if (F16 && !wide)
      convert<true>(r, s);
    else
      convert<false>(r, s);
    return wide;
  }
  template <bool HALF>
  __device__ __forceinline__ void convert(const RawKeys& r, const float (&s)[kHalves][D / 64]) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const uint32_t word = r.x[h][st / 4][st % 4];
        k[h][st] = cvt_eight<HALF>(word, s[h][st / 4]);
      }
  }

  struct Tile { u32x4 q[kSteps]; };
  __device__ __forceinline__ static void fetch_tile(Tile& x, const WeightParams& p, const Places& places, int tile) {
    const int lane = threadIdx.x & 63;
    const uint16_t* src = p.q + places.at[tile * 32 + (lane & 31)] + (lane >> 5) * (D / 2);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) x.q[st] = *reinterpret_cast<const u32x4*>(src + st * 8);
  }

  // rows: that the tile has (FULL: 32).  key0: the first of the keys (MASKED: some
  // row may not see all of them).
  template <bool WIDE, bool MASKED, bool FULL, class Places>
  __device__ __forceinline__ void add(const Tile& x, const Places& places, int tile, int rows, int key0, float c2) {
    const int lane = threadIdx.x & 63, half = lane >> 5;
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
      if (!FULL && 8 * a >= rows) break;
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
  f32x4 shift[4];
  __device__ __forceinline__ void clear() {  // of no rows
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) shift[a][i] = -__builtin_inff();
#pragma unroll
    for (int h = 0; h < kKeys / 32; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[h][i] = 0.f;
  }
  // registers i of 16
  __device__ __forceinline__ void form(Wave<D, F16>& w, int i, float c2) const {
#pragma unroll
    for (int h = 0; h < kKeys / 32; ++h)
      w.sum[h] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][i], c2, shift[i >> 2][i & 3]));
  }
  // The products of 32 rows in LDS (32 rows that give to every key), with the weights
  // of the tile before formed between them: the matrix cores and the vector ALU
  // work side by side.
  __device__ __forceinline__ void multiply(Wave<D, F16>& w, const char* q, const float* shifts, const Pending& before, float c2) {
    constexpr int kSteps = D / 16, kHalves = kKeys / 32, kAhead = 4;
    u32x4 a[kAhead];
#pragma unroll
    for (int st = 0; st < kAhead; ++st) a[st] = *reinterpret_cast<const u32x4*>(q + st * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) shift[i] = *reinterpret_cast<const f32x4*>(shifts + 8 * i);
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
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          if (n >= 2) w.sum[h] += y[h][e];
          if (n >= 1 && n <= kSlots) y[h][e] = __builtin_amdgcn_exp2f(x[h][e]);
          if (n < kSlots) {
            const int i = n * kEach + e;
            x[h][e] = __builtin_fmaf(before.s[h][i], c2, before.shift[i >> 2][i & 3]);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Pool slot of key j, the first of 16 of a block (the 16 have slots in a row).
__device__ __forceinline__ uint32_t slot_of(const WeightParams& p, const int32_t* table, int j) {
  const int id = min(max(table[j >> p.bs_shift], 0), p.num_blocks - 1);
  return ((uint32_t)id << p.bs_shift) + (j & (1 << p.bs_shift) - 1);
}

// Few rows.  Waves of a workgroup beside each other: on different KV heads (heads of them,
// so that whole rows of the cache are read at about the same time), then on the
// keys that follow.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2)
weights_kernel(const WeightParams p) {
  using W = Wave<D, F16>;
  constexpr int kHalves = kKeys / 32;
  __shared__ Places all_places[kWaves];
  __shared__ float all_sums[kWaves][kWeightBlocks * kKeys];
  __shared__ uint32_t all_slots[kWaves][kWeightBlocks * kKeys / 16];   // of every 16th key
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.y, split = blockIdx.z;
  const int beside = p.heads_beside, first_head = wave % beside;
  const int wave_keys = p.blocks * kKeys, group_keys = kWaves / beside * wave_keys;   // of the workgroup
  const int wave_key0 = blockIdx.x * group_keys + wave / beside * wave_keys;
  const Seq s(p, b);
  Places& places = all_places[wave];
  float* const sums = all_sums[wave];
  for (int i = lane; i < wave_keys; i += 64) sums[i] = 0.f;
  // this split's rows of each head
  const int64_t rows_all = (int64_t)s.n * p.group, tiles_all = (rows_all + 31) / 32;
  const int64_t from = tiles_all * split / p.splits * 32;
  const int64_t to = min(rows_all, tiles_all * (split + 1) / p.splits * 32);
  const int blocks = min((s.cap - wave_key0 + kKeys - 1) / kKeys, p.blocks);
  if (blocks > 0 && from < to) {
    const int32_t* table = p.bt + (int64_t)b * p.bt_stride;
    uint32_t* const slots = all_slots[wave];
    if (lane < blocks * (kKeys / 16)) slots[lane] = slot_of(p, table, min(wave_key0 + lane * 16, s.cap - 1) & ~15);
    __builtin_amdgcn_wave_barrier();
    const auto fetch = [&](typename W::RawKeys& raw, int block, int head) {
      uint32_t first[kHalves];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int i = block * kKeys + h * 32 + (lane & 31);
        first[h] = ((slots[i >> 4] + (i & 15)) * p.kv_heads + head) * (D / 32);
      }
      W::fetch_keys(raw, p, first);
    };
    W w;
    typename W::RawKeys raw;
    typename W::Tile x;
    fetch(raw, 0, first_head);
    for (int head = first_head; head < p.kv_heads; head += beside) {
      for (int64_t r0 = from; r0 < to; r0 += kChunk) {
        const int rows = (int)min(to - r0, (int64_t)kChunk), tiles = (rows + 31) / 32;
        __builtin_amdgcn_wave_barrier();
        bool left_out = false;               // a row that gives nothing, whatever its scores
        for (int i = 0; i < tiles * 32; i += 64) {
          const int r = min(i + lane, rows - 1);
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
          const int key0 = wave_key0 + block * kKeys;
          const bool wide = w.put_keys(raw);
          // the next block, or the first of the next rows or the next head
          const bool again = block + 1 == blocks, more_rows = r0 + kChunk < to;
          fetch(raw, again ? 0 : block + 1, again && !more_rows ? min(head + beside, p.kv_heads - 1) : head);
          if (most <= key0) continue;        // none of these rows sees it
#pragma unroll
          for (int h = 0; h < kHalves; ++h) w.sum[h] = 0.f;
#pragma nounroll
          for (int t = 0; t < tiles; ++t) {
            if (tiles > 1) W::fetch_tile(x, p, places, t);
            const int n = min(rows - t * 32, 32);
            const bool masked = some_left_out || s.seen((int)((r0 + t * 32) / p.group)) < key0 + kKeys;
            if (F16 && wide)
              w.template add<F16, true, false>(x, places, t, n, key0, p.c2);
            else if (masked)
              w.template add<false, true, false>(x, places, t, n, key0, p.c2);
            else if (n == 32)
              w.template add<false, false, true>(x, places, t, n, key0, p.c2);
            else
              w.template add<false, false, false>(x, places, t, n, key0, p.c2);
          }
          // the two halves' rows
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const float y = w.sum[h] + __shfl_xor(w.sum[h], 32);
            if (lane < 32) sums[block * kKeys + h * 32 + lane] += y;
          }
        }
      }
    }
  }
  // the heads beside each other
  __syncthreads();
  for (int i = tid; i < group_keys; i += kThreads) {
    const int key = blockIdx.x * group_keys + i;
    if (key >= p.max_ctx) break;
    float x = 0.f;
    for (int j = 0; j < beside; ++j) x += all_sums[i / wave_keys * beside + j][i % wave_keys];
    if (p.part)
      p.part[((int64_t)split * p.batch + b) * p.max_ctx + key] = x;
    else
      p.out[b * p.out_stride + key] = key < s.cap ? (p.before ? p.before[b * p.before_stride + key] + x : x) : 0.f;
  }
}

// Many rows: 64 at a time go through LDS to the workgroup's four waves, which have
// 64 keys each.  (Read from global memory by every wave for itself, 16 bytes of
// each of 32 rows at a time, they kept the address unit busy for most of the time.)
constexpr int kStageRows = 64;

template <int D>
struct __attribute__((aligned(16))) StageRows {
  static constexpr int kPitch = D * 2 + 16;  // bytes; free of bank conflicts
  char q[kStageRows * kPitch];
  float shift[kStageRows];
  int seen[kStageRows];
  int left_out;            // a row that gives nothing, whatever its scores
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2)
weights_wide_kernel(const WeightParams p) {
  using W = Wave<D, F16>;
  constexpr int kHalves = kKeys / 32, kGroupKeys = kWaves * kKeys;
  constexpr int kLoads = kStageRows * D * 2 / 16 / kThreads, kRowsALoad = kThreads / 8;
  __shared__ StageRows<D> stage[2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.y, split = blockIdx.z;
  // (the last keys first: their rows end among them, which takes longer)
  const int group_key0 = (gridDim.x - 1 - blockIdx.x) * kGroupKeys, key0 = group_key0 + wave * kKeys;
  const Seq s(p, b);
  W w;
#pragma unroll
  for (int h = 0; h < kHalves; ++h) w.sum[h] = 0.f;
  // this split's pieces of 64 rows, of all KV heads' end to end
  const int rows = s.n * p.group, pieces = (rows + kStageRows - 1) / kStageRows;
  const int64_t all = (int64_t)pieces * p.kv_heads;
  const int64_t begin = all * split / p.splits, end = all * (split + 1) / p.splits;
  if (group_key0 < s.cap && begin < end) {
    const int32_t* table = p.bt + (int64_t)b * p.bt_stride;
    uint32_t slot[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int j = min(key0 + h * 32 + (lane & 31), s.cap - 1);
      slot[h] = slot_of(p, table, j & ~15) + (j & 15);
    }
    // Rows that see some of the keys follow those that do not: the first such piece.
    const int64_t blind = min(max((int64_t)group_key0 - s.base, (int64_t)0), (int64_t)s.n);   // tokens
    const int first_piece = (int)(blind * p.group / kStageRows);
    int head = (int)(begin / pieces), piece = max((int)(begin - (int64_t)head * pieces), first_piece);
    const int last_head = (int)((end - 1) / pieces), last_piece = (int)(end - 1 - (int64_t)last_head * pieces);
    // (token, head of the group) of the rows that this thread loads, and of the one
    // whose lse wave 0's lanes load: from piece to piece they move by 64 rows
    const int step_t = kStageRows / p.group, step_h = kStageRows - step_t * p.group;
    struct Row {
      int t, h;
    };
    Row mine[kStageRows / kRowsALoad], of_lse, front;
    const auto place = [&](Row& x, int r) {
      x.t = r / p.group;
      x.h = r - x.t * p.group;
    };
    const auto place_all = [&] {
#pragma unroll
      for (int i = 0; i < kStageRows / kRowsALoad; ++i) place(mine[i], piece * kStageRows + i * kRowsALoad + tid / 8);
      place(of_lse, piece * kStageRows + lane);
      place(front, piece * kStageRows);
    };
    const auto move = [&](Row& x) {
      x.t += step_t;
      x.h += step_h;
      if (x.h >= p.group) {
        x.h -= p.group;
        ++x.t;
      }
    };
    // whether there is a piece at (head, piece); past a head's last, the next one's first
    bool more = true;
    const auto settle = [&](bool moved) {
      if (piece >= pieces) {
        piece = first_piece;
        ++head;
        moved = true;
      }
      more = piece < pieces && (head < last_head || (head == last_head && piece <= last_piece));
      if (more && moved) place_all();
    };
    settle(true);
    u32x4 raw[kLoads];
    float lse = 0.f;
    int seen = 0;
    const auto fetch = [&] {
      constexpr int kPieces = D / 64;        // of 128 bytes of a row
#pragma unroll
      for (int i = 0; i < kStageRows / kRowsALoad; ++i) {
        // (past the last row, the last token's)
        const int64_t token = s.first + min(mine[i].t, s.n - 1);
        const uint16_t* src = p.q + token * p.q_stride + (head * p.group + mine[i].h) * D + tid % 8 * 8;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) raw[i * kPieces + j] = *reinterpret_cast<const u32x4*>(src + j * 64);
      }
      if (wave == 0) {
        const int64_t token = s.first + min(of_lse.t, s.n - 1);
        lse = p.lse[token * (p.kv_heads * p.group) + head * p.group + of_lse.h];
        seen = of_lse.t < s.n ? s.seen(of_lse.t) : -1;   // (-1: no row)
      }
    };
    const auto put = [&](StageRows<D>& x) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        constexpr int kPieces = D / 64;
        *reinterpret_cast<u32x4*>(x.q + (i / kPieces * kRowsALoad + tid / 8) * StageRows<D>::kPitch +
                                  (i % kPieces * 8 + tid % 8) * 16) = raw[i];
      }
      if (wave == 0) {
        const bool gives = seen >= 0 && lse != -__builtin_inff();
        x.shift[lane] = gives ? -lse * kLog2e : -__builtin_inff();
        x.seen[lane] = gives ? seen : 0;
        const bool left_out = __any(seen >= 0 && !gives);
        if (lane == 0) x.left_out = left_out;
      }
    };
    if (more) fetch();
    int buffer = 0, have = -1;
    bool wide = false;
    Pending<D, F16> pending[2];
    pending[1].clear();
    const auto finish = [&] {
      // (nothing of it belongs ahead of the branch, where multiply's own would follow it)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) asm volatile("" : "+v"(pending[1].s[h]));
#pragma unroll
      for (int i = 0; i < 16; ++i) pending[1].form(w, i, p.c2);
    };
    while (more) {
      if (head != have) {
        have = head;
        uint32_t first[kHalves];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) first[h] = (slot[h] * p.kv_heads + head) * (D / 32);
        typename W::RawKeys keys;
        W::fetch_keys(keys, p, first);
        wide = w.put_keys(keys);
      }
      StageRows<D>& x = stage[buffer];
      put(x);
      const int n = min(rows - piece * kStageRows, kStageRows), front_seen = s.seen(front.t);
      ++piece;
#pragma unroll
      for (int i = 0; i < kStageRows / kRowsALoad; ++i) move(mine[i]);
      move(of_lse);
      move(front);
      settle(false);
      if (more) fetch();
      __syncthreads();
      // (one barrier a piece: before the buffer is written again, every wave has
      // passed the next piece's)
      buffer ^= 1;
      const bool masked = x.left_out || front_seen < key0 + kKeys;
      if (!masked && n == kStageRows && !(F16 && wide)) {
        const char* q = x.q + (lane & 31) * StageRows<D>::kPitch + (lane >> 5) * D;
        const float* shifts = x.shift + 4 * (lane >> 5);
        pending[0].multiply(w, q, shifts, pending[1], p.c2);
        pending[1].multiply(w, q + 32 * StageRows<D>::kPitch, shifts + 32, pending[0], p.c2);
        continue;
      }
      finish();
      pending[1].clear();
#pragma unroll
      for (int t = 0; t < kStageRows / 32; ++t) {
        if (t * 32 >= n) break;
        const char* q = x.q + (t * 32 + (lane & 31)) * StageRows<D>::kPitch + (lane >> 5) * D;
        typename W::Tile tile;
#pragma unroll
        for (int st = 0; st < D / 16; ++st) tile.q[st] = *reinterpret_cast<const u32x4*>(q + st * 16);
        if (F16 && wide)
          w.template add<F16, true, false>(tile, x, t, n - t * 32, key0, p.c2);
        else if (masked)
          w.template add<false, true, false>(tile, x, t, n - t * 32, key0, p.c2);
        else
          w.template add<false, false, false>(tile, x, t, n - t * 32, key0, p.c2);
      }
    }
    finish();
  }
  // the two halves' rows
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    const float x = w.sum[h] + __shfl_xor(w.sum[h], 32);
    const int key = key0 + h * 32 + lane;
    if (lane >= 32 || key >= p.max_ctx) continue;
    if (p.part)
      p.part[((int64_t)split * p.batch + b) * p.max_ctx + key] = x;
    else
      p.out[b * p.out_stride + key] = key < s.cap ? (p.before ? p.before[b * p.before_stride + key] + x : x) : 0.f;
  }
}

// Adds the splits' sums, in their order.
__global__ void __launch_bounds__(256)
weights_join_kernel(const WeightParams p) {
  const int key = blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
  if (key >= p.max_ctx) return;
  const int cap = min(max(p.ctx[b], 0), p.max_ctx);
  float x = 0.f;
  if (key < cap) {
    for (int i = 0; i < p.splits; ++i) x += p.part[((int64_t)i * p.batch + b) * p.max_ctx + key];
    if (p.before) x += p.before[b * p.before_stride + key];
  }
  p.out[b * p.out_stride + key] = x;
}

template <int D, bool F16>
hipError_t launch(const WeightParams& p, hipStream_t s) {
  if (p.blocks == 0) {
    constexpr int keys = kWaves * kKeys;
    weights_wide_kernel<D, F16><<<dim3((p.max_ctx + keys - 1) / keys, p.batch, p.splits), kThreads, 0, s>>>(p);
  } else {
    const int keys = kWaves / p.heads_beside * kKeys * p.blocks;
    weights_kernel<D, F16><<<dim3((p.max_ctx + keys - 1) / keys, p.batch, p.splits), kThreads, 0, s>>>(p);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.part) return e;
  weights_join_kernel<<<dim3((p.max_ctx + 255) / 256, p.batch), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_weights(int d, int f16, const WeightParams& p, hipStream_t s) {
  if (d == 128) return f16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return f16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

}  // namespace mqa
