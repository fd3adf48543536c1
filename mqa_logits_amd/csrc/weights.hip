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

// A wave has 32 * KT keys of a sequence, and goes through the rows of every KV
// head, 32 at a time: S[key, row] = K Q^T, A = 32 keys x 16 of D, B = 16 of D x
// 32 rows.  A lane's results are 16 keys of one row, and what it adds up over
// the rows stays in its registers; the 32 lanes of a key are added at the end.
template <int D, bool F16>
struct Wave {
  static constexpr int kSteps = D / 16;
  u32x4 k[kSteps];         // key l % 32, elements 16 st + 8 (l / 32) ..
  f32x16 sum;              // keys i % 4 + 8 (i / 4) + 4 (l / 32) of row l % 32

  // K of one KV head.  Whether some scale needs the wide products (fp16 queries).
  __device__ __forceinline__ bool load_keys(const WeightParams& p, uint32_t block, bool held) {
    const int half = (threadIdx.x & 63) >> 5;
    // element order of the contraction: a lane's 16-byte piece of a 32-element
    // block holds what it multiplies in two steps' halves
    bool wide = false;
    uint32_t s[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      s[c] = held ? p.k_sf[(uint64_t)block + c] : 127u;
      wide |= s[c] - kHalfLow > kHalfHigh - kHalfLow;
      if (s[c] > kLastScale) s[c] = 255;
    }
    wide = F16 && __any(wide);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(p.k + ((uint64_t)block << 4) + c * 16 + half * 8);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        k[2 * c + i] = wide || !F16 ? cvt_eight<false>(x[i], scale_of(s[c])) : cvt_eight<true>(x[i], scale_of(s[c]));
    }
    return wide;
  }

  struct Row {
    u32x4 q[kSteps];
    float shift;           // -lse, in octaves; -inf for a row that counts for nothing
    int seen;
  };

  __device__ __forceinline__ static void load_row(Row& x, const WeightParams& p, const Seq& s, int kv_head, int r, int rows) {
    const int half = (threadIdx.x & 63) >> 5;
    const int at = min(r, rows - 1), t = at / p.group;
    const int64_t token = s.first + t;
    const int head = kv_head * p.group + at - t * p.group;
    const uint16_t* src = p.q + token * p.q_stride + head * D + half * 16;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.q[2 * c + i] = *reinterpret_cast<const u32x4*>(src + c * 32 + i * 8);
        if (p.negate) x.q[2 * c + i] ^= 0x80008000u;
      }
    const float lse = p.lse[token * (p.kv_heads * p.group) + head];
    x.shift = r < rows && lse != -__builtin_inff() ? -lse * kLog2e : -__builtin_inff();
    x.seen = r < rows ? s.seen(t) : 0;
  }

  template <bool WIDE>
  __device__ __forceinline__ void add(const Row& x, int key0, bool masked, float c2) {
    const int half = (threadIdx.x & 63) >> 5;
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
    asm volatile("" : "+v"(s));              // (a product must not overlap its operands)
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
        s = mma<false>(k[st], hi, s);
        s = mma<false>(k[st], lo, s);
      } else {
        s = mma<F16>(k[st], x.q[st], s);
      }
    }
    // (the compiler was seen to read a product's result too early behind a branch)
    asm volatile("s_nop 7\n\ts_nop 7" : "+v"(s));
    if (masked) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c2, x.shift));
        sum[i] += key0 + (i & 3) + 8 * (i >> 2) + 4 * half < x.seen ? w : 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c2, x.shift));
    }
  }
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2)
weights_kernel(const WeightParams p) {
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.y, split = blockIdx.z;
  const int key0 = (blockIdx.x * kWaves + wave) * 32;
  if (key0 >= p.max_ctx) return;
  const Seq s(p, b);
  float* out = p.part ? p.part + ((int64_t)split * p.batch + b) * p.max_ctx : p.out + b * p.out_stride;
  Wave<D, F16> w;
#pragma unroll
  for (int i = 0; i < 16; ++i) w.sum[i] = 0.f;
  if (key0 < s.cap && s.n > 0) {
    const int j = min(key0 + (lane & 31), s.cap - 1);
    const int32_t* table = p.bt + (int64_t)b * p.bt_stride;
    const int id = min(max(table[j >> p.bs_shift], 0), p.num_blocks - 1);
    const uint32_t slot = ((uint32_t)id << p.bs_shift) + (j & (1 << p.bs_shift) - 1);
    const int rows = s.n * p.group, tiles = (rows + 31) / 32;
    // this split's tiles of all KV heads', end to end
    const int64_t all = (int64_t)tiles * p.kv_heads;
    int64_t at = all * split / p.splits;
    const int64_t end = all * (split + 1) / p.splits;
    while (at < end) {
      const int kv_head = (int)(at / tiles);
      int tile = (int)(at - (int64_t)kv_head * tiles);
      const int last = (int)min((int64_t)tiles, tile + end - at);
      at += last - tile;
      const bool wide = w.load_keys(p, (slot * p.kv_heads + kv_head) * (D / 32), true);
      typename Wave<D, F16>::Row x;
      for (; tile < last; ++tile) {
        // rows whose last sees none of the keys
        const int r = tile * 32;
        if (s.seen(min(r + 31, rows - 1) / p.group) <= key0) continue;
        w.load_row(x, p, s, kv_head, r + (lane & 31), rows);
        const bool masked = r + 32 > rows || s.seen(r / p.group) < key0 + 32;
        if (F16 && wide)
          w.template add<F16>(x, key0, masked, p.c2);
        else
          w.template add<false>(x, key0, masked, p.c2);
      }
    }
  }
  // the 32 lanes of a key: key i of 16 ends up in lane i of each half
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x = w.sum[i];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) x += __shfl_xor(x, off);
    mine = (lane & 31) == i ? x : mine;
  }
  const int i = lane & 31, key = key0 + (i & 3) + 8 * (i >> 2) + 4 * half;
  if (i < 16 && key < p.max_ctx) {
    if (p.part)
      out[key] = mine;
    else
      out[key] = key < s.cap ? (p.before ? p.before[b * p.before_stride + key] + mine : mine) : 0.f;
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
  constexpr int kKeys = 32 * kWaves;
  weights_kernel<D, F16><<<dim3((p.max_ctx + kKeys - 1) / kKeys, p.batch, p.splits), kThreads, 0, s>>>(p);
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
