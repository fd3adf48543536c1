// Softmax attention over a paged cache held in MXFP4 (gfx950), whole contexts
// or the columns a top-k selected, and the kernel that joins split contexts.
//
//   out[r, :] = sum_j p[r, j] v[j, :],  p[r, :] = softmax_j(scale <q[r, :], k[j, :]>)
//
// over the keys j that row r sees.  A row here is one (query token, head) pair
// of a sequence and a KV head: all next_n * group of them share the KV head's
// tokens (with selected columns: the group heads of one query token).
//
// One pass over the cache with a running maximum and sum, 32 keys and 16 * RT
// rows at a time per wave.  How a workgroup's four waves divide the work gives
// three kernels:
//   attention_kernel        16 or 32 rows of a KV head: the waves take the tiles
//                           in turn, and join their maxima, sums and
//                           accumulators through LDS at the end;
//   attention_heads_kernel  16 rows of each of four KV heads, one per wave, over
//                           the same keys;
//   attention_wide_kernel   128 rows of a KV head, 32 per wave, over the same
//                           keys, which each wave converts a quarter of.
// Both products are computed transposed so that nothing leaves the registers
// between them:
//
//   S^T[key, row] = K Q^T   A = 16 keys x 32 of D, B = 32 of D x 16 rows
//   O^T[d, row]  += V^T P^T A = 16 of D x 32 keys, B = 32 keys x 16 rows
//
// The order of the contracted index is free as long as A and B agree:
//   * D in K Q^T: lane group g (lanes 16g .. 16g+15) carries the D/4 elements
//     from g * D/4 on, so a lane's part of a key is one contiguous load of
//     packed e2m1 under one e8m0 scale;
//   * keys in V^T P^T: the accumulator layout leaves row l % 16 and keys
//     4g .. 4g+3 of both 16-key halves in lane l, which are taken as the
//     lane's eight B elements as they stand;
//   * V's m index: column c of product j is element c * D/16 + j, so a lane
//     loads D/16 adjacent elements of each of its eight keys, and its results
//     are D/4 adjacent elements of one row inside one scale block.
// e2m1 times a power of two is exact in bf16, so the conversion instruction
// (packed pair, scale applied) loses nothing; V's pairs (two elements of a key)
// become operand pairs (two keys of an element) with one byte permute each.
//
// q is bf16, or fp16 split exactly into two bf16 parts.  p is split into two bf16
// parts for the second product (2^-16 left), for either type of result: one part
// would round every weight by up to 2^-8 while the sum they are divided by keeps
// all bits, and with weights of one size that does not average out (values that
// are all 1 gave 0.996).  The second part costs bf16 calls that the matrix cores
// bound 15 to 23% (64 x 4 query tokens of 64 heads: 222 us, 180 with one) and
// others up to 6%.  The sum of p, the maximum and all accumulators are fp32.
//
// What bounds it.  With few rows the cache's bytes: (D/2 + D/32) * 2 per key and
// KV head.  With many the matrix cores and the vector ALU one after the other,
// which hardly overlap on this chip: 32 keys x 32 rows are 48 products (768
// cycles) and, with the keys converted by every wave, about 240 vector
// instructions (1000 cycles).  Measured: 64 x 4 query
// tokens of 64 heads over 1024..32768 keys 222 us, 0.64 PFLOP/s (matrix cores
// busy 42% of the time; every wave also reads a tile's 16 KB of operands from LDS
// for its 32 rows, about 40% of the time at 128 bytes a clock); 32 sequences of
// those lengths, 8 KV heads of 8 fp16 rows each, 138 us, 4.2 TB/s (busy 23%); one
// context of 131072 keys, 4 KV heads, 28 us; 2048 selected keys of 64 heads for
// 256 query tokens 49 us (busy 22%), for one 10.7.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "launch.hpp"

namespace mqa {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kAttnThreads = 64 * kWaves;   // two workgroups per compute unit, without spills
constexpr int kTile = 32;                    // keys per wave and step
// Scale bytes above this could overflow fp32 (6 * 2^126): they count as NaN.
constexpr uint32_t kLastScale = 252;
// The running maximum is set this many octaves above the largest score, and
// follows a new one only when that leaves a weight above 1; most tiles rescale
// nothing.  With weights of at most 1 the unnormalised sums of n keys stay within n
// times the largest value (set to the largest score itself and left 8 octaves
// behind, they overflowed fp32 for averages far inside it).
constexpr float kRoom = 8.f;
constexpr float kMostWeight = 1.f;
constexpr float kLowest = -0x1.fffffep127f;  // a maximum before any key (finite: no inf - inf)
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ bf16x8 as_bf16(u32x4 x) { return __builtin_bit_cast(bf16x8, x); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Byte SEL of w: two e2m1 elements times the scale, as packed bf16.
template <int SEL>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}

__device__ __forceinline__ u32x4 cvt_eight(uint32_t w, float scale) {
  return u32x4{cvt_pair<0>(w, scale), cvt_pair<1>(w, scale), cvt_pair<2>(w, scale),
               cvt_pair<3>(w, scale)};
}

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

// Byte i of w as a scale: rotated to the exponent field.  The conversions read
// that field alone (checked for every scale byte with random other bits).
__device__ __forceinline__ float byte_scale(uint32_t w, int i) {
  return __uint_as_float(__builtin_amdgcn_alignbit(w, w, 8 * i + 9));
}

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(a), as_bf16(b), c, 0, 0, 0);
}

// Reductions over the four lanes of a row (same l % 16).
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// A wave's tile as loaded: 16 + 16 keys.  Lane l takes D/4 elements of K and of
// V of key l % 16 (of both halves), so a load instruction covers whole cache
// lines, and the scale bytes of one key: of K in lanes 0 .. 31, of V in lanes
// 32 .. 63.  Single-byte or single-dword loads would serve fewer bytes for the
// same occupancy of the address unit, which bounded the kernel.
struct Raw {
  u32x4 k[2], v[2];       // [half] (D = 64: x, y)
  uint32_t s;             // D/32 scale bytes of key l % 32
};

// A 32-element block of the cache is 16 bytes of codes and one scale byte, so
// one number, the block's index, gives both addresses.  LDS holds the index of
// the first block (of KV head 0) of every key (SPARSE; kNoKey for one to pass
// over) or of every 16th key.
constexpr uint32_t kNoKey = 0xffffffffu;

template <int D, bool SPARSE>
struct Tiles {
  Bytes k, v, ks, vs;
  const uint32_t* lds;
  uint32_t key_blocks;                       // blocks from one key of the pool to the next
  uint32_t code;                             // the lane's byte offset from its key's first code

  __device__ __forceinline__ Tiles(const AttnParams& p, const uint32_t* at, int kv_head)
      : k((Bytes)p.k + kv_head * (D / 2)), v((Bytes)p.v + kv_head * (D / 2)),
        ks((Bytes)p.k_sf + kv_head * (D / 32)), vs((Bytes)p.v_sf + kv_head * (D / 32)), lds(at),
        key_blocks(p.kv_heads * (D / 32)) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    code = (SPARSE ? 0 : c * key_blocks) * 16 + g * (D / 8);
  }

  template <bool LANES>
  __device__ __forceinline__ static Bytes at(Bytes pool, uint32_t block) {
    const Bytes p = pool + ((uint64_t)block << 4);
    return LANES ? p : scalar(p);
  }

  template <bool SCALES = true>
  __device__ __forceinline__ void load(Raw& r, int tile) const {
    const int lane = threadIdx.x & 63, c = lane & 15;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t first = key_block(tile * kTile + half * 16 + (SPARSE ? c : 0));
      const Bytes kp = at<SPARSE>(k, first) + lanes(code), vp = at<SPARSE>(v, first) + lanes(code);
      if constexpr (D == 128) {
        r.k[half] = load_from<u32x4>(kp);
        r.v[half] = load_from<u32x4>(vp);
      } else {
        const u32x2 x = load_from<u32x2>(kp), y = load_from<u32x2>(vp);
        r.k[half] = u32x4{x[0], x[1], 0u, 0u};
        r.v[half] = u32x4{y[0], y[1], 0u, 0u};
      }
    }
    if constexpr (!SCALES) return;
    uint32_t first;                          // of key l % 32
    if constexpr (SPARSE) {
      first = key_block(tile * kTile + (lane & 31));
    } else {
      const uint32_t lo = key_block(tile * kTile), hi = key_block(tile * kTile + 16);
      first = (lane & 16 ? hi : lo) + c * key_blocks;
    }
    const Bytes sp = (lane & 32 ? vs : ks) + first;
    r.s = D == 128 ? load_from<uint32_t>(sp) : load_from<uint16_t>(sp);
  }

  // First block of any one key of the stage.
  __device__ __forceinline__ uint32_t key_first(int key) const {
    if constexpr (SPARSE) return key_block(key);
    return lds[key >> 4] + (key & 15) * key_blocks;
  }

  // First block of a key of the stage (SPARSE; any block for one to pass over)
  // or, wave-uniform, of the 16 keys from one on.
  __device__ __forceinline__ uint32_t key_block(int key) const {
    if constexpr (SPARSE) {
      const uint32_t b = lds[key];
      return b == kNoKey ? 0u : b;
    } else {
      return __builtin_amdgcn_readfirstlane(lds[key >> 4]);
    }
  }
};

// Rows' state of one wave: queries, running maximum and sum, accumulators.
template <int D, int RT, bool F16, bool QUERIES_IN_LDS>
struct Rows {
  static constexpr int kSteps = D / 32;      // products along D
  static constexpr int kCols = D / 16;       // 16-element column groups of V
  static constexpr int kParts = F16 ? 2 : 1;  // bf16 parts of a query
  static constexpr int kWeightParts = 2;     // and of a weight
  // the pitch of V's rows keeps both the 16-byte writes and the 4-byte reads
  // free of bank conflicts
  static constexpr int kPitch = D == 128 ? 80 : 40;
  static constexpr int kStageBytes = 256 + kTile * kPitch;
  struct Scores { f32x4 s[RT][2]; };         // [half]: keys 4g .. 4g+3 of row l % 16
  // Queries in LDS, shared by the waves, where registers are short.
  static constexpr bool kQueriesInLds = QUERIES_IN_LDS;
  static constexpr int kQueryWords = RT * kParts * kSteps * 64;
  u32x4 q[kQueriesInLds ? 1 : RT][kParts][kSteps];
  u32x4* q_lds;                              // [RT][kParts][kSteps][64 lanes]
  uint32_t* words;                           // the wave's staging of a tile: 64 scale words,
  char* values;                              // and V's rows of D/2 bytes
  f32x4 o[RT][kCols];
  float m[RT], l[RT];
  int seen[RT];                              // keys the lane's row sees
  int most;                                  // keys of the context
  uint32_t nan_rows;                         // bit rt: the lane's results are NaN

  __device__ __forceinline__ void clear() {
    nan_rows = 0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = kLowest;
      l[rt] = 0.f;
#pragma unroll
      for (int j = 0; j < kCols; ++j) o[rt][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }

  __device__ __forceinline__ u32x4 query(int rt, int part, int st) const {
    if constexpr (kQueriesInLds)
      return q_lds[((rt * kParts + part) * kSteps + st) * 64 + (threadIdx.x & 63)];
    else
      return q[rt][part][st];
  }

  // Scale words and V go through LDS to the lanes that need them.
  __device__ __forceinline__ void stage(const Raw& r) const {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    words[lane] = r.s;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      char* row = values + (half * 16 + c) * kPitch + g * (D / 8);
      if constexpr (D == 128)
        *reinterpret_cast<u32x4*>(row) = r.v[half];
      else
        *reinterpret_cast<u32x2*>(row) = u32x2{r.v[half][0], r.v[half][1]};
    }
    __builtin_amdgcn_wave_barrier();
  }

  __device__ __forceinline__ void scores(const Raw& r, Scores& x) const {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int half = 0; half < 2; ++half) x.s[rt][half] = f32x4{0.f, 0.f, 0.f, 0.f};
    float ks[2];
#pragma unroll
    for (int half = 0; half < 2; ++half)
      ks[half] = byte_scale(words[half * 16 + c], g * (D / 4) / 32);
    u32x4 y[2][kParts][RT];                  // queries of this step and the next
    const auto fetch = [&](int st) {
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) y[st & 1][part][rt] = query(rt, part, st);
    };
    fetch(0);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      if (st + 1 < kSteps) fetch(st + 1);
      if (kQueriesInLds) __builtin_amdgcn_sched_barrier(0);
      const u32x4 a = cvt_eight(r.k[0][st], ks[0]), b = cvt_eight(r.k[1][st], ks[1]);
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          x.s[rt][0] = mma(a, y[st & 1][part][rt], x.s[rt][0]);
          x.s[rt][1] = mma(b, y[st & 1][part][rt], x.s[rt][1]);
        }
    }
  }

  // The scales of keys that no row sees (MASKED) may hold anything and are read
  // as finite.  Others that are NaN spread: K's bytes over kLastScale become
  // the NaN byte, V's mark the rows that see their key and become 0.  first:
  // position of the tile's first key; places: the LDS entries of its keys
  // (SPARSE).  Returns whether some key may be hidden from some row.
  template <bool MASKED, bool SPARSE>
  __device__ __forceinline__ bool check_scales(Raw& r, int first, const uint32_t* places) {
    const int lane = threadIdx.x & 63;
    bool hidden = MASKED;
    if constexpr (MASKED) {
      const bool any = SPARSE ? places[lane & 31] != kNoKey : first + (lane & 31) < most;
      r.s = any ? r.s : 0u;
      if (SPARSE) hidden = !__all(any);
    }
    if (__builtin_expect(__any(has_nan(r.s)), 0))
      spread_nan<MASKED && !SPARSE>(r.s, first);
    return hidden;
  }

  // The compiler was seen to read a product's result right behind a branch,
  // before it is there; ahead of a branch, the products end here.
  __device__ __forceinline__ static void end_products(Scores& s) {
    if constexpr (RT == 1)
      asm volatile("s_nop 7" : "+v"(s.s[0][0]), "+v"(s.s[0][1]));
    else
      asm volatile("s_nop 7" : "+v"(s.s[0][0]), "+v"(s.s[0][1]), "+v"(s.s[RT - 1][0]), "+v"(s.s[RT - 1][1]));
  }

  template <bool BY_ROW>
  __device__ __forceinline__ void spread_nan(uint32_t& s, int first) {
#pragma nounroll
    for (int key = 0; key < kTile; ++key) mark_nan<BY_ROW>(__shfl(s, 32 + key), first + key);
    s = without_nan(s);
  }

  // A key's V scales mark the rows that see it, by the block of the lane's results.
  template <bool BY_ROW>
  __device__ __forceinline__ void mark_nan(uint32_t word, int key) {
    const uint32_t b = (word >> (8 * ((threadIdx.x & 63) / 16 * (D / 4) / 32))) & 0xffu;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (b > kLastScale && (!BY_ROW || key < seen[rt])) nan_rows |= 1u << rt;
  }

  __device__ __forceinline__ static bool has_nan(uint32_t s) {
    // some byte of s over 252: some byte of ~s under 3
    return ((~s - 0x03030303u) & s & 0x80808080u) != 0;
  }
  __device__ __forceinline__ static uint32_t without_nan(uint32_t s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t byte = 0xffu << (8 * i), b = (s >> (8 * i)) & 0xffu;
      if (b > kLastScale) s = threadIdx.x & 32 ? s & ~byte : s | byte;
    }
    return s;
  }

  // Keys that a row does not see leave its scores.
  template <bool SPARSE>
  __device__ __forceinline__ void mask(Scores& x, int first, const uint32_t* places) const {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      u32x4 four;
      if constexpr (SPARSE) four = *reinterpret_cast<const u32x4*>(places + half * 16 + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const bool use = SPARSE ? four[i] != kNoKey : first + half * 16 + 4 * g + i < seen[rt];
          x.s[rt][half][i] = use ? x.s[rt][half][i] : -__builtin_inff();
        }
    }
  }

  // One tile.
  template <bool MASKED, bool SPARSE>
  __device__ __forceinline__ void step(Raw& r, int first, const uint32_t* places, float c2) {
    Scores s;
    const bool hidden = check_scales<MASKED, SPARSE>(r, first, places);
    stage(r);
    scores(r, s);
    if constexpr (MASKED) {
      end_products(s);
      if (hidden) mask<SPARSE>(s, first, places);
    }
    accumulate(s, c2);
    __builtin_amdgcn_wave_barrier();         // the staging is read
  }

  // Weights of one row tile from its scores, packed for the second product.
  // Whether a maximum was left behind shows in the weights themselves; then
  // they are formed again.  One fused instruction scales and shifts a score; it
  // leaves the maximum's own rounding in the exponent, half an octave at 2^24
  // octaves, which is why scores may not be larger.  (Scaled and shifted apart,
  // 64 x 4 query tokens of 64 heads took 228 us instead of 222.)
  __device__ __forceinline__ void weights(const f32x4 (&x)[2], int rt, float c2, u32x4 (&p)[kWeightParts]) {
    float w[8];
    const auto form = [&] {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i >> 2][i & 3], c2, -m[rt]));
    };
    form();
    const float most = fmaxf(fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])),
                             fmaxf(fmaxf(w[4], w[5]), fmaxf(w[6], w[7])));
    if (__builtin_expect(__any(most > kMostWeight), 0)) {
      asm volatile("");                      // rare: nothing of it belongs before the branch
      const float best = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                               fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3]))) * c2;
      const float next = fmaxf(m[rt], row_max(best) + kRoom);
      const float f = __builtin_amdgcn_exp2f(m[rt] - next);
      m[rt] = next;
      l[rt] *= f;
#pragma unroll
      for (int j = 0; j < kCols; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[rt][j][i] *= f;
      form();
    }
    l[rt] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t hi = pack_bf16(w[2 * i], w[2 * i + 1]);
      p[0][i] = hi;
      p[1][i] = pack_bf16(w[2 * i] - bf16_lo(hi), w[2 * i + 1] - bf16_hi(hi));
    }
  }

  // From the staging: D/16 elements of keys 4g .. 4g+3 of both halves, and
  // their scales.
  __device__ __forceinline__ void read_values(uint32_t (&v)[8], float (&vs)[8]) const {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const char* row = values + ((i >> 2) * 16 + 4 * g + (i & 3)) * kPitch + c * (D / 32);
      v[i] = D == 128 ? *reinterpret_cast<const uint32_t*>(row) : *reinterpret_cast<const uint16_t*>(row);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(words + 32 + half * 16 + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) vs[4 * half + i] = byte_scale(w[i], c * (D / 16) / 32);
    }
  }

  // Operands of elements 2 SEL and 2 SEL + 1 of the lane's D/16.
  template <int SEL>
  __device__ __forceinline__ static void value_operands(const uint32_t (&v)[8], const float (&vs)[8],
                                                        u32x4& even, u32x4& odd) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = cvt_pair<SEL>(v[i], vs[i]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      even[w] = __builtin_amdgcn_perm(e[2 * w + 1], e[2 * w], 0x05040100);
      odd[w] = __builtin_amdgcn_perm(e[2 * w + 1], e[2 * w], 0x07060302);
    }
  }

  // The weighted sum of a tile's V.
  __device__ __forceinline__ void accumulate(const Scores& x, float c2) {
    uint32_t v[8];
    float vs[8];
    read_values(v, vs);
    u32x4 p[RT][kWeightParts];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) weights(x.s[rt], rt, c2, p[rt]);
    // in turn: interleaved, their operands would not fit the registers
    __builtin_amdgcn_sched_barrier(0);
    add_values<0>(v, vs, p);
    __builtin_amdgcn_sched_barrier(0);
    add_values<1>(v, vs, p);
    if constexpr (D == 128) {
      __builtin_amdgcn_sched_barrier(0);
      add_values<2>(v, vs, p);
      __builtin_amdgcn_sched_barrier(0);
      add_values<3>(v, vs, p);
    }
  }

  template <int SEL>
  __device__ __forceinline__ void add_values(const uint32_t (&v)[8], const float (&vs)[8],
                                             const u32x4 (&p)[RT][kWeightParts]) {
    u32x4 even, odd;
    value_operands<SEL>(v, vs, even, odd);
#pragma unroll
    for (int part = 0; part < kWeightParts; ++part)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        o[rt][2 * SEL] = mma(even, p[rt][part], o[rt][2 * SEL]);
        o[rt][2 * SEL + 1] = mma(odd, p[rt][part], o[rt][2 * SEL + 1]);
      }
  }

  // ---- operands in LDS, shared by the workgroup's waves (the wide kernel) ----

  static constexpr int kKeyOps = 2 * kSteps, kTileOps = kKeyOps + kCols;   // of 64 lanes x 16 bytes

  // The wave's tile into operands: K's [half][step], then V's [column group].
  __device__ __forceinline__ void convert(const Raw& r, u32x4* ops) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    values = reinterpret_cast<char*>(ops + kKeyOps * 64);      // V as loaded, where its operands will be
    stage(r);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float ks = byte_scale(words[half * 16 + c], g * (D / 4) / 32);
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
        ops[(half * kSteps + st) * 64 + lane] = cvt_eight(r.k[half][st], ks);
    }
    uint32_t v[8];
    float vs[8];
    read_values(v, vs);
    __builtin_amdgcn_wave_barrier();
    put_values<0>(v, vs, ops);
    put_values<1>(v, vs, ops);
    if constexpr (D == 128) {
      put_values<2>(v, vs, ops);
      put_values<3>(v, vs, ops);
    }
  }

  template <int SEL>
  __device__ __forceinline__ void put_values(const uint32_t (&v)[8], const float (&vs)[8], u32x4* ops) const {
    u32x4 even, odd;
    value_operands<SEL>(v, vs, even, odd);
    ops[(kKeyOps + 2 * SEL) * 64 + (threadIdx.x & 63)] = even;
    ops[(kKeyOps + 2 * SEL + 1) * 64 + (threadIdx.x & 63)] = odd;
  }

  // K's operands of a tile, read while the tile before it is worked on.
  struct KeyOps { u32x4 a[2][kSteps]; };
  __device__ __forceinline__ static void read_keys(KeyOps& k, const u32x4* ops) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
        k.a[half][st] = ops[(half * kSteps + st) * 64 + (threadIdx.x & 63)];
  }

  // One tile from its operands; k: its K's, then the next tile's.
  template <bool SPARSE>
  __device__ __forceinline__ void step_shared(KeyOps& k, const u32x4* ops, const u32x4* next, bool masked,
                                              int first, const uint32_t* places, float c2) {
    const int lane = threadIdx.x & 63;
    if constexpr (!kKeysAhead) read_keys(k, ops);
    Scores s;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int half = 0; half < 2; ++half) s.s[rt][half] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          s.s[rt][0] = mma(k.a[0][st], q[rt][part][st], s.s[rt][0]);
          s.s[rt][1] = mma(k.a[1][st], q[rt][part][st], s.s[rt][1]);
        }
    if constexpr (kKeysAhead) read_keys(k, next);
    end_products(s);
    if (masked) mask<SPARSE>(s, first, places);
    // V's operands, kAhead ahead of their products
    const u32x4* vops = ops + kKeyOps * 64 + lane;
    u32x4 a[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) a[j] = vops[j * 64];
    __builtin_amdgcn_sched_barrier(0);
    u32x4 p[RT][kWeightParts];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) weights(s.s[rt], rt, c2, p[rt]);
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
#pragma unroll
      for (int part = 0; part < kWeightParts; ++part)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) o[rt][j] = mma(a[j % kAhead], p[rt][part], o[rt][j]);
      if (j + kAhead < kCols) {
        a[j % kAhead] = vops[(j + kAhead) * 64];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // (as far as the registers go: fp16's queries take twice as many)
  static constexpr int kAhead = F16 && RT == 2 ? 2 : 4;
  static constexpr bool kKeysAhead = !(F16 && RT == 2);
};

template <bool F16>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
  if constexpr (F16) {
    const uint16_t x = __builtin_bit_cast(uint16_t, (_Float16)a);
    const uint16_t y = __builtin_bit_cast(uint16_t, (_Float16)b);
    return x | (uint32_t)y << 16;
  } else {
    return pack_bf16(a, b);
  }
}

// ---------------------------------------------------------------------------
// Work split
// ---------------------------------------------------------------------------
//
// A member is a group of rows of one KV head, or of four.  For every member the
// units (sequences; with selected columns, query tokens) are laid end to end in
// steps of 128 keys (four tiles; at least one step a unit), and the S steps are
// cut into equal pieces, one per worker, as many as the chip holds at a time (a
// worker per chunk of a unit left it idle for 40% of the time on contexts of
// 1024..32768 keys).  A worker walks its piece unit by unit.  A
// unit inside one piece is finished there; one cut by piece borders leaves a
// part in each: worker j writes the part that begins its piece to slot 2j, the
// one that ends it to slot 2j + 1.  The worker that begins a unit notes the
// unit's workers for the kernel that joins the parts.
constexpr int kStep = kTile * kWaves;

struct Split {
  int steps, workers;     // S; workers in use, of p.workers
  int each, more;         // steps per piece; the first `more` pieces have one more
  __device__ __forceinline__ Split(int s, const AttnParams& p) : steps(s) {
    workers = min(p.workers, s);
    each = s / workers;
    more = s - each * workers;
  }
  __device__ __forceinline__ int border(int j) const { return j * each + min(j, more); }
};

__device__ __forceinline__ int unit_length(const AttnParams& p, int unit) {
  return min(max(p.ctx[unit], 0), p.max_ctx);
}
__device__ __forceinline__ int unit_steps(int length) {
  return max((length + kStep - 1) / kStep, 1);
}

// Sum over the block, for every thread; buf holds one value per wave.
__device__ __forceinline__ int block_sum(int x, int* buf) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) x += __shfl_xor(x, off);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) x += buf[w];
  __syncthreads();
  return x;
}

// Members of one piece read the same tokens: they follow each other on one XCD.
// Pieces go round the XCDs; with selected columns each XCD has a run of them,
// because neighbouring query tokens select many of the same columns.
template <bool SPARSE>
__device__ __forceinline__ int worker_of(const AttnParams& p, int xcd, int turn) {
  return SPARSE ? xcd * ((p.workers + 7) / 8) + turn : turn * 8 + xcd;
}

// The unit being walked, and what its rows see.
template <bool SPARSE>
struct Unit {
  int raw_ctx, ctx, length;                  // keys of the context; entries to walk
  __device__ __forceinline__ Unit(const AttnParams& p, int unit) {
    raw_ctx = max(p.ctx[SPARSE ? unit / p.next_n : unit], 0);
    ctx = min(raw_ctx, p.max_ctx);
    length = SPARSE ? p.topk : ctx;
  }
  // keys that query token t sees
  __device__ __forceinline__ int seen(const AttnParams& p, int t) const {
    return min(max(raw_ctx - p.next_n + 1 + t, 0), ctx);
  }
};

// A worker's piece: the steps [at, end) from step unit_begin of `unit` on.
struct Piece {
  int begin, end, at;
  int unit, unit_begin;
  int steps, workers, each, more;

  // False for a worker that has none.  sums, found: LDS, 4 and 2 words.
  template <bool SPARSE>
  __device__ __forceinline__ bool find(const AttnParams& p, int worker, int* sums, int* found) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // (up to 64 units: every wave by itself, without a barrier)
    const bool few = SPARSE || p.units <= 64;
    int total = p.units * unit_steps(p.topk), mine = 0, scan = 0;
    if constexpr (!SPARSE) {
      if (few) {
        scan = mine = lane < p.units ? unit_steps(unit_length(p, lane)) : 0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const int x = __shfl_up(scan, off);
          if (lane >= off) scan += x;
        }
        total = __shfl(scan, 63);
      } else {
        total = 0;
        for (int b = tid; b < p.units; b += kAttnThreads) total += unit_steps(unit_length(p, b));
        total = block_sum(total, sums);
      }
    }
    const Split split(__builtin_amdgcn_readfirstlane(total), p);
    if (worker >= split.workers) return false;
    steps = split.steps;
    workers = split.workers;
    each = split.each;
    more = split.more;
    begin = at = split.border(worker);
    end = split.border(worker + 1);
    if constexpr (SPARSE) {
      unit = begin / unit_steps(p.topk);
      unit_begin = unit * unit_steps(p.topk);
      return true;
    }
    if (few) {
      const uint64_t here = __ballot(scan - mine <= begin && begin < scan);
      unit = __builtin_ctzll(here);
      unit_begin = __builtin_amdgcn_readlane(scan - mine, unit);
      return true;
    }
    int base = 0;
    for (int b0 = 0; base <= begin; b0 += kAttnThreads) {
      const int b = b0 + tid;
      mine = b < p.units ? unit_steps(unit_length(p, b)) : 0;
      scan = mine;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int x = __shfl_up(scan, off);
        if (lane >= off) scan += x;
      }
      if (lane == 63) sums[wave] = scan;
      __syncthreads();
      int first = base + scan - mine;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) first += sums[w];
        base += sums[w];
      }
      if (first <= begin && begin < first + mine) {
        found[0] = b;
        found[1] = first;
      }
      __syncthreads();
    }
    unit = __builtin_amdgcn_readfirstlane(found[0]);
    unit_begin = __builtin_amdgcn_readfirstlane(found[1]);
    return true;
  }

  // The kernel that joins the parts learns where a unit begun here has its own.
  __device__ __forceinline__ void note(const AttnParams& p, int worker, int unit_end) const {
    int2 n = make_int2(0, 1);                // first slot, parts
    if (at > unit_begin || unit_end > end) {
      const int head = more * (each + 1), last = unit_end - 1;
      const int owner = last < head ? last / (each + 1) : more + (last - head) / each;
      n = make_int2(2 * worker + (at == begin ? 0 : 1), owner - worker + 1);
    }
    p.notes[unit] = n;
  }
};

// The first cache blocks of keys [stage, stage_end) of a unit, into LDS.
template <int D, bool SPARSE>
__device__ __forceinline__ void fill_places(const AttnParams& p, uint32_t* blocks, int unit,
                                            int stage, int stage_end, int n_tiles, int seen_sparse) {
  constexpr int kEach = SPARSE ? 1 : 16;     // keys per entry
  const int32_t* table = p.bt + (int64_t)(SPARSE ? unit / p.next_n : unit) * p.bt_stride;
  const int32_t* index = SPARSE ? p.indices + (int64_t)unit * p.idx_stride : nullptr;
  for (int i = threadIdx.x; i < n_tiles * (kTile / kEach); i += kAttnThreads) {
    int j = stage + i * kEach;
    bool use = j < stage_end;
    if constexpr (SPARSE) {
      j = use ? index[j] : -1;
      use = j >= 0 && j < seen_sparse;
    }
    uint32_t first = SPARSE ? kNoKey : 0u;
    if (use) {
      const int id = min(max(table[j >> p.bs_shift], 0), p.num_blocks - 1);
      const uint32_t slot = ((uint32_t)id << p.bs_shift) + (j & ((1 << p.bs_shift) - 1));
      first = slot * p.kv_heads * (D / 32);
    }
    blocks[i] = first;
  }
}

// Row r of a unit's KV head: its query token of all, and its head.
struct RowAt {
  int token, head;
  template <bool SPARSE>
  __device__ __forceinline__ static RowAt of(const AttnParams& p, int unit, int kv_head, int r) {
    const int t = SPARSE ? 0 : r / p.group;
    return {SPARSE ? unit : unit * p.next_n + t, kv_head * p.group + (SPARSE ? r : r - t * p.group)};
  }
  __device__ __forceinline__ int64_t out(const AttnParams& p) const {
    return (int64_t)token * (p.kv_heads * p.group) + head;
  }
};

// The lane's piece st of a query, bf16; with F16 its two exact bf16 parts.
template <int D, bool F16>
__device__ __forceinline__ void load_query(const AttnParams& p, RowAt row, int st, u32x4& hi, u32x4& lo) {
  const int g = (threadIdx.x & 63) >> 4;
  const uint16_t* src = p.q + (int64_t)row.token * p.q_stride + row.head * D + g * (D / 4);
  hi = *reinterpret_cast<const u32x4*>(src + st * 8);
  if (p.negate) hi ^= 0x80008000u;
  if constexpr (F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = (float)__builtin_bit_cast(_Float16, (uint16_t)(hi[i] & 0xffff));
      const float y = (float)__builtin_bit_cast(_Float16, (uint16_t)(hi[i] >> 16));
      hi[i] = pack_bf16(x, y);
      // the part below bf16's eight bits; an infinity stays in hi alone
      const float rx = x - bf16_lo(hi[i]), ry = y - bf16_hi(hi[i]);
      lo[i] = pack_bf16(__builtin_isfinite(x) ? rx : 0.f, __builtin_isfinite(y) ? ry : 0.f);
    }
  }
}

// Scale words of four adjacent KV heads, one for each wave.  A thread loads the
// four of one key and pool (one piece instead of four) a step of 128 keys ahead
// of their use, through LDS to the waves: [step parity][head][pool][key].  The
// barrier of a step also keeps the waves together, on the same cache lines.
template <int D, bool SPARSE>
struct SharedScales {
  static constexpr int kWords = kWaves * 2 * kStep;      // of a step
  uint32_t* lds;                             // [2][kWords]
  const Tiles<D, SPARSE>& tiles;             // at the first of the four heads
  int n_tiles, wave;
  u32x4 next;

  __device__ __forceinline__ SharedScales(uint32_t* at, const Tiles<D, SPARSE>& t, int n, int w)
      : lds(at), tiles(t), n_tiles(n), wave(w) {
    __syncthreads();                         // the buffers' last use is over
    load(0);
    put(0);
    load(1);
    __syncthreads();
  }
  // At the first tile of a step: the next step's words are put down.
  __device__ __forceinline__ void turn(int step) {
    if (step > 0) __syncthreads();
    put(step + 1);
    load(step + 2);
  }
  __device__ __forceinline__ uint32_t word(int tile) const {
    const int lane = threadIdx.x & 63;
    return lds[(tile / kWaves & 1) * kWords + (wave * 2 + (lane >> 5)) * kStep + tile % kWaves * kTile +
               (lane & 31)];
  }
  __device__ __forceinline__ void load(int step) {
    const int pool = threadIdx.x / kStep;
    const int key = min(step * kStep + (int)threadIdx.x % kStep, n_tiles * kTile - 1);
    const uint32_t block = tiles.key_first(key);
    const Bytes from = (pool ? tiles.vs : tiles.ks) + block;
    if constexpr (D == 128) {
      next = load_from<u32x4>(from);
    } else {
      const u32x2 x = load_from<u32x2>(from);
      next = u32x4{x[0] & 0xffffu, x[0] >> 16, x[1] & 0xffffu, x[1] >> 16};
    }
  }
  __device__ __forceinline__ void put(int step) const {
    const int pool = threadIdx.x / kStep, key = threadIdx.x % kStep;
#pragma unroll
    for (int h = 0; h < kWaves; ++h) lds[(step & 1) * kWords + (h * 2 + pool) * kStep + key] = next[h];
  }
};

// A wave's tiles, every fourth, loaded two ahead (past the last, the last
// again, so that every load is unconditional).  Keys that some row does not see
// lie in the context's last 15 + 32, so only a wave's last tile can hold any.
template <int D, int RT, bool F16, bool QLDS, bool SPARSE>
__device__ __forceinline__ void walk(Rows<D, RT, F16, QLDS>& rows, const Tiles<D, SPARSE>& tiles,
                                     const uint32_t* blocks, int tile, int n_tiles, int stage, float c2) {
  const int last = tile + (n_tiles - 1 - tile) / kWaves * kWaves;
  Raw r[3];
  tiles.load(r[0], tile);
  tiles.load(r[1], min(tile + kWaves, last));
  const auto advance = [&](auto turn) {
    constexpr int i = decltype(turn)::value, ahead = (i + 2) % 3;
    if (QLDS) asm volatile("" ::: "memory");   // the queries are not kept in registers
    tiles.load(r[ahead], min(tile + 2 * kWaves, last));
    rows.template step<SPARSE, SPARSE>(r[i], 0, blocks + tile * kTile, c2);
    tile += kWaves;
  };
  while (tile < last) {
    advance(std::integral_constant<int, 0>{});
    if (tile >= last) {
      r[0] = r[1];
      break;
    }
    advance(std::integral_constant<int, 1>{});
    if (tile >= last) {
      r[0] = r[2];
      break;
    }
    advance(std::integral_constant<int, 2>{});
  }
  rows.template step<true, SPARSE>(r[0], stage + tile * kTile, blocks + tile * kTile, c2);
}

// Every tile, for a wave that has a KV head of its own: in steps of four, loaded
// three ahead, the scales from the workgroup's.  The last tiles, where keys may
// be hidden from some row (two at most) or a step is not whole, one by one.
template <int D, bool F16, bool SPARSE>
__device__ __forceinline__ void walk_all(Rows<D, 1, F16, false>& rows, const Tiles<D, SPARSE>& tiles,
                                         SharedScales<D, SPARSE>& scales, const uint32_t* blocks,
                                         int n_tiles, int stage, float c2) {
  static_assert(kWaves == 4, "a step is four tiles");
  const int last = n_tiles - 1, whole = (SPARSE ? n_tiles : max(n_tiles - 2, 0)) / 4 * 4;
  Raw r[4];
#pragma unroll
  for (int u = 0; u < 3; ++u) tiles.template load<false>(r[u], min(u, last));
  int tile = 0;
  for (; tile < whole; tile += 4) {
    scales.turn(tile / 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      tiles.template load<false>(r[(u + 3) % 4], min(tile + u + 3, last));
      r[u].s = scales.word(tile + u);
      rows.template step<SPARSE, SPARSE>(r[u], 0, blocks + (tile + u) * kTile, c2);
    }
  }
  for (; tile <= last; ++tile) {
    if (tile % 4 == 0) scales.turn(tile / 4);
    tiles.template load<false>(r[3], min(tile + 3, last));
    r[0].s = scales.word(tile);
    rows.template step<true, SPARSE>(r[0], stage + tile * kTile, blocks + tile * kTile, c2);
#pragma unroll
    for (int u = 0; u < 3; ++u) r[u] = r[u + 1];
  }
}

template <int D, int RT, bool F16, bool SPARSE>
__global__ void __launch_bounds__(kAttnThreads, 2)
attention_kernel(const AttnParams p) {
  constexpr int kRows = 16 * RT;
  constexpr int kPitch = D + 4;              // LDS floats per row of the join
  constexpr int kEach = SPARSE ? 1 : 16;     // keys per entry of `blocks`
  constexpr int kStage = SPARSE ? kAttnStageSparse : kAttnStage;   // keys staged at a time
  using State = Rows<D, RT, F16, RT == 2>;
  // the join's rows, or (before it) queries, places and scales
  constexpr int kPlaceBytes = kStage / kEach * 4, kQueryBytes = State::kQueriesInLds ? State::kQueryWords * 16 : 0;
  constexpr int kJoinBytes = kWaves * kRows * kPitch * 4, kLoopBytes = kQueryBytes + kPlaceBytes + kWaves * State::kStageBytes;
  __shared__ __attribute__((aligned(16))) char shared[kJoinBytes > kLoopBytes ? kJoinBytes : kLoopBytes];
  float* const join = reinterpret_cast<float*>(shared);
  u32x4* const queries = reinterpret_cast<u32x4*>(shared);
  uint32_t* const blocks = reinterpret_cast<uint32_t*>(shared + kQueryBytes);
  __shared__ float wave_m[kWaves][kRows], wave_l[kWaves][kRows];
  __shared__ int sums[kWaves], found[2];

  const int members = p.row_groups * p.kv_heads;
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int worker = worker_of<SPARSE>(p, xcd, idx / members), member = idx % members;
  const int kv_head = member / p.row_groups, row0 = member % p.row_groups * kRows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform, so its branches are too
  const int c = lane & 15, g = lane >> 4;
  const int unit_rows = SPARSE ? p.group : p.next_n * p.group;

  Piece piece;
  if (!piece.find<SPARSE>(p, worker, sums, found)) return;

  const Tiles<D, SPARSE> tiles(p, blocks, kv_head);
  State rows;
  rows.words = reinterpret_cast<uint32_t*>(shared + kQueryBytes + kPlaceBytes + wave * State::kStageBytes);
  rows.values = reinterpret_cast<char*>(rows.words + 64);
  rows.q_lds = queries;
  for (; piece.at < piece.end; ++piece.unit) {
    const int unit = piece.unit;
    const Unit<SPARSE> u(p, unit);
    const int unit_end = piece.unit_begin + unit_steps(u.length);
    const int begin = (piece.at - piece.unit_begin) * kStep;     // keys of this part
    const int end = min(u.length, (min(unit_end, piece.end) - piece.unit_begin) * kStep);
    const bool whole = piece.at == piece.unit_begin && unit_end <= piece.end;
    const int seen_sparse = SPARSE ? u.seen(p, unit % p.next_n) : 0;

    rows.clear();
    rows.most = u.ctx;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      // lanes past the last row repeat it; their results are dropped
      const int r = min(row0 + rt * 16 + c, unit_rows - 1);
      rows.seen[rt] = SPARSE ? seen_sparse : u.seen(p, r / p.group);
      const RowAt row = RowAt::of<SPARSE>(p, unit, kv_head, r);
#pragma unroll
      for (int st = 0; st < D / 32; ++st) {
        u32x4 hi, lo;
        load_query<D, F16>(p, row, st, hi, lo);
        if constexpr (State::kQueriesInLds) {
          // (every wave holds all row tiles' lanes; the first RT write one each)
          if (wave == rt) {
            queries[(rt * State::kParts * State::kSteps + st) * 64 + lane] = hi;
            if (F16) queries[((rt * State::kParts + State::kParts - 1) * State::kSteps + st) * 64 + lane] = lo;
          }
        } else {
          rows.q[rt][0][st] = hi;
          if (F16) rows.q[rt][State::kParts - 1][st] = lo;
        }
      }
    }

    for (int stage = begin; stage < end; stage += kStage) {
      const int stage_end = min(end, stage + kStage);
      const int n_tiles = (stage_end - stage + kTile - 1) / kTile;
      __syncthreads();                       // the last use of `blocks` is over
      fill_places<D, SPARSE>(p, blocks, unit, stage, stage_end, n_tiles, seen_sparse);
      __syncthreads();
      if (wave < n_tiles) walk(rows, tiles, blocks, wave, n_tiles, stage, p.c2);
    }

    // join the four waves
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      rows.l[rt] = row_sum(rows.l[rt]);
      if (g == 0) {
        wave_m[wave][rt * 16 + c] = rows.m[rt];
        wave_l[wave][rt * 16 + c] = rows.l[rt];
      }
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float m = kLowest;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) m = fmaxf(m, wave_m[w][rt * 16 + c]);
      const float f = __builtin_amdgcn_exp2f(rows.m[rt] - m);
      const bool is_nan = (rows.nan_rows >> rt) & 1;
      float* dst = join + (wave * kRows + rt * 16 + c) * kPitch + g * (D / 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          dst[i * (D / 16) + j] = is_nan ? __builtin_nanf("") : rows.o[rt][j][i] * f;
    }
    __syncthreads();
    const int64_t part_slot =
        ((int64_t)member * p.workers + worker) * 2 + (piece.at == piece.begin ? 0 : 1);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      // thread: D/16 adjacent elements of row tid / 16
      const int jr = tid >> 4, jc = (tid & 15) * (D / 16);
      const int r = row0 + rt * 16 + jr;
      if (r < unit_rows) {
        float mj = kLowest, lj = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mj = fmaxf(mj, wave_m[w][rt * 16 + jr]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
          lj += wave_l[w][rt * 16 + jr] * __builtin_amdgcn_exp2f(wave_m[w][rt * 16 + jr] - mj);
        float x[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          x[j] = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) x[j] += join[(w * kRows + rt * 16 + jr) * kPitch + jc + j];
        }
        if (whole) {
          const int64_t out_row = RowAt::of<SPARSE>(p, unit, kv_head, r).out(p);
          const float inv = lj == 0.f ? 0.f : 1.f / lj;
          uint32_t w[D / 32];
#pragma unroll
          for (int j = 0; j < D / 32; ++j) w[j] = pack_out<F16>(x[2 * j] * inv, x[2 * j + 1] * inv);
          uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + out_row * D + jc);
          if constexpr (D == 128)
            *reinterpret_cast<u32x4*>(dst) = u32x4{w[0], w[1], w[2], w[3]};
          else
            *reinterpret_cast<u32x2*>(dst) = u32x2{w[0], w[1]};
          if (p.lse && (tid & 15) == 0)
            p.lse[out_row] = lj == 0.f ? -__builtin_inff() : (mj + __builtin_log2f(lj)) * kLn2;
        } else {
          const int64_t part = part_slot * kRows + rt * 16 + jr;
          f32x4* dst = reinterpret_cast<f32x4*>(p.part_o + part * D + jc);
#pragma unroll
          for (int j = 0; j < D / 64; ++j)
            dst[j] = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
          if ((tid & 15) == 0) p.part_ml[part] = make_float2(mj, lj);
        }
      }
    }
    __syncthreads();                         // the join's LDS is read
    if (p.join && member == 0 && tid == 0 && piece.at == piece.unit_begin)
      piece.note(p, worker, unit_end);
    piece.at = piece.unit_begin = unit_end;
  }
}

// The results of a wave that has rows of its own, from row `first` of the KV
// head on: a lane has D/4 adjacent elements of row l % 16 of each row tile.
// part0: where its rows' parts go if the unit is cut.
template <bool SPARSE, int D, int RT, bool F16, bool QLDS>
__device__ __forceinline__ void store_rows(const AttnParams& p, const Rows<D, RT, F16, QLDS>& rows,
                                           bool whole, int unit, int kv_head, int unit_rows, int first,
                                           int64_t part0) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float m = rows.m[rt], l = row_sum(rows.l[rt]);
    const bool is_nan = (rows.nan_rows >> rt) & 1;
    int r = first + rt * 16 + c;
    asm volatile("" : "+v"(r));              // nothing derived from it is kept through the loops
    if (r < unit_rows) {
      if (whole) {
        const int64_t out_row = RowAt::of<SPARSE>(p, unit, kv_head, r).out(p);
        const float inv = is_nan ? __builtin_nanf("") : l == 0.f ? 0.f : 1.f / l;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + out_row * D + g * (D / 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[D / 32];
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            w[j] = pack_out<F16>(rows.o[rt][2 * j][i] * inv, rows.o[rt][2 * j + 1][i] * inv);
          if constexpr (D == 128)
            *reinterpret_cast<u32x4*>(dst + i * 4) = u32x4{w[0], w[1], w[2], w[3]};
          else
            *reinterpret_cast<u32x2*>(dst + i * 2) = u32x2{w[0], w[1]};
        }
        if (p.lse && g == 0)
          p.lse[out_row] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
      } else {
        const int64_t part = part0 + (r - first);
        f32x4* dst = reinterpret_cast<f32x4*>(p.part_o + part * D + g * (D / 4));
        const float one = is_nan ? __builtin_nanf("") : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < D / 64; ++j)
            dst[i * (D / 64) + j] =
                f32x4{rows.o[rt][4 * j][i] * one, rows.o[rt][4 * j + 1][i] * one,
                      rows.o[rt][4 * j + 2][i] * one, rows.o[rt][4 * j + 3][i] * one};
        if (g == 0) p.part_ml[part] = make_float2(m, l);
      }
    }
  }
}

// Several KV heads: the four waves take a KV head each and walk the same keys,
// so that a token's adjacent heads are read at about the same time and the
// cache lines and DRAM pages they share are fetched once.  (With a workgroup per
// KV head, 64 bytes of every token's row at a time, the loads alone ran at
// 3.7 TB/s on 8 heads, 32 sequences of 1024..32768 tokens; whole blocks are
// read at about 6.)  Every wave has rows of its own; nothing is joined.
template <int D, int RT, bool F16, bool SPARSE>
__global__ void __launch_bounds__(kAttnThreads, 2)
attention_heads_kernel(const AttnParams p) {
  constexpr int kRows = 16 * RT * kWaves;    // of a member: 16 * RT of each of its four heads
  constexpr int kEach = SPARSE ? 1 : 16;
  constexpr int kStage = SPARSE ? kAttnStageSparse : kAttnStage;
  using State = Rows<D, RT, F16, false>;
  __shared__ __attribute__((aligned(16))) uint32_t blocks[kStage / kEach];
  __shared__ __attribute__((aligned(16))) char staging[kWaves][State::kStageBytes];
  __shared__ uint32_t scales[2 * SharedScales<D, SPARSE>::kWords];
  __shared__ int sums[kWaves], found[2];

  const int members = p.row_groups * (p.kv_heads / kWaves);
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int worker = worker_of<SPARSE>(p, xcd, idx / members), member = idx % members;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kv_head = member / p.row_groups * kWaves + wave;   // (Hkv is a multiple of four)
  const int row0 = member % p.row_groups * 16 * RT;
  const int c = lane & 15;
  const int unit_rows = SPARSE ? p.group : p.next_n * p.group;

  Piece piece;
  if (!piece.find<SPARSE>(p, worker, sums, found)) return;

  const Tiles<D, SPARSE> tiles(p, blocks, kv_head), heads(p, blocks, kv_head - wave);
  State rows;
  rows.words = reinterpret_cast<uint32_t*>(staging[wave]);
  rows.values = staging[wave] + 256;
  for (; piece.at < piece.end; ++piece.unit) {
    const int unit = piece.unit;
    const Unit<SPARSE> u(p, unit);
    const int unit_end = piece.unit_begin + unit_steps(u.length);
    const int begin = (piece.at - piece.unit_begin) * kStep;
    const int end = min(u.length, (min(unit_end, piece.end) - piece.unit_begin) * kStep);
    const bool whole = piece.at == piece.unit_begin && unit_end <= piece.end;
    const int seen_sparse = SPARSE ? u.seen(p, unit % p.next_n) : 0;

    rows.clear();
    rows.most = u.ctx;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      int r = min(row0 + rt * 16 + c, unit_rows - 1);
      asm volatile("" : "+v"(r));
      rows.seen[rt] = SPARSE ? seen_sparse : u.seen(p, r / p.group);
      const RowAt row = RowAt::of<SPARSE>(p, unit, kv_head, r);
#pragma unroll
      for (int st = 0; st < D / 32; ++st)
        load_query<D, F16>(p, row, st, rows.q[rt][0][st], rows.q[rt][State::kParts - 1][st]);
    }
    for (int stage = begin; stage < end; stage += kStage) {
      const int stage_end = min(end, stage + kStage);
      const int n_tiles = (stage_end - stage + kTile - 1) / kTile;
      __syncthreads();                       // the last use of `blocks` is over
      fill_places<D, SPARSE>(p, blocks, unit, stage, stage_end, n_tiles, seen_sparse);
      __syncthreads();
      SharedScales<D, SPARSE> shared(scales, heads, n_tiles, wave);
      walk_all(rows, tiles, shared, blocks, n_tiles, stage, p.c2);
    }

    const int64_t part_slot =
        ((int64_t)member * p.workers + worker) * 2 + (piece.at == piece.begin ? 0 : 1);
    store_rows<SPARSE>(p, rows, whole, unit, kv_head, unit_rows, row0,
                       part_slot * kRows + wave * 16 * RT);
    if (p.join && member == 0 && tid == 0 && piece.at == piece.unit_begin)
      piece.note(p, worker, unit_end);
    piece.at = piece.unit_begin = unit_end;
  }
}

// Many rows on a KV head: each wave has 16 * RT rows of its own, and the four
// share the keys.  The matrix cores and the vector ALU hardly overlap, and with
// every wave converting the keys that it multiplies, the conversions take as
// long as the products of 32 rows.  Here a wave converts one of a step's four
// tiles for all four, into operands in LDS (16 KB a tile), and reads the others'
// from there.  No row is split over waves, so nothing is joined at the end.
template <int D, int RT, bool F16, bool SPARSE>
__global__ void __launch_bounds__(kAttnThreads, 2)
attention_wide_kernel(const AttnParams p) {
  constexpr int kRows = 16 * RT * kWaves;
  constexpr int kEach = SPARSE ? 1 : 16;
  constexpr int kStage = SPARSE ? kAttnStageSparse : kAttnStage;
  using State = Rows<D, RT, F16, false>;
  __shared__ u32x4 ops[kWaves][State::kTileOps * 64];
  __shared__ __attribute__((aligned(16))) uint32_t blocks[kStage / kEach];
  __shared__ __attribute__((aligned(16))) uint32_t words[kWaves][64];
  __shared__ uint32_t nan_words[kWaves][kTile], nan_flags[kWaves];
  __shared__ int sums[kWaves], found[2];

  const int members = p.row_groups * p.kv_heads;
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int worker = worker_of<SPARSE>(p, xcd, idx / members), member = idx % members;
  const int kv_head = member / p.row_groups, row0 = member % p.row_groups * kRows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15;
  const int unit_rows = SPARSE ? p.group : p.next_n * p.group;
  const int wave_row = row0 + wave * 16 * RT;

  Piece piece;
  if (!piece.find<SPARSE>(p, worker, sums, found)) return;

  const Tiles<D, SPARSE> tiles(p, blocks, kv_head);
  State rows;
  rows.words = words[wave];
  for (; piece.at < piece.end; ++piece.unit) {
    const int unit = piece.unit;
    const Unit<SPARSE> u(p, unit);
    const int unit_end = piece.unit_begin + unit_steps(u.length);
    const int begin = (piece.at - piece.unit_begin) * kStep;
    const int end = min(u.length, (min(unit_end, piece.end) - piece.unit_begin) * kStep);
    const bool whole = piece.at == piece.unit_begin && unit_end <= piece.end;
    const int seen_sparse = SPARSE ? u.seen(p, unit % p.next_n) : 0;
    // keys that all rows of the workgroup see (rows in order of t)
    const int least = SPARSE ? 0 : u.seen(p, row0 / p.group);

    rows.clear();
    rows.most = u.ctx;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      int r = min(wave_row + rt * 16 + c, unit_rows - 1);
      asm volatile("" : "+v"(r));            // nothing derived from it is kept through the loops
      rows.seen[rt] = SPARSE ? seen_sparse : u.seen(p, r / p.group);
      const RowAt row = RowAt::of<SPARSE>(p, unit, kv_head, r);
#pragma unroll
      for (int st = 0; st < D / 32; ++st)
        load_query<D, F16>(p, row, st, rows.q[rt][0][st], rows.q[rt][State::kParts - 1][st]);
    }

    for (int stage = begin; stage < end; stage += kStage) {
      const int stage_end = min(end, stage + kStage);
      const int n_tiles = (stage_end - stage + kTile - 1) / kTile;
      __syncthreads();                       // the last use of `blocks` is over
      fill_places<D, SPARSE>(p, blocks, unit, stage, stage_end, n_tiles, seen_sparse);
      __syncthreads();
      // a wave without a tile of its own in the last step repeats the last one
      Raw r;
      tiles.load(r, min(wave, n_tiles - 1));
      for (int tile0 = 0; tile0 < n_tiles; tile0 += kWaves) {
        const int own = min(tile0 + wave, n_tiles - 1);
        int half_lane = lane & 31;
        asm volatile("" : "+v"(half_lane));
        const bool any = SPARSE ? blocks[own * kTile + half_lane] != kNoKey
                                : stage + own * kTile + half_lane < rows.most;
        r.s = any ? r.s : 0u;
        __syncthreads();                     // the operands are read
        const bool bad = __any(State::has_nan(r.s));
        if (lane == 0) nan_flags[wave] = bad;
        if (__builtin_expect(bad, 0)) {
          if (lane & 32) nan_words[wave][half_lane] = r.s;
          r.s = State::without_nan(r.s);
        }
        rows.convert(r, ops[wave]);
        tiles.load(r, min(tile0 + kWaves + wave, n_tiles - 1));
        __syncthreads();
        const int n = min(n_tiles - tile0, kWaves);
        if (__builtin_expect(__any((lane < n ? nan_flags[lane & (kWaves - 1)] : 0u) != 0), 0)) {
          for (int w = 0; w < n; ++w)
            if (nan_flags[w])
              for (int key = 0; key < kTile; ++key)
                rows.template mark_nan<!SPARSE>(nan_words[w][key], stage + (tile0 + w) * kTile + key);
        }
        const bool masked = SPARSE || stage + (tile0 + kWaves) * kTile > least;
        typename State::KeyOps k;
        if constexpr (State::kKeysAhead) State::read_keys(k, ops[0]);
#pragma nounroll
        for (int w = 0; w < n; ++w)
          rows.template step_shared<SPARSE>(k, ops[w], ops[min(w + 1, n - 1)], masked,
                                            stage + (tile0 + w) * kTile,
                                            blocks + (tile0 + w) * kTile, p.c2);
      }
    }

    const int64_t part_slot =
        ((int64_t)member * p.workers + worker) * 2 + (piece.at == piece.begin ? 0 : 1);
    store_rows<SPARSE>(p, rows, whole, unit, kv_head, unit_rows, wave_row, part_slot * kRows + wave * 16 * RT);
    if (p.join && member == 0 && tid == 0 && piece.at == piece.unit_begin)
      piece.note(p, worker, unit_end);
    piece.at = piece.unit_begin = unit_end;
  }
}

// Joins the parts of the units that were cut: GROUPS groups of D/4 lanes (16
// bytes of a row each) per (query token, head).  Part 0 is in the noted slot,
// the next in slot 2j of the workers that follow.  Bound by the latency of its
// three loads in a row (note, maxima, rows), so a group keeps four parts in
// flight, and a block of one item covers 32 parts at a time.
template <int D, bool F16, int GROUPS>
__global__ void __launch_bounds__(256)
attention_join_kernel(const AttnParams p, int sparse) {
  constexpr int kLanes = D / 4, kBlockGroups = 256 / kLanes;
  static_assert(GROUPS == 1 || GROUPS == kBlockGroups, "one item per group or per block");
  __shared__ f32x4 part_x[GROUPS > 1 ? kBlockGroups : 1][kLanes];
  __shared__ float part_ml[GROUPS > 1 ? kBlockGroups : 1][2];
  const int group = threadIdx.x / kLanes, i = threadIdx.x % kLanes;
  const int64_t item = GROUPS > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kBlockGroups + group;
  if (item >= p.rows_heads) return;            // (no block of one item is partly out)
  const int heads = p.kv_heads * p.group;
  const int token = (int)(item / heads), head = (int)(item - (int64_t)token * heads);
  const int2 note = p.notes[sparse ? token : token / p.next_n];
  const int n = note.y;
  if (n <= 1) return;                          // written by its only worker
  const int kv_head = head / p.group;
  const int r = head % p.group + (sparse ? 0 : token % p.next_n * p.group);
  // a member's rows: of one KV head, or of member_heads of them
  const int rows = p.member_rows, rows_each = rows / p.member_heads;
  const int64_t base = (kv_head / p.member_heads * p.row_groups + r / rows_each) * (int64_t)p.workers * 2;
  const int row = kv_head % p.member_heads * rows_each + r % rows_each;
  const int first = GROUPS > 1 ? group : 0;
  constexpr int kStride = GROUPS;
  float m = kLowest, l = 0.f;
  f32x4 x{0.f, 0.f, 0.f, 0.f};
  for (int j0 = first; j0 < n; j0 += 4 * kStride) {
    float2 ml[4];
    f32x4 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = min(j0 + u * kStride, n - 1);
      const int64_t at = (base + (j == 0 ? note.x : ((note.x >> 1) + j) * 2)) * rows + row;
      ml[u] = p.part_ml[at];
      y[u] = reinterpret_cast<const f32x4*>(p.part_o + at * D)[i];
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = fmaxf(top, j0 + u * kStride < n ? ml[u].x : kLowest);
    const float f = __builtin_amdgcn_exp2f(m - top);
    m = top;
    l *= f;
    x *= f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j0 + u * kStride < n) {
        const float g = __builtin_amdgcn_exp2f(ml[u].x - m);
        l += ml[u].y * g;
        x += y[u] * g;
      }
    }
  }
  if constexpr (GROUPS > 1) {
    part_x[group][i] = x;
    if (i == 0) {
      part_ml[group][0] = m;
      part_ml[group][1] = l;
    }
    __syncthreads();
    if (group > 0) return;
    float top = kLowest;
#pragma unroll
    for (int w = 0; w < kBlockGroups; ++w) top = fmaxf(top, part_ml[w][0]);
    m = top;
    l = 0.f;
    x = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kBlockGroups; ++w) {
      const float g = __builtin_amdgcn_exp2f(part_ml[w][0] - m);
      l += part_ml[w][1] * g;
      x += part_x[w][i] * g;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<u32x2*>(p.out + item * D)[i] =
      u32x2{pack_out<F16>(x[0] * inv, x[1] * inv), pack_out<F16>(x[2] * inv, x[3] * inv)};
  if (p.lse && i == 0) p.lse[item] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
}

template <int D, bool F16, bool SPARSE>
hipError_t launch_rt(const AttnParams& p, hipStream_t s) {
  const int members = p.row_groups * (p.kv_heads / p.member_heads);
  const uint32_t grid = (uint32_t)((p.workers + 7) / 8 * 8 * members);
  if (p.member_heads > 1)
    attention_heads_kernel<D, 1, F16, SPARSE><<<grid, kAttnThreads, 0, s>>>(p);
  else if (p.member_rows == 16)
    attention_kernel<D, 1, F16, SPARSE><<<grid, kAttnThreads, 0, s>>>(p);
  else if (p.member_rows == 32)
    attention_kernel<D, 2, F16, SPARSE><<<grid, kAttnThreads, 0, s>>>(p);
  else
    attention_wide_kernel<D, 2, F16, SPARSE><<<grid, kAttnThreads, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.join) return e;
  constexpr int kPer = 256 / (D / 4);
  // few items: a block each, so that long contexts' many parts are read at once
  if (p.rows_heads <= 1024)
    attention_join_kernel<D, F16, kPer><<<(uint32_t)p.rows_heads, 256, 0, s>>>(p, SPARSE);
  else
    attention_join_kernel<D, F16, 1><<<(uint32_t)((p.rows_heads + kPer - 1) / kPer), 256, 0, s>>>(p, SPARSE);
  return hipGetLastError();
}

template <int D, bool F16>
hipError_t launch_form(const AttnParams& p, hipStream_t s) {
  return p.indices ? launch_rt<D, F16, true>(p, s) : launch_rt<D, F16, false>(p, s);
}

}  // namespace

hipError_t launch_attention(int d, int f16, const AttnParams& p, hipStream_t s) {
  if (d == 128) return f16 ? launch_form<128, true>(p, s) : launch_form<128, false>(p, s);
  return f16 ? launch_form<64, true>(p, s) : launch_form<64, false>(p, s);
}

}  // namespace mqa
