// Softmax attention over a paged cache held in MXFP4 (gfx950), whole contexts
// or the columns a top-k selected, and the kernel that joins split contexts.
//
//   out[r, :] = sum_j p[r, j] v[j, :],  p[r, :] = softmax_j(scale <q[r, :], k[j, :]>)
//
// over the keys j that row r sees.  A row here is one (query token, head) pair
// of a sequence and a KV head: all next_n * group of them share the KV head's
// tokens (with selected columns: the group heads of one query token).
//
// One pass over the cache with a running maximum and sum.  A workgroup of four
// waves takes 16 * RT rows and a chunk of keys; wave w walks the 32-key tiles
// w, w + 4, ... of the chunk with its own maximum, sum and accumulators, and
// the four join through LDS at the end.  Both products are computed transposed
// so that nothing leaves the registers between them:
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
// q is bf16, or fp16 split exactly into two bf16 parts.  p is rounded to bf16
// for the second product (relative 2^-8 at most, the size of the bf16 result's
// own rounding); with fp16 q it is split into two bf16 parts, because fp16
// results keep eleven bits.  The sum of p, the maximum and all accumulators are fp32.
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
// The running maximum follows a new one only when that leaves a weight above
// this; most tiles rescale nothing.
constexpr float kMostWeight = 256.f;
constexpr float kLowest = -3.0e38f;          // a maximum before any key
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
// the first block (of this KV head) of every key (SPARSE; kNoKey for one to
// pass over) or of every 16th key.
constexpr uint32_t kNoKey = 0xffffffffu;

template <int D, bool SPARSE>
struct Tiles {
  Bytes k, v, ks, vs;
  const uint32_t* lds;
  uint32_t key_blocks;                       // blocks from one key of the pool to the next
  uint32_t code;                             // the lane's byte offset from its key's first code

  __device__ __forceinline__ Tiles(const AttnParams& p, const uint32_t* at)
      : k((Bytes)p.k), v((Bytes)p.v), ks((Bytes)p.k_sf), vs((Bytes)p.v_sf), lds(at),
        key_blocks(p.kv_heads * (D / 32)) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    code = (SPARSE ? 0 : c * key_blocks) * 16 + g * (D / 8);
  }

  template <bool LANES>
  __device__ __forceinline__ static Bytes at(Bytes pool, uint32_t block) {
    const Bytes p = pool + ((uint64_t)block << 4);
    return LANES ? p : scalar(p);
  }

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
template <int D, int RT, bool F16>
struct Rows {
  static constexpr int kSteps = D / 32;      // products along D
  static constexpr int kCols = D / 16;       // 16-element column groups of V
  static constexpr int kParts = F16 ? 2 : 1;
  // staging: 64 scale words, then V's rows of D/2 bytes; the pitch keeps both
  // the 16-byte writes and the 4-byte reads free of bank conflicts
  static constexpr int kPitch = D == 128 ? 80 : 40;
  static constexpr int kStageBytes = 256 + kTile * kPitch;
  struct Scores { f32x4 s[RT][2]; };         // [half]: keys 4g .. 4g+3 of row l % 16
  // Queries in LDS, shared by the waves, where registers are short.
  static constexpr bool kQueriesInLds = RT == 2;
  static constexpr int kQueryWords = RT * kParts * kSteps * 64;
  u32x4 q[kQueriesInLds ? 1 : RT][kParts][kSteps];
  u32x4* q_lds;                              // [RT][kParts][kSteps][64 lanes]
  char* lds;                                 // the wave's staging of a tile (kStageBytes)
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
    reinterpret_cast<uint32_t*>(lds)[lane] = r.s;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      char* row = lds + 256 + (half * 16 + c) * kPitch + g * (D / 8);
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
      ks[half] = byte_scale(reinterpret_cast<const uint32_t*>(lds)[half * 16 + c], g * (D / 4) / 32);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const u32x4 a = cvt_eight(r.k[0][st], ks[0]), b = cvt_eight(r.k[1][st], ks[1]);
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const u32x4 y = query(rt, part, st);
          x.s[rt][0] = mma(a, y, x.s[rt][0]);
          x.s[rt][1] = mma(b, y, x.s[rt][1]);
        }
    }
  }

  // The scales of keys that no row sees (MASKED) may hold anything and are read
  // as finite.  Others that are NaN spread: K's bytes over kLastScale become
  // the NaN byte, V's mark the rows that see their key and become 0.  first:
  // position of the tile's first key; places: the LDS entries of its keys
  // (SPARSE).
  template <bool MASKED, bool SPARSE>
  __device__ __forceinline__ void check_scales(Raw& r, int first, const uint32_t* places) {
    const int lane = threadIdx.x & 63;
    if constexpr (MASKED) {
      const bool any = SPARSE ? places[lane & 31] != kNoKey : first + (lane & 31) < most;
      r.s = any ? r.s : 0u;
    }
    // some byte of s over 252: some byte of ~s under 3
    if (__builtin_expect(__any(((~r.s - 0x03030303u) & r.s & 0x80808080u) != 0), 0))
      spread_nan<MASKED && !SPARSE>(r.s, first);
  }

  template <bool BY_ROW>
  __device__ __forceinline__ void spread_nan(uint32_t& s, int first) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int shift = 8 * (g * (D / 4) / 32);            // the block of the lane's results
#pragma nounroll
    for (int key = 0; key < kTile; ++key) {
      const uint32_t b = (__shfl(s, 32 + key) >> shift) & 0xffu;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        if (b > kLastScale && (!BY_ROW || first + key < seen[rt])) nan_rows |= 1u << rt;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t byte = 0xffu << (8 * i), b = (s >> (8 * i)) & 0xffu;
      if (b > kLastScale) s = lane & 32 ? s & ~byte : s | byte;
    }
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
    check_scales<MASKED, SPARSE>(r, first, places);
    stage(r);
    scores(r, s);
    if constexpr (MASKED) mask<SPARSE>(s, first, places);
    accumulate(s, c2);
    __builtin_amdgcn_wave_barrier();         // the staging is read
  }

  // Weights of one row tile from its scores, packed for the second product.
  // Whether a maximum was left behind shows in the weights themselves; then
  // they are formed again.
  __device__ __forceinline__ void weights(const f32x4 (&x)[2], int rt, float c2, u32x4 (&p)[kParts]) {
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
      const float next = fmaxf(m[rt], row_max(best));
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
      if constexpr (F16)
        p[1][i] = pack_bf16(w[2 * i] - bf16_lo(hi), w[2 * i + 1] - bf16_hi(hi));
    }
  }

  // The weighted sum of a tile's V.
  __device__ __forceinline__ void accumulate(const Scores& x, float c2) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    uint32_t v[8];                           // D/16 elements of keys 4g .. 4g+3 of both halves
    float vs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const char* row = lds + 256 + ((i >> 2) * 16 + 4 * g + (i & 3)) * kPitch + c * (D / 32);
      v[i] = D == 128 ? *reinterpret_cast<const uint32_t*>(row) : *reinterpret_cast<const uint16_t*>(row);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(lds + (32 + half * 16 + 4 * g) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) vs[4 * half + i] = byte_scale(w[i], c * (D / 16) / 32);
    }
    u32x4 p[RT][kParts];
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

  // Elements 2 SEL and 2 SEL + 1 of the lane's D/16.
  template <int SEL>
  __device__ __forceinline__ void add_values(const uint32_t (&v)[8], const float (&vs)[8],
                                             const u32x4 (&p)[RT][kParts]) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = cvt_pair<SEL>(v[i], vs[i]);
    u32x4 even, odd;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      even[w] = __builtin_amdgcn_perm(e[2 * w + 1], e[2 * w], 0x05040100);
      odd[w] = __builtin_amdgcn_perm(e[2 * w + 1], e[2 * w], 0x07060302);
    }
#pragma unroll
    for (int part = 0; part < kParts; ++part)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        o[rt][2 * SEL] = mma(even, p[rt][part], o[rt][2 * SEL]);
        o[rt][2 * SEL + 1] = mma(odd, p[rt][part], o[rt][2 * SEL + 1]);
      }
  }
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
// A member is a KV head and a group of 16 * RT rows.  For every member the
// units (sequences; with selected columns, query tokens) are laid end to end in
// steps of 128 keys (one tile per wave; at least one step a unit), and the S
// steps are cut into equal pieces, one per worker, as many as the chip holds at
// a time but none below min_steps.  A worker walks its piece unit by unit.  A
// unit inside one piece is finished there; one cut by piece borders leaves a
// part in each: worker j writes the part that begins its piece to slot 2j, the
// one that ends it to slot 2j + 1.  The worker that begins a unit notes the
// unit's workers for the kernel that joins the parts.
constexpr int kStep = kTile * kWaves;

struct Split {
  int steps, workers;     // S; workers in use, of p.workers
  int each, more;         // steps per piece; the first `more` pieces have one more
  __device__ __forceinline__ Split(int s, const AttnParams& p) : steps(s) {
    workers = min(p.workers, max(s / p.min_steps, 1));
    each = s / workers;
    more = s - each * workers;
  }
  __device__ __forceinline__ int border(int j) const { return j * each + min(j, more); }
  __device__ __forceinline__ int owner(int step) const {
    const int head = more * (each + 1);
    return step < head ? step / (each + 1) : more + (step - head) / each;
  }
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

template <int D, int RT, bool F16, bool SPARSE>
__global__ void __launch_bounds__(kAttnThreads, 2)
attention_kernel(const AttnParams p) {
  constexpr int kRows = 16 * RT;
  constexpr int kPitch = D + 4;              // LDS floats per row of the join
  constexpr int kEach = SPARSE ? 1 : 16;     // keys per entry of `blocks`
  constexpr int kStage = SPARSE ? kAttnStageSparse : kAttnStage;   // keys staged at a time
  using State = Rows<D, RT, F16>;
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
  // members of one piece read the same tokens: on one XCD, one after the other
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int worker = idx / members * 8 + xcd, member = idx % members;
  const int kv_head = member / p.row_groups, row0 = member % p.row_groups * kRows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform, so its branches are too
  const int c = lane & 15, g = lane >> 4;
  const int unit_rows = SPARSE ? p.group : p.next_n * p.group;

  // the worker's piece, and the unit it begins in
  int unit, unit_begin;                      // unit_begin: its first step
  int total;
  if constexpr (SPARSE) {
    total = p.units * unit_steps(p.topk);
  } else {
    int sum = 0;
    for (int b = tid; b < p.units; b += kAttnThreads) sum += unit_steps(unit_length(p, b));
    total = block_sum(sum, sums);
  }
  const Split split(__builtin_amdgcn_readfirstlane(total), p);
  if (worker >= split.workers) return;
  const int piece_begin = split.border(worker), piece_end = split.border(worker + 1);
  if constexpr (SPARSE) {
    unit = piece_begin / unit_steps(p.topk);
    unit_begin = unit * unit_steps(p.topk);
  } else {
    int base = 0;
    for (int b0 = 0; base <= piece_begin; b0 += kAttnThreads) {
      const int b = b0 + tid;
      const int mine = b < p.units ? unit_steps(unit_length(p, b)) : 0;
      int scan = mine;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int x = __shfl_up(scan, off);
        if (lane >= off) scan += x;
      }
      if (lane == 63) sums[wave] = scan;
      __syncthreads();
      int at = base + scan - mine;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += sums[w];
        base += sums[w];
      }
      if (at <= piece_begin && piece_begin < at + mine) {
        found[0] = b;
        found[1] = at;
      }
      __syncthreads();
    }
    unit = __builtin_amdgcn_readfirstlane(found[0]);
    unit_begin = __builtin_amdgcn_readfirstlane(found[1]);
  }

  const Tiles<D, SPARSE> tiles(p, blocks);
  State rows;
  rows.lds = shared + kQueryBytes + kPlaceBytes + wave * State::kStageBytes;
  rows.q_lds = queries;
  for (int at = piece_begin; at < piece_end; ++unit) {
    const int seq = SPARSE ? unit / p.next_n : unit;
    const int raw_ctx = max(p.ctx[seq], 0);
    const int ctx = min(raw_ctx, p.max_ctx);
    const int length = SPARSE ? p.topk : ctx;
    const int unit_end = unit_begin + unit_steps(length);
    const int begin = (at - unit_begin) * kStep;                 // keys of this part
    const int end = min(length, (min(unit_end, piece_end) - unit_begin) * kStep);
    const bool whole = at == unit_begin && unit_end <= piece_end;
    // keys that query token t sees
    const auto seen_by = [&](int t) { return min(max(raw_ctx - p.next_n + 1 + t, 0), ctx); };
    const int seen_sparse = SPARSE ? seen_by(unit % p.next_n) : 0;

    rows.clear();
    rows.most = ctx;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      // lanes past the last row repeat it; their results are dropped
      const int r = min(row0 + rt * 16 + c, unit_rows - 1);
      const int t = SPARSE ? 0 : r / p.group;
      rows.seen[rt] = SPARSE ? seen_sparse : seen_by(t);
      const int token = SPARSE ? unit : unit * p.next_n + t;
      const int head = kv_head * p.group + (SPARSE ? r : r - t * p.group);
      const uint16_t* src = p.q + (int64_t)token * p.q_stride + head * D + g * (D / 4);
#pragma unroll
      for (int st = 0; st < D / 32; ++st) {
        u32x4 w = *reinterpret_cast<const u32x4*>(src + st * 8), lo;
        if (p.negate) w ^= 0x80008000u;
        if constexpr (F16) {
          u32x4 hi;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] & 0xffff));
            const float y = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
            hi[i] = pack_bf16(x, y);
            // the part below bf16's eight bits; an infinity stays in hi alone
            const float rx = x - bf16_lo(hi[i]), ry = y - bf16_hi(hi[i]);
            lo[i] = pack_bf16(__builtin_isfinite(x) ? rx : 0.f, __builtin_isfinite(y) ? ry : 0.f);
          }
          w = hi;
        }
        if constexpr (State::kQueriesInLds) {
          // (every wave holds all row tiles' lanes; the first RT write one each)
          if (wave == rt) {
            queries[(rt * State::kParts * State::kSteps + st) * 64 + lane] = w;
            if (F16) queries[((rt * State::kParts + State::kParts - 1) * State::kSteps + st) * 64 + lane] = lo;
          }
        } else {
          rows.q[rt][0][st] = w;
          if (F16) rows.q[rt][State::kParts - 1][st] = lo;
        }
      }
    }

    const int32_t* table = p.bt + (int64_t)seq * p.bt_stride;
    const int32_t* index = SPARSE ? p.indices + (int64_t)unit * p.idx_stride : nullptr;
    for (int stage = begin; stage < end; stage += kStage) {
      const int stage_end = min(end, stage + kStage);
      const int n_tiles = (stage_end - stage + kTile - 1) / kTile;
      __syncthreads();                       // the last use of `blocks` is over
      for (int i = tid; i < n_tiles * (kTile / kEach); i += kAttnThreads) {
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
          first = (slot * p.kv_heads + kv_head) * (D / 32);
        }
        blocks[i] = first;
      }
      __syncthreads();
      // The wave's tiles, loaded two ahead (past the last, the last again, so that
      // every load is unconditional).  Keys that some row does not see lie in
      // the context's last 15 + 32, so only a wave's last tile can hold any.
      if (wave < n_tiles) {
        const int last = wave + (n_tiles - 1 - wave) / kWaves * kWaves;
        Raw r[3];
        int tile = wave;
        tiles.load(r[0], tile);
        tiles.load(r[1], min(tile + kWaves, last));
        const auto advance = [&](auto turn) {
          constexpr int i = decltype(turn)::value, ahead = (i + 2) % 3;
          if (State::kQueriesInLds) asm volatile("" ::: "memory");   // not kept in registers
          tiles.load(r[ahead], min(tile + 2 * kWaves, last));
          rows.template step<SPARSE, SPARSE>(r[i], 0, blocks + tile * kTile, p.c2);
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
        rows.template step<true, SPARSE>(r[0], stage + tile * kTile, blocks + tile * kTile, p.c2);
      }
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
        ((int64_t)member * p.workers + worker) * 2 + (at == piece_begin ? 0 : 1);
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
          const int t = SPARSE ? 0 : r / p.group;
          const int64_t token = SPARSE ? unit : unit * p.next_n + t;
          const int head = kv_head * p.group + (SPARSE ? r : r - t * p.group);
          const int64_t out_row = token * (p.kv_heads * p.group) + head;
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
    if (p.workers > 1 && member == 0 && tid == 0 && at == unit_begin) {
      int2 note = make_int2(0, 1);           // first slot, parts
      if (!whole) note = make_int2(2 * worker + (at == piece_begin ? 0 : 1),
                                   split.owner(unit_end - 1) - worker + 1);
      p.notes[unit] = note;
    }
    at = unit_end;
    unit_begin = unit_end;
  }
}

// Joins the parts of the units that were cut: WAVES waves per (query token,
// head).  Part 0 is in the noted slot, the next in slot 2j of the workers that
// follow.
template <int D, bool F16, int WAVES>
__global__ void __launch_bounds__(256)
attention_join_kernel(const AttnParams p, int sparse) {
  constexpr int kItems = 4 / WAVES, kPer = D / 64;
  __shared__ float part_x[WAVES > 1 ? 4 : 1][D], part_l[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t item = (int64_t)blockIdx.x * kItems + wave / WAVES;
  const int mine = wave % WAVES;
  if (item >= p.rows_heads) return;            // (whole blocks when WAVES > 1)
  const int heads = p.kv_heads * p.group;
  const int token = (int)(item / heads), head = (int)(item % heads);
  const int unit = sparse ? token : token / p.next_n;
  const int2 note = p.notes[unit];
  const int n = note.y;
  if (n <= 1) return;                          // written by its only worker
  const int kv_head = head / p.group;
  const int r = head % p.group + (sparse ? 0 : token % p.next_n * p.group);
  const int rows = 16 * p.row_tiles;
  const int64_t member = kv_head * p.row_groups + r / rows;
  const int64_t base = member * p.workers * 2;
  const auto part = [&](int i) {
    const int64_t slot = base + (i == 0 ? note.x : ((note.x >> 1) + i) * 2);
    return slot * rows + r % rows;
  };
  float m = kLowest;
  for (int i = lane; i < n; i += 64) m = fmaxf(m, p.part_ml[part(i)].x);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
  float l = 0.f, x[kPer] = {};
#pragma unroll 4
  for (int i = mine; i < n; i += WAVES) {
    const int64_t at = part(i);
    const float2 ml = p.part_ml[at];
    const float f = __builtin_amdgcn_exp2f(ml.x - m);
    l += ml.y * f;
    const float* src = p.part_o + at * D + lane * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] += src[j] * f;
  }
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) part_x[wave][lane * kPer + j] = x[j];
    if (lane == 0) part_l[wave] = l;
    __syncthreads();
    if (wave > 0) return;
    for (int w = 1; w < WAVES; ++w) {
      l += part_l[w];
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] += part_x[w][lane * kPer + j];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if constexpr (D == 128)
    reinterpret_cast<uint32_t*>(p.out + item * D)[lane] = pack_out<F16>(x[0] * inv, x[1] * inv);
  else
    p.out[item * D + lane] = (uint16_t)pack_out<F16>(x[0] * inv, 0.f);
  if (p.lse && lane == 0) p.lse[item] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
}

template <int D, bool F16, bool SPARSE>
hipError_t launch_rt(const AttnParams& p, hipStream_t s) {
  const uint32_t grid = (uint32_t)((p.workers + 7) / 8 * 8 * p.row_groups * p.kv_heads);
  if (p.row_tiles == 1)
    attention_kernel<D, 1, F16, SPARSE><<<grid, kAttnThreads, 0, s>>>(p);
  else
    attention_kernel<D, 2, F16, SPARSE><<<grid, kAttnThreads, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.workers == 1) return e;
  if (p.rows_heads <= 2048)
    attention_join_kernel<D, F16, 4><<<(uint32_t)p.rows_heads, 256, 0, s>>>(p, SPARSE);
  else
    attention_join_kernel<D, F16, 1><<<(uint32_t)((p.rows_heads + 3) / 4), 256, 0, s>>>(p, SPARSE);
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
