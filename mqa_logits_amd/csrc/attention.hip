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

#include "launch.hpp"

namespace mqa {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kAttnThreads = 64 * kWaves;
constexpr int kTile = 32;                    // keys per wave and step
// Scale bytes above this could overflow fp32 (6 * 2^126): they count as NaN.
constexpr uint32_t kLastScale = 252;
// The running maximum follows a new one only when it is left this far behind
// (in powers of two): p stays below 2^8, and most tiles rescale nothing.
constexpr float kSlack = 8.f;
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

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

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

// A wave's tile as loaded: 16 + 16 keys.
template <int D>
struct Raw {
  u32x4 k[2];             // [half]: D/4 elements of key l % 16 (D = 64: x, y)
  uint32_t ks[2];         // their scale byte
  uint32_t v[8];          // [4 * half + i]: D/16 elements of key 4g + i
  uint32_t vs[8];         // their scale byte
};

template <int D, bool SPARSE>
struct Tiles {
  const uint8_t *k, *ks, *v, *vs;            // at this KV head
  int64_t row_bytes, sf_bytes;               // from one token to the next
  const int32_t* lds;                        // slots: per key (SPARSE) or per 16 keys

  __device__ __forceinline__ void load(Raw<D>& r, int tile) const {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    constexpr int kPart = D / 8;                          // bytes of a quarter of a row
    const int kblk = g * (D / 4) / 32, vblk = c * (D / 16) / 32;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint8_t *kp, *ksp;
      const uint8_t *vp[4], *vsp[4];
      if constexpr (SPARSE) {
        const int32_t* s = lds + tile * kTile + half * 16;
        const int64_t sk = max(s[c], 0);
        kp = k + sk * row_bytes;
        ksp = ks + sk * sf_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t sv = max(s[4 * g + i], 0);
          vp[i] = v + sv * row_bytes;
          vsp[i] = vs + sv * sf_bytes;
        }
      } else {
        const int64_t s = __builtin_amdgcn_readfirstlane(lds[tile * 2 + half]);
        kp = k + s * row_bytes + (int32_t)(c * row_bytes);
        ksp = ks + s * sf_bytes + (int32_t)(c * sf_bytes);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vp[i] = v + s * row_bytes + (int32_t)((4 * g + i) * row_bytes);
          vsp[i] = vs + s * sf_bytes + (int32_t)((4 * g + i) * sf_bytes);
        }
      }
      if constexpr (D == 128) {
        r.k[half] = *reinterpret_cast<const u32x4*>(kp + g * kPart);
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(kp + g * kPart);
        r.k[half] = u32x4{w[0], w[1], 0u, 0u};
      }
      r.ks[half] = ksp[kblk];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128)
          r.v[4 * half + i] = *reinterpret_cast<const uint32_t*>(vp[i] + c * 4);
        else
          r.v[4 * half + i] = *reinterpret_cast<const uint16_t*>(vp[i] + c * 2);
        r.vs[4 * half + i] = vsp[i][vblk];
      }
    }
  }
};

// Rows' state of one wave: queries, running maximum and sum, accumulators.
template <int D, int RT, bool F16>
struct Rows {
  static constexpr int kSteps = D / 32;      // products along D
  static constexpr int kCols = D / 16;       // 16-element column groups of V
  static constexpr int kParts = F16 ? 2 : 1;
  u32x4 q[RT][kParts][kSteps];
  f32x4 o[RT][kCols];
  float m[RT], l[RT];
  int seen[RT];                              // keys the lane's row sees
  uint32_t nan_rows;                         // bit rt: the lane's results are NaN

  // One tile.  first: position of its first key; full: every key is seen by
  // every row.  valid: bit 4 * half + i is set if key 4g + i of the half is
  // one to attend to (SPARSE).
  template <bool SPARSE>
  __device__ __forceinline__ void step(const Raw<D>& r, int first, bool full, uint32_t valid,
                                       float c2) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    // scores
    f32x4 s[RT][2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float ks = scale_of(r.ks[half] > kLastScale ? 255u : r.ks[half]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][half] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x4 a = cvt_eight(r.k[half][st], ks);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            s[rt][half] = mma(a, q[rt][part][st], s[rt][half]);
      }
    }
    // V scales: keys that no row sees may hold anything and are read as
    // finite; a scale that is NaN marks the rows that see its key
    uint32_t vs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) vs[i] = r.vs[i];
    if (!full) {
      int most = seen[0];
#pragma unroll
      for (int rt = 1; rt < RT; ++rt) most = max(most, seen[rt]);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) most = max(most, __shfl_xor(most, off));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = first + (i >> 2) * 16 + 4 * g + (i & 3);
        const bool use = SPARSE ? (valid >> i) & 1 : key < most;
        vs[i] = use ? vs[i] : 0u;
      }
    }
    uint32_t top = vs[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = max(top, vs[i]);
    if (__any(top > kLastScale)) {
      // the lane's results lie in scale block g * (D/4) / 32; lanes 16 gs +
      // (block * 32 / (D/16)) hold that block's bytes of keys 4 gs + i
      const int col = (g * (D / 4) / 32) * (512 / D);
      for (int gs = 0; gs < 4; ++gs)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = __shfl(vs[i], gs * 16 + col);
          const int key = first + (i >> 2) * 16 + 4 * gs + (i & 3);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            if (b > kLastScale && (SPARSE || key < seen[rt])) nan_rows |= 1u << rt;
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) vs[i] = vs[i] > kLastScale ? 0u : vs[i];
    }
    // softmax weights
    u32x4 p[RT][kParts];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = s[rt][i >> 2][i & 3] * c2;
      if (!full) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = first + (i >> 2) * 16 + 4 * g + (i & 3);
          const bool use = SPARSE ? (valid >> i) & 1 : key < seen[rt];
          x[i] = use ? x[i] : -__builtin_inff();
        }
      }
      float top_x = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top_x = fmaxf(top_x, fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      if (__any(top_x > m[rt] + kSlack)) {
        const float next = fmaxf(m[rt], row_max(top_x));
        const float f = __builtin_amdgcn_exp2f(m[rt] - next);
        m[rt] = next;
        l[rt] *= f;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[rt][j][i] *= f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __builtin_amdgcn_exp2f(x[i] - m[rt]);
        l[rt] += x[i];
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t hi = pack_bf16(x[2 * w], x[2 * w + 1]);
        p[rt][0][w] = hi;
        if constexpr (F16)
          p[rt][1][w] = pack_bf16(x[2 * w] - bf16_lo(hi), x[2 * w + 1] - bf16_hi(hi));
      }
    }
    // weighted sum of V
    add_values<0>(r, vs, p);
    add_values<1>(r, vs, p);
    if constexpr (D == 128) {
      add_values<2>(r, vs, p);
      add_values<3>(r, vs, p);
    }
  }

  // Elements 2 SEL and 2 SEL + 1 of the lane's D/16.
  template <int SEL>
  __device__ __forceinline__ void add_values(const Raw<D>& r, const uint32_t (&vs)[8],
                                             const u32x4 (&p)[RT][kParts]) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = cvt_pair<SEL>(r.v[i], scale_of(vs[i]));
    u32x4 even, odd;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      even[w] = __builtin_amdgcn_perm(e[2 * w + 1], e[2 * w], 0x05040100);
      odd[w] = __builtin_amdgcn_perm(e[2 * w + 1], e[2 * w], 0x07060302);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
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

// Workgroups that read the same tokens (row groups of a KV head, KV heads of a
// token) follow each other on one XCD, so the shared lines stay in its L2;
// such groups go round the eight XCDs.
__device__ __forceinline__ bool locate(const AttnParams& p, int& member, int& unit, int& chunk) {
  const int gs = p.row_groups * p.kv_heads;
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int group = idx / gs * 8 + xcd;
  member = idx % gs;
  if (group >= p.units * p.chunks) return false;
  unit = group % p.units;
  chunk = group / p.units;
  return true;
}

template <int D, int RT, bool F16, bool SPARSE>
__global__ void __launch_bounds__(kAttnThreads)
attention_kernel(const AttnParams p) {
  constexpr int kRows = 16 * RT;
  constexpr int kPitch = D + 4;              // LDS floats per row of the join
  __shared__ int32_t slots[SPARSE ? kAttnMaxChunk : kAttnMaxChunk / 16];
  __shared__ float join[kWaves * 16 * kPitch];
  __shared__ float wave_m[kWaves][kRows], wave_l[kWaves][kRows];

  int member, unit, chunk;
  if (!locate(p, member, unit, chunk)) return;
  const int kv_head = member / p.row_groups, row0 = member % p.row_groups * kRows;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;

  // unit: a sequence, or (SPARSE) a query token
  const int seq = SPARSE ? unit / p.next_n : unit;
  const int raw_ctx = max(p.ctx[seq], 0);
  const int ctx = min(raw_ctx, p.max_ctx);
  const int unit_rows = SPARSE ? p.group : p.next_n * p.group;
  // keys of query token t: those before raw_ctx - next_n + 1 + t
  const int t_sparse = SPARSE ? unit % p.next_n : 0;
  const int seen_sparse = min(max(raw_ctx - p.next_n + 1 + t_sparse, 0), ctx);
  const int length = SPARSE ? p.topk : ctx;
  const int begin = chunk * p.chunk;
  const int end = min(length, begin + p.chunk);
  if (chunk > 0 && begin >= length) return;
  const int n_chunks = max(1, (length + p.chunk - 1) / p.chunk);

  const int32_t* table = p.bt + (int64_t)seq * p.bt_stride;
  if constexpr (SPARSE) {
    const int32_t* index = p.indices + (int64_t)unit * p.idx_stride;
    const int padded = (end - begin + kTile - 1) / kTile * kTile;
    for (int i = tid; i < padded; i += kAttnThreads) {
      const int j = begin + i < end ? index[begin + i] : -1;
      int slot = -1;
      if (j >= 0 && j < seen_sparse) {
        const int id = min(max(table[j >> p.bs_shift], 0), p.num_blocks - 1);
        slot = (id << p.bs_shift) + (j & ((1 << p.bs_shift) - 1));
      }
      slots[i] = slot;
    }
  } else {
    const int n16 = (end - begin + kTile - 1) / kTile * 2;
    for (int i = tid; i < n16; i += kAttnThreads) {
      const int j = begin + i * 16;
      int slot = 0;
      if (j < end) {
        const int id = min(max(table[j >> p.bs_shift], 0), p.num_blocks - 1);
        slot = (id << p.bs_shift) + (j & ((1 << p.bs_shift) - 1));
      }
      slots[i] = slot;
    }
  }

  Rows<D, RT, F16> rows;
  rows.nan_rows = 0;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = row0 + rt * 16 + c;
    const int t = SPARSE ? 0 : r / p.group;
    const bool real = r < unit_rows;
    rows.seen[rt] = !real ? 0
                    : SPARSE ? seen_sparse
                             : min(max(raw_ctx - p.next_n + 1 + t, 0), ctx);
    rows.m[rt] = kLowest;
    rows.l[rt] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) rows.o[rt][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int token = SPARSE ? unit : unit * p.next_n + t;
    const int head = kv_head * p.group + (SPARSE ? r : r - t * p.group);
    const uint16_t* src = p.q + (int64_t)token * p.q_stride + head * D + g * (D / 4);
#pragma unroll
    for (int st = 0; st < D / 32; ++st) {
      u32x4 w{0u, 0u, 0u, 0u};
      if (real) w = *reinterpret_cast<const u32x4*>(src + st * 8);
      if (p.negate) w ^= 0x80008000u;
      if constexpr (F16) {
        u32x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] & 0xffff));
          const float b = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
          hi[i] = pack_bf16(a, b);
          // the part below bf16's eight bits; an infinity stays in hi alone
          const float ra = a - bf16_lo(hi[i]), rb = b - bf16_hi(hi[i]);
          lo[i] = pack_bf16(__builtin_isfinite(a) ? ra : 0.f, __builtin_isfinite(b) ? rb : 0.f);
        }
        rows.q[rt][0][st] = hi;
        rows.q[rt][1][st] = lo;
      } else {
        rows.q[rt][0][st] = w;
      }
    }
  }
  __syncthreads();

  // keys every row of the workgroup sees (rows in order of t)
  const int least = SPARSE ? 0 : min(max(raw_ctx - p.next_n + 1 + row0 / p.group, 0), ctx);
  const int head_off = kv_head * (D / 2), sf_off = kv_head * (D / 32);
  const Tiles<D, SPARSE> tiles{p.k + head_off, p.k_sf + sf_off, p.v + head_off, p.v_sf + sf_off,
                               (int64_t)p.kv_heads * (D / 2), (int64_t)p.kv_heads * (D / 32), slots};
  const int n_tiles = end > begin ? (end - begin + kTile - 1) / kTile : 0;
  Raw<D> now, next;
  if (wave < n_tiles) tiles.load(now, wave);
  for (int tile = wave; tile < n_tiles; tile += kWaves) {
    if (tile + kWaves < n_tiles) tiles.load(next, tile + kWaves);
    uint32_t valid = 0xff;
    bool full;
    if constexpr (SPARSE) {
      valid = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        valid |= (slots[tile * kTile + (i >> 2) * 16 + 4 * g + (i & 3)] >= 0 ? 1u : 0u) << i;
      full = false;
    } else {
      full = begin + (tile + 1) * kTile <= least;
    }
    rows.template step<SPARSE>(now, begin + tile * kTile, full, valid, p.c2);
    now = next;
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
    float* dst = join + (wave * 16 + c) * kPitch + g * (D / 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        dst[i * (D / 16) + j] = is_nan ? __builtin_nanf("") : rows.o[rt][j][i] * f;
    __syncthreads();
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
        for (int w = 0; w < kWaves; ++w) x[j] += join[(w * 16 + jr) * kPitch + jc + j];
      }
      const int t = SPARSE ? 0 : r / p.group;
      const int64_t token = SPARSE ? unit : unit * p.next_n + t;
      const int head = kv_head * p.group + (SPARSE ? r : r - t * p.group);
      const int64_t at = token * (p.kv_heads * p.group) + head;
      if (n_chunks == 1) {
        const float inv = lj == 0.f ? 0.f : 1.f / lj;
        uint32_t w[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) w[j] = pack_out<F16>(x[2 * j] * inv, x[2 * j + 1] * inv);
        uint32_t* dst_out = reinterpret_cast<uint32_t*>(p.out + at * D + jc);
        if constexpr (D == 128)
          *reinterpret_cast<u32x4*>(dst_out) = u32x4{w[0], w[1], w[2], w[3]};
        else
          *reinterpret_cast<u32x2*>(dst_out) = u32x2{w[0], w[1]};
        if (p.lse && (tid & 15) == 0)
          p.lse[at] = lj == 0.f ? -__builtin_inff() : (mj + __builtin_log2f(lj)) * kLn2;
      } else {
        const int64_t part = (int64_t)chunk * p.rows_heads + at;
        f32x4* dst_o = reinterpret_cast<f32x4*>(p.part_o + part * D + jc);
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
          dst_o[j] = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
        if ((tid & 15) == 0) p.part_ml[part] = make_float2(mj, lj);
      }
    }
    if (rt + 1 < RT) __syncthreads();
  }
}

// Joins the chunks of split contexts: one wave per (query token, head).
template <int D, bool F16>
__global__ void __launch_bounds__(256)
attention_join_kernel(const AttnParams p, int sparse) {
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (at >= p.rows_heads) return;
  const int token = (int)(at / (p.kv_heads * p.group));
  const int length = sparse ? p.topk : min(max(p.ctx[token / p.next_n], 0), p.max_ctx);
  const int n = (length + p.chunk - 1) / p.chunk;
  if (n <= 1) return;                          // written by the only chunk
  float m = kLowest;
  for (int i = lane; i < n; i += 64) m = fmaxf(m, p.part_ml[i * p.rows_heads + at].x);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
  float l = 0.f;
  constexpr int kPer = D / 64;
  float x[kPer] = {};
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 ml = p.part_ml[i * p.rows_heads + at];
    const float f = __builtin_amdgcn_exp2f(ml.x - m);
    l += ml.y * f;
    const float* src = p.part_o + (i * p.rows_heads + at) * D + lane * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] += src[j] * f;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if constexpr (D == 128) {
    reinterpret_cast<uint32_t*>(p.out + at * D)[lane] = pack_out<F16>(x[0] * inv, x[1] * inv);
  } else {
    p.out[at * D + lane] = (uint16_t)pack_out<F16>(x[0] * inv, 0.f);
  }
  if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
}

template <int D, bool F16, bool SPARSE>
hipError_t launch_rt(const AttnParams& p, hipStream_t s) {
  const int64_t groups = (int64_t)p.units * p.chunks;
  const int64_t grid = (groups + 7) / 8 * 8 * p.row_groups * p.kv_heads;
  if (p.row_tiles == 1)
    attention_kernel<D, 1, F16, SPARSE><<<(uint32_t)grid, kAttnThreads, 0, s>>>(p);
  else if (p.row_tiles == 2)
    attention_kernel<D, 2, F16, SPARSE><<<(uint32_t)grid, kAttnThreads, 0, s>>>(p);
  else
    attention_kernel<D, 4, F16, SPARSE><<<(uint32_t)grid, kAttnThreads, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.chunks == 1) return e;
  attention_join_kernel<D, F16><<<(uint32_t)((p.rows_heads + 3) / 4), 256, 0, s>>>(p, SPARSE);
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
