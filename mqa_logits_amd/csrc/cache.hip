// The paged cache's upkeep (gfx950): quantising writes of new rows, and block
// tables with slot maps from request lengths.
#include <hip/hip_runtime.h>

#include "launch.hpp"

namespace mqa {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// Quantising write
// ---------------------------------------------------------------------------
//
// A group of elements (32 along D; all D of a head for FP8) shares the scale
// 2^e with the least e for which no element exceeds the format's largest code:
//   amax = f * 2^k, f in [1, 2):  e = k - K      if f <= F
//                                     k - K + 1  otherwise,  top = F * 2^K
// (e2m1: 6 = 1.5 * 2^2; e4m3: 448 = 1.75 * 2^8).  Scaling by a power of two is
// exact, so a code is the round-to-nearest-even of the element itself: the
// conversion instructions take the scale as an operand and round once (checked
// over both formats' ties, subnormals and scale range).  A thread holds eight
// elements of one group; a group's maximum goes through 4 (MX) or D/8 (FP8)
// neighbouring lanes.  Reads and writes are whole 16-byte and 4- or 8-byte
// pieces of adjacent lanes; the kernel is bound by them: 32768 rows of 8 heads of
// 128 bf16 into MXFP4, with their values written back, take 25 us, 6.1 TB/s of
// 152 MB moved; 256 rows of 128 take the launch (3.5 us).

template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (TYPE == kF32) {
    const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    const f32x4 a = s[0], b = s[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kBF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] & 0xffff));
        x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
      }
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8]) {
  if constexpr (TYPE == kF32) {
    f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
    d[0] = f32x4{x[0], x[1], x[2], x[3]};
    d[1] = f32x4{x[4], x[5], x[6], x[7]};
  } else {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kBF16) {
        bf16x2 v;
        v[0] = (__bf16)x[2 * i];
        v[1] = (__bf16)x[2 * i + 1];
        w[i] = __builtin_bit_cast(uint32_t, v);
      } else {
        w[i] = __builtin_bit_cast(uint16_t, (_Float16)x[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x[2 * i + 1]) << 16;
      }
    }
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at) = w;
  }
}

constexpr uint32_t kInfBits = 0x7f800000u;

// Biased exponent byte of a group's scale from its largest magnitude's bits.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  constexpr uint32_t kFrac = FMT == 2 ? 0x400000u : 0x600000u;   // F = 1.5, 1.75
  constexpr int kExp = FMT == 2 ? 2 : 8;                         // K
  if (amax >= kInfBits) return 255;
  if (amax == 0) return 127;
  // subnormal maxima lie far below the least scale's range: any element of
  // theirs is below top * 2^low already
  const int k = (int)(amax >> 23);
  const int e = k - kExp + ((amax & 0x7fffffu) > kFrac ? 1 : 0);
  return (uint32_t)max(e, FMT == 0 ? 1 : 0);
}

template <int FMT, int D, int TYPE>
__global__ void __launch_bounds__(256) kv_write_kernel(const WriteParams p) {
  constexpr int kLanes = D / 8;                    // threads per head row
  constexpr int kGroup = FMT == 0 ? kLanes : 4;    // threads per scale
  const uint32_t item = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;   // below 2^31
  const uint32_t row = item / (uint32_t)p.heads;
  if (row >= p.rows) return;
  const int part = threadIdx.x % kLanes;
  const int head = (int)(item - row * p.heads);
  float x[8];
  load8<TYPE>(p.x, row * p.x_stride + head * p.x_head_stride + part * 8, x);
  const int64_t slot = p.slots[row];

  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = 1; off < kGroup; off <<= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off));
  const uint32_t byte = scale_byte<FMT>(amax);
  const bool fine = byte != 255;
  // byte 0 is 2^-127, which the conversions take by its exponent field
  const float scale = __uint_as_float((fine ? byte : 127u) << 23);
  if (!fine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
  }
  uint32_t code[2] = {0u, 0u};
  if constexpr (FMT == 2) {
    code[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[0], x[0], x[1], scale, 0);
    code[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[0], x[2], x[3], scale, 1);
    code[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[0], x[4], x[5], scale, 2);
    code[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code[0], x[6], x[7], scale, 3);
  } else {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      i16x2 c = {0, 0};
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[4 * w], x[4 * w + 1], scale, false);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[4 * w + 2], x[4 * w + 3], scale, true);
      code[w] = __builtin_bit_cast(uint32_t, c);
    }
  }
  if (slot >= 0 && slot < p.num_slots) {
    const int64_t at = slot * p.heads + head;
    if constexpr (FMT == 2) {
      *reinterpret_cast<uint32_t*>(p.pool + at * (D / 2) + part * 4) = code[0];
    } else {
      *reinterpret_cast<u32x2*>(p.pool + at * D + part * 8) = u32x2{code[0], code[1]};
    }
    if (part % kGroup == 0) {
      if constexpr (FMT == 0)
        p.scale[at] = fine ? scale : __builtin_nanf("");
      else
        p.sf[at * (D / 32) + part / 4] = (uint8_t)byte;
    }
  }
  if (p.values) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      f32x2 v;
      if constexpr (FMT == 2) {
        v = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 0)
            : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 1)
            : i == 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 2)
                     : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 3);
      } else {
        v = i & 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i >> 2], scale, true)
                  : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i >> 2], scale, false);
      }
      y[i] = v[0];
      y[i + 1] = v[1];
    }
    if (!fine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_nanf("");
    }
    store8<TYPE>(p.values, (int64_t)item * D + part * 8, y);
  }
}

template <int FMT, int D>
hipError_t launch_write_type(int type, const WriteParams& p, hipStream_t s) {
  const int64_t per = 256 / (D / 8);
  const uint32_t grid = (uint32_t)((p.rows * p.heads + per - 1) / per);
  if (type == kF32)
    kv_write_kernel<FMT, D, kF32><<<grid, 256, 0, s>>>(p);
  else if (type == kBF16)
    kv_write_kernel<FMT, D, kBF16><<<grid, 256, 0, s>>>(p);
  else
    kv_write_kernel<FMT, D, kF16><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_write_dim(int d, int type, const WriteParams& p, hipStream_t s) {
  return d == 128 ? launch_write_type<FMT, 128>(type, p, s) : launch_write_type<FMT, 64>(type, p, s);
}

// ---------------------------------------------------------------------------
// Block tables and slot maps
// ---------------------------------------------------------------------------
//
// Every block computes the two prefix sums over the batch by itself (new
// tokens, and blocks taken; at most 8192 lengths, from L2) instead of waiting
// for another kernel's, then fills its own stripe of the slots and of the
// table entries.  Slots in blocks of this step come straight from the free
// list, slots in older blocks from table entries that no block of this launch
// writes.  One launch, bound by the latency of its chain: lengths, sums, a
// binary search in LDS, one id: 5 us for 64 sequences, 7.9 us for 513 prompts of
// 480 thousand tokens.  A thread takes four slots at a time so that
// their searches and loads overlap (12.9 us for those prompts with eight slots one
// after the other).

constexpr int kSlotThreads = 512;
constexpr int kSlotMaxBatch = 8192;
constexpr int kSlotEach = 4;

struct SlotSums {
  int32_t token[kSlotMaxBatch + 1], block[kSlotMaxBatch + 1];
  int32_t old[kSlotMaxBatch];                 // tokens before this step
};

// The last b with start[b] <= k[u], for k[u] below start[n].
template <int N>
__device__ __forceinline__ void find_rows(const int32_t* start, int n, const int (&k)[N], int (&b)[N]) {
  int hi[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    b[u] = 0;
    hi[u] = n;
  }
  for (int left = n; left > 1; left = (left + 1) >> 1) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int mid = (b[u] + hi[u]) >> 1;
      const bool up = start[mid] <= k[u];
      b[u] = up ? mid : b[u];
      hi[u] = up ? hi[u] : mid;
    }
  }
}

// Blocks of n tokens (n + block_size may pass int32).
__device__ __forceinline__ int blocks_of(int n, int shift) {
  return (n >> shift) + ((n & ((1 << shift) - 1)) != 0);
}

__global__ void __launch_bounds__(kSlotThreads) kv_slots_kernel(const SlotParams p) {
  __shared__ SlotSums sums;
  __shared__ int32_t wave_tok[kSlotThreads / 64], wave_blk[kSlotThreads / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int in_block = (1 << p.bs_shift) - 1;
  int tok_base = 0, blk_base = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kSlotThreads) {
    const int b = b0 + t;
    int tok = 0, blk = 0, old = 0;
    if (b < p.batch) {
      const int len = min(max(p.ctx[b], 0), p.max_ctx);
      tok = min(max(p.new_lens[b], 0), len);
      old = len - tok;
      blk = blocks_of(len, p.bs_shift) - blocks_of(old, p.bs_shift);
    }
    int st = tok, sb = blk;                    // inclusive scans
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int a = __shfl_up(st, off), c = __shfl_up(sb, off);
      if (lane >= off) {
        st += a;
        sb += c;
      }
    }
    if (lane == 63) {
      wave_tok[wave] = st;
      wave_blk[wave] = sb;
    }
    __syncthreads();
    int before_t = tok_base, before_b = blk_base;
#pragma unroll
    for (int w = 0; w < kSlotThreads / 64; ++w) {
      if (w < wave) {
        before_t += wave_tok[w];
        before_b += wave_blk[w];
      }
      tok_base += wave_tok[w];
      blk_base += wave_blk[w];
    }
    if (b < p.batch) {
      sums.token[b] = before_t + st - tok;
      sums.block[b] = before_b + sb - blk;
      sums.old[b] = old;
    }
    __syncthreads();
  }
  if (t == 0) {
    sums.token[p.batch] = tok_base;
    sums.block[p.batch] = blk_base;
  }
  __syncthreads();

  if (blockIdx.x == 0) {
    for (int b = t; b <= p.batch; b += kSlotThreads) p.offsets[b] = sums.token[b];
    if (t == 0) p.taken[0] = blk_base;
  }
  const int64_t n_threads = (int64_t)gridDim.x * kSlotThreads;
  const int64_t me = (int64_t)blockIdx.x * kSlotThreads + t;
  // slots
  for (int64_t k0 = me; k0 < p.max_tokens; k0 += kSlotEach * n_threads) {
    int k[kSlotEach], b[kSlotEach];
    int64_t slot[kSlotEach];
#pragma unroll
    for (int u = 0; u < kSlotEach; ++u) k[u] = (int)min(k0 + u * n_threads, (int64_t)tok_base - 1);
    if (tok_base > 0) find_rows(sums.token, p.batch, k, b);
#pragma unroll
    for (int u = 0; u < kSlotEach; ++u) {
      slot[u] = -1;
      if (k0 + u * n_threads < tok_base) {
        const int old = sums.old[b[u]], pos = old + (k[u] - sums.token[b[u]]);
        const int first = blocks_of(old, p.bs_shift), j = pos >> p.bs_shift;
        const int at = sums.block[b[u]] + j - first;
        const int32_t* src = j < first ? p.bt + b[u] * p.bt_stride + j
                             : at < p.num_free ? p.free_ids + at : nullptr;
        const int id = src ? *src : -1;
        if (id >= 0 && id < p.num_blocks) slot[u] = ((int64_t)id << p.bs_shift) + (pos & in_block);
      }
    }
#pragma unroll
    for (int u = 0; u < kSlotEach; ++u)
      if (k0 + u * n_threads < p.max_tokens) p.slots[k0 + u * n_threads] = slot[u];
  }
  // table entries of the blocks taken
  for (int64_t k = me; k < blk_base; k += n_threads) {
    const int want[1] = {(int)k};
    int b[1];
    find_rows(sums.block, p.batch, want, b);
    const int first = blocks_of(sums.old[b[0]], p.bs_shift);
    p.bt[b[0] * p.bt_stride + first + ((int)k - sums.block[b[0]])] = k < p.num_free ? p.free_ids[k] : -1;
  }
}

}  // namespace

hipError_t launch_kv_write(int fmt, int d, int in_type, const WriteParams& p, hipStream_t s) {
  if (fmt == 0) return launch_write_dim<0>(d, in_type, p, s);
  if (fmt == 1) return launch_write_dim<1>(d, in_type, p, s);
  return launch_write_dim<2>(d, in_type, p, s);
}

hipError_t launch_kv_slots(const SlotParams& p, hipStream_t s) {
  // at most one block per compute unit: each repeats the prefix sums
  const int64_t per = kSlotEach * kSlotThreads;
  const int64_t want = ((int64_t)p.max_tokens + per - 1) / per;
  const uint32_t grid = (uint32_t)(want < 1 ? 1 : want > 256 ? 256 : want);
  kv_slots_kernel<<<grid, kSlotThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace mqa
