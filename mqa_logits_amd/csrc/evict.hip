// Eviction from a paged cache (gfx950): of every sequence longer than `keep`, the
// last `recent` tokens and the heaviest of the others are copied, in order, to
// blocks from a free list.
//
//   ranges   which columns the top-k chooses from: [0, ctx - recent)
//   (top-k)  the library's own, over the rows of weights
//   plan     one workgroup: new lengths, and where each sequence's blocks begin in
//            the free list and in the list of freed ones
//   move     tokens, weights, positions and tables, a chunk of a sequence per
//            workgroup.  Sources are only read, so nothing depends on the order.
#include <hip/hip_runtime.h>

#include "launch.hpp"

namespace mqa {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kPlanThreads = 1024;
constexpr int kThreads = 256;
constexpr int kChunk = 128;                  // tokens a workgroup moves

__device__ __forceinline__ int length(const EvictParams& p, int b) { return min(max(p.ctx[b], 0), p.max_ctx); }
__device__ __forceinline__ int blocks_of(const EvictParams& p, int n) { return (n + (1 << p.bs_shift) - 1) >> p.bs_shift; }

__global__ void __launch_bounds__(256) ranges_kernel(const EvictParams p) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= p.batch) return;
  const int n = length(p, b);
  p.k_start[b] = 0;
  p.k_end[b] = n > p.keep ? n - p.recent : 0;
}

// Exclusive sum over the block, and the total; sums: LDS, a word per wave.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t scan = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t y = __shfl_up((long long)scan, off);
    if (lane >= off) scan += y;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = scan;
  __syncthreads();
  int64_t before = scan - x;
  total = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w < wave) before += sums[w];
    total += sums[w];
  }
  return before;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const EvictParams p) {
  __shared__ int64_t sums[kPlanThreads / 64];
  int64_t taken = 0, freed = 0, total;
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const int n = b < p.batch ? length(p, b) : 0;
    const bool cut = n > p.keep;
    int chosen = 0;                          // tokens the top-k found before its padding
    if (cut && p.keep > p.recent) {
      const int32_t* row = p.kept + (int64_t)b * p.kept_stride;
      int hi = p.keep - p.recent;
      while (chosen < hi) {
        const int mid = (chosen + hi) >> 1;
        if (row[mid] >= 0) chosen = mid + 1; else hi = mid;
      }
    }
    const int64_t want = cut ? blocks_of(p, chosen + p.recent) : 0;
    const int64_t at = taken + block_scan(want, sums, total);
    taken += total;
    // left as it was if the list does not reach
    const bool moved = cut && at + want <= p.num_free;
    const int64_t back = freed + block_scan(moved ? blocks_of(p, n) : 0, sums, total);
    freed += total;
    if (b < p.batch) {
      p.plan[b] = EvictPlan{moved ? chosen : -1, cut, (int32_t)min(at, (int64_t)p.num_free), (int32_t)back};
      p.new_ctx[b] = moved ? chosen + p.recent : n;
    }
  }
  if (threadIdx.x == 0) {
    p.counts[0] = (int32_t)taken;
    p.counts[1] = (int32_t)freed;
  }
}

template <class T>
__device__ __forceinline__ void copy_rows(uint8_t* data, int64_t bytes, const int64_t* from, const int64_t* to, int tokens) {
  const int pieces = (int)(bytes / sizeof(T));
  for (int i = threadIdx.x; i < tokens * pieces; i += kThreads) {
    const int t = i / pieces, c = i - t * pieces;
    if (from[t] >= 0) *reinterpret_cast<T*>(data + to[t] * bytes + c * sizeof(T)) = *reinterpret_cast<const T*>(data + from[t] * bytes + c * sizeof(T));
  }
}

__global__ void __launch_bounds__(kThreads) move_kernel(const EvictParams p) {
  __shared__ int64_t from[kChunk], to[kChunk];
  const int b = blockIdx.y, tid = threadIdx.x;
  const EvictPlan plan = p.plan[b];
  const int n = length(p, b);
  const bool moved = plan.chosen >= 0;
  const int left = moved ? plan.chosen + p.recent : n;       // tokens afterwards
  const int32_t* table = p.bt + (int64_t)b * p.bt_stride;
  const int mask = (1 << p.bs_shift) - 1;
  const int first = blockIdx.x * kChunk;
  // tokens, positions and weights
  int32_t* kept = p.kept + (int64_t)b * p.kept_stride;
  if (tid < kChunk) {
    const int i = first + tid;
    int64_t src = -1, dst = -1;
    if (i < left) {
      const int at = !moved ? i : i < plan.chosen ? kept[i] : n - p.recent + (i - plan.chosen);
      if (moved) {
        const int id = table[at >> p.bs_shift], free_id = p.free_ids[plan.first + (i >> p.bs_shift)];
        if (id >= 0 && id < p.num_blocks && free_id >= 0 && free_id < p.num_blocks) {
          src = ((int64_t)id << p.bs_shift) + (at & mask);
          dst = ((int64_t)free_id << p.bs_shift) + (i & mask);
        }
      }
      if (i < p.keep && (!plan.cut || (moved && i >= plan.chosen))) kept[i] = at;
      if (i < p.max_ctx) p.new_weights[b * p.new_weights_stride + i] = p.weights[b * p.weights_stride + at];
    } else {
      if (i < p.keep && (!plan.cut || moved)) kept[i] = -1;
      if (i < p.max_ctx) p.new_weights[b * p.new_weights_stride + i] = 0.f;
    }
    if (plan.cut && !moved && i < p.keep) kept[i] = -1;
    from[tid] = src;
    to[tid] = dst;
  }
  __syncthreads();
  // this chunk's entries of the table, of the freed blocks
  const int entries = kChunk >> p.bs_shift, width = blocks_of(p, p.max_ctx);
  if (tid < entries) {
    const int e = blockIdx.x * entries + tid, held = blocks_of(p, n);
    if (e < width)
      p.new_bt[b * p.new_bt_stride + e] =
          e >= blocks_of(p, left) ? -1 : moved ? p.free_ids[plan.first + e] : table[e];
    if (moved && e < held) p.freed[plan.freed + e] = table[e];
  }
  // padding of the freed blocks' list: behind the last one
  const int64_t pad = p.counts[1] + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * entries + tid;
  if (tid < entries && pad < (int64_t)p.batch * width) p.freed[pad] = -1;
  const int tokens = min(left - first, kChunk);
  if (!moved || tokens <= 0) return;
  for (int i = 0; i < p.num_pools; ++i) {
    uint8_t* data = static_cast<uint8_t*>(p.pools[i].data);
    const int64_t bytes = p.pools[i].bytes;
    switch (p.pools[i].width) {
      case 16: copy_rows<u32x4>(data, bytes, from, to, tokens); break;
      case 8: copy_rows<u32x2>(data, bytes, from, to, tokens); break;
      case 4: copy_rows<uint32_t>(data, bytes, from, to, tokens); break;
      case 2: copy_rows<uint16_t>(data, bytes, from, to, tokens); break;
      default: copy_rows<uint8_t>(data, bytes, from, to, tokens);
    }
  }
}

}  // namespace

hipError_t launch_evict(const EvictParams& p, hipStream_t s) {
  ranges_kernel<<<(p.batch + 255) / 256, 256, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.keep > p.recent) {
    const TopkParams t{p.weights, p.weights_stride, p.k_start, p.k_end, p.batch, p.max_ctx, p.keep - p.recent,
                       p.kept, p.kept_stride};
    e = launch_topk(kF32, t, s);
    if (e != hipSuccess) return e;
  }
  plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = p.max_ctx > p.keep ? p.max_ctx : p.keep;
  move_kernel<<<dim3((rows + kChunk - 1) / kChunk, p.batch), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace mqa
