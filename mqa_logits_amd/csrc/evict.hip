// Eviction from a paged cache (gfx950): of every sequence longer than `keep`, the
// last `recent` tokens and the heaviest of the others are copied, in order, to
// blocks from a free list.
//
//   ranges   which columns the choice is made from: [0, ctx - recent)
//   (top-k)  the library's own, over the rows of weights; or, for a few long rows, a
//            radix selection over many workgroups (below)
//   plan     one workgroup: new lengths, and where each sequence's blocks begin in
//            the free list and in the list of freed ones
//   move     tokens, weights, positions and tables, a chunk of a sequence per
//            workgroup.  Sources are only read, so nothing depends on the order.
//
// Bound by the bytes: a kept token is read once and written once, a row of weights
// read a few times (from the L2 after the first).  Chosen tokens lie apart, so what a
// token has in a pool costs whole cache lines: with one KV head 64 bytes of K, 64 of
// V, 128 of the indexer's keys and three scales of 4 cost about 430 bytes of reads
// instead of 268.
//   64 sequences of up to 32768 tokens to 4096, one KV head and an index: 75 us, 61 where
//     the last-level cache still holds the pools from the call before
//     (top-k 25, plan 3 to 5, move 32: 178 MB of lines at 5.5 TB/s);
//   one of 131072 to 16384, eight KV heads: 40 us a call from Python, which its eight
//     launches bound (selection 24 us on the device, plan 3, move 9);
//   3 of up to 600 to 128: 28 us a call, the same with four (15 on the device).
#include <hip/hip_runtime.h>

#include "launch.hpp"

namespace mqa {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kPlanThreads = 1024;
constexpr int kThreads = 256;
constexpr int kChunk = 128;                  // tokens a workgroup moves at most
constexpr int kTail = 2048;                  // columns a workgroup writes down where no token stays
constexpr int kAhead = 4;                    // pieces a thread has in flight

__device__ __forceinline__ int length(const EvictParams& p, int b) { return min(max(p.ctx[b], 0), p.max_ctx); }
__device__ __forceinline__ int blocks_of(const EvictParams& p, int n) { return (n + (1 << p.bs_shift) - 1) >> p.bs_shift; }

// Also clears the selection's counts.
__global__ void __launch_bounds__(256) ranges_kernel(const EvictParams p, uint32_t* counts, int n_counts) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  for (int i = b; i < n_counts; i += gridDim.x * 256) counts[i] = 0;
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
  for (int w = 0; w < (int)blockDim.x / 64; ++w) {
    if (w < wave) before += sums[w];
    total += sums[w];
  }
  return before;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const EvictParams p) {
  __shared__ int64_t sums[kPlanThreads / 64];
  int64_t taken = 0, freed = 0, total;
  for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const int n = b < p.batch ? length(p, b) : 0;
    const bool cut = n > p.keep;
    int chosen = 0;                          // tokens the top-k found before its padding
    if (cut && p.keep > p.recent) {
      const int32_t* row = p.kept + (int64_t)b * p.kept_stride;
      int hi = p.keep - p.recent;
      if (row[hi - 1] >= 0) chosen = hi;     // (as good as always)
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

// ---------------------------------------------------------------------------
// Selection from a few long rows
// ---------------------------------------------------------------------------
//
// The k-th largest key of a row, from its highest bits down: three launches count the
// keys by 11, 11 and 10 bits of those that agree with what is known of it.  (Counts
// of integers do not depend on the order in which they are added.)  Then every
// workgroup counts what its columns give, and writes them behind the others'.
// Whole evictions in a graph, by the top-k's workgroup a row and by this, an eighth of
// the columns kept: one row of 16384 columns 17 us against 27, of 32768 24 against 27,
// of 40000 48 against 27, of 131072 124 against 29; 64 rows of 16384 21 against 35, of
// 33000 47 against 48, of 65536 90 against 62; 96 of 40000 65 against 63, 256 95 against 115.
constexpr int kSelectThreads = 256, kEach = 8, kColumns = kSelectThreads * kEach;   // of a workgroup
constexpr int kBins = 2048;
constexpr int kSelectRows = 64, kSelectFrom = 32768;   // rows at most, of more columns than that

struct Choice {
  uint32_t key;              // the least that is taken
  uint32_t equal;            // how many equal to it
};

// What is known of that key after a pass: its highest bits, and how many of the keys
// that agree with them are taken (~0: every candidate is, there are fewer).
struct Known {
  uint32_t high, left;
};

struct SelectParams {
  EvictParams e;
  Known* known;              // [batch][2]: after the first pass, the second
  uint32_t* bins;            // [batch][3][kBins]
  uint2* counts;             // [batch][groups]: columns above the key, equal to it
  Choice* choice;            // [batch]
  int groups;
};

// Ascending unsigned order of the values (by IEEE total order); -inf is no candidate.
__device__ __forceinline__ uint32_t order(uint32_t bits) { return bits ^ (uint32_t((int32_t)bits >> 31) | 0x80000000u); }
constexpr uint32_t kNoBits = 0xff800000u;

// What is known once PASSES passes have counted; the row's first workgroup leaves it
// for the next launch.
template <int PASSES>
__device__ __forceinline__ Known known(const SelectParams& p, int b, int k) {
  if constexpr (PASSES == 0) return Known{0, (uint32_t)k};
  __shared__ uint32_t sums[kSelectThreads / 64], found[2];
  constexpr int kMine = kBins / kSelectThreads;
  const uint32_t* bins = p.bins + ((int64_t)b * 3 + PASSES - 1) * kBins;
  Known now{0, (uint32_t)k};
  if constexpr (PASSES > 1) now = p.known[b * 2 + PASSES - 2];
  if (now.left != ~0u) {
    // bins from the last down, kMine for each thread
    const int first = kBins - 1 - (int)threadIdx.x * kMine;
    uint32_t mine[kMine], sum = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) sum += mine[i] = bins[first - i];
    uint32_t scan = sum;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t y = __shfl_up(scan, off);
      if (lane >= off) scan += y;
    }
    if (threadIdx.x == 0) {
      found[0] = 0;
      found[1] = ~0u;
    }
    if (lane == 63) sums[wave] = scan;
    __syncthreads();
    uint32_t above = scan - sum;
    for (int w = 0; w < wave; ++w) above += sums[w];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (above < now.left && now.left <= above + mine[i]) {
        found[0] = first - i;
        found[1] = now.left - above;
      }
      above += mine[i];
    }
    __syncthreads();
    now.high = now.high << (PASSES == 3 ? 10 : 11) | found[0];
    now.left = found[1];
  }
  if (PASSES < 3 && blockIdx.x == 0 && threadIdx.x == 0) p.known[b * 2 + PASSES - 1] = now;
  return now;
}

// This workgroup's columns: thread's i-th of kEach is first + (i / 4 * 256 + tid) * 4 + i % 4.
__device__ __forceinline__ int column(int first, int i) {
  return first + (i / 4 * kSelectThreads + (int)threadIdx.x) * 4 + i % 4;
}
__device__ __forceinline__ void load_columns(const float* row, int first, int n, uint32_t (&bits)[kEach]) {
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = column(first, i);
    bits[i] = j < n ? __float_as_uint(row[j]) : kNoBits;
  }
}

template <int PASS>
__global__ void __launch_bounds__(kSelectThreads) count_bits_kernel(const SelectParams p) {
  __shared__ uint32_t bins[kBins];
  const int b = blockIdx.y, first = blockIdx.x * kColumns, n = p.e.k_end[b];
  if (first >= n) return;
  uint32_t bits[kEach];
  load_columns(p.e.weights + (int64_t)b * p.e.weights_stride, first, n, bits);
  for (int i = threadIdx.x; i < kBins; i += kSelectThreads) bins[i] = 0;
  const Known now = known<PASS>(p, b, p.e.keep - p.e.recent);
  if (now.left == ~0u) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t key = order(bits[i]);
    const bool agrees = PASS == 0 || key >> (PASS == 1 ? 21 : 10) == now.high;
    if (bits[i] != kNoBits && agrees)
      atomicAdd(&bins[PASS == 0 ? key >> 21 : PASS == 1 ? key >> 10 & 0x7ffu : key & 0x3ffu], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kSelectThreads)
    if (bins[i]) atomicAdd(&p.bins[((int64_t)b * 3 + PASS) * kBins + i], bins[i]);
}

__global__ void __launch_bounds__(kSelectThreads) count_columns_kernel(const SelectParams p) {
  __shared__ uint32_t above[kSelectThreads / 64], equal[kSelectThreads / 64];
  const int b = blockIdx.y, first = blockIdx.x * kColumns, n = p.e.k_end[b];
  if (first >= n) return;
  uint32_t bits[kEach];
  load_columns(p.e.weights + (int64_t)b * p.e.weights_stride, first, n, bits);
  const Known last = known<3>(p, b, p.e.keep - p.e.recent);
  const Choice c{last.left == ~0u ? 0 : last.high, last.left};   // (0: no key is below)
  uint32_t g = 0, e = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t key = order(bits[i]);
    g += bits[i] != kNoBits && key > c.key;
    e += bits[i] != kNoBits && key == c.key;
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    g += __shfl_xor(g, off);
    e += __shfl_xor(e, off);
  }
  if ((threadIdx.x & 63) == 0) {
    above[threadIdx.x >> 6] = g;
    equal[threadIdx.x >> 6] = e;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    g = e = 0;
    for (int w = 0; w < kSelectThreads / 64; ++w) {
      g += above[w];
      e += equal[w];
    }
    p.counts[(int64_t)b * p.groups + blockIdx.x] = make_uint2(g, e);
    if (blockIdx.x == 0) p.choice[b] = c;
  }
}

__global__ void __launch_bounds__(kSelectThreads) write_columns_kernel(const SelectParams p) {
  __shared__ uint2 sums[kSelectThreads / 64];
  const int b = blockIdx.y, first = blockIdx.x * kColumns, n = p.e.k_end[b], tid = threadIdx.x;
  int32_t* kept = p.e.kept + (int64_t)b * p.e.kept_stride;
  const int k = p.e.keep - p.e.recent, groups = (n + kColumns - 1) / kColumns;
  const Choice c = n > 0 ? p.choice[b] : Choice{0, 0};
  const auto all = [&](uint2 x) {            // over the workgroup
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      x.x += __shfl_xor(x.x, off);
      x.y += __shfl_xor(x.y, off);
    }
    __syncthreads();
    if ((tid & 63) == 0) sums[tid >> 6] = x;
    __syncthreads();
    x = make_uint2(0, 0);
    for (int w = 0; w < kSelectThreads / 64; ++w) {
      x.x += sums[w].x;
      x.y += sums[w].y;
    }
    return x;
  };
  // columns of the groups before this one, and of all
  uint2 mine = make_uint2(0, 0), total = mine;
  for (int i = tid; i < groups; i += kSelectThreads) {
    const uint2 x = p.counts[(int64_t)b * p.groups + i];
    total.x += x.x;
    total.y += x.y;
    if (i < (int)blockIdx.x) {
      mine.x += x.x;
      mine.y += x.y;
    }
  }
  uint2 before = all(mine);
  total = all(total);
  const uint32_t chosen = total.x + min(total.y, c.equal);
  // behind them: -1
  for (int i = (int)chosen + blockIdx.x * kSelectThreads + tid; i < k; i += gridDim.x * kSelectThreads) kept[i] = -1;
  if (first >= n) return;
  uint32_t bits[kEach];
  load_columns(p.e.weights + (int64_t)b * p.e.weights_stride, first, n, bits);
#pragma unroll
  for (int part = 0; part < kEach / 4; ++part) {
    // 1024 columns, four in a row for each thread: what the threads before give
    uint2 own = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = bits[part * 4 + i], key = order(x);
      own.x += x != kNoBits && key > c.key;
      own.y += x != kNoBits && key == c.key;
    }
    uint2 scan = own;
    const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t gx = __shfl_up(scan.x, off), gy = __shfl_up(scan.y, off);
      if (lane >= off) {
        scan.x += gx;
        scan.y += gy;
      }
    }
    __syncthreads();
    if (lane == 63) sums[wave] = scan;
    __syncthreads();
    uint2 at = make_uint2(before.x + scan.x - own.x, before.y + scan.y - own.y);
    for (int w = 0; w < kSelectThreads / 64; ++w) {
      if (w < wave) {
        at.x += sums[w].x;
        at.y += sums[w].y;
      }
      before.x += sums[w].x;
      before.y += sums[w].y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = bits[part * 4 + i], key = order(x);
      const bool up = x != kNoBits && key > c.key, same = x != kNoBits && key == c.key;
      if (up || (same && at.y < c.equal)) kept[at.x + min(at.y, c.equal)] = column(first, part * 4 + i);
      at.x += up;
      at.y += same;
    }
  }
}

template <class T>
__device__ __forceinline__ void copy_rows(uint8_t* data, int64_t bytes, const int64_t* from, const int64_t* to, int tokens) {
  const int pieces = (int)(bytes / sizeof(T)), more = kThreads / pieces, rest = kThreads - more * pieces;
  int t = threadIdx.x / pieces, c = threadIdx.x - t * pieces;    // token, piece of it
  while (t < tokens) {
    T x[kAhead];
    int64_t at[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t source = t < tokens ? from[t] : -1;
      at[u] = -1;
      if (source >= 0) {
        x[u] = *reinterpret_cast<const T*>(data + source * bytes + c * sizeof(T));
        at[u] = to[t] * bytes + c * sizeof(T);
      }
      t += more;
      c += rest;
      if (c >= pieces) {
        c -= pieces;
        ++t;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (at[u] >= 0) *reinterpret_cast<T*>(data + at[u]) = x[u];
  }
}

// movers: workgroups of `chunk` tokens each, as far as tokens stay.  Those after them
// have kTail columns each of what is only written down: weights, table, positions.
__global__ void __launch_bounds__(kThreads) move_kernel(const EvictParams p, int chunk, int movers) {
  __shared__ int64_t from[kChunk], to[kChunk];
  const int b = blockIdx.y, tid = threadIdx.x;
  const bool tail = (int)blockIdx.x >= movers, records = blockIdx.z == 0;
  if (tail && !records) return;
  const int first = tail ? movers * chunk + (blockIdx.x - movers) * kTail : blockIdx.x * chunk;
  const int columns = tail ? kTail : chunk;
  const EvictPlan plan = p.plan[b];
  const int n = length(p, b);
  const bool moved = plan.chosen >= 0;
  const int left = moved ? plan.chosen + p.recent : n;       // tokens afterwards
  const int32_t* table = p.bt + (int64_t)b * p.bt_stride;
  const int mask = (1 << p.bs_shift) - 1;
  // tokens, positions and weights
  int32_t* kept = p.kept + (int64_t)b * p.kept_stride;
  for (int c = tid; c < columns; c += kThreads) {
    const int i = first + c;
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
      if (records && i < p.keep && (!plan.cut || (moved && i >= plan.chosen))) kept[i] = at;
      if (records && i < p.max_ctx) p.new_weights[b * p.new_weights_stride + i] = p.weights[b * p.weights_stride + at];
    } else {
      if (records && i < p.keep && (!plan.cut || moved)) kept[i] = -1;
      if (records && i < p.max_ctx) p.new_weights[b * p.new_weights_stride + i] = 0.f;
    }
    if (records && plan.cut && !moved && i < p.keep) kept[i] = -1;
    if (!tail) {
      from[c] = src;
      to[c] = dst;
    }
  }
  __syncthreads();
  // these columns' entries of the table, of the freed blocks
  const int width = blocks_of(p, p.max_ctx), entry = blocks_of(p, first), entries = blocks_of(p, first + columns) - entry;
  if (records && tid < entries) {
    const int e = entry + tid, held = blocks_of(p, n);
    if (e < width)
      p.new_bt[b * p.new_bt_stride + e] =
          e >= blocks_of(p, left) ? -1 : moved ? p.free_ids[plan.first + e] : table[e];
    if (moved && e < held) p.freed[plan.freed + e] = table[e];
  }
  // padding of the freed blocks' list: behind the last one
  const int64_t pad = p.counts[1] + (int64_t)blockIdx.y * width + entry + tid;
  if (records && tid < entries && entry + tid < width && pad < (int64_t)p.batch * width) p.freed[pad] = -1;
  const int tokens = min(left - first, chunk);
  if (tail || !moved || tokens <= 0) return;
  for (int i = blockIdx.z; i < p.num_pools; i += gridDim.z) {
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

namespace {
bool selects(int32_t batch, int32_t max_ctx) { return batch <= kSelectRows && max_ctx > kSelectFrom; }
int groups_of(int32_t max_ctx) { return (max_ctx + kColumns - 1) / kColumns; }
}  // namespace

int64_t evict_workspace(int32_t batch, int32_t max_ctx) {
  int64_t bytes = (int64_t)batch * (int64_t)(sizeof(EvictPlan) + 8);
  if (selects(batch, max_ctx))
    bytes += batch * ((int64_t)sizeof(Choice) + 2 * (int64_t)sizeof(Known) + 3 * kBins * 4 + groups_of(max_ctx) * (int64_t)sizeof(uint2));
  return bytes;
}

hipError_t launch_evict(EvictParams p, hipStream_t s) {
  p.plan = static_cast<EvictPlan*>(p.workspace);
  p.k_start = reinterpret_cast<int32_t*>(p.plan + p.batch);
  p.k_end = p.k_start + p.batch;
  const bool choose = p.keep > p.recent && p.max_ctx > p.keep, select = choose && selects(p.batch, p.max_ctx);
  SelectParams c{};
  if (select) {
    c.choice = reinterpret_cast<Choice*>(p.k_end + p.batch);
    c.known = reinterpret_cast<Known*>(c.choice + p.batch);
    c.counts = reinterpret_cast<uint2*>(c.known + 2 * p.batch);
    c.groups = groups_of(p.max_ctx);
    c.bins = reinterpret_cast<uint32_t*>(c.counts + (int64_t)p.batch * c.groups);
    c.e = p;
  }
  const int n_counts = select ? p.batch * 3 * kBins : 0;
  ranges_kernel<<<select ? p.batch * 24 : (p.batch + 255) / 256, 256, 0, s>>>(p, c.bins, n_counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (select) {
    const dim3 grid(c.groups, p.batch);
    count_bits_kernel<0><<<grid, kSelectThreads, 0, s>>>(c);
    count_bits_kernel<1><<<grid, kSelectThreads, 0, s>>>(c);
    count_bits_kernel<2><<<grid, kSelectThreads, 0, s>>>(c);
    count_columns_kernel<<<grid, kSelectThreads, 0, s>>>(c);
    write_columns_kernel<<<grid, kSelectThreads, 0, s>>>(c);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else if (choose) {
    const TopkParams t{p.weights, p.weights_stride, p.k_start, p.k_end, p.batch, p.max_ctx, p.keep - p.recent,
                       p.kept, p.kept_stride};
    e = launch_topk(kF32, t, s);
    if (e != hipSuccess) return e;
  }
  plan_kernel<<<1, p.batch < kPlanThreads ? (p.batch + 63) / 64 * 64 : kPlanThreads, 0, s>>>(p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = p.max_ctx > p.keep ? p.max_ctx : p.keep;
  // Fewer tokens for a workgroup until there are two for each CU, then one for each
  // pool (one sequence cut to 16384 tokens of 1088 bytes in four pools: 17.2 us with
  // 32 tokens for a workgroup, 12.5 with its pools apart).  Otherwise one for all
  // pools, that finds its tokens' places once (64 sequences, six pools: 37 us, apart 66).
  const int tokens = p.keep < p.max_ctx ? p.keep : p.max_ctx;
  const auto wanted = [&](int n) { return (int64_t)p.batch * ((tokens + n - 1) / n); };
  int chunk = kChunk;
  while (chunk > 32 && wanted(chunk) < 512) chunk /= 2;
  const bool apart = wanted(chunk) < 1024 && p.num_pools > 1;
  const int movers = (tokens + chunk - 1) / chunk;
  const int tails = rows > movers * chunk ? (rows - movers * chunk + kTail - 1) / kTail : 0;
  move_kernel<<<dim3(movers + tails, p.batch, apart ? p.num_pools : 1), kThreads, 0, s>>>(p, chunk, movers);
  return hipGetLastError();
}

}  // namespace mqa
