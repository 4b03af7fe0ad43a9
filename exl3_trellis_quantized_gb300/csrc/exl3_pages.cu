// exl3_pages.cu -- a step's packing, positions, slots and page tables from the
// requests' lengths, and the pages of ended requests given back.
//
// Request b brings n_b new tokens.  Its place among the packed rows is the sum of
// the n before it, the pages it lacks are need_b = max(0, ceil((len_b + n_b) /
// page) - held_b), and it takes them from the top of the stack of free pages,
// after the needs of the requests before it: two prefix sums, then one
// search and one lookup a token.  The sums saturate at 2^30 (min(a + b, 2^30) of
// numbers from 0 to 2^30 is associative), so they stay in 32 bits whatever the lengths;
// rows and stacks are fewer, so what has saturated never fits.
//
// Bound by latency: a step's few hundred KB at the most are nothing, the chain launch,
// lengths, two sums of a block, search, table, store is what counts.  So it is one
// launch: one block, or for many rows a cluster of eight that all do the sums (the
// lengths come out of L2) and share the rows; the state may be updated in
// place, so block 0 writes it after a barrier of the cluster.
//   61 requests, 66 rows (0.4 ns of DRAM time)                3.4 us; in a cluster of eight 4.3
//   203 requests with prompts, 17400 rows, pages of 64        7.1 us; in one, two and four blocks 15.2, 11.2 and 8.5
//   2001 requests, 10010 rows, pages of 16, too few free      7.2 us; one block 11.1; blocks of 256 threads 13.2
//   250 requests, half of which end (some 7000 pages)         5.0 us; in one, two and four blocks 10.2, 7.6 and 5.6
#include "exl3_attn.h"

namespace exl3 {
namespace {

constexpr int kMost = 1 << 30;   // where sums saturate
constexpr int kPer = 2;          // requests a thread
constexpr int kThreads = 1024;   // at most
constexpr int kChunk = kPer * kThreads;

// Of 0 .. 2^30 each.  Two that are saturated make 2^31, which only the unsigned sum holds.
__device__ __forceinline__ int sat_add(int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)kMost); }
__device__ __forceinline__ int clamped(int x, int hi) { return max(0, min(x, hi)); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums before each of this thread's kPer values (in thread order), and the block's sum.  `part` is shared memory for 32.
__device__ __forceinline__ int block_sums(const int (&v)[kPer], int (&before)[kPer], int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int own = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    before[i] = own;
    own = sat_add(own, v[i]);
  }
  int inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = sat_add(inc, p);
  }
  int prev = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) prev = 0;
  __syncthreads();  // whoever read `part` before is done
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int w = lane < warps ? part[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w = sat_add(w, p);
  }
  const int all = __shfl_sync(0xffffffffu, w, 31);
  const int base = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) before[i] = sat_add(sat_add(base, prev), before[i]);
  return all;
}

// The last of `count` rising numbers that is at or below x (the first is).
__device__ __forceinline__ int last_at_or_below(const int* from, int count, int x) {
  int lo = 0, n = count;
  while (n > 1) {
    const int half = n >> 1;
    if (from[lo + half] <= x) lo += half, n -= half;
    else n = half;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const KvPlanArgs a) {
  __shared__ int part[32];
  __shared__ int s_start[kChunk];   // first row of each request
  __shared__ int s_len[kChunk];     // cached tokens
  __shared__ int s_held[kChunk];    // pages held; bit 31: not granted
  __shared__ int s_before[kChunk];  // pages that the requests before it take
  const int tid = threadIdx.x, threads = blockDim.x, chunk = kPer * threads;
  const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
  const int total = (int)a.total, width = a.t.table_width, shift = a.t.page_shift, mask = (1 << shift) - 1;
  const int free_pages = clamped(*a.t.free_count, a.t.capacity);
  int rows = 0, pages = 0;  // of the requests before this chunk
  int taken = 0;
  for (int b0 = 0; b0 < a.t.batch; b0 += chunk) {
    const int here = min(chunk, a.t.batch - b0);
    int n[kPer], len[kPer], held[kPer], need[kPer], start[kPer], before[kPer];
    bool can[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = b0 + kPer * tid + i;
      const bool there = b < a.t.batch;
      n[i] = there ? clamped(a.new_lens[b], total + 1) : 0;  // more never fit
      len[i] = there ? clamped(a.t.kv_lens[b], width << shift) : 0;
      held[i] = there ? clamped(a.t.held[b], width) : 0;
    }
    const int chunk_rows = block_sums(n, start, part);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      start[i] = sat_add(rows, start[i]);
      const int want = (len[i] + n[i] + mask) >> shift;
      can[i] = start[i] + n[i] <= total && want <= width;
      need[i] = can[i] && n[i] > 0 ? max(0, want - held[i]) : 0;
    }
    const int chunk_pages = block_sums(need, before, part);
    int gave = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      before[i] = sat_add(pages, before[i]);
      const bool granted = can[i] && (need[i] == 0 || sat_add(before[i], need[i]) <= free_pages);
      if (!granted) need[i] = 0;
      if (need[i] > 0) gave = before[i] + need[i];
      can[i] = granted;
      const int at = kPer * tid + i;
      s_start[at] = start[i];
      s_len[at] = len[i];
      s_held[at] = granted ? held[i] : held[i] | (int)0x80000000;
      s_before[at] = before[i];
      if (rank == 0 && at < here) {
        const int b = b0 + at;
        a.cu_q[b] = min(start[i], total);
        a.granted[b] = granted ? 1 : 0;
      }
    }
    // pages up to the last that is given: those that are form the beginning of the list
    taken = max(taken, __reduce_max_sync(0xffffffffu, gave));
    __syncthreads();
    if ((tid & 31) == 0) part[tid >> 5] = taken;
    __syncthreads();
    {
      const int w = (tid & 31) < (threads >> 5) ? part[tid & 31] : 0;
      taken = __reduce_max_sync(0xffffffffu, w);
    }
    if (ranks > 1) cluster_barrier();  // every block has read the old lengths of these requests
    if (rank == 0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = b0 + kPer * tid + i;
        if (b < a.t.batch) {
          a.kv_lens_out[b] = can[i] ? len[i] + n[i] : len[i];
          a.held_out[b] = held[i] + need[i];
        }
      }
    }
    // the table's new entries
    for (int p = pages + rank * threads + tid; p < taken; p += ranks * threads) {
      const int r = last_at_or_below(s_before, here, p);
      a.t.table[(int64_t)(b0 + r) * width + (s_held[r] & 0x7FFFFFFF) + p - s_before[r]] = a.t.free_pages[free_pages - 1 - p];
    }
    // positions and slots
    const int end = min(sat_add(rows, chunk_rows), total);
    for (int t = rows + rank * threads + tid; t < end; t += ranks * threads) {
      const int r = last_at_or_below(s_start, here, t);
      const int pos = s_len[r] + t - s_start[r];
      a.positions[t] = pos;
      int64_t slot = -1;
      if (s_held[r] >= 0) {
        const int j = pos >> shift, k = j - s_held[r];
        const int id = k < 0 ? a.t.table[(int64_t)(b0 + r) * width + j] : a.t.free_pages[free_pages - 1 - (s_before[r] + k)];
        if (id >= 0) slot = ((int64_t)id << shift) + (pos & mask);
      }
      a.slots[t] = slot;
    }
    rows = sat_add(rows, chunk_rows);
    pages = sat_add(pages, chunk_pages);
    __syncthreads();  // the shared arrays are read before the next chunk's
  }
  rows = min(rows, total);
  for (int t = rows + rank * threads + tid; t < total; t += ranks * threads) {
    a.positions[t] = 0;
    a.slots[t] = -1;
  }
  if (rank == 0 && tid == 0) {
    a.cu_q[a.t.batch] = rows;
  }
  if (ranks > 1) cluster_barrier();  // every block has read the count
  else __syncthreads();
  if (rank == 0 && tid == 0) *a.free_count_out = free_pages - taken;
}

__global__ void __launch_bounds__(kThreads) kv_release_kernel(const KvReleaseArgs a) {
  __shared__ int part[32];
  __shared__ int s_keep[kChunk];    // first page that is given back
  __shared__ int s_before[kChunk];  // pages that the requests before it give back
  const int tid = threadIdx.x, threads = blockDim.x, chunk = kPer * threads;
  const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
  const int width = a.t.table_width;
  const int free_pages = clamped(*a.t.free_count, a.t.capacity), room = a.t.capacity - free_pages;
  int pages = 0;
  for (int b0 = 0; b0 < a.t.batch; b0 += chunk) {
    const int here = min(chunk, a.t.batch - b0);
    int len[kPer], held[kPer], give[kPer], before[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = b0 + kPer * tid + i;
      const bool there = b < a.t.batch, ended = there && a.ended[b] != 0;
      const int h = there ? clamped(a.t.held[b], width) : 0;
      const int keep = ended && a.shared != nullptr ? clamped(a.shared[b], h) : 0;
      len[i] = ended || !there ? 0 : a.t.kv_lens[b];
      held[i] = ended ? 0 : h;
      give[i] = ended ? h - keep : 0;
      s_keep[kPer * tid + i] = keep;
    }
    const int all = block_sums(give, before, part);
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_before[kPer * tid + i] = sat_add(pages, before[i]);
    __syncthreads();
    if (ranks > 1) cluster_barrier();  // every block has read the old state of these requests
    if (rank == 0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = b0 + kPer * tid + i;
        if (b < a.t.batch) {
          a.kv_lens_out[b] = len[i];
          a.held_out[b] = held[i];
        }
      }
    }
    const int end = min(sat_add(pages, all), room);
    for (int p = pages + rank * threads + tid; p < end; p += ranks * threads) {
      const int r = last_at_or_below(s_before, here, p);
      a.t.free_pages[free_pages + p] = a.t.table[(int64_t)(b0 + r) * width + s_keep[r] + p - s_before[r]];
    }
    pages = sat_add(pages, all);
    __syncthreads();
  }
  if (ranks > 1) cluster_barrier();  // every block has read the count
  else __syncthreads();
  if (rank == 0 && tid == 0) *a.free_count_out = free_pages + min(pages, room);
}

template <typename Args>
cudaError_t launch(void (*kernel)(const Args), const Args& a, int64_t requests, int64_t work, cudaStream_t stream) {
  const int64_t most = requests > work ? requests : work;
  cudaLaunchConfig_t cfg = {};
  const unsigned threads = most <= 256 ? 256u : most <= 512 ? 512u : 1024u;
  const unsigned blocks = work > 4 * kThreads ? 8u : work > kThreads ? 4u : 1u;
  cfg.gridDim = dim3(blocks, 1u, 1u);
  cfg.blockDim = dim3(threads, 1u, 1u);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  return launch<KvPlanArgs>(kv_plan_kernel, a, a.t.batch, a.total, stream);
}
cudaError_t launch_kv_release(const KvReleaseArgs& a, cudaStream_t stream) {
  // (how many pages come back only the GPU knows: some dozens a request)
  return launch<KvReleaseArgs>(kv_release_kernel, a, a.t.batch, (int64_t)a.t.batch * 32, stream);
}

}  // namespace exl3
