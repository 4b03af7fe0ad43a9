// exl3_attn_shared.cu -- attention of sequences whose first keys are the same:
// what comes before and after the row-tile and token kernels.
//
// With P the keys that a group of sequences shares, a query's softmax splits into
// two sums,
//     out = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2),  m = max(m1, m2),
// one over the keys before P and one over its sequence's own.  Every query of
// the group sees all of the first, so the group's query tokens are the rows of one
// product with the prefix: it is read once for all of them, by tcgen05 row tiles
// (exl3_attn_tile.cu).  The own keys go the way of the paged call: few rows a
// sequence through the token kernel (exl3_attn_token.cu), which runs beside the
// prefixes' kernel, more of them through row tiles of the same launch.  All of them
// leave (m, l, o) in fp32, which the join here adds up in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "exl3_attn.h"
#include "exl3_attn_seq.cuh"
#include "exl3_sm100.cuh"

namespace exl3 {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Groups and starts.  The prefix that is used: whole tiles of keys that every query of the group sees, none for a group
// with queries of fewer than two sequences.  One warp a group.
constexpr int kPrepThreads = 256;
__global__ void __launch_bounds__(kPrepThreads) shared_prep_kernel(const AttnArgs a, const int32_t* cu_groups,
                                                                   const int32_t* prefix_lens, int4* group, int32_t* start) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x; b < a.batch; b += kPrepThreads) start[b] = 0;
  __syncthreads();
  const int room = a.table_width << a.cache.page_shift;
  for (int g = threadIdx.x >> 5; g < a.groups; g += kPrepThreads / 32) {
    const int s0 = max(0, min(cu_groups[g], a.batch)), s1 = max(s0, min(cu_groups[g + 1], a.batch));
    int keys = max(0, min(prefix_lens[g], room)), first = INT32_MAX, queries = 0;
    for (int b = s0 + lane; b < s1; b += 32) {
      const int c0 = max(0, a.cu_q[b]), c1 = min(a.cu_q[b + 1], (int)a.total_q);
      if (c1 <= c0) continue;
      const int kl = max(0, min(a.kv_lens[b], room));
      keys = min(keys, max(0, kl - (c1 - c0) + 1));  // what its first query sees
      first = min(first, b);
      ++queries;
    }
    keys = __reduce_min_sync(0xffffffffu, keys);
    first = __reduce_min_sync(0xffffffffu, first);
    queries = __reduce_add_sync(0xffffffffu, queries);
    keys = queries < 2 || keys < kLeastPrefix ? 0 : keys / kPrefixKeys * kPrefixKeys;
    if (keys > 0)
      for (int b = s0 + lane; b < s1; b += 32) start[b] = keys;
    if (lane == 0) {
      const int total = (int)a.total_q, c0 = max(0, min(a.cu_q[s0], total)), c1 = max(c0, min(a.cu_q[s1], total));
      group[g] = make_int4(c0, c1 - c0, keys, keys > 0 ? first : 0);
    }
  }
}

// A row's running sum of parts.
template <int PER>
struct Sum {
  float m = kNegInf, l = 0.0f, o[PER] = {};
  __device__ __forceinline__ void add(const float2& ml, const float (&v)[PER]) {
    if (ml.x == kNegInf) {
      l += ml.y;  // 0, or NaN
      return;
    }
    const float top = fmaxf(m, ml.x);
    const float f = m == kNegInf ? 0.0f : ex2(m - top), f1 = ex2(ml.x - top);
    l = (m == kNegInf ? l : l * f) + ml.y * f1;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] * f + v[i] * f1;
    m = top;
  }
};

template <int PER>
__device__ __forceinline__ void load_row(float (&v)[PER], const float* src) {
#pragma unroll
  for (int i = 0; i < PER; i += 2) {
    const float2 w = *reinterpret_cast<const float2*>(src + i);
    v[i] = w.x, v[i + 1] = w.y;
  }
}

// One warp has a row's sum: out of the rotated basis, divided, stored.
template <int D, bool QUANT>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const Sum<D / 32>& s, int64_t tok, int head, int lane) {
  constexpr int PER = D / 32;
  const float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;
  float o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = s.o[i] * inv;
  if constexpr (QUANT) {
#pragma unroll
    for (int st = 1; st < PER; st *= 2)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (!(i & st)) {
          const float x = o[i], y = o[i + st];
          o[i] = x + y, o[i + st] = x - y;
        }
#pragma unroll
    for (int st = 1; st < 32; st *= 2)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float x = __shfl_xor_sync(0xffffffffu, o[i], st);
        o[i] = (lane & st) ? x - o[i] : o[i] + x;
      }
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] *= 8.0f / D;
  }
  uint16_t* dst = static_cast<uint16_t*>(a.out) + tok * a.out_token_stride + head * a.out_head_stride + PER * lane;
#pragma unroll
  for (int i = 0; i < PER; i += 2) {
    if (a.bf16) *reinterpret_cast<__nv_bfloat162*>(dst + i) = __floats2bfloat162_rn(o[i], o[i + 1]);
    else *reinterpret_cast<__half2*>(dst + i) = __floats2half2_rn(o[i], o[i + 1]);
  }
}

// Few rows a sequence: one block an item (sequence and key head) and row; its warps take the parts in turn (those of the
// prefix, then its own: one, or those of the ranges that cut the item), four loads at a time, then one joins the warps.
constexpr int kWarps = 8, kAhead = 4;
template <int D, bool QUANT>
__global__ void __launch_bounds__(32 * kWarps) shared_token_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 32;
  __shared__ float so[kWarps][D];
  __shared__ float2 sml[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.heads / a.kv_heads;
  const int r = blockIdx.y, b = blockIdx.x / a.kv_heads, h = blockIdx.x % a.kv_heads;
  const Seq s = load_seq<true>(a, b);
  // units before this sequence, and of the call
  int64_t total = 0, before = 0;
  for (int i = lane; i < a.batch; i += 32) {
    const int n = load_seq<true>(a, i).weight();
    total += n;
    before += i < b ? n : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  total *= a.kv_heads;
  const int64_t first = before * a.kv_heads + (int64_t)h * s.weight() + kItemUnits, last = first + s.units - 1;
  const int64_t grid = a.ctas;
  const bool there = r < s.q_len * group;
  int64_t c0 = 0, c1 = 0;  // the CTA of a unit is the last whose range begins at or before it
  if (there) {
    c0 = ((first + 1) * grid - 1) / total;
    c1 = ((last + 1) * grid - 1) / total;
  }
  pdl_wait();
  if (!there) return;
  const int tok = r / group, head = h * group + r - tok * group;
  const int64_t row = (s.q0 + tok) * a.heads + head, rows = a.total_q * a.heads;
  const int shared = s.first > 0 ? a.prefix_splits : 0;  // s.first: the prefix
  const int64_t parts = shared + (c1 - c0 + 1);
  Sum<PER> sum;
  for (int64_t p = warp; p < parts; p += kWarps * kAhead) {
    float2 ml[kAhead];
    float v[kAhead][PER];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int64_t i = p + x * kWarps;
      ml[x] = make_float2(kNegInf, 0.0f);
      if (i >= parts) continue;
      if (i < shared || c0 == c1) {
        const int64_t at = (i < shared ? i : a.prefix_splits) * rows + row;
        ml[x] = a.part_ml[at];
        load_row(v[x], a.part_o + at * D + PER * lane);
      } else {
        const int64_t cc = c0 + i - shared;
        const int64_t begin = total * cc / grid, end = total * (cc + 1) / grid;
        if (begin >= end) continue;
        const int64_t at = (2 * cc + (begin <= first ? 1 : 0)) * kTokenRows + r;
        ml[x] = a.cut_ml[at];
        load_row(v[x], a.cut_o + at * D + PER * lane);
      }
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) sum.add(ml[x], v[x]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) so[warp][PER * lane + i] = sum.o[i];
  if (lane == 0) sml[warp] = make_float2(sum.m, sum.l);
  __syncthreads();
  if (warp != 0) return;
  Sum<PER> all;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    float v[PER];
    load_row(v, &so[w][PER * lane]);
    all.add(sml[w], v);
  }
  finish_row<D, QUANT>(a, all, s.q0 + tok, head, lane);
}

// Row tiles: one warp a row.
template <int D, bool QUANT>
__global__ void __launch_bounds__(256) shared_tile_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), rows = a.total_q * a.heads;
  pdl_wait();
  if (row >= rows) return;
  const int64_t tok = row / a.heads;
  // only the tokens of a sequence have parts, and those of its prefix only where it has one
  int start = -1;
  for (int b = lane; b < a.batch; b += 32) {
    const int64_t c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
    if (tok >= c0 && tok < c1) start = max(start, __ldcg(a.start + b));
  }
  start = __reduce_max_sync(0xffffffffu, start);
  if (start < 0) return;
  const int end = a.prefix_splits + a.splits;
  Sum<PER> sum;
  for (int p = start > 0 ? 0 : a.prefix_splits; p < end; p += kAhead) {
    float2 ml[kAhead];
    float v[kAhead][PER];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      ml[x] = make_float2(kNegInf, 0.0f);
      if (p + x >= end) continue;
      const int64_t at = (p + x) * rows + row;
      ml[x] = a.part_ml[at];
      load_row(v[x], a.part_o + at * D + PER * lane);
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) sum.add(ml[x], v[x]);
  }
  finish_row<D, QUANT>(a, sum, tok, (int)(row - tok * a.heads), lane);
}

}  // namespace

cudaError_t launch_shared_prep(const AttnArgs& a, const int32_t* cu_groups, const int32_t* prefix_lens, cudaStream_t stream) {
  shared_prep_kernel<<<1, kPrepThreads, 0, stream>>>(a, cu_groups, prefix_lens, const_cast<int4*>(a.group), const_cast<int32_t*>(a.start));
  return cudaGetLastError();
}

cudaError_t launch_shared_join(const AttnArgs& a, bool token, cudaStream_t stream) {
  const bool quant = kv_quantised(a.cache.format), wide = a.head_dim == 128;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256u, 1u, 1u);
  cfg.gridDim = token ? dim3((unsigned)(a.batch * a.kv_heads), (unsigned)(a.max_q * (a.heads / a.kv_heads)), 1u)
                      : dim3((unsigned)((a.total_q * a.heads + 7) / 8), 1u, 1u);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  using Kernel = void (*)(const AttnArgs);
  static constexpr Kernel kernels[2][2][2] = {
      {{shared_tile_join_kernel<64, false>, shared_tile_join_kernel<64, true>},
       {shared_tile_join_kernel<128, false>, shared_tile_join_kernel<128, true>}},
      {{shared_token_join_kernel<64, false>, shared_token_join_kernel<64, true>},
       {shared_token_join_kernel<128, false>, shared_token_join_kernel<128, true>}}};
  return cudaLaunchKernelEx(&cfg, kernels[token][wide][quant], a);
}

}  // namespace exl3
