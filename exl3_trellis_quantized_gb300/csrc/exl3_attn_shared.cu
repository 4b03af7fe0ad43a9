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

// What the workspace holds beside the parts.
struct SharedState {
  SharedGroup* group;
  int2* seq;
  int64_t* units;
  int32_t* items;
};

// Sums before each thread's value, in thread order, after those that came before (`carry`, which moves on).
__device__ __forceinline__ int64_t block_sums(int64_t v, int64_t* part, int64_t* carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t p = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += p;
  }
  __syncthreads();
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < warps; ++w) {
    const int64_t p = part[w];
    if (w < warp) before += p;
    all += p;
  }
  before += *carry + inc - v;
  *carry += all;
  return before;
}

// Groups, starts, items and units from the lengths, in one block.
//
// The prefix that is used: whole tiles of keys that every query of the group sees, none for a group with queries of
// fewer than two sequences.
//
// Parts.  Each row tile's keys go to ceil(blocks / u) CTAs, u blocks of 64 keys at the most; u is the same for all, so
// that long and short prefixes make items of about one length.  Of 32 sizes u (the longest prefix in 1 to 32) the one
// that a model of the time likes best: an item takes 0.85 us a block and 4 us; up to 152 items the longest counts, more
// are taken up in turn, so all of them by 152 and 0.7 of the last; and what the parts cost to write and join.
constexpr int kPrepThreads = 256;
constexpr float kSms = 152.0f;
__global__ void __launch_bounds__(kPrepThreads) shared_prep_kernel(const AttnArgs a, const int32_t* cu_groups,
                                                                   const int32_t* prefix_lens, const SharedState s, int token) {
  __shared__ int64_t part[kPrepThreads / 32];
  __shared__ int longest;
  __shared__ int unit;
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int per = 2 * a.tile_tokens;
  for (int b = tid; b < a.batch; b += kPrepThreads) s.seq[b] = make_int2(0, -1);
  if (tid == 0) longest = 0;
  __syncthreads();
  const int room = a.table_width << a.cache.page_shift, total = (int)a.total_q;
  for (int g = tid >> 5; g < a.groups; g += kPrepThreads / 32) {  // one warp a group
    const int s0 = max(0, min(cu_groups[g], a.batch)), s1 = max(s0, min(cu_groups[g + 1], a.batch));
    int keys = max(0, min(prefix_lens[g], room)), first = INT32_MAX, queries = 0;
    for (int b = s0 + lane; b < s1; b += 32) {
      const int c0 = max(0, a.cu_q[b]), c1 = min(a.cu_q[b + 1], total);
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
      for (int b = s0 + lane; b < s1; b += 32) s.seq[b] = make_int2(keys, g);
    if (lane == 0) {
      const int c0 = max(0, min(a.cu_q[s0], total)), c1 = max(c0, min(a.cu_q[s1], total));
      s.group[g] = {c0, c1 - c0, keys, keys > 0 ? first : 0, 0, 0};
      atomicMax(&longest, keys);
    }
  }
  __syncthreads();
  if (tid < 32) {
    // a lane a size
    const int most = longest / 64, u = max(4, (most + lane) / (lane + 1) + 1 & ~1);
    float items = 0.0f, blocks = 0.0f;
    for (int g = 0; g < a.groups; ++g) {
      const int keys = s.group[g].keys / 64, tiles = keys > 0 ? (s.group[g].tokens + per - 1) / per : 0;
      items += (float)(tiles * a.kv_heads) * (float)((keys + u - 1) / u);
      blocks += (float)(tiles * a.kv_heads) * (float)keys;
    }
    const float one = 0.85f * (float)u + 4.0f;
    float us = items <= kSms ? one : (0.85f * blocks + 4.0f * items) / kSms + 0.7f * one;
    us += items * (float)(kPrefixRows * a.head_dim) * 8.0f / 8.0e6f;
    if (items > (float)a.prefix_ctas) us = __builtin_huge_valf();  // (the first size has an item a row tile: always room)
    float best = us;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
    const uint32_t hit = __ballot_sync(0xffffffffu, us == best);
    if (lane == __ffs(hit) - 1) unit = u;
  }
  __syncthreads();
  int64_t carry = 0;
  for (int g0 = 0; g0 < a.groups; g0 += kPrepThreads) {
    const int g = g0 + tid;
    int tiles = 0, parts = 0;
    if (g < a.groups) {
      const int keys = s.group[g].keys / 64;
      tiles = keys > 0 ? (s.group[g].tokens + per - 1) / per : 0;
      parts = (keys + unit - 1) / unit;
    }
    const int64_t before = block_sums((int64_t)tiles * a.kv_heads * parts, part, &carry);
    if (g < a.groups) {
      s.group[g].item = (int)before;
      s.group[g].parts = parts;
    }
  }
  if (tid == 0) s.items[0] = (int)min(carry, (int64_t)a.prefix_ctas);
  if (!token) return;
  carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPrepThreads) {
    const int b = b0 + tid;
    const int64_t before = block_sums(b < a.batch ? load_seq<true>(a, b).weight() : 0, part, &carry);
    if (b < a.batch) s.units[b] = before;
  }
  if (tid == 0) s.units[a.batch] = carry;
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

// The part of row (tok, head) in the first of its prefix items; the next parts lie kPrefixRows rows on.
__device__ __forceinline__ int64_t prefix_row(const AttnArgs& a, const SharedGroup& g, int tok, int h, int head, int group) {
  const int per = 2 * a.tile_tokens, t = tok - g.q0, tiles = (g.tokens + per - 1) / per, tile = t / per;
  const int64_t item = g.item + ((int64_t)(tiles - 1 - tile) * a.kv_heads + h) * g.parts;  // last tiles come first
  return item * kPrefixRows + (t - tile * per) * group + head;
}
__device__ __forceinline__ SharedGroup load_group(const SharedGroup* g) {
  return {__ldcg(&g->q0), __ldcg(&g->tokens), __ldcg(&g->keys), __ldcg(&g->lead), __ldcg(&g->item), __ldcg(&g->parts)};
}

// The join: WARPS warps a row take its parts in turn (those of the prefix, then its own), kAhead loads at a time; with
// more than one, the first joins them.  Every query token of a sequence has its rows here; the sequence is found from
// cu_q.  TOKEN: own parts of the token kernel, one, or those of the ranges that cut the item.
constexpr int kAhead = 6;
template <int D, bool QUANT, bool TOKEN, int WARPS>
__global__ void __launch_bounds__(256) shared_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 32, ROWS = 8 / WARPS;  // rows of a block
  __shared__ float so[WARPS > 1 ? WARPS : 1][D];
  __shared__ float2 sml[WARPS > 1 ? WARPS : 1];
  const int warp = (threadIdx.x >> 5) % WARPS, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (threadIdx.x >> 5) / WARPS, rows = a.total_q * a.heads;
  const int group = a.heads / a.kv_heads;
  const int tok = (int)(row / a.heads), head = (int)(row - (int64_t)tok * a.heads), h = head / group;
  int b = -1;
  if (row < rows) {
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int i = b0 + lane;
      const uint32_t hit = __ballot_sync(0xffffffffu, i < a.batch && tok >= a.cu_q[i] && tok < a.cu_q[i + 1]);
      if (hit) {
        b = b0 + __ffs(hit) - 1;
        break;
      }
    }
  }
  pdl_wait();
  if (b < 0) return;  // a token of no sequence (the whole block, where warps share a row)
  const int g = __ldcg(&a.seq[b].y);
  int shared = 0;
  int64_t at0 = 0;
  if (g >= 0) {
    const SharedGroup sg = load_group(a.group + g);
    shared = sg.parts;
    at0 = prefix_row(a, sg, tok, h, head - h * group, group);
  }
  int64_t own = a.splits, c0 = 0, total = 0, first = 0;
  int r = 0;
  if constexpr (TOKEN) {
    const Seq s = load_seq<true>(a, b);
    r = (tok - (int)s.q0) * group + head - h * group;
    if (r >= s.q_len * group) return;  // more tokens than max_q
    total = __ldcg(a.units + a.batch) * a.kv_heads;
    first = __ldcg(a.units + b) * a.kv_heads + (int64_t)h * s.weight() + kItemUnits;
    const int64_t last = first + s.units - 1;
    // the CTA of a unit is the last whose range begins at or before it
    c0 = ((first + 1) * a.ctas - 1) / total;
    own = ((last + 1) * a.ctas - 1) / total - c0 + 1;
  }
  const int64_t parts = shared + own;
  Sum<PER> sum;
  for (int64_t p = warp; p < parts; p += WARPS * kAhead) {
    float2 ml[kAhead];
    float v[kAhead][PER];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int64_t i = p + x * WARPS, j = i - shared;
      ml[x] = make_float2(kNegInf, 0.0f);
      if (i >= parts) continue;
      const float* o = a.own_o;
      const float2* l = a.own_ml;
      int64_t at = j * rows + row;
      if (j < 0) {
        o = a.prefix_o, l = a.prefix_ml, at = at0 + i * kPrefixRows;
      } else if (TOKEN && own > 1) {
        const int64_t cc = c0 + j, begin = total * cc / a.ctas;
        if (begin >= total * (cc + 1) / a.ctas) continue;
        o = a.cut_o, l = a.cut_ml, at = (2 * cc + (begin <= first ? 1 : 0)) * kTokenRows + r;
      }
      ml[x] = l[at];
      load_row(v[x], o + at * D + PER * lane);
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) sum.add(ml[x], v[x]);
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) so[warp][PER * lane + i] = sum.o[i];
    if (lane == 0) sml[warp] = make_float2(sum.m, sum.l);
    __syncthreads();
    if (warp != 0) return;
    sum = Sum<PER>();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      float v[PER];
      load_row(v, &so[w][PER * lane]);
      sum.add(sml[w], v);
    }
  }
  finish_row<D, QUANT>(a, sum, tok, head, lane);
}

}  // namespace

cudaError_t launch_shared_prep(const AttnArgs& a, const int32_t* cu_groups, const int32_t* prefix_lens, bool token,
                               cudaStream_t stream) {
  const SharedState s = {const_cast<SharedGroup*>(a.group), const_cast<int2*>(a.seq), const_cast<int64_t*>(a.units),
                         const_cast<int32_t*>(a.items)};
  shared_prep_kernel<<<1, kPrepThreads, 0, stream>>>(a, cu_groups, prefix_lens, s, token ? 1 : 0);
  return cudaGetLastError();
}

namespace {
template <int D, bool QUANT>
cudaError_t launch_join(const AttnArgs& a, bool token, cudaStream_t stream) {
  const int64_t rows = a.total_q * a.heads;
  // few rows: eight warps each
  const bool wide = rows <= 152 * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256u, 1u, 1u);
  cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + 7) / 8), 1u, 1u);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (token)
    return wide ? cudaLaunchKernelEx(&cfg, shared_join_kernel<D, QUANT, true, 8>, a)
                : cudaLaunchKernelEx(&cfg, shared_join_kernel<D, QUANT, true, 1>, a);
  return wide ? cudaLaunchKernelEx(&cfg, shared_join_kernel<D, QUANT, false, 8>, a)
              : cudaLaunchKernelEx(&cfg, shared_join_kernel<D, QUANT, false, 1>, a);
}
}  // namespace

cudaError_t launch_shared_join(const AttnArgs& a, bool token, cudaStream_t stream) {
  const bool quant = kv_quantised(a.cache.format);
  if (a.head_dim == 64) return quant ? launch_join<64, true>(a, token, stream) : launch_join<64, false>(a, token, stream);
  return quant ? launch_join<128, true>(a, token, stream) : launch_join<128, false>(a, token, stream);
}

}  // namespace exl3
