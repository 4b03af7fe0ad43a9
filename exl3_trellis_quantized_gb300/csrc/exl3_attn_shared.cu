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
//
// What bounds it: for single tokens DRAM (own keys) and what an item of row tiles takes before its first scores and for
// its results, 10 us (codes: 18), so the prefix goes into few items that run while the own keys are read; for long
// chunks the row tiles' softmax and, over codes, their conversion, as in a paged call.
//   64 sequences, 1 to 2000 own keys behind 8192, one token, 32 and 8 heads of 128, 16 bits
//     68.2 us (a paged call 160): 317 MB, 4640 GB/s; lengths 5 us, then prefix 50 and own keys 47 beside each other, join 6
//   24 and 9 sequences behind 6011 and 30000, 6 alone, 1 to 3 tokens, 40 and 8 heads, 8 bits   68.0 us (187)
//   7 chunks of 1 to 700 tokens behind 16000, 32 and 8 heads, 4 bits   479 us (522), 992 TFLOP/s
// Halves of a row tile that take blocks in turn leave a part each: meeting in shared memory, as a paged call's do, costs
// an item 2 us.  A row's parts are found before the wait for them (found after it 71.7 us in the second case), from a
// group and sequence read once a token (once a head: 486 us in the third).
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
  int4* counts;
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

// Groups, starts, units and items from the lengths, in one block.
//
// The prefix that is used: whole tiles of keys that every query of the group sees, none for a group with queries of
// fewer than two sequences.
//
// Parts.  Each row tile's keys go to ceil(blocks / u) CTAs, u blocks of 64 keys at the most; u is the same for all, so
// that long and short prefixes make items of about one length.  Of 32 sizes u (the longest prefix in 1 to 32) the one
// that a model of the time likes best.  An item takes `block` us a block (`joint` where its rows fill one tile, whose
// halves take blocks in turn) and `fixed` us.
//   With the token kernel, own keys take `unit` us a unit and SM, and all of them at least their bytes at what DRAM
// gives.  Up to 128 items leave SMs for it, so both run at the same time and the longer counts; else one follows the
// other.  64 sequences of 1 to 2000 own keys behind 8192 shared ones, 32 and 8 heads of 128, 16 bits: 85, 70, 70, 71, 76,
// 81 and (one after the other) 80 us with the prefix in 2, 3, 5, 6, 8, 12 and 16 parts.
//   Without, up to 152 items the longest counts; more are taken up in turn: all of them by 152, and 0.7 of the last.
// And every item's rows are written and joined, at 4 TB/s.
//   The rates are those that split best beside own keys, not a block's own time, which over keys out of L2 is 0.46 us for a
// tile of up to 128 rows and 0.79 for two (codes 0.79 and 0.95; heads of 64 0.34 and 0.64, codes 0.65 and 0.87): with these
// in their place the case above takes 88 us for 70, 39 sequences of 40 heads behind 8-bit prefixes 75 for 69.
//   Own keys in row tiles are of a few parts too where the call has few items (the host says how many at the most, for a
// sequence that shares nothing), each sequence by its own length: 36 tokens alone over 31510 keys 29 us and 240 in one part
// (a paged call 28), 74 groups of one or two behind 8000 to 16000 8-bit keys, 24 rows a sequence, 151 and 290 us (212).
constexpr int kPrepThreads = 256;
constexpr int kSms = 152, kMostBeside = 128;
struct SharedCosts {
  float block, joint, fixed, unit, unit_dram;  // us
  int token, per_sm;  // the token kernel takes the own keys, so many CTAs an SM
};
// What the lengths say is loaded once, into shared memory as far as that goes (kHeldSeqs sequences, kHeldGroups groups): this
// block stands before everything else, and its time is its chain of loads (5.3 us with the lengths read where they are used).
constexpr int kHeldSeqs = 1024, kHeldGroups = 256;
__global__ void __launch_bounds__(kPrepThreads) shared_prep_kernel(const AttnArgs a, const int32_t* cu_groups,
                                                                   const int32_t* prefix_lens, const SharedState s,
                                                                   const SharedCosts cost) {
  __shared__ int64_t part[kPrepThreads / 32];
  __shared__ int h_q[kHeldSeqs + 1], h_kv[kHeldSeqs];  // first query tokens and lengths
  __shared__ int2 h_seq[kHeldSeqs];                    // what s.seq will hold
  __shared__ int h_group[kHeldGroups + 1], h_prefix[kHeldGroups];
  __shared__ int2 h_size[kHeldGroups];                 // blocks and tokens
  __shared__ int longest, longest_own, unit;
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int per = 2 * a.tile_tokens, room = a.table_width << a.cache.page_shift, total = (int)a.total_q;
  const bool held = a.batch <= kHeldSeqs;
  auto clamped = [](int x, int hi) { return max(0, min(x, hi)); };
  for (int b = tid; b <= min(a.batch, kHeldSeqs); b += kPrepThreads) {
    h_q[b] = clamped(a.cu_q[b], total);
    if (b < min(a.batch, kHeldSeqs)) {
      h_kv[b] = clamped(a.kv_lens[b], room);
      h_seq[b] = make_int2(0, -1);
    }
  }
  for (int g = tid; g <= min(a.groups, kHeldGroups); g += kPrepThreads) {
    h_group[g] = clamped(cu_groups[g], a.batch);
    if (g < min(a.groups, kHeldGroups)) h_prefix[g] = clamped(prefix_lens[g], room);
  }
  if (!held)
    for (int b = tid; b < a.batch; b += kPrepThreads) s.seq[b] = make_int2(0, -1);
  if (tid == 0) longest = longest_own = 0;
  __syncthreads();
  auto first_q = [&](int b) { return held ? h_q[b] : clamped(a.cu_q[b], total); };
  auto length = [&](int b) { return held ? h_kv[b] : clamped(a.kv_lens[b], room); };
#pragma unroll 1
  for (int g = tid >> 5; g < a.groups; g += kPrepThreads / 32) {  // one warp a group
    const int s0 = g <= kHeldGroups ? h_group[g] : clamped(cu_groups[g], a.batch);
    const int s1 = max(s0, g < kHeldGroups ? h_group[g + 1] : clamped(cu_groups[g + 1], a.batch));
    int keys = g < kHeldGroups ? h_prefix[g] : clamped(prefix_lens[g], room), first = INT32_MAX, queries = 0;
#pragma unroll 1
    for (int b = s0 + lane; b < s1; b += 32) {
      const int n = first_q(b + 1) - first_q(b);
      if (n <= 0) continue;
      keys = min(keys, max(0, length(b) - n + 1));  // what its first query sees
      first = min(first, b);
      ++queries;
    }
    keys = __reduce_min_sync(0xffffffffu, keys);
    first = __reduce_min_sync(0xffffffffu, first);
    queries = __reduce_add_sync(0xffffffffu, queries);
    keys = queries < 2 || keys < kLeastPrefix ? 0 : keys / kPrefixKeys * kPrefixKeys;
    if (keys > 0)
      for (int b = s0 + lane; b < s1; b += 32) (held ? h_seq : s.seq)[b] = make_int2(keys, g);
    if (lane == 0) {
      const int q0 = first_q(s0), q1 = max(q0, first_q(s1));
      s.group[g] = {q0, q1 - q0, keys, keys > 0 ? first : 0, 0, 0};
      if (g < kHeldGroups) h_size[g] = make_int2(keys / 64, q1 - q0);
      atomicMax(&longest, keys / 64);
    }
  }
  __syncthreads();
  auto sizes = [&](int g) { return g < kHeldGroups ? h_size[g] : make_int2(s.group[g].keys / 64, s.group[g].tokens); };
  int64_t units = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += kPrepThreads) {
    const int b = b0 + tid;
    int weight = 0;
    if (b < a.batch) {
      const int2 seq = held ? h_seq[b] : s.seq[b];
      if (held) s.seq[b] = seq;
      // as load_seq has it
      if (first_q(b + 1) > first_q(b)) weight = max(1, (length(b) - seq.x + kTokenUnit - 1) / kTokenUnit) + kItemUnits;
    }
    if (a.splits > 1 && weight > 0) atomicMax(&longest_own, weight - kItemUnits);
    if (cost.token) {
      const int64_t before = block_sums(weight, part, &units);
      if (b < a.batch) s.units[b] = before;
    }
  }
  if (cost.token && tid == 0) s.units[a.batch] = units;
  if (tid < 32) {
    // a lane a size
    const int u = max(4, ((longest + lane) / (lane + 1) + 1) & ~1);
    float items = 0.0f, us = 0.0f, one = 0.0f;
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      const int2 n = sizes(g);
      if (n.x == 0) continue;
      const float tiles = (float)((n.y + per - 1) / per * a.kv_heads), block = n.y <= a.tile_tokens ? cost.joint : cost.block;
      const float parts = (float)((n.x + u - 1) / u);
      items += tiles * parts;
      us += tiles * ((float)n.x * block + parts * cost.fixed);
      one = fmaxf(one, (float)min(n.x, u) * block + cost.fixed);
    }
    const float sms = (float)kSms, all = items <= sms ? one : us / sms + 0.7f * one;
    const float n = (float)units * a.kv_heads, beside = items <= (float)kMostBeside ? sms - items : sms;
    const float own = cost.token ? fmaxf(n * cost.unit / beside, n * cost.unit_dram) : 0.0f;
    us = cost.token && items <= (float)kMostBeside ? fmaxf(one, own) : all + own;
    us += items * (float)(kPrefixRows * a.head_dim) * 8.0f / 4.0e6f;
    if (items > (float)a.prefix_ctas) us = __builtin_huge_valf();  // (the first size has an item a row tile: always room)
    float best = us;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
    const uint32_t hit = __ballot_sync(0xffffffffu, us == best);
    if (lane == __ffs(hit) - 1) unit = u;
  }
  __syncthreads();
  int64_t items = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < a.groups; g0 += kPrepThreads) {
    const int g = g0 + tid;
    int tiles = 0, parts = 0;
    if (g < a.groups) {
      const int2 n = sizes(g);
      tiles = n.x > 0 ? (n.y + per - 1) / per : 0;
      parts = tiles > 0 ? (n.x + unit - 1) / unit : 0;
    }
    const int64_t n = (int64_t)tiles * a.kv_heads * parts, before = block_sums(n, part, &items);
    if (g < a.groups) {
      // (groups that overlap, which the call does not allow, may be more than there is room for: those have no parts)
      const bool room_left = before + n <= a.prefix_ctas;
      s.group[g].item = room_left ? (int)before : 0;
      s.group[g].parts = room_left ? parts : 0;
    }
  }
  if (tid == 0) {
    const int n = (int)min(items, (int64_t)a.prefix_ctas);
    const int beside = n <= kMostBeside ? (kSms - n) * cost.per_sm : kSms * cost.per_sm;
    // (row tiles: parts of own keys, no shorter than those of prefixes, beside which they run)
    const int own = a.splits > 1 ? max(max(8, unit), (longest_own + a.splits - 1) / a.splits) : INT32_MAX / 2;
    s.counts[0] = make_int4(n, min(a.ctas, beside), own, 0);
  }
}

// A row's running sum of parts: eight values a lane.
struct Sum {
  float m = kNegInf, l = 0.0f, o[8] = {};
  __device__ __forceinline__ void add(const float2& ml, const float (&v)[8]) {
    if (ml.x == kNegInf) {
      l += ml.y;  // 0, or NaN
      return;
    }
    const float top = fmaxf(m, ml.x);
    const float f = m == kNegInf ? 0.0f : ex2(m - top), f1 = ex2(ml.x - top);
    l = (m == kNegInf ? l : l * f) + ml.y * f1;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * f + v[i] * f1;
    m = top;
  }
};

__device__ __forceinline__ void load_row(float (&v)[8], const float* src) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>(src + i);
    v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
  }
}

// A row's sum, held by D/8 lanes: out of the rotated basis, divided, stored (a whole warp; nothing where not `there`).
template <int D, bool QUANT>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const Sum& s, int64_t tok, int head, int l, bool there) {
  const float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = s.o[i] * inv;
  if constexpr (QUANT) {
#pragma unroll
    for (int st = 1; st < 8; st *= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(i & st)) {
          const float x = o[i], y = o[i + st];
          o[i] = x + y, o[i + st] = x - y;
        }
#pragma unroll
    for (int st = 1; st < D / 8; st *= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = __shfl_xor_sync(0xffffffffu, o[i], st);
        o[i] = (l & st) ? x - o[i] : o[i] + x;
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= 8.0f / D;
  }
  if (!there) return;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
    const __half2 y = __floats2half2_rn(o[2 * i], o[2 * i + 1]);
    w[i] = a.bf16 ? *reinterpret_cast<const uint32_t*>(&x) : *reinterpret_cast<const uint32_t*>(&y);
  }
  uint16_t* dst = static_cast<uint16_t*>(a.out) + tok * a.out_token_stride + head * a.out_head_stride + 8 * l;
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The part of row (tok, head) in the first of its prefix items.  The next item's lies kPrefixRows rows on; where the
// item's rows fill one tile (twice: it has halves with a part each) half of that.
__device__ __forceinline__ int64_t prefix_row(const AttnArgs& a, const SharedGroup& g, int tok, int h, int head, int group, bool* twice) {
  const int per = 2 * a.tile_tokens, t = max(0, min(tok - g.q0, g.tokens - 1)), tiles = (g.tokens + per - 1) / per, tile = t / per;
  const int64_t item = g.item + ((int64_t)(tiles - 1 - tile) * a.kv_heads + h) * g.parts;  // last tiles come first
  *twice = g.tokens - tile * per <= a.tile_tokens;
  return item * kPrefixRows + (t - tile * per) * group + head;
}
__device__ __forceinline__ SharedGroup load_group(const SharedGroup* g) {
  return {__ldcg(&g->q0), __ldcg(&g->tokens), __ldcg(&g->keys), __ldcg(&g->lead), __ldcg(&g->item), __ldcg(&g->parts)};
}

// Where a row's parts lie.
template <bool TOKEN>
struct Parts {
  // Of the token's sequence: its group (keys 0: none) and, with the token kernel, its own items.
  SharedGroup group;
  Seq seq;
  int64_t units, total;
  int ctas;
  // Those of the prefix and those of its own keys: the first, how many, rows from one to the next.
  int64_t prefix0, own0;
  int shared, own, step, own_parts;
  int64_t own_step;
  bool cut;  // its own come from ranges that cut the item (token kernel)
  int64_t c0;
  __device__ __forceinline__ void open(const AttnArgs& a, int b) {
    const int g = __ldcg(&a.seq[b].y);
    if constexpr (TOKEN) {
      seq = load_seq<true>(a, b);
      ctas = __ldcg(&a.counts->y);
      total = __ldcg(a.units + a.batch) * a.kv_heads;
      units = __ldcg(a.units + b) * a.kv_heads;
    } else {
      own_parts = shared_own_parts(a, b, __ldcg(a.counts).z);
    }
    group = g >= 0 ? load_group(a.group + g) : SharedGroup{0, 0, 0, 0, 0, 0};
  }
  // Of row (tok, head); false where there are none.
  __device__ __forceinline__ bool find(const AttnArgs& a, int tok, int head) {
    const int heads = a.heads / a.kv_heads, h = head / heads;
    shared = step = 0;
    prefix0 = 0;
    if (group.keys > 0) {
      bool twice;
      prefix0 = prefix_row(a, group, tok, h, head - h * heads, heads, &twice);
      shared = twice ? 2 * group.parts : group.parts;
      step = twice ? kPrefixRows / 2 : kPrefixRows;
    }
    own0 = (int64_t)tok * a.heads + head;
    own = own_parts;
    own_step = a.total_q * a.heads;
    cut = false;
    if constexpr (TOKEN) {
      const int r = (tok - (int)seq.q0) * heads + head - h * heads;
      if (r >= seq.q_len * heads) return false;  // more tokens than max_q
      const int64_t first = units + (int64_t)h * seq.weight() + kItemUnits;
      // the CTA of a unit is the last whose range begins at or before it
      c0 = ((first + 1) * ctas - 1) / total;
      own = (int)(((first + seq.units) * ctas - 1) / total - c0) + 1;
      cut = own > 1;
      // two places a CTA, the second for an item that its range does not begin in: the first of the row's CTAs
      if (cut) own0 = (2 * c0 + 1) * kTokenRows + r, own_step = 2 * kTokenRows;
    }
    return true;
  }
  // Part i's output (null: it has none) and statistics.
  __device__ __forceinline__ const float* at(const AttnArgs& a, int i, int d, const float2** ml) const {
    int64_t n;
    if (i < shared) {
      n = prefix0 + (int64_t)i * step;
      *ml = a.prefix_ml + n;
      return a.prefix_o + n * d;
    }
    const int j = i - shared;
    n = own0 + j * own_step;
    if (!TOKEN || !cut) {
      *ml = a.own_ml + n;
      return a.own_o + n * d;
    }
    if (total < ctas && total * (c0 + j) / ctas == total * (c0 + j + 1) / ctas) return nullptr;  // an empty range
    if (j > 0) n -= kTokenRows;
    *ml = a.cut_ml + n;
    return a.cut_o + n * d;
  }
};
// The sequence of a token, -1 for none (a whole warp).
__device__ __forceinline__ int find_sequence(const AttnArgs& a, int tok, int lane) {
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int i = b0 + lane;
    const uint32_t hit = __ballot_sync(0xffffffffu, i < a.batch && tok >= a.cu_q[i] && tok < a.cu_q[i + 1]);
    if (hit) return b0 + __ffs(hit) - 1;
  }
  return -1;
}

// The joins.  A row is held by D/8 lanes, eight values each, its parts kAhead loads at a time: those of the prefix, then
// its own.  Many rows: a block takes one token, finds its parts once, and its lane groups take the heads in turn.
// Few rows: a block takes one row, and its lane groups the parts in turn.
constexpr int kAhead = 4;
constexpr int kJoinThreads = 256;
template <int D, bool QUANT, bool TOKEN>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const AttnArgs a) {
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x & 31, l = threadIdx.x % LANES;
  const int tok = (int)blockIdx.x;
  const int b = find_sequence(a, tok, lane);
  // whole warps go round, for the shuffles of the last step
  const int step = gridDim.y * (kJoinThreads / LANES);
  int head = blockIdx.y * (kJoinThreads / LANES) + threadIdx.x / LANES;
  // (the first kernel of the call is done when the one before this has started: only the parts are waited for)
  Parts<TOKEN> parts;
  if (b >= 0) parts.open(a, b);
  bool there = b >= 0 && head < a.heads && parts.find(a, tok, head);
  pdl_wait();
  if (b < 0) return;
  for (int head0 = head - lane / LANES; head0 < a.heads; head0 += step) {
    Sum sum;
    const int n = there ? parts.shared + parts.own : 0;
    for (int i = 0; i < n; i += kAhead) {
      float2 ml[kAhead];
      float v[kAhead][8];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const float2* pml;
        ml[x] = make_float2(kNegInf, 0.0f);
        const float* po = i + x < n ? parts.at(a, i + x, D, &pml) : nullptr;
        if (po == nullptr) continue;
        ml[x] = *pml;
        load_row(v[x], po + 8 * l);
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) sum.add(ml[x], v[x]);
    }
    finish_row<D, QUANT>(a, sum, tok, head, l, there);
    head += step;
    there = head < a.heads && parts.find(a, tok, head);
  }
}
template <int D, bool QUANT, bool TOKEN>
__global__ void __launch_bounds__(kJoinThreads) shared_join_row_kernel(const AttnArgs a) {
  constexpr int LANES = D / 8, TEAMS = kJoinThreads / LANES;
  __shared__ __align__(16) float so[TEAMS][D];
  __shared__ float2 sml[TEAMS];
  const int lane = threadIdx.x & 31, l = threadIdx.x % LANES, team = threadIdx.x / LANES;
  const int tok = (int)blockIdx.x, head = (int)blockIdx.y;
  const int b = find_sequence(a, tok, lane);
  Parts<TOKEN> parts;
  if (b >= 0) parts.open(a, b);
  const bool there = b >= 0 && parts.find(a, tok, head);
  pdl_wait();
  if (!there) return;
  const int n = parts.shared + parts.own;
  Sum sum;
  for (int i = team; i < n; i += TEAMS) {
    const float2* pml;
    const float* po = parts.at(a, i, D, &pml);
    if (po == nullptr) continue;
    float v[8];
    load_row(v, po + 8 * l);
    sum.add(*pml, v);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4*>(&so[team][8 * l + i]) = make_float4(sum.o[i], sum.o[i + 1], sum.o[i + 2], sum.o[i + 3]);
  if (l == 0) sml[team] = make_float2(sum.m, sum.l);
  __syncthreads();
  if (threadIdx.x >= 32) return;
  // one warp, whose lane groups do the same
  Sum all;
#pragma unroll 4
  for (int t = 0; t < TEAMS; ++t) {
    float v[8];
    load_row(v, &so[t][8 * l]);
    all.add(sml[t], v);
  }
  finish_row<D, QUANT>(a, all, tok, head, l, threadIdx.x < LANES);
}

}  // namespace

cudaError_t launch_shared_prep(const AttnArgs& a, const int32_t* cu_groups, const int32_t* prefix_lens, bool token,
                               cudaStream_t stream) {
  const SharedState s = {const_cast<SharedGroup*>(a.group), const_cast<int2*>(a.seq), const_cast<int64_t*>(a.units),
                         const_cast<int4*>(a.counts)};
  const bool quant = kv_quantised(a.cache.format), few = a.max_q * (a.heads / a.kv_heads) <= 8;
  const float wide = (float)a.head_dim / 128.0f;
  SharedCosts cost = {};
  cost.block = (quant ? 1.3f : 1.05f) * wide;
  cost.joint = 0.72f * wide;
  cost.fixed = quant ? 18.0f : 11.0f;
  cost.unit = (few ? 0.6f : 0.7f) * wide;
  cost.unit_dram = (float)(128 * kv_row_bytes(a.cache.format, a.head_dim)) / 5.3e6f;
  cost.token = token ? 1 : 0;
  cost.per_sm = token_ctas_per_sm(a.max_q * (a.heads / a.kv_heads));
  shared_prep_kernel<<<1, kPrepThreads, 0, stream>>>(a, cu_groups, prefix_lens, s, cost);
  return cudaGetLastError();
}

cudaError_t launch_shared_join(const AttnArgs& a, bool token, cudaStream_t stream) {
  const int quant = kv_quantised(a.cache.format), wide = a.head_dim == 128, teams = kJoinThreads / (a.head_dim / 8);
  const int64_t rows = a.total_q * a.heads;
  const bool few = rows <= kSms * 4 && a.heads <= 65535;
  // a block a token, or while that leaves SMs idle a token's heads over several
  const int heads = (a.heads + teams - 1) / teams;
  const unsigned y = few ? (unsigned)a.heads : (unsigned)(a.total_q >= 4 * kSms ? 1 : heads);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kJoinThreads, 1u, 1u);
  cfg.gridDim = dim3((unsigned)a.total_q, y, 1u);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  using Kernel = void (*)(const AttnArgs);
  static constexpr Kernel kernels[2][2][2][2] = {
      {{{shared_join_kernel<64, false, false>, shared_join_kernel<64, false, true>},
        {shared_join_kernel<64, true, false>, shared_join_kernel<64, true, true>}},
       {{shared_join_kernel<128, false, false>, shared_join_kernel<128, false, true>},
        {shared_join_kernel<128, true, false>, shared_join_kernel<128, true, true>}}},
      {{{shared_join_row_kernel<64, false, false>, shared_join_row_kernel<64, false, true>},
        {shared_join_row_kernel<64, true, false>, shared_join_row_kernel<64, true, true>}},
       {{shared_join_row_kernel<128, false, false>, shared_join_row_kernel<128, false, true>},
        {shared_join_row_kernel<128, true, false>, shared_join_row_kernel<128, true, true>}}}};
  return cudaLaunchKernelEx(&cfg, kernels[few][wide][quant][token], a);
}

}  // namespace exl3
