// exl3_attn_tile.cu -- causal attention of many query rows: whole prompts over
// packed keys and values, and chunks of new tokens over the paged cache.
//
// Rows.  The query heads of a group share their keys, so the rows of a sequence
// and key head are its query tokens times the group's heads, token major: one
// CTA takes two tiles of 128 (the M of the MMA), as many whole tokens as fit into
// each, and reads each key and value once for all of them.  (Whole tokens make a
// row tile one box of a tensor copy: with a thread loading and storing a row, the
// two took 10000 cycles an item, half of a 512-token prompt's time.)
//
// Per block of 64 keys and 128 rows:
//     S = Q K^T            tcgen05.mma, both operands in shared memory, S in tensor memory
//     m' = max(m, S c),  P = 2^(S c - m'),  l += sum P    (c = scale * log2 e; one thread a row)
//     O += P V             tcgen05.mma, P from tensor memory (written over S), V from shared memory
// The running maximum is only raised when it has grown by more than 8 (log2):
// until then P stays below 2^8, l and O are held relative to the old maximum
// in fp32, and O in tensor memory needs no rescaling.  P rounds to the operand
// type; l sums the unrounded values in fp32.
//
// What bounds it: the tensor core (4 * 128 * 64 * D operations a block) once there
// are a few hundred rows a sequence.  Each row tile has two buffers of scores, so
// the products of the next block run under a block's softmax, and a warp of its
// own issues them.  (Blocks of 128 keys have products that read less shared memory,
// but leave room for one buffer a tile: then each tile's products and softmax wait
// for one another, and 16384 tokens of 32 heads took 1529 us.)
//
// Measured (query heads, key heads of 128; rates by the multiply-adds that the mask leaves):
//   one prompt of 16384 tokens, 32 and 8 heads, bf16           1400 us: 1570 TFLOP/s, 82% of a large matrix product's;
//     in a loop that runs into the power limit 1510 to 1540 us, 76%
//   ten prompts of 1 to 2048 tokens, 40 and 8 heads            144 us: 920 TFLOP/s; an item has 8 to 32 blocks of
//     about 0.95 us each, and its diagonal blocks, first scores and output (2 to 4.5 us) weigh more
//   512 tokens over 32768 16-bit keys, 32 and 8 heads          220 us: 1240 TFLOP/s; 64 items in seven parts each, three
//     a CTA of 73 blocks, and about 15 us for the parts' results and their join
//   chunks of 129 to 700 tokens and single ones over up to 15000 8-bit keys, window 4096, 96 and 8 heads
//     229 us: 885 TFLOP/s; four warps make fp16 rows of the codes, four passes' codes loaded ahead (one after the other:
//     246), and an output costs 4 to 12 us
// The kernels over 16-bit rows spill 12 bytes a thread beside their 168 registers; those over codes spill none.
// What holds the first below the peak is the products themselves: with the softmax reduced to passing the barriers on,
// the same prompt takes 1331 us.  A score product of N = 64 reads its 128 rows of q from shared memory for half the
// operations that N = 128 would have (48 cycles instead of 32 a k16 step), and a commit, a wait and the next issue leave
// gaps that two row tiles only partly fill.
//
// A CTA with no more than 128 rows gives both halves the same rows and every
// other block of keys each, and joins them at the end.  With few row tiles the keys are
// also split over CTAs, and attn_tile_join_kernel joins the parts.
//
// The grid has a CTA an item, but one CTA an SM takes item after item: when its
// loader has issued an item's last copies it cancels a CTA that has not started
// (clusterlaunchcontrol) and takes its item, so the copies and first scores of the
// next item run under the last softmax and the output of the one before, and the
// order of the items stays the hardware's.
//
// Roles: warps 0-3 and 4-7 softmax of row tiles 0 and 1 (a thread a row), warps 8
// and 10 issue their MMAs, warp 9 takes the items and issues the copies of keys and values
// into a ring of slots, warp 11 those of q; for the quantised cache formats it copies the codes and
// scales into a ring of their own, and warps 12-15 turn them into fp16 rows.
// Quantised rows stay in the rotated basis (see exl3_rope_cache.cu): q is rotated
// on its way into shared memory and the output on its way out, each a transform
// within a thread.  Keys, values and q round to fp16 there, 2^-11 of each entry at the most, below the codes' own
// steps, in units of powers of two: a row's of q, and of every 16 keys and 16 values, by their largest scale, which
// nothing can pass.  A group's key unit is a factor of its scores, its value unit an addend of its exponents, so groups
// of any sizes meet (one unit an item, from its first tile's scales, made a later row of 2000 times the scale
// infinite).  (With bf16 rows the results are as exact as 64-bit sums rounded to bf16; with fp16 rows the error is
// 0.0006 (4 bits) to 0.0009 (8 bits) of the result's norm, of which rounding the result is 0.0002.  A second fp16
// term of q, as few rows have it, would take 64 KB of shared memory that the rings need, and twice the score products.)
//
// Tensor memory: S of row tile i at columns 128 i and 128 i + 64, O at 256 + 128 i.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "exl3_attn.h"
#include "exl3_attn_seq.cuh"
#include "exl3_sm100.cuh"

namespace exl3 {
namespace {

// Compiled once for whole sequences and once for sequences that begin with their group's keys.  Then an item is a row
// tile of a group's query tokens over the group's prefix, or of a sequence's own tokens over its own keys, and its
// result stays a part (over a quantised cache in the rotated basis) for a join of all parts of a row.
#ifdef EXL3_ATTN_SHARED
constexpr bool kShared = true;
#else
constexpr bool kShared = false;
#endif

enum Source { kPacked = 0, kPaged16 = 1, kPaged8 = 2, kPaged4 = 3 };
constexpr int kKeys = 128;      // keys of a copy (a tile)
constexpr int kBlock = 64;      // keys of a step
constexpr int kTileRows = 128;  // rows of a tile; a CTA has two tiles
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kSlack = 8.0f;

constexpr int kUnitKeys = 16;   // keys that share a unit (quantised formats)
// What the fp16 operands of a tile of a quantised cache are in units of: powers of two for every 16 keys and values.
struct Units {
  int k[kKeys / kUnitKeys], v[kKeys / kUnitKeys];  // log2
};
// A group's largest scale lies in [2^kScaleTop, 2^(kScaleTop + 1)) of its unit: codes then reach 2^15, and scales 2^24
// times smaller still have all their bits.  No unit is below 2^kLeastUnit, so that sums of weights, which the values'
// units divide, stay within fp32; the format's least scale, 2^-100, has its bits in that unit too.
constexpr int kScaleTop = 7, kLeastUnit = -90;
// Weights over a quantised cache may reach 2^15 (2^8 by the maximum's slack), so that those far below the largest are
// still normal fp16 numbers.
constexpr float kRoom = 7.0f;

template <int D, int SRC>
struct TileCfg {
  static constexpr bool kQuant = SRC >= kPaged8;
  static constexpr int kConverters = kQuant ? 4 : 0;   // warps 12-15
  static constexpr int kThreads = kQuant ? 512 : 384;  // whole groups of four warps, for the register split
  // Registers a thread of each group of four warps.  The kernel is launched with 168 (384 threads) or 128 (512); what
  // the softmax warps gain is what the others give up.
  static constexpr int kLaunchRegs = kQuant ? 128 : 168;
  static constexpr int kSoftmaxRegs = kQuant ? 192 : 208;
  static constexpr int kIssueRegs = kQuant ? 72 : 88;
  static constexpr int kConvertRegs = 56;
  static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs + (kQuant ? 128 * kConvertRegs : 0) <= kLaunchRegs * kThreads,
                "the split draws on the registers of the launch");
  static constexpr int kSlot = kKeys * D * 2;
  static constexpr int kSlots = D == 64 ? 8 : kQuant ? 4 : 5;
  // codes and scales of 128 keys or values as they lie in the cache
  static constexpr int kRowBytes = SRC == kPaged8 ? D : D / 2;
  static constexpr int kCodes = kKeys * kRowBytes;
  static constexpr int kRaw = kCodes + kKeys * 2;
  static constexpr int kRaws = !kQuant ? 0 : kRaw > 16 * 1024 ? 2 : 3;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileRows * D * 2;
  static constexpr int kRawRing = kRing + kSlots * kSlot;
  static constexpr int kCtrl = kRawRing + kRaws * kRaw;  // barriers, items, a joint item's exponents, tiles' units
  static constexpr int kSmem = 1024 + kCtrl + 1280 + (kQuant ? kSlots / 2 * (int)sizeof(Units) : 0);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kSmem > 114 * 1024, "one CTA an SM: each allocates all of tensor memory");
  static_assert(kRing >= kTileRows * D * 4, "q's room holds a tile's output for the join");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// One look at a barrier's phase: SPIN answers at once, else after as long as the hardware holds a waiting thread.
// (With a suspend-time hint waiting warps woke late: 16384 tokens of 32 heads took 1600 us instead of 1411.)
template <bool SPIN>
__device__ __forceinline__ bool bar_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (SPIN) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  }
  return ok != 0;
}
// mbar_wait in few instructions: the many waits of this kernel are code that its warps walk through once a block.
template <bool SPIN = false>
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t b = smem_u32(bar);
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t tries = 0; !bar_poll<SPIN>(b, parity); ++tries) {
    if ((tries & 255u) != 0) continue;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitTimeoutNs) {
      atomicOr(&g_device_error, kErrWaitTimeout);
      return false;
    }
  }
  return true;
}
// Two fp32 multiply-adds / adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Ask for a CTA of this grid that has not started: 16 bytes of answer at `answer`, completing on `bar`.
__device__ __forceinline__ void cancel_cta(uint32_t answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(smem_u32(bar))
               : "memory");
}
// Its index, or -1 when there is none left.
__device__ __forceinline__ int cancelled_cta(uint32_t answer) {
  int x;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%1];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n mov.b32 %0, -1;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n}\n"
      : "=r"(x)
      : "r"(answer)
      : "memory");
  return x;
}
// Bytes on their way into L2; address and size as for a bulk copy.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Sixteen lanes of tensor memory, eight 32-bit columns a piece: lane t gets columns 2 (t % 4), + 1 of rows t / 4 (first
// two registers of a piece) and t / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr)
               : "memory");
}
// Instruction descriptor, kind::f16 with fp32 accumulators: operand types at bits 7 and 10 (1: bf16), B transposed
// (N contiguous in shared memory) at bit 16.
__host__ __device__ constexpr uint32_t idesc(bool bf16, int m, int n, bool b_n_major) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
// Descriptor of an operand whose contiguous axis is N, 128-byte swizzled: rows of 64 values, eight rows (of k) an
// atom of 1024 bytes (stride offset), `lead` bytes from one block of 64 columns to the next (leading offset).
__device__ __forceinline__ uint64_t sdesc_n_major(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Byte offset of 16-byte chunk c (of D/8) of row r in a [128][D] operand: halves of 64 columns, 128-byte swizzled.
__device__ __forceinline__ uint32_t row_chunk(int r, int c) {
  return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Position of value i of a row among the operand's columns: the 4-bit codes come out of a word as the pairs
// (0, 4) (1, 5) (2, 6) (3, 7), and stay in that order in keys, values and q alike.
template <int SRC>
__device__ __forceinline__ constexpr int column_value(int c) {
  return SRC == kPaged4 ? (c & ~7) + ((c & 1) << 2) + ((c >> 1) & 3) : c;
}
// In-thread Hadamard transform of a row.
template <int D>
__device__ __forceinline__ void hadamard_row(float (&v)[D]) {
#pragma unroll
  for (int s = 1; s < D; s *= 2)
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (!(i & s)) {
        const float x = v[i], y = v[i + s];
        v[i] = x + y;
        v[i + s] = x - y;
      }
}

struct TileMaps {
  CUtensorMap q, k, v;
};

// What a CTA works on at a time.
struct Span {  // blocks of one half: b0, b0 + step, ... below b1 (b1 <= b0: none)
  int b0, b1, step;
};
struct Item {
  int64_t q0;        // first packed query token of the sequence
  int kvh, first;    // key head; position of the sequence's first query token
  int tok0, toks;    // query tokens of the item within the sequence
  int kv_len;
  int base;          // first key of block 0
  int b, split;
  int joint;         // both halves on the same rows, blocks in turn
  Span span[2];
  int jlo, jhi;      // key tiles (two blocks each) that a half uses
  int tail;          // the key tile that the length ends in, where its value rows past the end must be made zeros; or -1
  int lead;          // rows of key tile 0 before the first that the item's queries see: value rows to be made zeros too
  int done;          // no item
#ifdef EXL3_ATTN_SHARED
  // where the rows' parts go: row part_row + token (in the sequence or group) * part_stride + head (in the group)
  float* part_o;
  float2* part_ml;
  int64_t part_row;
  int part_stride;
  int merge;  // the halves of a joint item meet in shared memory; else each leaves a part of its own
#endif
};
__device__ __forceinline__ bool merges(const Item& it) {
#ifdef EXL3_ATTN_SHARED
  return it.merge != 0;
#else
  return it.joint != 0;
#endif
}

// Whether value rows of key tile j must be made zeros: a weight of zero does not hide what is not finite.
__device__ __forceinline__ bool mend_values(int j, int tail, int lead) { return j == tail || (j == 0 && lead > 0); }

// Blocks of n0 .. n1 that half i of the item uses.
__device__ Span half_span(const AttnArgs& a, const Item& it, int n0, int n1, int i) {
  if (it.joint) return Span{min(n0 + ((n0 & 1) ^ i), n1), n1, 2};  // half 0 the even blocks
  const int t0 = it.tok0 + i * a.tile_tokens;
  const int t1 = min(t0 + a.tile_tokens, it.tok0 + it.toks) - 1;
  const int lo = a.window > 0 ? max(0, it.first + t0 - a.window + 1) : 0;
  if (t1 < t0 || it.first + t1 < lo) return Span{n0, n0, 1};
  const int s0 = max(n0, (lo - it.base) / kBlock), s1 = min(n1, (it.first + t1 - it.base) / kBlock + 1);
  return s0 < s1 ? Span{s0, s1, 1} : Span{n0, n0, 1};
}

#ifdef EXL3_ATTN_SHARED
// The item of CTA index idx (a whole warp); false past the last.  The prefixes' row tiles come first, then those of the
// sequences' own keys.
template <int SRC>
__device__ bool find_item(const AttnArgs& a, int lane, int64_t idx, Item* it) {
  const int per = 2 * a.tile_tokens, group = a.heads / a.kv_heads;
  const int4 counts = __ldcg(a.counts);
  const int prefix_items = counts.x;
  const bool prefix = idx < prefix_items;
  if (!prefix && a.splits == 0) return false;  // own keys go through the token kernel
  // Items come in lists, one a group or (own keys) a sequence: of each its row tiles, of each its key heads, of each its
  // parts.  In 32 bits: a grid has no more.
  int place = prefix ? (int)idx : (int)idx - prefix_items, base = 0;
  const int lists = prefix ? a.groups : a.batch, total = (int)a.total_q;
#pragma unroll 1
  for (int b0 = 0; b0 < lists; b0 += 32) {
    const int b = b0 + lane;
    int c0 = 0, n = 0, keys = 0, seq = b, parts = 1;
    if (b < lists) {
      if (prefix) {
        const SharedGroup* g = a.group + b;
        c0 = __ldcg(&g->q0), n = __ldcg(&g->tokens), keys = __ldcg(&g->keys), seq = __ldcg(&g->lead), parts = __ldcg(&g->parts);
        if (keys == 0) n = 0;
      } else {
        c0 = max(0, min(a.cu_q[b], total));
        n = max(0, min(a.cu_q[b + 1], total) - c0);
        keys = max(0, min(a.kv_lens[b], a.table_width << a.cache.page_shift));
        parts = shared_own_parts(a, b, counts.z);
      }
    }
    const int tiles = (n + per - 1) / per, here = tiles * a.kv_heads * parts;
    int inc = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += p;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + inc > place);
    if (hit) {
      const int at = __ffs(hit) - 1;
      place -= base + __shfl_sync(0xffffffffu, inc - here, at);
      const int count = __shfl_sync(0xffffffffu, tiles, at), splits = __shfl_sync(0xffffffffu, parts, at);
      const int q_len = __shfl_sync(0xffffffffu, n, at);
      const int q0 = __shfl_sync(0xffffffffu, c0, at);
      it->q0 = q0;
      it->b = __shfl_sync(0xffffffffu, seq, at);
      it->kv_len = __shfl_sync(0xffffffffu, keys, at);
      const int split = place % splits;
      place /= splits;
      it->kvh = place % a.kv_heads;
      it->tok0 = (count - 1 - place / a.kv_heads) * per;
      it->toks = min(per, q_len - it->tok0);
      it->split = split;
      it->part_o = prefix ? a.prefix_o : a.own_o;
      it->part_ml = prefix ? a.prefix_ml : a.own_ml;
      it->part_stride = prefix ? group : a.heads;
      it->part_row = prefix ? idx * kPrefixRows - it->tok0 * group : (split * a.total_q + q0) * a.heads + it->kvh * group;
      // every query of a group sees all of the prefix: as if it stood behind it
      it->first = prefix ? it->kv_len - 1 : it->kv_len - q_len;
      it->joint = it->toks <= a.tile_tokens;
      it->merge = it->joint && !prefix;
      // whole tiles of keys, so that no page is cut by a tile's first key
      const int lo = prefix ? 0 : __ldcg(&a.seq[it->b].x);
      const int p1 = min(it->first + it->tok0 + it->toks, it->kv_len) - 1;
      it->base = lo;
      it->lead = 0;
      const int blocks = p1 >= lo ? (p1 - lo) / kBlock + 1 : 0;
      // in whole tiles of two blocks, so that none is copied twice
      // (2^24 pairs at the most, and 32 parts: below 2^31)
      const int pairs = (blocks + 1) >> 1;
      const int n0 = 2 * (pairs * split / splits), n1 = min(blocks, 2 * (pairs * (split + 1) / splits));
      it->span[0] = half_span(a, *it, n0, n1, 0);
      it->span[1] = half_span(a, *it, n0, n1, 1);
      const Span s0 = it->span[0], s1 = it->span[1];
      const bool use0 = s0.b0 < s0.b1, use1 = s1.b0 < s1.b1;
      it->jlo = (use0 && use1 ? min(s0.b0, s1.b0) : use0 ? s0.b0 : use1 ? s1.b0 : 0) >> 1;
      it->jhi = ((use0 && use1 ? max(s0.b1, s1.b1) : use0 ? s0.b1 : use1 ? s1.b1 : 0) + 1) >> 1;
      const int over = it->kv_len - lo;
      it->tail = (over & 15) != 0 && over / kKeys >= it->jlo && over / kKeys < it->jhi ? over / kKeys : -1;
      it->done = 0;
      return true;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

#else
// The item of CTA index idx (a whole warp); false past the last row tile.
template <int SRC>
__device__ bool find_item(const AttnArgs& a, int lane, int64_t idx, Item* it) {
  const int per = 2 * a.tile_tokens;  // tokens of an item
  it->split = (int)(idx % a.splits);
  idx /= a.splits;
  it->kvh = (int)(idx % a.kv_heads);
  const int64_t tile = idx / a.kv_heads;
  // the sequence that holds row tile `tile`
  int64_t base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int b = b0 + lane;
    int64_t c0 = 0, n = 0;
    if (b < a.batch) {
      c0 = a.cu_q[b];
      c0 = c0 < 0 ? 0 : c0 > a.total_q ? a.total_q : c0;
      const int64_t c1 = a.cu_q[b + 1] > a.total_q ? a.total_q : a.cu_q[b + 1];
      n = c1 > c0 ? c1 - c0 : 0;
    }
    const int tiles = ((int)n + per - 1) / per;
    int64_t inc = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += p;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + inc > tile);
    if (hit) {
      const int at = __ffs(hit) - 1;
      const int64_t before = base + __shfl_sync(0xffffffffu, inc - tiles, at);
      const int count = __shfl_sync(0xffffffffu, tiles, at);
      const int q_len = (int)__shfl_sync(0xffffffffu, n, at);
      it->q0 = __shfl_sync(0xffffffffu, c0, at);
      it->b = b0 + at;
      // a sequence's last row tiles see the most keys and go first
      it->tok0 = (count - 1 - (int)(tile - before)) * per;
      it->toks = min(per, q_len - it->tok0);
      it->kv_len = q_len;
      if constexpr (SRC != kPacked) {
        const int64_t room = (int64_t)a.table_width << a.cache.page_shift;
        const int64_t kl = a.kv_lens[it->b];
        it->kv_len = (int)(kl < 0 ? 0 : kl > room ? room : kl);
      }
      it->first = it->kv_len - q_len;
      it->joint = it->toks <= a.tile_tokens;
      // positions of the item's first and last token
      const int p0 = it->first + it->tok0, p1 = p0 + it->toks - 1;
      int lo = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
      const int seen = lo;
      if constexpr (SRC != kPacked) {
        // whole pages (or 128 keys of a larger one), so that a page is never cut by a tile's first key
        const int align = a.cache.page_shift < 7 ? 1 << a.cache.page_shift : kKeys;
        lo &= ~(align - 1);
      }
      it->base = lo;
      it->lead = seen - lo;
      const int blocks = p1 >= lo ? (p1 - lo) / kBlock + 1 : 0;
      const int from = min(it->lead / kBlock, blocks);  // blocks before the first key are nobody's
      const int n0 = from + (int)((int64_t)(blocks - from) * it->split / a.splits);
      const int n1 = from + (int)((int64_t)(blocks - from) * (it->split + 1) / a.splits);
      it->span[0] = half_span(a, *it, n0, n1, 0);
      it->span[1] = half_span(a, *it, n0, n1, 1);
      // the spans of two non-empty halves overlap or touch
      const Span s0 = it->span[0], s1 = it->span[1];
      const bool use0 = s0.b0 < s0.b1, use1 = s1.b0 < s1.b1;
      it->jlo = (use0 && use1 ? min(s0.b0, s1.b0) : use0 ? s0.b0 : use1 ? s1.b0 : 0) >> 1;
      it->jhi = ((use0 && use1 ? max(s0.b1, s1.b1) : use0 ? s0.b1 : use1 ? s1.b1 : 0) + 1) >> 1;
      // a weight of zero times what a page or the next sequence holds past the length need not be zero
      const int over = it->kv_len - lo;
      it->tail = (over & 15) != 0 && over / kKeys >= it->jlo && over / kKeys < it->jhi ? over / kKeys : -1;
      it->done = 0;
      return true;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

#endif

// D: head size.  BF16: operand type (fp16 for the quantised formats).
template <int D, int SRC, bool BF16>
__global__ void __launch_bounds__(TileCfg<D, SRC>::kThreads, 1)
    attn_tile_kernel(const __grid_constant__ TileMaps maps, const __grid_constant__ AttnArgs a) {
  using C = TileCfg<D, SRC>;
  constexpr int NS = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* data = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* base = data + C::kCtrl;
  uint64_t* kvfull = reinterpret_cast<uint64_t*>(base);  // [NS] slot filled
  uint64_t* kvempty = kvfull + 8;                        // [NS] slot read by the MMAs
  uint64_t* rawfull = kvempty + 8;                       // [kRaws] codes and scales landed
  uint64_t* rawempty = rawfull + 4;                      // [kRaws] converted
  uint64_t* qfull = rawempty + 4;                        // [2] a half's q in shared memory
  uint64_t* sfull = qfull + 2;                           // [2][2] a half's scores in a buffer of tensor memory
  uint64_t* pfull = sfull + 4;                           // [2][2] weights in tensor memory, O rescaled
  uint64_t* pvdone = pfull + 4;                          // [2] a block's weights times values added to O
  uint64_t* ofull = pvdone + 2;                          // [2] every MMA of a half's item done
  uint64_t* ifull = ofull + 2;                           // [2] item published
  uint64_t* iempty = ifull + 2;                          // [2] and read by every warp
  uint64_t* jfull = iempty + 2;                          // joint item: half 1's output in shared memory
  uint64_t* jfree = jfull + 1;                           // and read by half 0
  uint64_t* vfix = jfree + 1;                            // [NS] value rows that no query sees are zeros
  uint64_t* qraw = vfix + 8;                             // [2] a half's q as it is (quantised formats: still to be rotated)
  uint64_t* qempty = qraw + 2;                           // [2] a half's scores of an item are done
  uint64_t* clc = qempty + 2;                              // answer to a cancel request
  uint64_t* mdrain = clc + 1;                            // [2] MMAs issued before a wait gave up
  uint64_t* jopen = mdrain + 2;                          // joint item: half 0 is done with q's room
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(jopen + 1);
  uint8_t* answer = base + 496;                          // 16 bytes
  Item* items = reinterpret_cast<Item*>(base + 512);     // [2]
  float* jlse = reinterpret_cast<float*>(base + 768);    // [128] joint item: log2 of half 1's sums
  Units* units = reinterpret_cast<Units*>(base + 1280);  // [NS / 2] quantised: of the tile whose values are in slot 2x + 1
  static_assert(((2 * 8 + 2 * 4) + (8 + 28)) * 8 + 4 <= 496 && 512 + 2 * sizeof(Item) <= 768, "control area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.heads / a.kv_heads;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kvfull[s], C::kQuant ? C::kConverters : 1);
      mbar_init(&kvempty[s], 2);
      mbar_init(&vfix[s], 1);
    }
    for (int s = 0; s < C::kRaws; ++s) {
      mbar_init(&rawfull[s], 1);
      mbar_init(&rawempty[s], C::kConverters);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], C::kQuant ? 4 : 1);
      mbar_init(&qraw[i], 1);
      mbar_init(&qempty[i], 1);
      mbar_init(&sfull[2 * i], 1);
      mbar_init(&sfull[2 * i + 1], 1);
      mbar_init(&pvdone[i], 1);
      mbar_init(&pfull[2 * i], 4);
      mbar_init(&pfull[2 * i + 1], 4);
      mbar_init(&ofull[i], 1);
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 11 + C::kConverters);
      mbar_init(&mdrain[i], 1);
    }
    mbar_init(jopen, 4);
    mbar_init(jfull, 4);
    mbar_init(jfree, 4);
    mbar_init(clc, 1);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (kShared) {
    pdl_wait();  // groups and starts
    pdl_launch_dependents();
  }

  // The n-th item, as every warp but the loader reads it; false when there is none (or a wait gave up).
  auto read_item = [&](uint32_t n, Item* it) {
    if (!bar_wait(&ifull[n & 1], (n >> 1) & 1u)) return false;
    *it = items[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&iempty[n & 1]);
    return it->done == 0;
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ---------------- softmax: a thread a row ----------------
    const int i = warp >> 2;
    const int r = 32 * (warp & 3) + lane;  // row of the tile, lane of tensor memory
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + 128 * i;  // buffer 0
    const uint32_t o_col = tmem + lanes + 256 + 128 * i;
    float c = a.scale_log2;  // quantised: times the unit of q's row, and a group's times the unit of its keys
    uint32_t tiles = 0;      // quantised: key tiles of the items before
#ifdef EXL3_ATTN_SHARED
    // Rotate the half's q where the copy has put it: LPQ lanes a row, chunk LPQ x + l of eight values the x-th of lane l, and
    // only rows that there are.  (A thread a row is 1400 instructions in a line, which an item that runs once has to fetch
    // first.  Of four and eight lanes the better by measurement, with issuing warps that looked at their barriers over and
    // over: 1600 tokens over 16000 8-bit keys 435 and 424 us, 4-bit ones 438 and 444; heads of 64 356 and 359.  Without that
    // the ones taken are 415, 418 us.)
    auto rotate_q = [&](const Item& x, uint32_t parity) {
      if (!bar_wait(&qraw[i], parity)) return false;
      constexpr int LPQ = D == 128 && SRC == kPaged8 ? 8 : 4;  // lanes of a row
      constexpr int N = D / LPQ, RP = 32 / LPQ;                // values a lane; rows a warp takes at a time
      const uint32_t at = smem_u32(data + C::kQ) + (uint32_t)i * (kTileRows * D * 2);
      const int l = lane % LPQ, rows = min(a.tile_tokens, x.toks - (x.joint ? 0 : i * a.tile_tokens)) * group;
#pragma unroll 1
      for (int p = 0; p < 32 / RP; ++p) {
        const int first = 32 * (warp & 3) + p * RP;
        if (first >= rows) break;
        float v[N];
#pragma unroll
        for (int y = 0; y < N / 8; ++y) {
          uint32_t w[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(at + row_chunk(first + lane / LPQ, LPQ * y + l))
                       : "memory");
          if (a.bf16) {
#pragma unroll
            for (int z = 0; z < 4; ++z) v[8 * y + 2 * z] = __uint_as_float(w[z] << 16), v[8 * y + 2 * z + 1] = __uint_as_float(w[z] & 0xFFFF0000u);
          } else {
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[z]));
              v[8 * y + 2 * z] = f.x, v[8 * y + 2 * z + 1] = f.y;
            }
          }
        }
        hadamard_row<N>(v);  // every bit of the place in a chunk and of the lane's chunk
#pragma unroll
        for (int st = 1; st < LPQ; st *= 2)
#pragma unroll
          for (int y = 0; y < N; ++y) {
            const float o = __shfl_xor_sync(0xffffffffu, v[y], st);
            v[y] = (l & st) ? o - v[y] : v[y] + o;
          }
        float top = 0.0f;
#pragma unroll
        for (int y = 0; y < N; ++y) top = fmaxf(top, fabsf(v[y]));
#pragma unroll
        for (int st = 1; st < LPQ; st *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, st));
        // in units of a power of two near its largest value, so that fp16 holds rows of any size alike
        const uint32_t e = unit_exponent(top);
        const float unit = __shfl_sync(0xffffffffu, power(e), LPQ * (lane % RP));
        if (lane / RP == p) c = a.scale_log2 * (unit * (8.0f / D));  // this thread's row
        const float f = power(254 - e);
#pragma unroll
        for (int y = 0; y < N / 8; ++y) {
          uint32_t w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            w[z] = pack2<false>(v[8 * y + column_value<SRC>(2 * z)] * f, v[8 * y + column_value<SRC>(2 * z + 1)] * f);
          sts128(at + row_chunk(first + lane / LPQ, LPQ * y + l), w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[i]);
      return true;
    };
#else
    // Rotate the half's q where the copy has put it, a thread a row.
    auto rotate_q = [&](const Item&, uint32_t parity) {
      if (!bar_wait(&qraw[i], parity)) return false;
      const uint32_t at = smem_u32(data + C::kQ) + (uint32_t)i * (kTileRows * D * 2);
      float v[D];
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at + row_chunk(r, x))
                     : "memory");
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (a.bf16) {
            v[8 * x + 2 * y] = __uint_as_float(w[y] << 16);
            v[8 * x + 2 * y + 1] = __uint_as_float(w[y] & 0xFFFF0000u);
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[y]));
            v[8 * x + 2 * y] = f.x;
            v[8 * x + 2 * y + 1] = f.y;
          }
        }
      }
      hadamard_row<D>(v);
      // in units of a power of two near its largest value, so that fp16 holds rows of any size alike
      float top = 0.0f;
#pragma unroll
      for (int x = 0; x < D; ++x) top = fmaxf(top, fabsf(v[x]));
      const uint32_t e = unit_exponent(top);
      c = a.scale_log2 * (power(e) * (8.0f / D));
      const float f = power(254 - e);
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        uint32_t w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          w[y] = pack2<false>(v[column_value<SRC>(8 * x + 2 * y)] * f, v[column_value<SRC>(8 * x + 2 * y + 1)] * f);
        sts128(at + row_chunk(r, x), w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[i]);
      return true;
    };
#endif
    auto used = [&](const Item& x) { return i ? x.span[1].b0 < x.span[1].b1 : x.span[0].b0 < x.span[0].b1; };

    Item it;
    uint32_t n = 0, jphase = 0;
    uint32_t blocks = 0;  // of this half so far: the buffers and their phases
    uint32_t oph = 0;     // phase of this half's outputs (an item without blocks of it has none)
    bool have = read_item(n, &it);
    uint32_t qph = 0;
    // this thread's row: query token (from the half's first) and head (of the group); none past the tile's whole tokens
    const int row_tok = r / group, row_head = r - row_tok * group;
    if (C::kQuant && have && used(it)) {
      have = rotate_q(it, qph);
      qph ^= 1u;
    }
    while (have) {
      bool ok = true;
      const int tok = it.tok0 + (it.joint ? 0 : i * a.tile_tokens) + row_tok;  // in the sequence
      const bool there = row_tok < a.tile_tokens && tok < it.tok0 + it.toks;
      const Span sp = i ? it.span[1] : it.span[0];
      const int pos = it.first + tok;
      const int lim = pos - it.base;                                            // last key it sees, from the item's first key
      const int low = a.window > 0 ? max(0, pos - a.window + 1) - it.base : 0;  // first
      float m = kNegInf;
      float2 l0 = make_float2(0.0f, 0.0f), l1 = make_float2(0.0f, 0.0f);
      bool any = false;
#pragma unroll 1
      for (int b = sp.b0; b < sp.b1; b += sp.step, ++blocks) {
        const uint32_t buf = blocks & 1u;
        ok = bar_wait(&sfull[2 * i + buf], blocks >> 1 & 1u);
        if (!ok) break;
        tc_fence_after();
        int ek[4] = {}, ev[4] = {};  // quantised: this block's units
        if constexpr (C::kQuant) {
          const uint32_t t = tiles + (uint32_t)((b >> 1) - it.jlo), x = t % (NS / 2);
          ok = bar_wait(&kvfull[2 * x + 1], t / (NS / 2) & 1u);  // they come with the tile's values
          if (!ok) break;
          const int4 k4 = *reinterpret_cast<const int4*>(units[x].k + 4 * (b & 1));
          const int4 v4 = *reinterpret_cast<const int4*>(units[x].v + 4 * (b & 1));
          ek[0] = k4.x, ek[1] = k4.y, ek[2] = k4.z, ek[3] = k4.w;
          ev[0] = v4.x, ev[1] = v4.y, ev[2] = v4.z, ev[3] = v4.w;
        }
        float s[kBlock];
        const uint32_t col = s_col + kBlock * buf;
#pragma unroll
        for (int x = 0; x < kBlock; x += 32) tmem_ld_32x32b_x32(col + x, *reinterpret_cast<uint32_t(*)[32]>(&s[x]));
        tmem_ld_wait();
        const int k0 = b * kBlock;
        if (__any_sync(0xffffffffu, k0 + kBlock - 1 > lim || k0 < low)) {
          const int hi = lim - k0, lo = low - k0;
#pragma unroll
          for (int x = 0; x < kBlock; ++x)
            if (x > hi || x < lo) s[x] = kNegInf;
        }
        float t[4];
        float top;
        float cg[4];  // quantised: factor of a group's scores
        if constexpr (C::kQuant) {
          // The values' units go into the exponents: weight times unit is what the product with the values needs, and
          // what the maximum is taken of.
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float* x = s + kUnitKeys * y;
            t[y] = max3(max3(x[0], x[1], x[2]), x[3], x[4]);
            const float u = max3(max3(x[5], x[6], x[7]), x[8], x[9]), v = max3(max3(x[10], x[11], x[12]), x[13], x[14]);
            t[y] = fmaxf(max3(t[y], u, v), x[15]);
            cg[y] = fmaxf(c * power(127 + ek[y]), 1.1754944e-38f);  // not 0: a masked score stays -inf
            t[y] = fmaf(t[y], cg[y], (float)ev[y]);
          }
          top = fmaxf(max3(t[0], t[1], t[2]), t[3]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) t[x] = max3(s[x], s[x + 4], s[x + 8]);
#pragma unroll
          for (int x = 12; x < 60; x += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y) t[y] = max3(t[y], s[x + y], s[x + y + 4]);
          top = fmaxf(max3(t[0], t[1], t[2]), max3(max3(t[3], s[60], s[61]), s[62], s[63])) * c;
        }
        const bool up = top > m + kSlack;
        if (__any_sync(0xffffffffu, up)) {
          const float f = up ? ex2(m - top) : 1.0f;
          m = up ? top : m;
          l0.x *= f, l0.y *= f, l1.x *= f, l1.y *= f;
          if (any) {
            ok = bar_wait(&pvdone[i], (blocks & 1u) ^ 1u);  // the block before this one is in O
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(o_col + x, o);
              tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st_x32(o_col + x, o);
            }
          }
        }
        any = true;
        // nothing seen yet: all scores are -inf, any finite reference does
        const float ref = m == kNegInf ? 0.0f : C::kQuant ? m - kRoom : m;
        uint32_t w[32];
        constexpr int kGroup = C::kQuant ? kUnitKeys : kBlock;
#pragma unroll
        for (int y = 0; y < 32; y += kGroup / 2) {
          const int gi = y / (kUnitKeys / 2);
          const float cf = C::kQuant ? cg[gi] : c, mf = C::kQuant ? (float)ev[gi] - ref : -ref;
          const float2 cc = make_float2(cf, cf), mm = make_float2(mf, mf);
          float2 g0 = C::kQuant ? make_float2(0.0f, 0.0f) : l0, g1 = C::kQuant ? make_float2(0.0f, 0.0f) : l1;
#pragma unroll
          for (int z = y; z < y + kGroup / 2; z += 2) {
            const float* x = s + 2 * z;
            float2 p = fma2(make_float2(x[0], x[1]), cc, mm), q = fma2(make_float2(x[2], x[3]), cc, mm);
            p.x = ex2(p.x), p.y = ex2(p.y), q.x = ex2(q.x), q.y = ex2(q.y);
            g0 = add2(g0, p);
            g1 = add2(g1, q);
            w[z] = pack2<BF16>(p.x, p.y);
            w[z + 1] = pack2<BF16>(q.x, q.y);
          }
          if constexpr (C::kQuant) {
            const float inv = power(127 - ev[gi]);  // the sum is of the weights alone
            l0 = fma2(g0, make_float2(inv, inv), l0);
            l1 = fma2(g1, make_float2(inv, inv), l1);
          } else {
            l0 = g0, l1 = g1;
          }
        }
        tmem_st_x32(col, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[2 * i + buf]);
      }

      float l = (l0.x + l0.y) + (l1.x + l1.y);
      if (C::kQuant) {
        m -= kRoom;  // what l and O are held relative to
        tiles += (uint32_t)(it.jhi - it.jlo);
      }
      Item next;
      have = ok && read_item(n + 1, &next);

      // ---- the rows' output.  Tensor memory is read sixteen rows at a time, a quad of lanes two of them: of rows
      // g and g + 8 a lane gets columns 8x + 2q, + 1.
      const int g = lane >> 2, q = lane & 3;
      if (used(it)) {
        ok = ok && bar_wait(&ofull[i], oph);
        oph ^= 1u;
      }
      // A joint item's meeting place is q's room, of both halves: half 1 may write there once half 0's products of this
      // item and of those before it are done.  (A look at half 0's ofull cannot tell: half 0 may be an item behind,
      // whose phase of that barrier has the other parity, or have no blocks here.)
      const bool merge = merges(it);
      if (merge) {
        if (i == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(jopen);
        } else if (ok) {
          ok = bar_wait(jopen, jphase);
        }
      }
      tc_fence_after();
      // this thread's row: its own part times f0, a joint item's other half's (already divided by its sum) times f1
      float f0 = 1.0f, f1 = 0.0f;
      if (ok && merge && i == 0) {
        ok = bar_wait(jfull, jphase);
        const float other = jlse[r];
        const float both = fmaxf(m, other);
        // a half without a maximum saw nothing (its sum is 0) or nothing but NaN (its sum is NaN)
        f0 = m == kNegInf ? (l == 0.0f ? 0.0f : l) : ex2(m - both);
        f1 = other == kNegInf ? 0.0f : ex2(other - both);
        l = l * f0 + f1;
        m = both;
      }
      const bool partial = (kShared || a.splits > 1) && !(merge && i == 1);
      if (!partial) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that saw no key gives zeros
        f0 *= inv, f1 *= inv;
      }
      if (!any) f0 = 0.0f;
      float* jo = reinterpret_cast<float*>(data + C::kQ) + r;  // [D][128]: a thread a column
      if (ok && merge && i == 1) jlse[r] = m + log2f(l);
#ifdef EXL3_ATTN_SHARED
      // half 1 of a joint item that does not meet half 0: its part lies a tile's rows on
      const int64_t part_row = it.part_row + (i == 1 && it.joint && !merge ? kTileRows : 0);
      if (ok && partial && there) it.part_ml[part_row + (int64_t)tok * it.part_stride + row_head] = make_float2(m, l);
#else
      const int64_t row = (it.q0 + tok) * a.heads + it.kvh * group + row_head;
      if (ok && partial && there) a.part_ml[(int64_t)it.split * a.total_q * a.heads + row] = make_float2(m, l);
#endif
#pragma unroll 1
      for (int h = 0; ok && h < 2; ++h) {
        float o[D / 2];  // o[4x + 2e + y]: row 16h + 8e + g of the warp, column 8x + 2q + y
        if (any) {
#pragma unroll
          for (int x = 0; x < D / 2; x += 16)
            tmem_ld_16x256b_x4(o_col + ((uint32_t)(16 * h) << 16) + 2 * x, *reinterpret_cast<uint32_t(*)[16]>(&o[x]));
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int x = 0; x < D / 2; ++x) o[x] = 0.0f;
        }
        if constexpr (C::kQuant && !kShared) {
          // Back out of the rotated basis.  Column 8x + 2q + y of the operands holds value 8x + 2q + y, or for the 4-bit
          // codes' order 8x + 4y + q: its bits are this lane's q, y and x.
#pragma unroll
          for (int x = 0; x < D / 2; x += 2) {
            const float u = o[x], v = o[x + 1];
            o[x] = u + v, o[x + 1] = u - v;
          }
#pragma unroll
          for (int st = 1; st < 4; st *= 2)
#pragma unroll
            for (int x = 0; x < D / 2; ++x) {
              const float u = __shfl_xor_sync(0xffffffffu, o[x], st);
              o[x] = (q & st) ? u - o[x] : o[x] + u;
            }
#pragma unroll
          for (int st = 4; st < D / 2; st *= 2)
#pragma unroll
            for (int x = 0; x < D / 2; ++x)
              if (!(x & st)) {
                const float u = o[x], v = o[x + st];
                o[x] = u + v, o[x + st] = u - v;
              }
#pragma unroll
          for (int x = 0; x < D / 2; ++x) o[x] *= 8.0f / D;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int src = 16 * h + 8 * e + g;  // lane whose row this is
          const float s0 = __shfl_sync(0xffffffffu, f0, src), s1 = __shfl_sync(0xffffffffu, f1, src);
          const int rtok = __shfl_sync(0xffffffffu, tok, src), rhead = __shfl_sync(0xffffffffu, row_head, src);
          const bool rthere = __shfl_sync(0xffffffffu, (int)there, src) != 0;
#pragma unroll
          for (int x = 2 * e; x < D / 2; x += 4) o[x] *= s0, o[x + 1] *= s0;
          if (merge) {
            float* at = jo + h * (D / 2) * kTileRows;
            if (i == 1) {
#pragma unroll
              for (int x = 2 * e; x < D / 2; x += 4) at[x * kTileRows] = o[x], at[(x + 1) * kTileRows] = o[x + 1];
              continue;
            }
#pragma unroll
            for (int x = 2 * e; x < D / 2; x += 4) {
              o[x] = fmaf(at[x * kTileRows], s1, o[x]);
              o[x + 1] = fmaf(at[(x + 1) * kTileRows], s1, o[x + 1]);
            }
          }
          if (partial) {
#ifdef EXL3_ATTN_SHARED
            float* dst = it.part_o + (part_row + (int64_t)rtok * it.part_stride + rhead) * D;
#else
            float* dst = a.part_o + (((int64_t)it.split * a.total_q + it.q0 + rtok) * a.heads + it.kvh * group + rhead) * D;
#endif
#pragma unroll
            for (int x = 0; x < D / 8; ++x) {
              if (!rthere) continue;
              if constexpr (SRC == kPaged4) {
                dst[8 * x + q] = o[4 * x + 2 * e];
                dst[8 * x + 4 + q] = o[4 * x + 2 * e + 1];
              } else {
                *reinterpret_cast<float2*>(dst + 8 * x + 2 * q) = make_float2(o[4 * x + 2 * e], o[4 * x + 2 * e + 1]);
              }
            }
          } else {
            uint16_t* dst = static_cast<uint16_t*>(a.out) + (it.q0 + rtok) * a.out_token_stride +
                            (int64_t)(it.kvh * group + rhead) * a.out_head_stride;
            const bool to_bf16 = C::kQuant ? a.bf16 != 0 : BF16;
            auto two = [&](float u, float v) { return to_bf16 ? pack2<true>(u, v) : pack2<false>(u, v); };
#pragma unroll
            for (int x = 0; x < D / 8; x += 4) {
              // four pieces of eight columns; the quad's transpose gives lane q the whole of piece x + q
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                float u = o[4 * (x + y) + 2 * e], v = o[4 * (x + y) + 2 * e + 1];
                if constexpr (SRC == kPaged4) {
                  // values q and 4 + q of the piece: swap with the neighbour for two next to each other
                  const float give = (q & 1) ? u : v;
                  const float take = __shfl_xor_sync(0xffffffffu, give, 1);
                  if (q & 1) u = take;  // lane 1, 3: values 4 + q - 1, 4 + q
                  else v = take;        // lane 0, 2: values q, q + 1
                }
                w[y] = two(u, v);
              }
#pragma unroll
              for (int st = 1; st < 4; st *= 2)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (!(y & st)) {
                    const uint32_t give = (q & st) ? w[y] : w[y + st];
                    const uint32_t take = __shfl_xor_sync(0xffffffffu, give, st);
                    if (q & st) w[y] = take;
                    else w[y + st] = take;
                  }
              // w[y]: what lane y had of piece x + q
              if constexpr (SRC == kPaged4) {
                // lanes 0 and 2 had values 0, 1 and 2, 3; lanes 1 and 3 values 4, 5 and 6, 7
                const uint32_t t = w[1];
                w[1] = w[2], w[2] = t;
              }
              if (rthere) *reinterpret_cast<uint4*>(dst + 8 * (x + q)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      if (merge) {
        fence_proxy_async_smem();  // the next q is copied over what was written and read here
        __syncwarp();
        if (lane == 0) mbar_arrive(i ? jfull : jfree);
        if (ok && i == 1) ok = bar_wait(jfree, jphase);
        jphase ^= 1u;
      }
      tc_fence_before();
      if (C::kQuant && ok && have && used(next)) {
        ok = rotate_q(next, qph);
        qph ^= 1u;
      }
      have = have && ok;
      it = next;
      ++n;
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
    if (warp == 8 || warp == 10) {
      // ---------------- MMA issue: a warp a half ----------------
      // Looking at a barrier over and over takes issue slots, which the conversion of codes wants (1600 tokens over 16000
      // 4-bit keys, shared: 426 us with it and 418 without; 16-bit ones 340 and 358).
      constexpr bool SPIN = !(kShared && C::kQuant);
      // The MMAs' descriptors are taken from uniform registers.  What comes out of shared memory is the same in every
      // lane but not known to be: it goes through a warp reduction, whose result is.
      constexpr uint32_t kIdS = idesc(BF16, 128, kBlock, false);
      constexpr uint32_t kIdO = idesc(BF16, 128, D, true);
      auto uni = [](int x) { return (int)__reduce_or_sync(0xffffffffu, (unsigned)x); };
      const int i = uni(warp == 10);
      const uint64_t qd = sdesc_sw128(smem_u32(data + C::kQ)) + (uint64_t)(i * (kTileRows * D * 2 >> 4));
      const uint64_t kd0 = sdesc_sw128(smem_u32(data + C::kRing));
      const uint64_t vd0 = sdesc_n_major(smem_u32(data + C::kRing), kKeys * 128);
      const uint32_t tm = (uint32_t)uni((int)tmem) + 128 * i;  // this half's scores and weights; its output 256 columns on
      const uint32_t one = elect_one();
      bool ok = true;
      uint32_t n = 0, qph = 0, blocks = 0;
      uint32_t fph = 0;  // phases of the slots' vfix (a bit a slot)
      // The ring holds K(jlo), V(jlo), K(jlo + 1), ... of each item: where the next tile's keys and values lie.
      uint32_t slot[2] = {0u, 1u}, sph[2] = {0u, 0u};
      auto next_slot = [&](int value) {
        slot[value] += 2;
        if (slot[value] >= NS) {
          slot[value] -= NS;
          sph[value] ^= 1u;
        }
      };
      while (ok) {
        Item it;
        if (!__all_sync(0xffffffffu, read_item(n, &it))) break;
        ++n;
        const int b0 = uni(i ? it.span[1].b0 : it.span[0].b0), b1 = uni(i ? it.span[1].b1 : it.span[0].b1), step = uni(it.joint) + 1;
        const int jlo = uni(it.jlo), jhi = uni(it.jhi), tail = uni(it.tail), lead = uni(it.lead), keys = uni(it.kv_len - it.base);
        int kt = jlo, vt = jlo;  // tiles whose keys / values come next
        // Tiles that this half does not use, before its first and after its last: released once they are filled, so that
        // releases stay in step with fills, and in the ring's order.
        auto skip = [&](int upto) {
#pragma unroll 1
          for (; ok && kt < upto; ++kt, ++vt) {
#pragma unroll
            for (int value = 0; value < 2; ++value) {
              ok = bar_wait<SPIN>(&kvfull[slot[value]], sph[value]) && ok;
              if (one) mbar_arrive(&kvempty[slot[value]]);
              if (value && mend_values(vt, tail, lead)) fph ^= 1u << slot[1];
              next_slot(value);
            }
            ok = __all_sync(0xffffffffu, ok);
          }
        };
        skip(b0 < b1 ? b0 >> 1 : jhi);
        if (b0 < b1) {
          ok = bar_wait<SPIN>(&qfull[i], qph) && ok;
          qph ^= 1u;
        }
        // Scores run a block ahead of weights times values: turn b has the scores of block b and the values of the one
        // before.
#pragma unroll 1
        for (int b = b0; b < b1 + step && b0 < b1; b += step) {
          if (b < b1) {
            const uint32_t s = slot[0], buf = blocks & 1u;
            ok = bar_wait<SPIN>(&kvfull[s], sph[0]) && ok;
            tc_fence_after();
            const uint64_t kd = kd0 + (uint64_t)(s * (C::kSlot >> 4) + (b & 1) * (kBlock * 128 >> 4));
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              if (one)
                tc_mma_f16(tm + kBlock * buf, qd + (uint64_t)(((k >> 2) * (kTileRows * 128) + (k & 3) * 32) >> 4),
                           kd + (uint64_t)(((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4), kIdS, k > 0);
              __syncwarp();
            }
            if (one) tc_commit(&sfull[2 * i + buf]);
            if (b + step >= b1 && one) tc_commit(&qempty[i]);
            if (b + step >= b1 || (b + step) >> 1 != b >> 1) {  // the tile's last scores
              if (one) tc_commit(&kvempty[s]);
              next_slot(0);
              ++kt;
            }
            __syncwarp();
          }
          if (b > b0) {
            const int pb = b - step;
            const uint32_t s = slot[1], g = blocks - 1, buf = g & 1u;
            ok = bar_wait<SPIN>(&kvfull[s], sph[1]) && ok;
            if (!C::kQuant && mend_values(vt, tail, lead)) ok = bar_wait<SPIN>(&vfix[s], fph >> s & 1u) && ok;
            // keys past the length take no part: whole steps of 16 are left out
            const int steps = (min(kBlock, keys - pb * kBlock) + 15) >> 4;
            const uint64_t vd = vd0 + (uint64_t)(s * (C::kSlot >> 4) + (pb & 1) * (kBlock * 128 >> 4));
            const uint32_t pd = tm + kBlock * buf;
            const bool held = pb > b0;
            ok = bar_wait<SPIN>(&pfull[2 * i + buf], g >> 1 & 1u) && ok;
            tc_fence_after();
            if (steps == 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (one) tc_mma_f16_ta(tm + 256, pd + 8 * k, vd + (uint64_t)(k * (2048 >> 4)), kIdO, held || k > 0);
                __syncwarp();
              }
            } else {
#pragma unroll 1
              for (int k = 0; k < steps; ++k) {
                if (one) tc_mma_f16_ta(tm + 256, pd + 8 * k, vd + (uint64_t)(k * (2048 >> 4)), kIdO, held || k > 0);
                __syncwarp();
              }
            }
            if (one) tc_commit(&pvdone[i]);
            if (b >= b1 || b >> 1 != pb >> 1) {  // the tile's last values
              if (one) tc_commit(&kvempty[s]);
              if (mend_values(vt, tail, lead)) fph ^= 1u << s;
              next_slot(1);
              ++vt;
            }
            __syncwarp();
          }
          ++blocks;
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (b0 < b1) {
          --blocks;  // the last turn had values only
          if (one) tc_commit(&ofull[i]);
          __syncwarp();
        }
        skip(jhi);
      }
      if (!ok) {
        // what was issued must be done before the CTA's memory goes
        if (one) tc_commit(&mdrain[i]);
        __syncwarp();
        bar_wait<SPIN>(&mdrain[i], 0u);
      }
      tc_fence_before();
    } else if (warp == 9) {
      // ---------------- items, and copies of keys and values ----------------
      constexpr int NR = C::kQuant ? C::kRaws : NS;
      uint64_t* full = C::kQuant ? rawfull : kvfull;
      uint64_t* empty = C::kQuant ? rawempty : kvempty;
      bool ok = true, more = true;
      uint32_t n = 0, asks = 0;
      int64_t filled = 0;
      int idx = (int)blockIdx.x;
      int page_rows = kKeys;  // keys of one copy
      if constexpr (SRC != kPacked) page_rows = min(kKeys, 1 << a.cache.page_shift);
      if (!C::kQuant && lane == 0) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
      }
      while (ok && more) {
        Item it;
        const bool valid = find_item<SRC>(a, lane, idx, &it);
        if (valid) {
          ok = bar_wait(&iempty[n & 1], ((n >> 1) & 1u) ^ 1u);
          if (!ok) break;
          if (lane == 0) {
            items[n & 1] = it;
            mbar_arrive(&ifull[n & 1]);
          }
          __syncwarp();
          ++n;
#ifdef EXL3_ATTN_SHARED
          // Cache rows of the next two tiles' copies: their page ids come, and for codes their bytes are on the way into L2
          // (the ring of codes holds two tiles' sides), while the tile before them is copied.
          int64_t ahead[2] = {-1, -1};
#pragma unroll 1
          for (int j = it.jlo - 2; ok && j < it.jhi; ++j) {
            const int64_t here = ahead[0];
            ahead[0] = ahead[1];
            ahead[1] = -1;  // no page of the cache
            const int key = it.base + (j + 2) * kKeys + lane * page_rows;
            if (j + 2 < it.jhi && lane * page_rows < kKeys && key < it.kv_len) {
              const int id = a.table[(int64_t)it.b * a.table_width + (key >> a.cache.page_shift)];
              if (id >= 0 && id < a.cache.num_pages) {
                const int64_t row = (((int64_t)id * a.kv_heads + it.kvh) << a.cache.page_shift) + (key & ((1 << a.cache.page_shift) - 1));
                ahead[1] = row;
                if constexpr (C::kQuant) {
                  prefetch_l2(a.cache.k + row * C::kRowBytes, (uint32_t)(page_rows * C::kRowBytes));
                  prefetch_l2(a.cache.v + row * C::kRowBytes, (uint32_t)(page_rows * C::kRowBytes));
                  prefetch_l2(a.cache.k_scale + row, (uint32_t)(page_rows * 2));
                  prefetch_l2(a.cache.v_scale + row, (uint32_t)(page_rows * 2));
                }
              }
            }
            if (j < it.jlo) continue;
            const int t = it.base + j * kKeys;
            const int copies = (min(kKeys, it.kv_len - t) + page_rows - 1) / page_rows;
            bool page_ok = true;
            int64_t row = here;  // cache row of this lane's copy
            if (lane < copies) {
              page_ok = here >= 0;
              if (!page_ok) row = C::kQuant ? 0 : (a.cache.num_pages * a.kv_heads) << a.cache.page_shift;
            }
#else
          for (int j = it.jlo; ok && j < it.jhi; ++j) {
            const int t = it.base + j * kKeys;
            int64_t row = 0;  // cache row of this lane's copy (paged)
            int copies = 1;
            bool page_ok = true;
            if constexpr (SRC != kPacked) {
              copies = (min(kKeys, it.kv_len - t) + page_rows - 1) / page_rows;
              if (lane < copies) {
                const int key = t + lane * page_rows;
                const int id = a.table[(int64_t)it.b * a.table_width + (key >> a.cache.page_shift)];
                page_ok = id >= 0 && id < a.cache.num_pages;
                // an id outside the cache: past the map's last row, which reads as zeros (16 bits); page 0's codes
                // with scales of zero
                row = page_ok ? (((int64_t)id * a.kv_heads + it.kvh) << a.cache.page_shift) +
                                    (key & ((1 << a.cache.page_shift) - 1))
                              : C::kQuant ? 0 : (a.cache.num_pages * a.kv_heads) << a.cache.page_shift;
              }
            }
#endif
#pragma unroll
            for (int value = 0; value < 2; ++value) {
              if (!ok) break;
              const int s = (int)(filled % NR);
              const uint32_t ph = (uint32_t)(filled / NR) & 1u;
              ok = bar_wait(&empty[s], ph ^ 1u);
              if (!ok) break;
              ++filled;
              if constexpr (!C::kQuant) {
                uint8_t* dst = data + C::kRing + s * C::kSlot;
                const CUtensorMap* map = value ? &maps.v : &maps.k;
                if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(copies * page_rows * D * 2));
                __syncwarp();
                if (lane < copies) {
#pragma unroll
                  for (int h = 0; h < D / 64; ++h) {
                    if constexpr (SRC == kPacked)
                      tma_tile3d_g2s(dst + h * (kKeys * 128), map, 64 * h, it.kvh, (int)(it.q0 + t), &full[s]);
                    else
                      tma_tile3d_g2s(dst + h * (kKeys * 128) + lane * page_rows * 128, map, 64 * h, 0, (int)row, &full[s]);
                  }
                }
                __syncwarp();
                if (value && mend_values(j, it.tail, it.lead)) {
                  ok = bar_wait(&full[s], ph);
                  if (!ok) break;
                  auto zeros = [&](int from, int to) {
                    for (int x = lane; x < (to - from) * (D / 8); x += 32)
                      sts128(smem_u32(dst) + row_chunk(from + x / (D / 8), x % (D / 8)), 0u, 0u, 0u, 0u);
                  };
                  // from the length to the next multiple of 16 keys of the tile (the products' step); and from the block
                  // that the first key lies in to it
                  const int keys = it.kv_len - t;
                  if (j == it.tail) zeros(keys, (keys + 15) & ~15);
                  if (j == 0) zeros(it.lead & ~(kBlock - 1), it.lead);
                  fence_proxy_async_smem();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&vfix[s]);
                }
              } else {
                uint8_t* dst = data + C::kRawRing + s * C::kRaw;
                const int bad = __popc(__ballot_sync(0xffffffffu, !page_ok));
                if (bad > 0) {
                  if (!page_ok) {
                    for (int x = 0; x < page_rows * 2; x += 16)
                      sts128(smem_u32(dst + C::kCodes + lane * page_rows * 2 + x), 0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                  }
                  __syncwarp();
                }
                if (lane == 0)
                  mbar_arrive_expect_tx(&full[s], (uint32_t)(copies * page_rows * (C::kRowBytes + 2) - bad * page_rows * 2));
                __syncwarp();
                if (lane < copies) {
                  tma_bulk_g2s(dst + lane * page_rows * C::kRowBytes, (value ? a.cache.v : a.cache.k) + row * C::kRowBytes,
                               (uint32_t)(page_rows * C::kRowBytes), &full[s]);
                  if (page_ok)
                    tma_bulk_g2s(dst + C::kCodes + lane * page_rows * 2, (value ? a.cache.v_scale : a.cache.k_scale) + row,
                                 (uint32_t)(page_rows * 2), &full[s]);
                }
                __syncwarp();
              }
            }
          }
        }
        if (!ok) break;
        // the next item: a CTA that has not started yet
        if (lane == 0) {
          fence_proxy_async_smem();  // the last answer has been read before this one is written
          mbar_arrive_expect_tx(clc, 16u);
          cancel_cta(smem_u32(answer), clc);
        }
        __syncwarp();
        ok = bar_wait(clc, asks & 1u);
        ++asks;
        if (!ok) break;
        idx = cancelled_cta(smem_u32(answer));
        __syncwarp();
        more = idx >= 0;
      }
      // no item left (after a wait that gave up, the readers' own waits give up)
      if (ok && bar_wait(&iempty[n & 1], ((n >> 1) & 1u) ^ 1u)) {
        if (lane == 0) {
          items[n & 1].done = 1;
          mbar_arrive(&ifull[n & 1]);
        }
        __syncwarp();
      }
      drain_ring(full, NR, filled);
    } else if (warp == 11) {
      // ---------------- copies of q ----------------
      uint64_t* landed = C::kQuant ? qraw : qfull;
      const uint32_t bytes = (uint32_t)(a.tile_tokens * group * D * 2);
      if (lane == 0) prefetch_tensormap(&maps.q);
      bool ok = true;
      Item it;
      uint32_t n = 0, eph = 3u, jph = 0, filled[2] = {0u, 0u};  // eph: phases of qempty (a bit a half); nothing to wait for at first
      bool joint = false;                                       // the item before: its halves met in q's room
      while (ok && read_item(n, &it)) {
        ++n;
        if (joint) {
          ok = bar_wait(jfree, jph);
          jph ^= 1u;
        }
        joint = merges(it);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ok || it.span[i].b0 >= it.span[i].b1) continue;
          ok = bar_wait(&qempty[i], eph >> i & 1u);
          eph ^= 1u << i;
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&landed[i], bytes);
            const int tok = (int)it.q0 + it.tok0 + (it.joint ? 0 : i * a.tile_tokens);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_tile3d_g2s(data + C::kQ + i * (kTileRows * D * 2) + h * (kTileRows * 128), &maps.q, 64 * h, it.kvh * group, tok,
                             &landed[i]);
          }
          ++filled[i];
          __syncwarp();
        }
      }
      for (int i = 0; i < 2; ++i) drain_ring(&landed[i], 1, filled[i]);
    }
  } else if constexpr (C::kQuant) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kConvertRegs));
    // ---------------- codes to fp16 rows ----------------
    constexpr int LPR = C::kRowBytes / 16;  // lanes of a row
    constexpr int RPP = 32 / LPR;           // rows a warp takes at a time
    constexpr int NP = 32 / RPP;            // passes over the warp's 32 rows
    // passes whose codes are read at a time
    constexpr int AHEAD = kShared && SRC == kPaged4 ? 2 : NP < 4 ? NP : 4;
    const int lw = warp - 12, sub = lane % LPR;
    bool ok = true;
    Item it;
    uint32_t n = 0, raw = 0, filled = 0;
    static_assert(kUnitKeys == 16, "a warp's 32 rows are two groups");
    while (ok && read_item(n, &it)) {
      int ek[2] = {};  // units of this warp's two groups of the tile's keys
      for (int x = 0; ok && x < 2 * (it.jhi - it.jlo); ++x, ++raw, ++filled) {
        const uint32_t rs = raw % C::kRaws, s = filled % NS;
        ok = bar_wait(&rawfull[rs], raw / C::kRaws & 1u);
        if (!ok) break;
        const int at = (it.jlo + (x >> 1)) * kKeys + 32 * lw + lane;  // row 32 lw + lane of the tile, from the item's first key
        const uint32_t src = smem_u32(data + C::kRawRing) + rs * C::kRaw;
        const uint32_t dst = smem_u32(data + C::kRing) + s * C::kSlot;
        uint32_t ww[AHEAD][4];
        auto load = [&](int p) {
#pragma unroll
          for (int y = 0; y < AHEAD; ++y)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(ww[y][0]), "=r"(ww[y][1]), "=r"(ww[y][2]), "=r"(ww[y][3])
                         : "r"(src + (32 * lw + (p + y) * RPP + lane / LPR) * C::kRowBytes + 16 * sub)
                         : "memory");
        };
        // that row's scale in units of its group's, from the group's largest scale; 0 past the length and before the first
        // key that the item sees, which makes zeros of any codes
        uint16_t s16;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s16) : "r"(src + C::kCodes + 2 * (32 * lw + lane)) : "memory");
        load(0);
        uint32_t scale = at < it.kv_len - it.base && at >= it.lead ? (uint32_t)s16 << 16 : 0u;
        // A row of zeros has the scale 1, which would set the unit although nothing is in it: taken as 0.
        if (__any_sync(0xffffffffu, scale == 0x3F800000u)) {
          constexpr uint32_t kZero = SRC == kPaged8 ? 0x80808080u : 0x88888888u;
          uint32_t codes = scale == 0x3F800000u ? 0u : 1u;
#pragma unroll 1
          for (int y = 0; y < LPR; ++y) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(src + (32 * lw + lane) * C::kRowBytes + 16 * y)
                         : "memory");
            codes |= (w[0] ^ kZero) | (w[1] ^ kZero) | (w[2] ^ kZero) | (w[3] ^ kZero);
          }
          if (codes == 0u) scale = 0u;
        }
        const uint32_t mag = (scale & 0x7FFFFFFFu) < 0x7F800000u ? scale & 0x7FFFFFFFu : 0u;  // a NaN row does not count
        int e[2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
          e[y] = max((int)(__reduce_max_sync(0xffffffffu, lane >> 4 == y ? mag : 0u) >> 23) - 127 - kScaleTop, kLeastUnit);
        const float sf = __uint_as_float(scale) * power(127 - (lane >> 4 ? e[1] : e[0]));
        const uint32_t mine = pack2<false>(sf, sf);
        ok = bar_wait(&kvempty[s], (filled / NS & 1u) ^ 1u);
        if (!ok) break;
        if (!(x & 1)) {
          ek[0] = e[0], ek[1] = e[1];
        } else if (lane == 0) {
          units[s >> 1].k[2 * lw] = ek[0], units[s >> 1].k[2 * lw + 1] = ek[1];
          units[s >> 1].v[2 * lw] = e[0], units[s >> 1].v[2 * lw + 1] = e[1];
        }
        // behind shared prefixes as a loop: items that run once have to fetch its instructions first, and the softmax's share
        // their cache (4 bits: 7 chunks over 16000 keys 486 us instead of 490; 8 bits: 39 sequences 67.4 instead of 69.7)
        constexpr int STEP = kShared ? AHEAD : NP;
#pragma unroll 1
        for (int p0 = 0; p0 < NP; p0 += STEP)
#pragma unroll
        for (int pp = 0; pp < STEP; ++pp) {
          const int p = p0 + pp, rr = 32 * lw + p * RPP + lane / LPR;
          if (p > 0 && pp % AHEAD == 0) load(p);
          const uint32_t(&w4)[4] = ww[pp % AHEAD];
          const uint32_t sh = __shfl_sync(0xffffffffu, mine, rr & 31);
          if constexpr (SRC == kPaged8) {
            uint32_t h[8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              h[2 * y] = hmul2(hsub2(__byte_perm(w4[y], 0x64646464u, 0x4140), 0x64806480u), sh);
              h[2 * y + 1] = hmul2(hsub2(__byte_perm(w4[y], 0x64646464u, 0x4342), 0x64806480u), sh);
            }
            sts128(dst + row_chunk(rr, 2 * sub), h[0], h[1], h[2], h[3]);
            sts128(dst + row_chunk(rr, 2 * sub + 1), h[4], h[5], h[6], h[7]);
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t h[4];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const uint32_t w = w4[y] >> (8 * z);
                h[2 * z] = hmul2(hsub2((w & 0x000F000Fu) | 0x64006400u, 0x64086408u), sh);
                h[2 * z + 1] = hmul2(hfma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u), sh);
              }
              sts128(dst + row_chunk(rr, 4 * sub + y), h[0], h[1], h[2], h[3]);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&kvfull[s]);
          mbar_arrive(&rawempty[rs]);
        }
      }
      ++n;
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// Joins the parts of split key ranges (at most 16): a warp a row, parts in order,
// the loads of four parts ahead of their sums (512 tokens of 32 heads in seven
// parts: 3 us off the call, a load at a time took 20; eight or sixteen ahead gained less).
constexpr int kJoinParts = 4;
template <int D>
__global__ void __launch_bounds__(256) attn_tile_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t n = a.total_q * a.heads;
  if (row >= n) return;
  const int64_t tok = row / a.heads;
  // only the tokens of a sequence have parts
  bool mine = false;
  for (int b = lane; b < a.batch; b += 32) {
    const int64_t c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
    mine = mine || (tok >= c0 && tok < c1);
  }
  if (!__any_sync(0xffffffffu, mine)) return;
  // a lane a part: its maximum and sum, then its factor
  const float2 ml = lane < a.splits ? a.part_ml[lane * n + row] : make_float2(kNegInf, 0.0f);
  float top = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // a part without a maximum has a sum of 0, or NaN, and its output is not looked at
  const float factor = ml.x == kNegInf ? 0.0f : ex2(ml.x - top);
  const float part = ml.x == kNegInf ? ml.y : ml.y * factor;
  float l = 0.0f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.0f;
  for (int s0 = 0; s0 < a.splits; s0 += kJoinParts) {
    float v[kJoinParts][PER];
#pragma unroll
    for (int y = 0; y < kJoinParts; ++y) {
      const bool in = s0 + y < a.splits && __shfl_sync(0xffffffffu, ml.x, s0 + y) != kNegInf;
      const float* src = a.part_o + ((s0 + y) * n + row) * D + PER * lane;
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        const float2 w = in ? *reinterpret_cast<const float2*>(src + i) : make_float2(0.0f, 0.0f);
        v[y][i] = w.x, v[y][i + 1] = w.y;
      }
    }
#pragma unroll
    for (int y = 0; y < kJoinParts; ++y) {
      const float f = __shfl_sync(0xffffffffu, factor, s0 + y);
      l += __shfl_sync(0xffffffffu, part, s0 + y);
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = fmaf(v[y][i], f, o[i]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + tok * a.out_token_stride +
                  (row - tok * a.heads) * a.out_head_stride + PER * lane;
#pragma unroll
  for (int i = 0; i < PER; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        a.bf16 ? pack2<true>(o[i] * inv, o[i + 1] * inv) : pack2<false>(o[i] * inv, o[i + 1] * inv);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Rows of D 16-bit values as 3-D {D, heads, tokens}; a copy takes 64 columns of box_tokens tokens of box_heads heads.
cudaError_t make_map(CUtensorMap* map, const void* data, int d, int64_t heads, int64_t tokens, int64_t head_stride,
                     int64_t token_stride, int box_heads, int box_tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(data), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int SRC, bool BF16>
cudaError_t launch_tile(const AttnArgs& a, cudaStream_t stream, bool own = true) {
  using C = TileCfg<D, SRC>;
  TileMaps maps = {};
  const int group = a.heads / a.kv_heads;
  cudaError_t e = make_map(&maps.q, a.q.data, D, a.heads, a.total_q, a.q.head_stride, a.q.token_stride, group, a.tile_tokens);
  if (e != cudaSuccess) return e;
  if constexpr (SRC == kPacked) {
    e = make_map(&maps.k, a.k.data, D, a.kv_heads, a.total_q, a.k.head_stride, a.k.token_stride, 1, kKeys);
    if (e == cudaSuccess) e = make_map(&maps.v, a.v.data, D, a.kv_heads, a.total_q, a.v.head_stride, a.v.token_stride, 1, kKeys);
  } else if constexpr (SRC == kPaged16) {
    const int64_t rows = (a.cache.num_pages * a.kv_heads) << a.cache.page_shift;
    const int box = a.cache.page_shift < 7 ? 1 << a.cache.page_shift : kKeys;
    e = make_map(&maps.k, a.cache.k, D, 1, rows, D, D, 1, box);
    if (e == cudaSuccess) e = make_map(&maps.v, a.cache.v, D, 1, rows, D, D, 1, box);
  }
  if (e != cudaSuccess) return e;
  // the register split waits for registers that a launch with fewer would never have
  e = allow_smem<attn_tile_kernel<D, SRC, BF16>>(C::kSmem, C::kLaunchRegs);
  if (e != cudaSuccess) return e;
  if constexpr (kShared) {
    const int64_t tiles = shared_tiles(a.total_q, a.batch, 2 * a.tile_tokens);
    const int64_t blocks = a.prefix_ctas + (own ? tiles * a.splits * a.kv_heads : 0);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1u, 1u);
    cfg.blockDim = dim3(C::kThreads, 1u, 1u);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tile_kernel<D, SRC, BF16>, maps, a);
  } else {
    // items: no more than all tokens' and one partly filled for each sequence
    const int64_t tiles = a.total_q / (2 * a.tile_tokens) + (a.total_q < a.batch ? a.total_q : a.batch);
    const int64_t blocks = tiles * a.kv_heads * a.splits;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    attn_tile_kernel<D, SRC, BF16><<<(unsigned)blocks, C::kThreads, C::kSmem, stream>>>(maps, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.splits == 1) return e;
    attn_tile_join_kernel<D><<<(unsigned)((a.total_q * a.heads + 7) / 8), 256, 0, stream>>>(a);
    return cudaGetLastError();
  }
}

template <int D>
cudaError_t launch_tile_d(const AttnArgs& a, bool paged, cudaStream_t stream, bool own = true) {
  if constexpr (!kShared) {
    if (!paged) return a.bf16 ? launch_tile<D, kPacked, true>(a, stream) : launch_tile<D, kPacked, false>(a, stream);
  }
  switch (a.cache.format) {
    case kKvF16: return launch_tile<D, kPaged16, false>(a, stream, own);
    case kKvBf16: return launch_tile<D, kPaged16, true>(a, stream, own);
    case kKvInt8: return launch_tile<D, kPaged8, false>(a, stream, own);
    default: return launch_tile<D, kPaged4, false>(a, stream, own);
  }
}

}  // namespace

#ifdef EXL3_ATTN_SHARED
cudaError_t launch_attn_tile_shared(const AttnArgs& a, bool own, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_tile_d<64>(a, true, stream, own) : launch_tile_d<128>(a, true, stream, own);
}

cudaError_t take_device_error_attn_shared(uint32_t* flags) { return take_tu_device_error(flags); }
#else
cudaError_t launch_attn_tile(const AttnArgs& a, bool paged, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_tile_d<64>(a, paged, stream) : launch_tile_d<128>(a, paged, stream);
}

cudaError_t take_device_error_attn(uint32_t* flags) { return take_tu_device_error(flags); }
#endif

}  // namespace exl3
