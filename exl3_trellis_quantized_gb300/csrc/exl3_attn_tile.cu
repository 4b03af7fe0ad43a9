// exl3_attn_tile.cu -- causal attention of many query rows: whole prompts over
// packed keys and values, and chunks of new tokens over the paged cache.
//
// Rows.  The query heads of a group share their keys, so the rows of a sequence
// and key head are its query tokens times the group's heads, token major: one
// CTA takes 256 of them (two tiles of 128, the M of the MMA) whatever the group
// size, and reads each key and value once for all of them.
//
// Per tile of 128 keys and 128 rows:
//     S = Q K^T            tcgen05.mma, both operands in shared memory, S in tensor memory
//     m' = max(m, S c),  P = 2^(S c - m'),  l += sum P    (c = scale * log2 e; one thread a row)
//     O += P V             tcgen05.mma, P from tensor memory (written over S), V from shared memory
// The running maximum is only raised when it has grown by more than 8 (log2):
// until then P stays below 2^8, l and O are held relative to the old maximum
// in fp32, and O in tensor memory needs no rescaling.  P rounds to the operand
// type; l sums the unrounded values in fp32.
//
// What bounds it: the tensor core (4 * 128 * 128 * D operations a tile) once there
// are a few hundred rows a sequence.  The two row tiles take turns: while one's
// softmax runs the tensor core works for the other.  A CTA with no more than 128
// rows gives both halves the same rows and every other key tile each, and joins
// them at the end.  With few row tiles the keys are also split over CTAs, and
// attn_tile_join_kernel joins the parts.
//
// Roles: warps 0-3 and 4-7 softmax of row tiles 0 and 1 (a thread a row), warp 8
// issues the MMAs, warp 9 issues the tensor copies of keys and values into a
// ring of slots; for the quantised cache formats warps 12-15 load the codes and
// write them as fp16 rows into the same ring.  Quantised rows stay in the
// rotated basis (see exl3_rope_cache.cu): q is rotated on its way into shared
// memory and the output on its way out, each a transform within a thread.
//
// Tensor memory: S of both tiles at columns 0 and 128, O at 256 and 384.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "exl3_attn.h"
#include "exl3_sm100.cuh"

namespace exl3 {
namespace {

enum Source { kPacked = 0, kPaged16 = 1, kPaged8 = 2, kPaged4 = 3 };
constexpr int kKeys = 128;      // keys of a tile
constexpr int kTileRows = 128;  // rows of a tile; a CTA has two tiles
constexpr int kItemRows = 2 * kTileRows;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kSlack = 8.0f;

template <int D, int SRC>
struct TileCfg {
  static constexpr bool kQuant = SRC >= kPaged8;
  static constexpr int kLoaders = kQuant ? 4 : 1;
  static constexpr int kFirstLoader = kQuant ? 12 : 9;
  static constexpr int kThreads = kQuant ? 512 : 384;  // whole groups of four warps, for the register split
  // Registers a thread of each group of four warps.  The kernel is launched with 168 (384 threads) or 128 (512); what
  // the softmax warps gain is what the others give up.
  static constexpr int kLaunchRegs = kQuant ? 128 : 168;
  static constexpr int kSoftmaxRegs = kQuant ? 192 : 208;
  static constexpr int kIssueRegs = kQuant ? 40 : 88;
  static constexpr int kLoaderRegs = 88;
  static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs + (kQuant ? 128 * kLoaderRegs : 0) <= kLaunchRegs * kThreads,
                "the split draws on the registers of the launch");
  static constexpr int kSlot = kKeys * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileRows * D * 2;
  static constexpr int kCtrl = 1024;
  static constexpr int kSmem = 1024 + kCtrl + kRing + kSlots * kSlot;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kSmem > 114 * 1024, "one CTA an SM: each allocates all of tensor memory");
  static_assert(kSlots * kSlot >= kTileRows * D * 4 + kTileRows * 8, "the ring holds a tile's output for the join");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  CUtensorMap k, v;
};

// What one CTA works on.
struct Item {
  int64_t q0;        // first packed query token of the sequence
  int kvh, first;    // key head; position of the sequence's first query token
  int row0, rows;    // rows of the item within the sequence and head
  int kv_len;
  int base;          // first key of key tile 0
  int j0, j1;        // key tiles of this CTA
  bool joint;        // both halves on the same rows, key tiles in turn
  int b, split;
};

struct Span {  // key tiles of one half: j0, j0 + step, ... below j1 (j1 <= j0: none)
  int j0, j1, step;
  __device__ __forceinline__ bool has(int j) const { return j >= j0 && j < j1 && (step == 1 || ((j - j0) & 1) == 0); }
};

template <int SRC>
__device__ bool find_item(const AttnArgs& a, int lane, Item* it) {
  const int group = a.heads / a.kv_heads;
  int64_t idx = blockIdx.x;
  it->split = (int)(idx % a.splits);
  idx /= a.splits;
  it->kvh = (int)(idx % a.kv_heads);
  int64_t tile = idx / a.kv_heads;
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
    const int64_t tiles = (n * group + kItemRows - 1) / kItemRows;
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
      const int64_t count = __shfl_sync(0xffffffffu, tiles, at);
      const int q_len = (int)__shfl_sync(0xffffffffu, n, at);
      it->q0 = __shfl_sync(0xffffffffu, c0, at);
      it->b = b0 + at;
      // a sequence's last row tiles see the most keys and go first
      const int64_t t = count - 1 - (tile - before);
      it->row0 = (int)(t * kItemRows);
      const int64_t left = (int64_t)q_len * group - it->row0;
      it->rows = left < kItemRows ? (int)left : kItemRows;
      it->kv_len = q_len;
      if constexpr (SRC != kPacked) {
        const int64_t room = (int64_t)a.table_width << a.cache.page_shift;
        const int64_t kl = a.kv_lens[it->b];
        it->kv_len = (int)(kl < 0 ? 0 : kl > room ? room : kl);
      }
      it->first = it->kv_len - q_len;
      it->joint = it->rows <= kTileRows;
      // keys that the item's first row sees first, and that its last row sees last
      const int p0 = it->first + it->row0 / group, p1 = it->first + (it->row0 + it->rows - 1) / group;
      int lo = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
      if constexpr (SRC != kPacked) {
        // whole pages (or 128 keys of a larger one), so that a page is never cut by a tile's first key
        const int align = a.cache.page_shift < 7 ? 1 << a.cache.page_shift : kKeys;
        lo &= ~(align - 1);
      }
      it->base = lo;
      const int tiles_k = p1 >= lo ? (p1 - lo) / kKeys + 1 : 0;
      it->j0 = (int)((int64_t)tiles_k * it->split / a.splits);
      it->j1 = (int)((int64_t)tiles_k * (it->split + 1) / a.splits);
      return true;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

// Key tiles of half i of the item.
__device__ Span half_span(const AttnArgs& a, const Item& it, int i) {
  if (it.joint) return Span{min(it.j0 + i, it.j1), it.j1, 2};
  const int group = a.heads / a.kv_heads;
  const int r0 = it.row0 + i * kTileRows;
  const int r1 = min(r0 + kTileRows, it.row0 + it.rows) - 1;
  const int p0 = it.first + r0 / group, p1 = it.first + r1 / group;
  const int lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
  if (r1 < r0 || p1 < lo) return Span{it.j0, it.j0, 1};
  const int s0 = max(it.j0, (lo - it.base) / kKeys), s1 = min(it.j1, (p1 - it.base) / kKeys + 1);
  return s0 < s1 ? Span{s0, s1, 1} : Span{it.j0, it.j0, 1};
}

// D: head size.  BF16: operand type (fp16 for the quantised formats).
template <int D, int SRC, bool BF16>
__global__ void __launch_bounds__(TileCfg<D, SRC>::kThreads, 1)
    attn_tile_kernel(const __grid_constant__ TileMaps maps, const __grid_constant__ AttnArgs a) {
  using C = TileCfg<D, SRC>;
  constexpr int NS = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* kvfull = reinterpret_cast<uint64_t*>(base);  // slot filled
  uint64_t* kvempty = kvfull + NS;                       // slot read by the MMAs
  uint64_t* qfull = kvempty + NS;                        // [2] a row tile's q in shared memory
  uint64_t* sfull = qfull + 2;                           // [2] scores in tensor memory
  uint64_t* pfull = sfull + 2;                           // [2] weights in tensor memory, O rescaled
  uint64_t* ofull = pfull + 2;                           // [2] every MMA of a tile done
  uint64_t* vfix = ofull + 2;                            // the last value slot's rows past the length are zeros
  uint64_t* mdrain = vfix + 1;                           // MMAs issued before a wait gave up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 1);
  uint8_t* data = base + C::kCtrl;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (SRC != kPacked) pdl_launch_dependents();  // the join may be scheduled; it waits for this grid
  Item it;
  if (!find_item<SRC>(a, lane, &it)) return;  // the whole block: past the last row tile
  const int group = a.heads / a.kv_heads;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kvfull[s], C::kQuant ? C::kLoaders : 1);
      mbar_init(&kvempty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 4);
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
      mbar_init(&ofull[i], 1);
    }
    mbar_init(vfix, 1);
    mbar_init(mdrain, 1);
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
  const Span sp0 = half_span(a, it, 0), sp1 = half_span(a, it, 1);
  // the tiles that a half uses; the spans of two non-empty halves overlap or touch
  const bool use0 = sp0.j0 < sp0.j1, use1 = sp1.j0 < sp1.j1;
  const int jlo = use0 && use1 ? min(sp0.j0, sp1.j0) : use0 ? sp0.j0 : use1 ? sp1.j0 : 0;
  const int jhi = use0 && use1 ? max(sp0.j1, sp1.j1) : use0 ? sp0.j1 : use1 ? sp1.j1 : 0;
  // the length ends inside key tile `tail`: its value rows past the end must be zeros (a weight of zero times what a
  // page or the next sequence holds there need not be zero)
  const int tail = (it.kv_len - it.base) % kKeys != 0 ? (it.kv_len - it.base) / kKeys : -1;
  const bool fix = !C::kQuant && tail >= jlo && tail < jhi && (it.kv_len & 15) != ((it.base & 15));

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ---------------- softmax: a thread a row ----------------
    const int i = warp >> 2;
    const Span sp = i ? sp1 : sp0;
    const int r = 32 * (warp & 3) + lane;  // row of the tile, lane of tensor memory
    const int row = (it.joint ? 0 : i * kTileRows) + r;
    const bool there = row < it.rows;
    const int tok = (it.row0 + (there ? row : it.rows - 1)) / group;
    const int head = it.kvh * group + (it.row0 + (there ? row : it.rows - 1)) - tok * group;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + 128 * i;
    const uint32_t o_col = tmem + lanes + 256 + 128 * i;
    bool ok = true;

    {  // q into shared memory
      const uint16_t* src =
          static_cast<const uint16_t*>(a.q.data) + (it.q0 + tok) * a.q.token_stride + (int64_t)head * a.q.head_stride;
      const uint32_t dst = smem_u32(data + C::kQ) + (uint32_t)i * (kTileRows * D * 2);
      if constexpr (!C::kQuant) {
        uint4 w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = there ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) sts128(dst + row_chunk(r, c), w[c].x, w[c].y, w[c].z, w[c].w);
      } else {
        float v[D];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = there ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (a.bf16) {
              v[8 * c + 2 * x] = __uint_as_float(ww[x] << 16);
              v[8 * c + 2 * x + 1] = __uint_as_float(ww[x] & 0xFFFF0000u);
            } else {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[x]));
              v[8 * c + 2 * x] = f.x;
              v[8 * c + 2 * x + 1] = f.y;
            }
          }
        }
        hadamard_row<D>(v);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = pack2<false>(v[column_value<SRC>(8 * c + 2 * x)] * (8.0f / D),
                                v[column_value<SRC>(8 * c + 2 * x + 1)] * (8.0f / D));
          sts128(dst + row_chunk(r, c), w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[i]);
    }

    const int pos = it.first + tok;
    const int lim = pos - it.base;                                             // last key it sees, from the item's first key
    const int low = a.window > 0 ? max(0, pos - a.window + 1) - it.base : 0;   // first
    const float c = a.scale_log2;
    float m = kNegInf;
    float2 l0 = make_float2(0.0f, 0.0f), l1 = make_float2(0.0f, 0.0f);
    uint32_t phase = 0;
    bool any = false;
    for (int j = sp.j0; ok && j < sp.j1; j += sp.step) {
      ok = mbar_wait(&sfull[i], phase);
      phase ^= 1u;
      if (!ok) break;
      tc_fence_after();
      float s[kKeys];
#pragma unroll
      for (int x = 0; x < kKeys; x += 32) tmem_ld_32x32b_x32(s_col + x, *reinterpret_cast<uint32_t(*)[32]>(&s[x]));
      tmem_ld_wait();
      const int k0 = j * kKeys;
      if (__any_sync(0xffffffffu, k0 + kKeys - 1 > lim || k0 < low)) {
        const int hi = lim - k0, lo = low - k0;
#pragma unroll
        for (int x = 0; x < kKeys; ++x)
          if (x > hi || x < lo) s[x] = kNegInf;
      }
      float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
      for (int x = 4; x < kKeys; x += 4) {
        t0 = fmaxf(t0, s[x]);
        t1 = fmaxf(t1, s[x + 1]);
        t2 = fmaxf(t2, s[x + 2]);
        t3 = fmaxf(t3, s[x + 3]);
      }
      const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * c;
      const bool up = top > m + kSlack;
      if (__any_sync(0xffffffffu, up)) {
        const float f = up ? ex2(m - top) : 1.0f;
        m = up ? top : m;
        l0.x *= f, l0.y *= f, l1.x *= f, l1.y *= f;
        if (any) {
          // the scores' barrier also stands for the previous tile's P V, so O is complete
#pragma unroll
          for (int x = 0; x < D; x += 32) {
            uint32_t w[32];
            tmem_ld_32x32b_x32(o_col + x, w);
            tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 32; ++y) w[y] = __float_as_uint(__uint_as_float(w[y]) * f);
            tmem_st_x32(o_col + x, w);
          }
        }
      }
      any = true;
      const float ref = m == kNegInf ? 0.0f : m;  // nothing seen yet: all scores are -inf, any finite reference does
      const float2 cc = make_float2(c, c), mm = make_float2(-ref, -ref);
#pragma unroll
      for (int x = 0; x < kKeys; x += 64) {
        uint32_t w[32];
#pragma unroll
        for (int y = 0; y < 32; y += 2) {
          float2 p = fma2(make_float2(s[x + 2 * y], s[x + 2 * y + 1]), cc, mm);
          float2 n = fma2(make_float2(s[x + 2 * y + 2], s[x + 2 * y + 3]), cc, mm);
          p.x = ex2(p.x), p.y = ex2(p.y), n.x = ex2(n.x), n.y = ex2(n.y);
          l0 = add2(l0, p);
          l1 = add2(l1, n);
          w[y] = pack2<BF16>(p.x, p.y);
          w[y + 1] = pack2<BF16>(n.x, n.y);
        }
        tmem_st_x32(s_col + x / 2, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[i]);
    }

    // ---- the row's output
    float l = (l0.x + l0.y) + (l1.x + l1.y);
    float o[D];
#pragma unroll
    for (int x = 0; x < D; ++x) o[x] = 0.0f;
    // in a joint item the other half's MMAs still read the ring that the join writes
    if (ok && jhi > jlo) {
      if (sp.j1 > sp.j0 || it.joint) ok = mbar_wait(&ofull[i], 0u);
      if (ok && it.joint) ok = mbar_wait(&ofull[i ^ 1], 0u);
    }
    if (ok && any) {
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < D; x += 32) tmem_ld_32x32b_x32(o_col + x, *reinterpret_cast<uint32_t(*)[32]>(&o[x]));
      tmem_ld_wait();
    }
    if (it.joint) {
      float* jo = reinterpret_cast<float*>(data + C::kRing);  // [D][128]: a thread a column, no bank conflicts
      float2* jml = reinterpret_cast<float2*>(jo + D * kTileRows);
      if (i == 1 && ok) {
#pragma unroll
        for (int x = 0; x < D; ++x) jo[x * kTileRows + r] = o[x];
        jml[r] = make_float2(m, l);
      }
      named_barrier(1, 256);  // both halves come here, also after a wait gave up
      if (i == 0 && ok) {
        const float2 other = jml[r];
        const float both = fmaxf(m, other.x);
        const float f0 = m == kNegInf ? 0.0f : ex2(m - both), f1 = other.x == kNegInf ? 0.0f : ex2(other.x - both);
        l = l * f0 + other.y * f1;
#pragma unroll
        for (int x = 0; x < D; ++x) o[x] = o[x] * f0 + jo[x * kTileRows + r] * f1;
        m = both;
      }
    }
    if (ok && there && !(it.joint && i == 1)) {
      const int64_t grow = (it.q0 + tok) * a.heads + head;
      if (a.splits > 1) {
        const int64_t prow = (int64_t)it.split * a.total_q * a.heads + grow;
        a.part_ml[prow] = make_float2(m, l);
        if (m != kNegInf) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + prow * D);
#pragma unroll
          for (int x = 0; x < D / 4; ++x) dst[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      } else {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that saw no key gives zeros
        uint16_t* dst = static_cast<uint16_t*>(a.out) + (it.q0 + tok) * a.out_token_stride + (int64_t)head * a.out_head_stride;
        if constexpr (C::kQuant) {
          float v[D];
#pragma unroll
          for (int x = 0; x < D; ++x) v[column_value<SRC>(x)] = o[x];
          hadamard_row<D>(v);
#pragma unroll
          for (int x = 0; x < D; ++x) o[x] = v[x] * (8.0f / D);
        }
#pragma unroll
        for (int x = 0; x < D; x += 8) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float p = o[x + 2 * y] * inv, n = o[x + 2 * y + 1] * inv;
            w[y] = (C::kQuant ? a.bf16 != 0 : BF16) ? pack2<true>(p, n) : pack2<false>(p, n);
          }
          *reinterpret_cast<uint4*>(dst + x) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    tc_fence_before();
  } else if (warp < 12) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
   if (warp == 8) {
    // ---------------- MMA issue ----------------
    constexpr uint32_t kIdS = idesc(BF16, 128, 128, false);
    constexpr uint32_t kIdO = idesc(BF16, 128, D, true);
    const uint32_t qaddr = smem_u32(data + C::kQ), ring = smem_u32(data + C::kRing);
    bool ok = true;
    int pend[2] = {-1, -1};     // key tile whose P V is due
    uint32_t pph[2] = {0u, 0u};
    bool started[2] = {false, false};
    const uint32_t one = elect_one();
    // slots are filled in the order K(jlo), V(jlo), K(jlo + 1), ...
    auto slot_of = [&](int j, int value) { return (2 * (j - jlo) + value) % NS; };
    auto phase_of = [&](int j, int value) { return (uint32_t)((2 * (j - jlo) + value) / NS) & 1u; };
    auto values = [&](int i) {  // P V of half i's pending tile
      const int j = pend[i];
      const int s = slot_of(j, 1);
      if (!mbar_wait(&kvfull[s], phase_of(j, 1))) return false;
      if (fix && j == tail && !mbar_wait(vfix, 0u)) return false;
      if (!mbar_wait(&pfull[i], pph[i])) return false;
      pph[i] ^= 1u;
      tc_fence_after();
      // keys past the length take no part: whole steps of 16 are left out
      const int keys = min(kKeys, it.kv_len - it.base - j * kKeys);
      const int steps = (keys + 15) >> 4;
      const uint64_t vd = sdesc_n_major(ring + (uint32_t)s * C::kSlot, kKeys * 128);
      for (int k = 0; k < steps; ++k) {
        if (one)
          tc_mma_f16_ta(tmem + 256 + 128 * i, tmem + 128 * i + 8 * k, vd + (uint64_t)(k * (2048 >> 4)), kIdO,
                        started[i] || k > 0);
      }
      started[i] = true;
      pend[i] = -1;
      const Span& other = i ? sp0 : sp1;
      // the slot is free once every half that uses it has read it; half 1 comes after half 0
      if (i == 1 || !other.has(j)) {
        if (one) tc_commit(&kvempty[s]);
      }
      return true;
    };
    for (int j = jlo; ok && j < jhi; ++j) {
      const int s = slot_of(j, 0);
      ok = mbar_wait(&kvfull[s], phase_of(j, 0));
      for (int i = 0; ok && i < 2; ++i) {
        const Span& sp = i ? sp1 : sp0;
        if (!sp.has(j)) {
          // past this half's last tile: its values go before the other half's release their slot
          if (pend[i] >= 0 && j >= sp.j1) ok = values(i);
          continue;
        }
        if (pend[i] >= 0) ok = values(i);
        else ok = mbar_wait(&qfull[i], 0u);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = sdesc_sw128(qaddr + (uint32_t)i * (kTileRows * D * 2));
        const uint64_t kd = sdesc_sw128(ring + (uint32_t)s * C::kSlot);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = (uint64_t)(((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4);
          if (one) tc_mma_f16(tmem + 128 * i, qd + off, kd + off, kIdS, k > 0);
        }
        if (one) tc_commit(&sfull[i]);
        pend[i] = j;
      }
      if (ok && one) tc_commit(&kvempty[s]);
    }
    for (int i = 0; ok && i < 2; ++i)
      if (pend[i] >= 0) ok = values(i);
    if (ok) {
      if (one) {
        tc_commit(&ofull[0]);
        tc_commit(&ofull[1]);
      }
    } else {
      // what was issued must be done before the CTA's memory goes
      if (one) tc_commit(mdrain);
      mbar_wait(mdrain, 0u);
    }
    tc_fence_before();
   } else if (!C::kQuant && warp == C::kFirstLoader) {
    // ---------------- tensor copies of keys and values ----------------
    bool ok = true;
    int64_t n = 0;
    int page_rows = kKeys;  // keys of one copy
    if constexpr (SRC == kPaged16) page_rows = min(kKeys, 1 << a.cache.page_shift);
    if (lane == 0) {
      prefetch_tensormap(&maps.k);
      prefetch_tensormap(&maps.v);
    }
    for (int j = jlo; ok && j < jhi; ++j) {
      const int t = it.base + j * kKeys;
      int64_t row = 0;  // cache row of this lane's copy (paged)
      int copies = 1;
      if constexpr (SRC == kPaged16) {
        copies = (min(kKeys, it.kv_len - t) + page_rows - 1) / page_rows;
        if (lane < copies) {
          const int key = t + lane * page_rows;
          const int id = a.table[(int64_t)it.b * a.table_width + (key >> a.cache.page_shift)];
          // an id outside the cache reads as zeros (past the map's last row)
          row = id >= 0 && id < a.cache.num_pages
                    ? (((int64_t)id * a.kv_heads + it.kvh) << a.cache.page_shift) + (key & ((1 << a.cache.page_shift) - 1))
                    : (a.cache.num_pages * a.kv_heads) << a.cache.page_shift;
        }
      }
      for (int value = 0; value < 2; ++value, ++n) {
        const int s = (int)(n % NS);
        ok = mbar_wait(&kvempty[s], ((uint32_t)(n / NS) & 1u) ^ 1u);
        if (!ok) break;
        uint8_t* dst = data + C::kRing + s * C::kSlot;
        const CUtensorMap* map = value ? &maps.v : &maps.k;
        if (lane == 0) mbar_arrive_expect_tx(&kvfull[s], (uint32_t)(copies * page_rows * D * 2));
        __syncwarp();
        if (lane < copies) {
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            if constexpr (SRC == kPacked)
              tma_tile3d_g2s(dst + h * (kKeys * 128), map, 64 * h, it.kvh, (int)(it.q0 + t), &kvfull[s]);
            else
              tma_tile3d_g2s(dst + h * (kKeys * 128) + lane * page_rows * 128, map, 64 * h, 0, (int)row, &kvfull[s]);
          }
        }
        __syncwarp();
        if (fix && value && j == tail) {
          // zeros from the length to the next multiple of 16 keys of the tile
          ok = mbar_wait(&kvfull[s], (uint32_t)(n / NS) & 1u);
          if (!ok) {
            ++n;
            break;
          }
          const int keys = it.kv_len - t, upto = (keys + 15) & ~15;
          const uint32_t d32 = smem_u32(dst);
          for (int x = lane; x < (upto - keys) * (D / 8); x += 32) {
            const int rr = keys + x / (D / 8), cc = x % (D / 8);
            sts128(d32 + row_chunk(rr, cc), 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(vfix);
        }
      }
    }
    drain_ring(kvfull, NS, n);
   }
  } else if constexpr (C::kQuant) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLoaderRegs));
    // ---------------- codes to fp16 rows ----------------
    constexpr int RB = SRC == kPaged8 ? D : D / 2;   // bytes of a cached row
    constexpr int LPR = RB / 16;                     // lanes of a row
    constexpr int RPP = 32 / LPR;                    // rows a warp loads at a time
    constexpr int NP = 32 / RPP;                     // such loads for the warp's 32 rows
    const int lw = warp - C::kFirstLoader;
    bool ok = true;
    int64_t n = 0;
    const int sub = lane % LPR;
    auto page_of = [&](int j) {  // page of the 16-key group lane & 7 of tile j
      const int key = it.base + j * kKeys + 16 * (lane & 7);
      int id = -1;
      if (j < jhi && key < it.kv_len) id = a.table[(int64_t)it.b * a.table_width + (key >> a.cache.page_shift)];
      return id < a.cache.num_pages ? id : -1;
    };
    uint4 code[NP];
    uint32_t scale[NP];  // both halves: the row's scale as fp16, 0 past the length
    auto fetch = [&](int j, int value, int pid) {
      const uint8_t* src = value ? a.cache.v : a.cache.k;
      const uint16_t* ss = value ? a.cache.v_scale : a.cache.k_scale;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int rr = 32 * lw + p * RPP + lane / LPR;
        const int id = __shfl_sync(0xffffffffu, pid, rr >> 4);
        const int key = it.base + j * kKeys + rr;
        code[p] = make_uint4(0u, 0u, 0u, 0u);
        scale[p] = 0u;
        if (id >= 0 && key < it.kv_len && j < jhi) {
          const int64_t row = (((int64_t)id * a.kv_heads + it.kvh) << a.cache.page_shift) + (key & ((1 << a.cache.page_shift) - 1));
          code[p] = __ldg(reinterpret_cast<const uint4*>(src + row * RB + 16 * sub));
          scale[p] = (uint32_t)__ldg(ss + row) << 16;
        }
      }
    };
    int pid = page_of(jlo), pid_next = page_of(jlo + 1);
    fetch(jlo, 0, pid);
    for (int j = jlo; ok && j < jhi; ++j) {
      for (int value = 0; value < 2; ++value, ++n) {
        const int s = (int)(n % NS);
        ok = mbar_wait(&kvempty[s], ((uint32_t)(n / NS) & 1u) ^ 1u);
        if (!ok) break;
        const uint32_t dst = smem_u32(data + C::kRing) + (uint32_t)s * C::kSlot;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int rr = 32 * lw + p * RPP + lane / LPR;
          const uint32_t ww[4] = {code[p].x, code[p].y, code[p].z, code[p].w};
          const bool none = scale[p] == 0u;  // past the length or no page: zeros
          const float sf = __uint_as_float(scale[p]);
          const uint32_t sh = pack2<false>(sf, sf);
          if constexpr (SRC == kPaged8) {
            uint32_t h[8];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              h[2 * x] = hmul2(hsub2(__byte_perm(ww[x], 0x64646464u, 0x4140), 0x64806480u), sh);
              h[2 * x + 1] = hmul2(hsub2(__byte_perm(ww[x], 0x64646464u, 0x4342), 0x64806480u), sh);
            }
            if (none) {
#pragma unroll
              for (int x = 0; x < 8; ++x) h[x] = 0u;
            }
            sts128(dst + row_chunk(rr, 2 * sub), h[0], h[1], h[2], h[3]);
            sts128(dst + row_chunk(rr, 2 * sub + 1), h[4], h[5], h[6], h[7]);
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t h[4];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t w = ww[x] >> (8 * y);
                h[2 * y] = hmul2(hsub2((w & 0x000F000Fu) | 0x64006400u, 0x64086408u), sh);
                h[2 * y + 1] = hmul2(hfma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u), sh);
              }
              if (none) h[0] = h[1] = h[2] = h[3] = 0u;
              sts128(dst + row_chunk(rr, 4 * sub + x), h[0], h[1], h[2], h[3]);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kvfull[s]);
        // the next rows' loads are in flight while the next slot is waited for
        if (value == 0) {
          fetch(j, 1, pid);
        } else {
          pid = pid_next;
          pid_next = page_of(j + 2);
          fetch(j + 1, 0, pid);
        }
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// Joins the parts of split key ranges: a warp a row, parts in order.
template <int D>
__global__ void __launch_bounds__(256) attn_tile_join_kernel(const AttnArgs a, int quant) {
  constexpr int PER = D / 32;
  pdl_wait();
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
  float top = kNegInf;
  for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_ml[s * n + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float l = 0.0f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = a.part_ml[s * n + row];
    if (ml.x == kNegInf) {
      l += ml.y;  // 0, or NaN
      continue;
    }
    const float f = ex2(ml.x - top);
    l = fmaf(ml.y, f, l);
    const float* src = a.part_o + (s * n + row) * D + PER * lane;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = fmaf(src[i], f, o[i]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (quant) {
    // lane `lane` holds columns PER * lane ..; put the values of 4-bit rows back in order
    __shared__ float sv[8][D];
    float* v = sv[threadIdx.x >> 5];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = PER * lane + i;
      v[quant == kPaged4 ? column_value<kPaged4>(c) : c] = o[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = v[PER * lane + i];
#pragma unroll
    for (int st = 1; st < PER; st *= 2)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (!(i & st)) {
          const float x = o[i], y = o[i + st];
          o[i] = x + y;
          o[i + st] = x - y;
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

// Rows of D 16-bit values as 3-D {D, heads, tokens}; a copy takes 64 columns of box_rows tokens of one head.
cudaError_t make_map(CUtensorMap* map, const void* data, int d, int64_t heads, int64_t tokens, int64_t head_stride,
                     int64_t token_stride, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(data), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int SRC, bool BF16>
cudaError_t launch_tile(const AttnArgs& a, cudaStream_t stream) {
  using C = TileCfg<D, SRC>;
  TileMaps maps = {};
  cudaError_t e = cudaSuccess;
  if constexpr (SRC == kPacked) {
    e = make_map(&maps.k, a.k.data, D, a.kv_heads, a.total_q, a.k.head_stride, a.k.token_stride, kKeys);
    if (e == cudaSuccess) e = make_map(&maps.v, a.v.data, D, a.kv_heads, a.total_q, a.v.head_stride, a.v.token_stride, kKeys);
  } else if constexpr (SRC == kPaged16) {
    const int64_t rows = (a.cache.num_pages * a.kv_heads) << a.cache.page_shift;
    const int box = a.cache.page_shift < 7 ? 1 << a.cache.page_shift : kKeys;
    e = make_map(&maps.k, a.cache.k, D, 1, rows, D, D, box);
    if (e == cudaSuccess) e = make_map(&maps.v, a.cache.v, D, 1, rows, D, D, box);
  }
  if (e != cudaSuccess) return e;
  // the register split waits for registers that a launch with fewer would never have
  e = allow_smem<attn_tile_kernel<D, SRC, BF16>>(C::kSmem, C::kLaunchRegs);
  if (e != cudaSuccess) return e;
  // row tiles: no more than all rows' and one partly filled for each sequence
  const int64_t group = a.heads / a.kv_heads;
  const int64_t tiles = a.total_q * group / kItemRows + (a.total_q < a.batch ? a.total_q : a.batch);
  const int64_t blocks = tiles * a.kv_heads * a.splits;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  attn_tile_kernel<D, SRC, BF16><<<(unsigned)blocks, C::kThreads, C::kSmem, stream>>>(maps, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.total_q * a.heads + 7) / 8), 1u, 1u);
  cfg.blockDim = dim3(256u, 1u, 1u);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_tile_join_kernel<D>, a, C::kQuant ? SRC : 0);
}

template <int D>
cudaError_t launch_tile_d(const AttnArgs& a, bool paged, cudaStream_t stream) {
  if (!paged) return a.bf16 ? launch_tile<D, kPacked, true>(a, stream) : launch_tile<D, kPacked, false>(a, stream);
  switch (a.cache.format) {
    case kKvF16: return launch_tile<D, kPaged16, false>(a, stream);
    case kKvBf16: return launch_tile<D, kPaged16, true>(a, stream);
    case kKvInt8: return launch_tile<D, kPaged8, false>(a, stream);
    default: return launch_tile<D, kPaged4, false>(a, stream);
  }
}

}  // namespace

cudaError_t launch_attn_tile(const AttnArgs& a, bool paged, cudaStream_t stream) {
  return a.head_dim == 64 ? launch_tile_d<64>(a, paged, stream) : launch_tile_d<128>(a, paged, stream);
}

cudaError_t take_device_error_attn(uint32_t* flags) { return take_tu_device_error(flags); }

}  // namespace exl3
