// exl3_attn_token.cu -- attention of a few query rows a sequence (single tokens,
// drafted tokens) over the paged cache, and the join of split results.
//
// One item is a sequence and a key head; its rows are the query tokens times
// the group's query heads (at most 16).  Scores, the running maximum and sum, and
// the output accumulate in one pass over the keys:
//     m' = max(m, s),  l' = l 2^(m - m') + sum 2^(s - m'),  o' = o 2^(m - m') + sum 2^(s - m') v.
// Every cached byte is read once and meets 2 * 16 multiply-adds a value at the
// most, so DRAM bounds it, and after that the instructions that turn codes into
// operands.  The keys and values are the M = 16 operand of mma.m16n8k16 and the
// rows the N = 8 one (S' = K Q', O' = V' P'): with up to eight rows, the usual
// decode step, no multiply-add, exponential or register goes to rows that are not
// there (with the rows as M = 16, the first case below took 201 us).  The codes go
// from shared memory to operands in registers without a 16-bit copy in between.
//
// Measured, 32 query and 8 key heads of 128:
//   48 sequences of 0 to 16384 keys, one token each, 8 bits   126 us, 713 MB: 5650 GB/s, 83% of a copy's
//   8 sequences of 9000 to 32768 keys, 1 to 4 tokens, 4 bits, fp16 queries
//     94 us, 216 MB: 2300 GB/s; two CTAs an SM (246 registers) issue what the widening of four-bit codes and
//     the second term take.  Three CTAs of fewer registers 118 us, pairs of warps on one ring 123 us.
//   one sequence of 4097 keys, one token, 16 bits             12.4 us, 16.8 MB: the chain lengths, page ids,
//     copies, join of the two launches
//
// Split.  The work is the list of all items' units of 64 keys, cut into one
// equal range a CTA (whatever the sequences' lengths are), so a range may begin
// and end inside items; an item counts a few units more than it has, for what
// beginning and ending one costs.  Each CTA works the cuts out from kv_lens by
// itself.  An item inside one range is finished there; one that is cut leaves
// (m, l, o) of its parts in the workspace, which attn_token_join_kernel joins in
// order.  Inside a CTA four warps take turns at the range's steps, each with its
// own ring of asynchronous copies and its own (m, l, o), joined at the item's end.
//
// Quantised rows stay in the rotated basis (see exl3_rope_cache.cu): q is
// rotated by the D-point Hadamard transform times 8/D once, the output once, and
// each row held in units of a power of two near its largest value.  The
// rotated q is not exact in fp16: for fp16 queries it goes in as two fp16 terms
// (22 bits), since one alone moved the outputs by 1.7 times their own rounding
// (bf16 outputs round eight times coarser: one term).
// A key's scale multiplies its score in fp32.  A value's scale goes into the
// exponent: the weight 2^(s + log2 scale - m), with m the maximum of the same sum,
// is at most 2^8 whatever the scales are, so rounding it to fp16 loses nothing by
// range; the sum l takes the weight divided by the scale.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "exl3_attn.h"
#include "exl3_ptx.cuh"
#include "exl3_sm100.cuh"

namespace exl3 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kNegInf = -__builtin_huge_valf();
// The reference of the exponents moves only when the maximum has grown by more
// than this (log2), so most steps rescale nothing; weights stay below 2^8.
constexpr float kSlack = 8.0f;
// What an item's beginning and end cost, in units of keys (for the cuts).
constexpr int kItemUnits = 4;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
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
__device__ __forceinline__ float to_f32(uint16_t e, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)e << 16) : __half2float(__ushort_as_half(e));
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Transpose of an 8x8 matrix of 16-bit values held as fragments.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The larger, or NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return __uint_as_float((uint32_t)v << 16);
}
// Two scores times a factor and two units, plus an addend, two numbers an instruction.
__device__ __forceinline__ void scale2(float& x, float& y, float factor, const float (&unit)[2], float add) {
  asm("{\n .reg .b64 s, f, u, a;\n mov.b64 s, {%0, %1};\n mov.b64 f, {%2, %2};\n mov.b64 u, {%3, %4};\n mov.b64 a, {%5, %5};\n"
      " mul.rn.f32x2 f, f, u;\n fma.rn.f32x2 s, s, f, a;\n mov.b64 {%0, %1}, s;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(factor), "f"(unit[0]), "f"(unit[1]), "f"(add));
}
// Two bytes (offset codes) widened by the pattern of 1024: {1024 + c0, 1024 + c1} - 1152.
__device__ __forceinline__ uint32_t bytes_to_h2(uint32_t w, uint32_t sel) {
  return hsub2(__byte_perm(w, 0x64646464u, sel), 0x64806480u);
}
// Nibbles at bits 0 and 16 / 4 and 20 of w, minus 8.
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) { return hsub2((w & 0x000F000Fu) | 0x64006400u, 0x64086408u); }
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) {
  return hfma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);  // / 16 - 72
}

// What a sequence asks for: its packed query tokens, its cached length, and its units of 64 keys.
struct Seq {
  int64_t q0;
  int q_len, kv_len;
  int first;  // first key that any row sees
  int lo;     // first key of the first unit
  int units;  // 0: no query tokens
  // units that the cuts count for one of its items: kItemUnits, then the units
  __device__ __forceinline__ int weight() const { return units == 0 ? 0 : units + kItemUnits; }
};
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  Seq s;
  const int64_t c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
  s.q0 = c0 < 0 ? 0 : c0 > a.total_q ? a.total_q : c0;
  const int64_t n = (c1 > a.total_q ? a.total_q : c1) - s.q0;
  s.q_len = n < 0 ? 0 : n > a.max_q ? a.max_q : (int)n;
  const int64_t room = (int64_t)a.table_width << a.cache.page_shift;
  const int64_t kl = a.kv_lens[b];
  s.kv_len = (int)(kl < 0 ? 0 : kl > room ? room : kl);
  const int64_t first = a.window > 0 ? (int64_t)s.kv_len - s.q_len - a.window + 1 : 0;
  s.first = first > 0 ? (int)first : 0;
  s.lo = s.first / kTokenUnit * kTokenUnit;
  // a sequence without keys still has a unit: its rows are zeros
  const int u = (s.kv_len - s.lo + kTokenUnit - 1) / kTokenUnit;
  s.units = s.q_len == 0 ? 0 : u < 1 ? 1 : u;
  return s;
}

// All units of the call (one warp; every lane gets the sum).
__device__ int64_t total_units(const AttnArgs& a, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < a.batch; b += 32) sum += load_seq(a, b).weight();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * a.kv_heads;
}
// The sequence that holds unit u, and the units of the sequences before it.
__device__ int find_seq(const AttnArgs& a, int lane, int64_t u, int64_t* before) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int64_t n = b0 + lane < a.batch ? (int64_t)load_seq(a, b0 + lane).weight() * a.kv_heads : 0;
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += p;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + inc > u);
    if (hit) {
      const int at = __ffs(hit) - 1;
      *before = base + __shfl_sync(0xffffffffu, inc - n, at);
      return b0 + at;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  *before = base;
  return a.batch;
}

// FMT: KvFormat.  NR: tiles of eight rows.  TWO: the rotated q in two terms.
template <int FMT, int D, int NR, bool TWO>
struct TokenCfg {
  static constexpr bool kQuant = kv_quantised(FMT);
  static constexpr bool kBf16 = FMT == kKvBf16;  // operand type of the MMAs (fp16 for the quantised formats)
  static constexpr int kRows = 8 * NR;
  static constexpr int kCtas = token_ctas_per_sm(kRows);
  static constexpr int kRow = kv_row_bytes(FMT, D);
  static constexpr int kStep = kRow >= 256 ? 16 : 32;  // keys a warp takes at a time
  static constexpr int kSide = kStep * kRow;           // bytes of a step's keys (or values)
  static constexpr int kScales = kQuant ? 4 * kStep : 0;
  static constexpr int kStage = 2 * kSide + kScales;
  static constexpr int kStages = kSide >= 4096 ? 2 : 4;
  static constexpr int kRing = kStages * kStage;           // a warp's
  static constexpr int kJoin = kRows * D * 4 + kRows * 8;  // a warp's (o, m, l) at an item's end
  static constexpr int kWarpBytes = ((kRing > kJoin ? kRing : kJoin) + 127) / 128 * 128;
  static constexpr int kQBytes = kQuant ? 2 * kRows * D * 2 : 0;  // the rotated q and the fragments of its second term
  static constexpr int kUnits = kWarps * kWarpBytes + kQBytes;    // [kRows] of the rotated q's rows: unit times 8/D and the scale
  static constexpr int kSmem = kUnits + (kQuant ? 4 * kRows : 0);
  static constexpr int kChunks = kRow / 16;  // 16-byte chunks of a row
  static constexpr int kTpr = kThreads / kRows;  // threads of a row where the CTA works on whole rows
  static constexpr int kPer = D / kTpr;          // and values of each
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory");
};
// Hadamard transform of a row held as PER consecutive values by TPR neighbouring threads.
template <int PER, int TPR>
__device__ __forceinline__ void hadamard_threads(float (&v)[PER], int part) {
#pragma unroll
  for (int st = 1; st < PER; st *= 2)
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!(i & st)) {
        const float x = v[i], y = v[i + st];
        v[i] = x + y;
        v[i + st] = x - y;
      }
#pragma unroll
  for (int st = 1; st < TPR; st *= 2)
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float x = __shfl_xor_sync(0xffffffffu, v[i], st);
      v[i] = (part & st) ? x - v[i] : v[i] + x;
    }
}

// Byte offset of chunk c of row r of a step's keys or values.  The permutations
// keep the eight or sixteen lanes of one shared-memory access on different
// banks, both for the keys' reads (neighbouring rows) and the values' (every
// other row).
template <int ROW>
__device__ __forceinline__ uint32_t ring_offset(int r, int c) {
  if constexpr (ROW >= 256) return (uint32_t)(r * ROW + ((c ^ (r & 7)) << 4));
  if constexpr (ROW == 128) return (uint32_t)(r * 128 + ((c ^ (r & 6) ^ ((r & 1) << 2)) << 4));
  if constexpr (ROW == 64)
    return (uint32_t)((r >> 1) * 128 + (((r ^ (r >> 2)) & 1) << 6) + ((c ^ (r & 2)) << 4));
  return (uint32_t)(r * ROW + (c << 4));
}

template <int FMT, int D, int NR, bool TWO>
__global__ void __launch_bounds__(kThreads, token_ctas_per_sm(8 * NR)) attn_token_kernel(const AttnArgs a) {
  using C = TokenCfg<FMT, D, NR, TWO>;
  constexpr bool BF16 = C::kBf16;
  constexpr int KS = D / 16;        // k16 steps of the scores
  constexpr int NK = C::kStep / 16;  // 16-key tiles of a step
  constexpr int ND = D / 16;        // 16-row tiles of the output (transposed)
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int group = a.heads / a.kv_heads;
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
  pdl_launch_dependents();  // the join may be scheduled; it waits for this grid

  const int64_t total = total_units(a, lane);
  const int64_t grid = gridDim.x;
  int64_t u = total * blockIdx.x / grid;
  const int64_t u_end = total * (blockIdx.x + 1) / grid;
  if (u >= u_end) return;
  int64_t before;
  int b = find_seq(a, lane, u, &before);

  while (u < u_end) {
    Seq s = load_seq(a, b);
    while (s.units == 0) s = load_seq(a, ++b);  // there is a unit left, so a sequence that has it
    const int weight = s.weight();
    const int64_t in_seq = u - before;
    const int h = (int)(in_seq / weight);
    const int at0 = (int)(in_seq - (int64_t)h * weight);
    const int64_t room = u_end - u;
    const int at1 = room < weight - at0 ? at0 + (int)room : weight;
    const int32_t* pages = a.table + (int64_t)b * a.table_width;
    u += at1 - at0;
    if (at1 == weight && h == a.kv_heads - 1) {
      before += (int64_t)weight * a.kv_heads;
      ++b;
    }
    const int unit0 = max(0, at0 - kItemUnits), unit1 = max(0, at1 - kItemUnits);
    if (unit0 == unit1) continue;  // nothing but what the item's beginning counts
    const int rows = s.q_len * group;
    const int t0 = s.lo + unit0 * kTokenUnit;
    const int t1 = min(s.kv_len, s.lo + unit1 * kTokenUnit);
    const int steps = t1 > t0 ? (t1 - t0 + C::kStep - 1) / C::kStep : 0;

    // ---- page ids of this warp's next 32 steps, one step a lane
    constexpr int PG = C::kStep / 16;  // a step's 16-key groups, each inside one page
    int pid[PG];
    auto load_pids = [&](int first) {  // first: this warp's step index (in its own steps) of lane 0
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        const int t = t0 + (warp + kWarps * (first + lane)) * C::kStep + 16 * i;
        pid[i] = -1;
        if (t < t1 && t + 16 > s.first) pid[i] = pages[t >> a.cache.page_shift];
        if (pid[i] >= a.cache.num_pages) pid[i] = -1;
      }
    };
    const int mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;
    int pid_base = 0;
    load_pids(0);

    // ---- the query rows' loads, in flight with the page ids'
    uint32_t qb[NR][KS][2];  // B fragments: row 8n + g, values 16k + 2q, + 1 and + 8, + 9; zeros past the last row
    constexpr int QW = C::kQuant ? C::kPer / 2 : 1;
    uint32_t qraw[QW];
    const int jr = threadIdx.x / C::kTpr, part = threadIdx.x % C::kTpr;  // row and part where the CTA works on rows
    if constexpr (!C::kQuant) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int r = 8 * n + g;
        const uint16_t* src = nullptr;
        if (r < rows) {
          const int tok = r / group;
          src = static_cast<const uint16_t*>(a.q.data) + (s.q0 + tok) * a.q.token_stride +
                (int64_t)(h * group + r - tok * group) * a.q.head_stride;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qb[n][k][0] = src ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q) : 0u;
          qb[n][k][1] = src ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * q) : 0u;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < QW; ++i) qraw[i] = 0u;
      if (jr < rows) {
        const int tok = jr / group;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            static_cast<const uint16_t*>(a.q.data) + (s.q0 + tok) * a.q.token_stride +
            (int64_t)(h * group + jr - tok * group) * a.q.head_stride + part * C::kPer);
#pragma unroll
        for (int i = 0; i < QW; ++i) qraw[i] = src[i];
      }
    }

    auto issue = [&](int i) {  // copies of this warp's step i into slot i % stages
      if (i < mine) {
        if (i - pid_base >= 32) {
          pid_base += 32;
          load_pids(pid_base);
        }
        const uint32_t dst = ring + (uint32_t)(i % C::kStages) * C::kStage;
        const int t = t0 + (warp + kWarps * i) * C::kStep;
        int64_t base[PG];  // cache row of each 16-key group's first key
        bool ok[PG];
#pragma unroll
        for (int p = 0; p < PG; ++p) {
          const int id = __shfl_sync(0xffffffffu, pid[p], i - pid_base);
          ok[p] = id >= 0;
          base[p] = (((int64_t)(ok[p] ? id : 0) * a.kv_heads + h) << a.cache.page_shift) +
                    (ok[p] ? (t + 16 * p) & ((1 << a.cache.page_shift) - 1) : 0);
        }
#pragma unroll
        for (int j = 0; j < C::kStep * C::kChunks / 32; ++j) {
          const int idx = j * 32 + lane;
          const int r = idx / C::kChunks, c = idx % C::kChunks;
          const int p = PG == 1 ? 0 : r >> 4;
          // rows outside the keys seen come as zeros, so no weight ever meets what a page holds there
          const bool there = (p ? ok[PG - 1] : ok[0]) && t + r < t1 && t + r >= s.first;
          const int64_t row = (p ? base[PG - 1] : base[0]) + (there ? (r & 15) : 0);
          const uint32_t off = ring_offset<C::kRow>(r, c);
          cp_async16(dst + off, a.cache.k + row * C::kRow + 16 * c, there);
          cp_async16(dst + C::kSide + off, a.cache.v + row * C::kRow + 16 * c, there);
        }
        if constexpr (C::kQuant) {
          // 32 bytes of scales a group and side
          if (lane < 4 * PG) {
            const int side = lane >= 2 * PG, i16 = lane % (2 * PG), p = i16 >> 1;
            const uint16_t* src = (side ? a.cache.v_scale : a.cache.k_scale) + (p ? base[PG - 1] : base[0]) + 8 * (i16 & 1);
            cp_async16(dst + 2 * C::kSide + side * 2 * C::kStep + 16 * i16, src, p ? ok[PG - 1] : ok[0]);
          }
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) issue(i);

    float unit[NR][2];  // of the scores of rows 8n + 2q, + 1 over a quantised cache: the rotated q's units, 8/D and the scale
    // the second term of the rotated q, only for fp16 queries: [n][k][lane] fragments
    const uint32_t qlo = smem_u32(smem) + kWarps * C::kWarpBytes + C::kRows * D * 2;
    if constexpr (C::kQuant) {
      // rotate, to fp16 in shared memory, one term after the other
      uint16_t* qs = reinterpret_cast<uint16_t*>(smem + kWarps * C::kWarpBytes);
      float v[C::kPer];
#pragma unroll
      for (int i = 0; i < QW; ++i) {
        v[2 * i] = to_f32((uint16_t)(qraw[i] & 0xFFFFu), a.bf16 != 0);
        v[2 * i + 1] = to_f32((uint16_t)(qraw[i] >> 16), a.bf16 != 0);
      }
      hadamard_threads<C::kPer, C::kTpr>(v, part);
      // in units of a power of two near the row's largest value, so that fp16 holds any q
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < C::kPer; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
      for (int st = 1; st < C::kTpr; st *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, st));
      const uint32_t e = unit_exponent(top);
      float* units = reinterpret_cast<float*>(smem + C::kUnits);
      if (part == 0) units[jr] = a.scale_log2 * (8.0f / D) * power(e);
#pragma unroll
      for (int i = 0; i < C::kPer; ++i) v[i] *= power(254u - e);
      // fragments in the order in which the codes come out of their words
      auto fragments = [&](uint32_t (&dst)[KS][2], int n) {
        const uint16_t* src = qs + (8 * n + g) * D;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if constexpr (FMT == kKvInt8) {
            // lane q holds values 16q .. 16q + 15 (of each 64), four a k16 step
            const uint32_t* w = reinterpret_cast<const uint32_t*>(src + (k >> 2) * 64 + 16 * q + 4 * (k & 3));
            dst[k][0] = w[0];
            dst[k][1] = w[1];
          } else {
            // lane q holds values (D/4)q .. , eight a word, pairs (0, 4) (1, 5) then (2, 6) (3, 7)
            const int d = (D / 4) * q + 8 * (k >> 1) + 2 * (k & 1);
            dst[k][0] = (uint32_t)src[d] | (uint32_t)src[d + 4] << 16;
            dst[k][1] = (uint32_t)src[d + 1] | (uint32_t)src[d + 5] << 16;
          }
        }
      };
      if constexpr (TWO) {
#pragma unroll
        for (int i = 0; i < C::kPer; i += 2) {
          const uint32_t hi = pack2<false>(v[i], v[i + 1]);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          *reinterpret_cast<uint32_t*>(qs + jr * D + part * C::kPer + i) = pack2<false>(v[i] - f.x, v[i + 1] - f.y);
        }
        __syncthreads();
        // warp w makes the fragments of tiles w, w + 4, ...
        if (warp < NR) {
          uint32_t tmp[KS][2];
          fragments(tmp, warp);
#pragma unroll
          for (int k = 0; k < KS; ++k)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qlo + (uint32_t)((warp * KS + k) * 32 + lane) * 8), "r"(tmp[k][0]), "r"(tmp[k][1])
                         : "memory");
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < C::kPer; i += 2) *reinterpret_cast<uint32_t*>(qs + jr * D + part * C::kPer + i) = pack2<false>(v[i], v[i + 1]);
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        fragments(qb[n], n);
        const float2 u = *reinterpret_cast<const float2*>(units + 8 * n + 2 * q);
        unit[n][0] = u.x, unit[n][1] = u.y;
      }
    }

    // ---- this lane's rows 8n + 2q, + 1: what they see, and their running softmax
    int pos[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) pos[n][i] = s.kv_len - s.q_len + min(8 * n + 2 * q + i, rows - 1) / group;
    const int lim_all = min(s.kv_len - s.q_len, t1 - 1);  // keys up to here are seen by every row
    const int low_all = a.window > 0 ? max(0, s.kv_len - a.window) : 0;
    float m[NR][2], l[NR][2];
    float o[NR][ND][4];  // rows of the output's tile j: values (see the write below), columns: rows 2q, 2q + 1
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      m[n][0] = m[n][1] = kNegInf;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < ND; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
    }

    for (int i = 0; i < mine; ++i) {
      issue(i + C::kStages - 1);
      cp_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t kb = ring + (uint32_t)(i % C::kStages) * C::kStage;
      const uint32_t vb = kb + C::kSide;
      const int t = t0 + (warp + kWarps * i) * C::kStep;

      // ---- scores of keys 16x + g (elements 0, 1) and 16x + g + 8 (2, 3)
      float sc[NK][NR][4];
#pragma unroll
      for (int x = 0; x < NK; ++x) {
#pragma unroll
        for (int n = 0; n < NR; ++n) sc[x][n][0] = sc[x][n][1] = sc[x][n][2] = sc[x][n][3] = 0.0f;
        if constexpr (!C::kQuant) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4];
            ldmatrix_x4(kb + ring_offset<C::kRow>(16 * x + (lane & 15), 2 * k + (lane >> 4)), r);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              mma16816<BF16>(sc[x][n], r, qb[n][k][0], qb[n][k][1]);
            }
          }
        }
      }
      if constexpr (C::kQuant) {
        constexpr int WORDS = FMT == kKvInt8 ? 4 : D / 32;        // words of a row a lane takes at a time
        constexpr int KW = FMT == kKvInt8 ? 4 : KS;               // k16 steps that they make
#pragma unroll
        for (int k0 = 0; k0 < KS; k0 += KW) {
          uint32_t w[NK][2][WORDS];
#pragma unroll
          for (int x = 0; x < NK; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int row = 16 * x + g + 8 * y;
              if constexpr (WORDS == 4) {
                const uint4 v = lds128(kb + ring_offset<C::kRow>(row, (FMT == kKvInt8 ? k0 : 0) + q));
                w[x][y][0] = v.x, w[x][y][1] = v.y, w[x][y][2] = v.z, w[x][y][3] = v.w;
              } else {
                const uint2 v = lds64(kb + ring_offset<C::kRow>(row, q >> 1) + 8 * (q & 1));
                w[x][y][0] = v.x, w[x][y][1] = v.y;
              }
            }
#pragma unroll
          for (int k = 0; k < KW; ++k) {
            uint32_t r[NK][4];
#pragma unroll
            for (int x = 0; x < NK; ++x) {
              if constexpr (FMT == kKvInt8) {
                r[x][0] = bytes_to_h2(w[x][0][k], 0x4140), r[x][1] = bytes_to_h2(w[x][1][k], 0x4140);
                r[x][2] = bytes_to_h2(w[x][0][k], 0x4342), r[x][3] = bytes_to_h2(w[x][1][k], 0x4342);
              } else {
                const uint32_t u0 = w[x][0][k >> 1] >> (8 * (k & 1)), u1 = w[x][1][k >> 1] >> (8 * (k & 1));
                r[x][0] = nib_lo(u0), r[x][1] = nib_lo(u1), r[x][2] = nib_hi(u0), r[x][3] = nib_hi(u1);
              }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) {
#pragma unroll
              for (int x = 0; x < NK; ++x) mma16816<false>(sc[x][n], r[x], qb[n][k0 + k][0], qb[n][k0 + k][1]);
              if constexpr (TWO) {
                const uint2 lo = lds64(qlo + (uint32_t)((n * KS + k0 + k) * 32 + lane) * 8);
#pragma unroll
                for (int x = 0; x < NK; ++x) mma16816<false>(sc[x][n], r[x], lo.x, lo.y);
              }
            }
          }
        }
      }

      // ---- scale, mask, running maximum
      float rv[NK][2];  // quantised: 1 / value scale of this lane's keys
      bool ones = false;  // a value scale of exactly 1 among them
#pragma unroll
      for (int x = 0; x < NK; ++x) {
        if constexpr (C::kQuant) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t at = kb + 2 * C::kSide + 2 * (16 * x + 8 * y + g);
            const float kc = lds_bf16(at);
            // a NaN scale (a row that reads back as NaN) stays one
            const float vc = max_nan(lds_bf16(at + 2 * C::kStep), 7.888609052210118e-31f);
            ones = ones || vc == 1.0f;
            const float lv = lg2(vc);
            rv[x][y] = rcp(vc);
#pragma unroll
            for (int n = 0; n < NR; ++n) scale2(sc[x][n][2 * y], sc[x][n][2 * y + 1], kc, unit[n], lv);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[x][n][c] *= a.scale_log2;
        }
      }
      if constexpr (C::kQuant) {
        // A row of zeros has the scale 1, which would lift the maximum over smaller rows' weights although nothing is in
        // it: its weight goes into the sum alone, by a scale of 2^-80.
        if (__any_sync(0xffffffffu, ones)) {
          constexpr uint32_t kZero = FMT == kKvInt8 ? 0x80808080u : 0x88888888u;
#pragma unroll
          for (int x = 0; x < NK; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int row = 16 * x + 8 * y + g;
              uint32_t codes = lds_bf16(kb + 2 * C::kSide + 2 * C::kStep + 2 * row) == 1.0f ? 0u : 1u;
#pragma unroll
              for (int ch = 0; ch < C::kChunks; ch += 4) {
                if (ch + q >= C::kChunks) continue;
                const uint4 w = lds128(vb + ring_offset<C::kRow>(row, ch + q));
                codes |= (w.x ^ kZero) | (w.y ^ kZero) | (w.z ^ kZero) | (w.w ^ kZero);
              }
              codes |= __shfl_xor_sync(0xffffffffu, codes, 1);
              codes |= __shfl_xor_sync(0xffffffffu, codes, 2);
              if (codes == 0u) {
                rv[x][y] = power(127 + 80);
#pragma unroll
                for (int n = 0; n < NR; ++n) sc[x][n][2 * y] -= 80.0f, sc[x][n][2 * y + 1] -= 80.0f;
              }
            }
        }
      }
      if (t + C::kStep - 1 > lim_all || t < low_all) {
#pragma unroll
        for (int x = 0; x < NK; ++x)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = t + 16 * x + g + 8 * (c >> 1);
#pragma unroll
            for (int n = 0; n < NR; ++n)
              if (key > min(pos[n][c & 1], t1 - 1) || (a.window > 0 && key <= pos[n][c & 1] - a.window)) sc[x][n][c] = kNegInf;
            if constexpr (C::kQuant) {
              // seen by no row: its scale may be anything
              if (key > lim_all + s.q_len - 1 || key < s.first) rv[x][c >> 1] = 0.0f;
            }
          }
      }
      float top[NR][2];
      bool up = false;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v = kNegInf;
#pragma unroll
          for (int x = 0; x < NK; ++x) v = fmaxf(v, fmaxf(sc[x][n][c], sc[x][n][c + 2]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          top[n][c] = v;
          up = up || v > m[n][c] + kSlack;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float f[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const bool u1 = top[n][c] > m[n][c] + kSlack;
            f[c] = u1 ? ex2(m[n][c] - top[n][c]) : 1.0f;
            m[n][c] = u1 ? top[n][c] : m[n][c];
            l[n][c] *= f[c];
          }
#pragma unroll
          for (int j = 0; j < ND; ++j) {
            o[n][j][0] *= f[0];
            o[n][j][1] *= f[1];
            o[n][j][2] *= f[0];
            o[n][j][3] *= f[1];
          }
        }
      }

      // ---- weights, and weights times values
#pragma unroll
      for (int x = 0; x < NK; ++x) {
        uint32_t pb[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // a row that has seen nothing yet has only -inf scores; any finite reference gives it zero weights
            const float ref = m[n][c & 1] == kNegInf ? 0.0f : m[n][c & 1];
            sc[x][n][c] = ex2(sc[x][n][c] - ref);
            l[n][c & 1] = C::kQuant ? fmaf(sc[x][n][c], rv[x][c >> 1], l[n][c & 1]) : l[n][c & 1] + sc[x][n][c];
          }
          pb[n][0] = movmatrix(pack2<BF16>(sc[x][n][0], sc[x][n][1]));
          pb[n][1] = movmatrix(pack2<BF16>(sc[x][n][2], sc[x][n][3]));
        }
        if constexpr (!C::kQuant) {
#pragma unroll
          for (int j = 0; j < ND; ++j) {
            uint32_t r[4];
            const int row = 16 * x + (lane & 7) + ((lane >> 4) << 3);
            ldmatrix_x4_trans(vb + ring_offset<C::kRow>(row, 2 * j + ((lane >> 3) & 1)), r);
#pragma unroll
            for (int n = 0; n < NR; ++n) mma16816<BF16>(o[n][j], r, pb[n][0], pb[n][1]);
          }
        } else {
          // this lane's keys 2q, 2q + 1, 2q + 8, 2q + 9 of the sixteen, its D/8 values from (D/8) g on
          constexpr int VB = C::kRow / 8;  // bytes a lane takes of a row
          uint32_t w[4][VB / 4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int row = 16 * x + 2 * q + (y & 1) + 8 * (y >> 1);
            const int at = VB * g;
            const uint32_t addr = vb + ring_offset<C::kRow>(row, at >> 4) + (at & 15);
            if constexpr (VB == 16) {
              const uint4 v = lds128(addr);
              w[y][0] = v.x, w[y][1] = v.y, w[y][2] = v.z, w[y][3] = v.w;
            } else if constexpr (VB == 8) {
              const uint2 v = lds64(addr);
              w[y][0] = v.x, w[y][1] = v.y;
            } else {
              w[y][0] = lds32(addr);
            }
          }
          // tile j's rows g and g + 8 are this lane's values 2j and 2j + 1
#pragma unroll
          for (int y = 0; y < VB / 4; ++y) {
            if constexpr (FMT == kKvInt8) {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                // {a, b, a', b'} of two neighbouring values, then each pair widened
                const uint32_t lo = __byte_perm(w[0][y], w[1][y], z ? 0x7362 : 0x5140);
                const uint32_t hi = __byte_perm(w[2][y], w[3][y], z ? 0x7362 : 0x5140);
                const uint32_t r[4] = {bytes_to_h2(lo, 0x4140), bytes_to_h2(lo, 0x4342), bytes_to_h2(hi, 0x4140),
                                       bytes_to_h2(hi, 0x4342)};
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                  mma16816<false>(o[n][2 * y + z], r, pb[n][0], pb[n][1]);
                }
              }
            } else {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                // four values of key a below the same four of key b
                const uint32_t lo = __byte_perm(w[0][y], w[1][y], z ? 0x7632 : 0x5410);
                const uint32_t hi = __byte_perm(w[2][y], w[3][y], z ? 0x7632 : 0x5410);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t r[4] = {nib_lo(lo >> (8 * e)), nib_hi(lo >> (8 * e)), nib_lo(hi >> (8 * e)),
                                         nib_hi(hi >> (8 * e))};
#pragma unroll
                  for (int n = 0; n < NR; ++n) {
                    mma16816<false>(o[n][4 * y + 2 * z + e], r, pb[n][0], pb[n][1]);
                  }
                }
              }
            }
          }
        }
      }
      __syncwarp();  // every lane is done with the slot that the next issue refills
    }
    cp_wait<0>();

    // ---- join the warps' results
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], 4);
        l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], 8);
        l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], 16);
      }
    __syncthreads();
    {
      float* wo = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);
      float2* wml = reinterpret_cast<float2*>(wo + C::kRows * D);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int j = 0; j < ND; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int d = C::kQuant ? (D / 8) * g + 2 * j + (c >> 1) : 16 * j + g + 8 * (c >> 1);
            wo[(8 * n + 2 * q + (c & 1)) * D + d] = o[n][j][c];
          }
        if (g == 0) {
          wml[8 * n + 2 * q] = make_float2(m[n][0], l[n][0]);
          wml[8 * n + 2 * q + 1] = make_float2(m[n][1], l[n][1]);
        }
      }
    }
    __syncthreads();
    {
      constexpr int PER = C::kPer;
      float2 ml[kWarps];
      float top = kNegInf, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = reinterpret_cast<const float2*>(smem + w * C::kWarpBytes + C::kRows * D * 4)[jr];
        top = fmaxf(top, ml[w].x);
      }
      float v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // a warp without a maximum saw nothing (its sum is 0) or nothing but NaN (its sum is NaN)
        const float f = ml[w].x == kNegInf ? (ml[w].y == 0.0f ? 0.0f : ml[w].y) : ex2(ml[w].x - top);
        sum = fmaf(ml[w].y, f, sum);
        const float4* wo = reinterpret_cast<const float4*>(smem + w * C::kWarpBytes + (jr * D + part * PER) * 4);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
          const float4 x = wo[i];
          v[4 * i] = fmaf(x.x, f, v[4 * i]);
          v[4 * i + 1] = fmaf(x.y, f, v[4 * i + 1]);
          v[4 * i + 2] = fmaf(x.z, f, v[4 * i + 2]);
          v[4 * i + 3] = fmaf(x.w, f, v[4 * i + 3]);
        }
      }
      if (unit0 == 0 && unit1 == s.units) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if constexpr (C::kQuant) {
          hadamard_threads<PER, C::kTpr>(v, part);
#pragma unroll
          for (int i = 0; i < PER; ++i) v[i] *= 8.0f / D;
        }
        if (jr < rows) {
          const int tok = jr / group;
          uint16_t* dst = static_cast<uint16_t*>(a.out) + (s.q0 + tok) * a.out_token_stride +
                          (int64_t)(h * group + jr - tok * group) * a.out_head_stride + part * PER;
#pragma unroll
          for (int i = 0; i < PER; i += 4) {
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float x = v[i + 2 * j] * inv, y = v[i + 2 * j + 1] * inv;
              w[j] = a.bf16 ? pack2<true>(x, y) : pack2<false>(x, y);
            }
            *reinterpret_cast<uint2*>(dst + i) = make_uint2(w[0], w[1]);
          }
        }
      } else if (jr < rows) {
        // a range begins inside at most one item and ends inside at most one
        const int64_t slot = 2 * (int64_t)blockIdx.x + (unit0 == 0 ? 1 : 0);
        float4* dst = reinterpret_cast<float4*>(a.part_o + (slot * kTokenRows + jr) * D + part * PER);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (part == 0) a.part_ml[slot * kTokenRows + jr] = make_float2(top, sum);
      }
    }
    __syncthreads();  // the next item's copies refill what was read here
  }
}

// Joins the parts of the items that were cut: one block an item and row; its
// warps take the parts in turn, four loads at a time, then one joins the warps in
// order.  The order is fixed by the lengths, so results repeat.
constexpr int kJoinWarps = 8;
template <int D, bool QUANT>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_token_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 32;
  constexpr int AHEAD = 4;
  __shared__ float so[kJoinWarps][D];
  __shared__ float2 sml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.heads / a.kv_heads;
  const int r = blockIdx.y;
  const int b = blockIdx.x / a.kv_heads, h = blockIdx.x % a.kv_heads;
  const Seq s = load_seq(a, b);
  const int rows = s.q_len * group;
  // units before this sequence, and of the call
  int64_t total = 0, before = 0;
  for (int i = lane; i < a.batch; i += 32) {
    const int n = load_seq(a, i).weight();
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
  // the CTA of a unit is the last whose range begins at or before it
  int64_t c0 = 0, c1 = 0;
  if (r < rows) {
    c0 = ((first + 1) * grid - 1) / total;
    c1 = ((last + 1) * grid - 1) / total;
  }
  // every block waits, cut item or not: the end of this grid then stands for the end of both
  pdl_wait();
  if (c0 == c1) return;  // no such row, or not cut
  float m = kNegInf, l = 0.0f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.0f;
  for (int64_t c = c0 + warp; c <= c1; c += kJoinWarps * AHEAD) {
    float2 ml[AHEAD];
    float v[AHEAD][PER];
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      const int64_t cc = c + x * kJoinWarps;
      const int64_t begin = total * cc / grid, end = total * (cc + 1) / grid;
      ml[x] = make_float2(kNegInf, 0.0f);
      if (cc <= c1 && begin < end) {
        const int64_t slot = 2 * cc + (begin <= first ? 1 : 0);
        ml[x] = a.part_ml[slot * kTokenRows + r];
        const float* src = a.part_o + (slot * kTokenRows + r) * D + PER * lane;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[x][i] = src[i];
      }
    }
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      if (ml[x].x == kNegInf) {
        l += ml[x].y;  // 0, or NaN
        continue;
      }
      const float top = fmaxf(m, ml[x].x);
      const float f = m == kNegInf ? 0.0f : ex2(m - top), f1 = ex2(ml[x].x - top);
      l = (m == kNegInf ? l : l * f) + ml[x].y * f1;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = o[i] * f + v[x][i] * f1;
      m = top;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) so[warp][PER * lane + i] = o[i];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  if (warp != 0) return;
  float top = kNegInf, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sml[w].x);
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = sml[w].x == kNegInf ? (sml[w].y == 0.0f ? 0.0f : sml[w].y) : ex2(sml[w].x - top);
    sum = fmaf(sml[w].y, f, sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = fmaf(so[w][PER * lane + i], f, o[i]);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if constexpr (QUANT) {
    hadamard_threads<PER, 32>(o, lane);
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] *= 8.0f / D;
  }
  const int tok = r / group;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + (s.q0 + tok) * a.out_token_stride +
                  (int64_t)(h * group + r - tok * group) * a.out_head_stride + PER * lane;
#pragma unroll
  for (int i = 0; i < PER; i += 2) {
    const uint32_t w = a.bf16 ? pack2<true>(o[i] * inv, o[i + 1] * inv) : pack2<false>(o[i] * inv, o[i + 1] * inv);
    *reinterpret_cast<uint32_t*>(dst + i) = w;
  }
}

template <int FMT, int D, int NR, bool TWO>
cudaError_t launch_token(const AttnArgs& a, cudaStream_t stream) {
  using C = TokenCfg<FMT, D, NR, TWO>;
  cudaError_t e = allow_smem<attn_token_kernel<FMT, D, NR, TWO>>(C::kSmem);
  if (e != cudaSuccess) return e;
  attn_token_kernel<FMT, D, NR, TWO><<<(unsigned)a.ctas, kThreads, C::kSmem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int rows = a.max_q * (a.heads / a.kv_heads);
  cfg.gridDim = dim3((unsigned)(a.batch * a.kv_heads), (unsigned)rows, 1u);
  cfg.blockDim = dim3(32u * kJoinWarps, 1u, 1u);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_token_join_kernel<D, C::kQuant>, a);
}
template <int FMT, bool TWO>
cudaError_t launch_token_fmt(const AttnArgs& a, cudaStream_t stream) {
  const bool small = a.max_q * (a.heads / a.kv_heads) <= 8;
  if (a.head_dim == 64) return small ? launch_token<FMT, 64, 1, TWO>(a, stream) : launch_token<FMT, 64, 2, TWO>(a, stream);
  return small ? launch_token<FMT, 128, 1, TWO>(a, stream) : launch_token<FMT, 128, 2, TWO>(a, stream);
}

}  // namespace

cudaError_t launch_attn_token(const AttnArgs& a, cudaStream_t stream) {
  switch (a.cache.format) {
    case kKvF16: return launch_token_fmt<kKvF16, false>(a, stream);
    case kKvBf16: return launch_token_fmt<kKvBf16, false>(a, stream);
    case kKvInt8: return a.bf16 ? launch_token_fmt<kKvInt8, false>(a, stream) : launch_token_fmt<kKvInt8, true>(a, stream);
    case kKvInt4: return a.bf16 ? launch_token_fmt<kKvInt4, false>(a, stream) : launch_token_fmt<kKvInt4, true>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace exl3
