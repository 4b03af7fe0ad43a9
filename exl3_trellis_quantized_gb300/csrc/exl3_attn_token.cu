// exl3_attn_token.cu -- attention of a few query rows a sequence (single tokens,
// drafted tokens) over the paged cache, and the join of split results.
//
// One item is a sequence and a key head; its rows are the query tokens times
// the group's query heads (at most 16, the M of mma.m16n8k16).  Scores, the
// running maximum and sum, and the output accumulate in one pass over the keys:
//     m' = max(m, s),  l' = l 2^(m - m') + sum 2^(s - m'),  o' = o 2^(m - m') + sum 2^(s - m') v.
// Every cached byte is read once and meets 2 * 16 multiply-adds a value at the
// most, so DRAM bounds it: the tensor work is far below even the warp-level
// MMA rate, whose fragments let the quantised formats go from shared memory to
// operands in registers without a 16-bit copy.
//
// Split.  The work is the list of all items' units of 64 keys, cut into one
// equal range a CTA (whatever the sequences' lengths are), so a range may begin
// and end inside items.  Each CTA works the cuts out from kv_lens by itself.  An
// item inside one range is finished there; one that is cut leaves (m, l, o) of
// its parts in the workspace, which attn_token_join_kernel joins in order.
// Inside a CTA four warps take turns at the range's steps, each with its own
// ring of asynchronous copies and its own (m, l, o), joined at the item's end.
//
// Quantised rows stay in the rotated basis (see exl3_rope_cache.cu): q is
// rotated by the D-point Hadamard transform times 8/D once, the output once.
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
  for (int b = lane; b < a.batch; b += 32) sum += load_seq(a, b).units;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * a.kv_heads;
}
// The sequence that holds unit u, and the units of the sequences before it.
__device__ int find_seq(const AttnArgs& a, int lane, int64_t u, int64_t* before) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int64_t n = b0 + lane < a.batch ? (int64_t)load_seq(a, b0 + lane).units * a.kv_heads : 0;
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

// FMT: KvFormat.  BF16: operand type of the MMAs (fp16 for the quantised formats).
template <int FMT, int D>
struct TokenCfg {
  static constexpr bool kQuant = kv_quantised(FMT);
  static constexpr bool kBf16 = FMT == kKvBf16;
  static constexpr int kRow = kv_row_bytes(FMT, D);
  static constexpr int kStep = kRow >= 256 ? 16 : 32;  // keys a warp takes at a time
  static constexpr int kSide = kStep * kRow;           // bytes of a step's keys (or values)
  static constexpr int kScales = kQuant ? 4 * kStep : 0;
  static constexpr int kStage = 2 * kSide + kScales;
  static constexpr int kStages = kSide >= 4096 ? 3 : 5;
  static constexpr int kRing = kStages * kStage;                    // a warp's
  static constexpr int kJoin = kTokenRows * D * 4 + kTokenRows * 8;  // a warp's (o, m, l) at an item's end
  static constexpr int kWarpBytes = ((kRing > kJoin ? kRing : kJoin) + 127) / 128 * 128;
  static constexpr int kQBytes = kQuant ? kTokenRows * D * 2 : 0;
  static constexpr int kSmem = kWarps * kWarpBytes + kQBytes;
  static constexpr int kChunks = kRow / 16;  // 16-byte chunks of a row
};

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

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 2) attn_token_kernel(const AttnArgs a) {
  using C = TokenCfg<FMT, D>;
  constexpr bool BF16 = C::kBf16;
  constexpr int KS = D / 16;       // k16 steps of the scores
  constexpr int NT = C::kStep / 8;  // 8-key tiles of a step
  constexpr int ND = D / 8;        // 8-column tiles of the output
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
    const int64_t in_seq = u - before;
    const int h = (int)(in_seq / s.units);
    const int unit0 = (int)(in_seq - (int64_t)h * s.units);
    const int64_t room = u_end - u;
    const int unit1 = room < s.units - unit0 ? unit0 + (int)room : s.units;
    const int rows = s.q_len * group;
    const int t0 = s.lo + unit0 * kTokenUnit;
    const int t1 = min(s.kv_len, s.lo + unit1 * kTokenUnit);
    const int steps = t1 > t0 ? (t1 - t0 + C::kStep - 1) / C::kStep : 0;
    const int32_t* pages = a.table + (int64_t)b * a.table_width;

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
          const bool there = (PG == 1 ? ok[0] : p ? ok[PG - 1] : ok[0]) && t + r < t1 && t + r >= s.first;
          const int64_t row = (PG == 1 || p == 0 ? base[0] : base[PG - 1]) + (there ? (r & 15) : 0);
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

    // ---- the query rows as A fragments; the rows past the last are zeros
    uint32_t qa[KS][4];
    if constexpr (!C::kQuant) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        const uint16_t* src = nullptr;
        if (r < rows) {
          const int tok = r / group;
          src = static_cast<const uint16_t*>(a.q.data) + (s.q0 + tok) * a.q.token_stride +
                (int64_t)(h * group + r - tok * group) * a.q.head_stride;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qa[k][half] = src ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q) : 0u;
          qa[k][half + 2] = src ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * q) : 0u;
        }
      }
    } else {
      // eight threads a row, D/8 values each: rotate, times 8/D, to fp16 in shared memory
      constexpr int PER = D / 8;
      uint16_t* qs = reinterpret_cast<uint16_t*>(smem + kWarps * C::kWarpBytes);
      const int r = threadIdx.x >> 3, part = threadIdx.x & 7;
      float v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = 0.0f;
      if (r < rows) {
        const int tok = r / group;
        const uint16_t* src = static_cast<const uint16_t*>(a.q.data) + (s.q0 + tok) * a.q.token_stride +
                              (int64_t)(h * group + r - tok * group) * a.q.head_stride + part * PER;
#pragma unroll
        for (int i = 0; i < PER; i += 8) {
          const uint4 w = *reinterpret_cast<const uint4*>(src + i);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i + 2 * j] = to_f32((uint16_t)(ww[j] & 0xFFFFu), a.bf16 != 0);
            v[i + 2 * j + 1] = to_f32((uint16_t)(ww[j] >> 16), a.bf16 != 0);
          }
        }
      }
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
      for (int st = 1; st < 8; st *= 2)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const float o = __shfl_xor_sync(0xffffffffu, v[i], st);
          v[i] = (part & st) ? o - v[i] : v[i] + o;
        }
#pragma unroll
      for (int i = 0; i < PER; i += 2)
        *reinterpret_cast<uint32_t*>(qs + r * D + part * PER + i) = pack2<false>(v[i] * (8.0f / D), v[i + 1] * (8.0f / D));
      __syncthreads();
      // fragments in the order in which the codes come out of their words
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint16_t* src = qs + (g + 8 * half) * D;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if constexpr (FMT == kKvInt8) {
            // lane q holds values 16q .. 16q + 15 (of each 64), four a k16 step
            const int d = (k >> 2) * 64 + 16 * q + 4 * (k & 3);
            qa[k][half] = *reinterpret_cast<const uint32_t*>(src + d);
            qa[k][half + 2] = *reinterpret_cast<const uint32_t*>(src + d + 2);
          } else {
            // lane q holds values (D/4)q .. , eight a word, pairs (0, 4) (1, 5) then (2, 6) (3, 7)
            const int d = (D / 4) * q + 8 * (k >> 1) + 2 * (k & 1);
            qa[k][half] = (uint32_t)src[d] | (uint32_t)src[d + 4] << 16;
            qa[k][half + 2] = (uint32_t)src[d + 1] | (uint32_t)src[d + 5] << 16;
          }
        }
      }
    }

    // ---- the two rows of this lane: what they see, and their running softmax
    int lim[2], low[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(g + 8 * i, rows - 1);
      const int pos = s.kv_len - s.q_len + r / group;
      lim[i] = min(pos, t1 - 1);
      low[i] = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    }
    const int lim_all = min(s.kv_len - s.q_len, t1 - 1);  // keys up to here are seen by every row
    const int low_all = a.window > 0 ? max(0, s.kv_len - a.window) : 0;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};
    float o[ND][4];
#pragma unroll
    for (int j = 0; j < ND; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;

    for (int i = 0; i < mine; ++i) {
      issue(i + C::kStages - 1);
      cp_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t kb = ring + (uint32_t)(i % C::kStages) * C::kStage;
      const uint32_t vb = kb + C::kSide;
      const int t = t0 + (warp + kWarps * i) * C::kStep;

      // ---- scores
      float sc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.0f;
      if constexpr (!C::kQuant) {
#pragma unroll
        for (int j = 0; j < NT; j += 2)
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4];
            const int row = 8 * j + (lane & 7) + ((lane >> 4) << 3);
            ldmatrix_x4(kb + ring_offset<C::kRow>(row, 2 * k + ((lane >> 3) & 1)), r);
            mma16816<BF16>(sc[j], qa[k], r[0], r[1]);
            mma16816<BF16>(sc[j + 1], qa[k], r[2], r[3]);
          }
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int row = 8 * j + g;
          if constexpr (FMT == kKvInt8) {
#pragma unroll
            for (int k4 = 0; k4 < KS / 4; ++k4) {
              const uint4 w = lds128(kb + ring_offset<C::kRow>(row, 4 * k4 + q));
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma16816<false>(sc[j], qa[4 * k4 + k], bytes_to_h2(ww[k], 0x4140),
                                bytes_to_h2(ww[k], 0x4342));
            }
          } else {
            uint32_t ww[D / 32];
            if constexpr (D == 128) {
              const uint4 w = lds128(kb + ring_offset<C::kRow>(row, q));
              ww[0] = w.x, ww[1] = w.y, ww[2] = w.z, ww[3] = w.w;
            } else {
              const uint2 w = lds64(kb + ring_offset<C::kRow>(row, q >> 1) + 8 * (q & 1));
              ww[0] = w.x, ww[1] = w.y;
            }
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              mma16816<false>(sc[j], qa[2 * k], nib_lo(ww[k]), nib_hi(ww[k]));
              mma16816<false>(sc[j], qa[2 * k + 1], nib_lo(ww[k] >> 8), nib_hi(ww[k] >> 8));
            }
          }
        }
      }

      // ---- scale, mask, running maximum
      float rv[NT][2];  // quantised: 1 / value scale of this lane's keys
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (C::kQuant) {
          const uint32_t ks = lds32(kb + 2 * C::kSide + 2 * (8 * j + 2 * q));
          const uint32_t vs = lds32(kb + 2 * C::kSide + 2 * C::kStep + 2 * (8 * j + 2 * q));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float kc = __uint_as_float(c ? ks & 0xFFFF0000u : ks << 16) * a.scale_log2;
            const float vc = fmaxf(__uint_as_float(c ? vs & 0xFFFF0000u : vs << 16), 7.888609052210118e-31f);
            // fmaxf drops a NaN scale (a row that reads back as NaN); the sum with the raw scale keeps it
            const float nan = __uint_as_float(c ? vs & 0xFFFF0000u : vs << 16) * 0.0f;
            const float lv = lg2(vc) + nan;
            rv[j][c] = __frcp_rn(vc);
            sc[j][c] = fmaf(sc[j][c], kc, lv);
            sc[j][c + 2] = fmaf(sc[j][c + 2], kc, lv);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[j][c] *= a.scale_log2;
        }
      }
      if (t + C::kStep - 1 > lim_all || t < low_all) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = t + 8 * j + 2 * q + (c & 1);
            if (key > lim[c >> 1] || key < low[c >> 1]) sc[j][c] = kNegInf;
          }
      }
      float top[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        top[0] = fmaxf(top[0], fmaxf(sc[j][0], sc[j][1]));
        top[1] = fmaxf(top[1], fmaxf(sc[j][2], sc[j][3]));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      }
      const bool up0 = top[0] > m[0] + kSlack, up1 = top[1] > m[1] + kSlack;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float f0 = up0 ? ex2(m[0] - top[0]) : 1.0f, f1 = up1 ? ex2(m[1] - top[1]) : 1.0f;
        m[0] = up0 ? top[0] : m[0];
        m[1] = up1 ? top[1] : m[1];
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int j = 0; j < ND; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
      }
      // a row that has seen nothing yet has only -inf scores; any finite reference gives it zero weights
      const float ref0 = m[0] == kNegInf ? 0.0f : m[0], ref1 = m[1] == kNegInf ? 0.0f : m[1];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sc[j][c] = ex2(sc[j][c] - ref0);
          sc[j][c + 2] = ex2(sc[j][c + 2] - ref1);
          if constexpr (C::kQuant) {
            l[0] = fmaf(sc[j][c], rv[j][c], l[0]);
            l[1] = fmaf(sc[j][c + 2], rv[j][c], l[1]);
          } else {
            l[0] += sc[j][c];
            l[1] += sc[j][c + 2];
          }
        }
      }

      // ---- weights times values
#pragma unroll
      for (int k = 0; k < C::kStep / 16; ++k) {
        const uint32_t pa[4] = {pack2<BF16>(sc[2 * k][0], sc[2 * k][1]), pack2<BF16>(sc[2 * k][2], sc[2 * k][3]),
                                pack2<BF16>(sc[2 * k + 1][0], sc[2 * k + 1][1]),
                                pack2<BF16>(sc[2 * k + 1][2], sc[2 * k + 1][3])};
        if constexpr (!C::kQuant) {
#pragma unroll
          for (int j = 0; j < ND; j += 2) {
            uint32_t r[4];
            const int row = 16 * k + (lane & 15);
            ldmatrix_x4_trans(vb + ring_offset<C::kRow>(row, j + (lane >> 4)), r);
            mma16816<BF16>(o[j], pa, r[0], r[1]);
            mma16816<BF16>(o[j + 1], pa, r[2], r[3]);
          }
        } else {
          // this lane's keys 2q, 2q + 1, 2q + 8, 2q + 9 of the sixteen, its D/8 values from (D/8) g on
          constexpr int VB = C::kRow / 8;  // bytes a lane takes of a row
          uint32_t w[4][VB / 4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = 16 * k + 2 * q + (x & 1) + 8 * (x >> 1);
            const int at = VB * g;
            const uint32_t addr = vb + ring_offset<C::kRow>(row, at >> 4) + (at & 15);
            if constexpr (VB == 16) {
              const uint4 v = lds128(addr);
              w[x][0] = v.x, w[x][1] = v.y, w[x][2] = v.z, w[x][3] = v.w;
            } else if constexpr (VB == 8) {
              const uint2 v = lds64(addr);
              w[x][0] = v.x, w[x][1] = v.y;
            } else {
              w[x][0] = lds32(addr);
            }
          }
#pragma unroll
          for (int y = 0; y < VB / 4; ++y) {
            if constexpr (FMT == kKvInt8) {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                // {a, b, a', b'} of two neighbouring values, then each pair widened
                const uint32_t lo = __byte_perm(w[0][y], w[1][y], z ? 0x7362 : 0x5140);
                const uint32_t hi = __byte_perm(w[2][y], w[3][y], z ? 0x7362 : 0x5140);
                mma16816<false>(o[4 * y + 2 * z], pa, bytes_to_h2(lo, 0x4140), bytes_to_h2(hi, 0x4140));
                mma16816<false>(o[4 * y + 2 * z + 1], pa, bytes_to_h2(lo, 0x4342), bytes_to_h2(hi, 0x4342));
              }
            } else {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                // four values of key a below the same four of key b
                const uint32_t lo = __byte_perm(w[0][y], w[1][y], z ? 0x7632 : 0x5410);
                const uint32_t hi = __byte_perm(w[2][y], w[3][y], z ? 0x7632 : 0x5410);
                mma16816<false>(o[8 * y + 4 * z], pa, nib_lo(lo), nib_lo(hi));
                mma16816<false>(o[8 * y + 4 * z + 1], pa, nib_hi(lo), nib_hi(hi));
                mma16816<false>(o[8 * y + 4 * z + 2], pa, nib_lo(lo >> 8), nib_lo(hi >> 8));
                mma16816<false>(o[8 * y + 4 * z + 3], pa, nib_hi(lo >> 8), nib_hi(hi >> 8));
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
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    __syncthreads();
    {
      float* wo = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);
      float2* wml = reinterpret_cast<float2*>(wo + kTokenRows * D);
#pragma unroll
      for (int j = 0; j < ND; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = 2 * q + (c & 1);
          const int d = C::kQuant ? (D / 8) * n + j : 8 * j + n;
          wo[(g + 8 * (c >> 1)) * D + d] = o[j][c];
        }
      if (q == 0) {
        wml[g] = make_float2(m[0], l[0]);
        wml[g + 8] = make_float2(m[1], l[1]);
      }
    }
    __syncthreads();
    {
      constexpr int PER = D / 8;
      const int r = threadIdx.x >> 3, part = threadIdx.x & 7;
      float2 ml[kWarps];
      float top = kNegInf, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = reinterpret_cast<const float2*>(smem + w * C::kWarpBytes + kTokenRows * D * 4)[r];
        top = fmaxf(top, ml[w].x);
      }
      float v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ml[w].x == kNegInf ? 0.0f : ex2(ml[w].x - top);
        sum = fmaf(ml[w].y, f, sum);
        const float4* wo = reinterpret_cast<const float4*>(smem + w * C::kWarpBytes + (r * D + part * PER) * 4);
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
          for (int st = 1; st < 8; st *= 2)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              const float x = __shfl_xor_sync(0xffffffffu, v[i], st);
              v[i] = ((part & st) ? x - v[i] : v[i] + x);
            }
#pragma unroll
          for (int i = 0; i < PER; ++i) v[i] *= 8.0f / D;
        }
        if (r < rows) {
          const int tok = r / group;
          uint16_t* dst = static_cast<uint16_t*>(a.out) + (s.q0 + tok) * a.out_token_stride +
                          (int64_t)(h * group + r - tok * group) * a.out_head_stride + part * PER;
#pragma unroll
          for (int i = 0; i < PER; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x = v[i + 2 * j] * inv, y = v[i + 2 * j + 1] * inv;
              w[j] = a.bf16 ? pack2<true>(x, y) : pack2<false>(x, y);
            }
            *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else if (r < rows) {
        // a range begins inside at most one item and ends inside at most one
        const int64_t slot = 2 * (int64_t)blockIdx.x + (unit0 == 0 ? 1 : 0);
        float4* dst = reinterpret_cast<float4*>(a.part_o + (slot * kTokenRows + r) * D + part * PER);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (part == 0) a.part_ml[slot * kTokenRows + r] = make_float2(top, sum);
      }
    }
    __syncthreads();  // the next item's copies refill what was read here
    u += unit1 - unit0;
    if (unit1 == s.units && h == a.kv_heads - 1) {
      before += (int64_t)s.units * a.kv_heads;
      ++b;
    }
  }
}

// Joins the parts of the items that were cut: one block an item and row, its
// warps take the parts in turn (all their loads in flight), then one joins the
// warps in order.  The order is fixed by the lengths, so results repeat.
constexpr int kJoinWarps = 4;
template <int D, bool QUANT>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_token_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 32;
  __shared__ float so[kJoinWarps][D];
  __shared__ float2 sml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.heads / a.kv_heads;
  const int r = blockIdx.y;
  // every block waits, cut item or not: the end of this grid then stands for the end of both
  pdl_wait();
  const int b = blockIdx.x / a.kv_heads, h = blockIdx.x % a.kv_heads;
  const Seq s = load_seq(a, b);
  const int rows = s.q_len * group;
  if (r >= rows) return;
  // units before this sequence, and of the call
  int64_t total = 0, before = 0;
  for (int i = lane; i < a.batch; i += 32) {
    const int n = load_seq(a, i).units;
    total += n;
    before += i < b ? n : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  total *= a.kv_heads;
  const int64_t first = before * a.kv_heads + (int64_t)h * s.units, last = first + s.units - 1;
  const int64_t grid = a.ctas;
  // the CTA of a unit is the last whose range begins at or before it
  const int64_t c0 = ((first + 1) * grid - 1) / total, c1 = ((last + 1) * grid - 1) / total;
  if (c0 == c1) return;  // not cut
  float m = kNegInf, l = 0.0f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.0f;
  for (int64_t c = c0 + warp; c <= c1; c += kJoinWarps) {
    const int64_t begin = total * c / grid, end = total * (c + 1) / grid;
    if (begin == end) continue;
    const int64_t slot = 2 * c + (begin <= first ? 1 : 0);
    const float2 ml = a.part_ml[slot * kTokenRows + r];
    float v[PER];
    const float* src = a.part_o + (slot * kTokenRows + r) * D + PER * lane;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = src[i];
    if (ml.x == kNegInf) continue;
    const float top = fmaxf(m, ml.x);
    const float f = m == kNegInf ? 0.0f : ex2(m - top), f1 = ex2(ml.x - top);
    l = l * f + ml.y * f1;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] * f + v[i] * f1;
    m = top;
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
    const float f = sml[w].x == kNegInf ? 0.0f : ex2(sml[w].x - top);
    sum = fmaf(sml[w].y, f, sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = fmaf(so[w][PER * lane + i], f, o[i]);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if constexpr (QUANT) {
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
  const int tok = r / group;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + (s.q0 + tok) * a.out_token_stride +
                  (int64_t)(h * group + r - tok * group) * a.out_head_stride + PER * lane;
#pragma unroll
  for (int i = 0; i < PER; i += 2) {
    const uint32_t w = a.bf16 ? pack2<true>(o[i] * inv, o[i + 1] * inv) : pack2<false>(o[i] * inv, o[i + 1] * inv);
    *reinterpret_cast<uint32_t*>(dst + i) = w;
  }
}

template <int FMT, int D>
cudaError_t launch_token(const AttnArgs& a, cudaStream_t stream) {
  using C = TokenCfg<FMT, D>;
  cudaError_t e = cudaFuncSetAttribute(attn_token_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  attn_token_kernel<FMT, D><<<(unsigned)a.ctas, kThreads, C::kSmem, stream>>>(a);
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

}  // namespace

cudaError_t launch_attn_token(const AttnArgs& a, cudaStream_t stream) {
#define EXL3_TOKEN(F)                                            \
  case F: return a.head_dim == 64 ? launch_token<F, 64>(a, stream) : launch_token<F, 128>(a, stream);
  switch (a.cache.format) {
    EXL3_TOKEN(kKvF16)
    EXL3_TOKEN(kKvBf16)
    EXL3_TOKEN(kKvInt8)
    EXL3_TOKEN(kKvInt4)
    default: return cudaErrorInvalidValue;
  }
#undef EXL3_TOKEN
}

}  // namespace exl3
