// exl3_rope_cache.cu -- rotary positions, and keys and values written into and
// read back from the paged cache.
//
// Rotation of the pair (a, b) at position p with frequency f:
//     (a cos t - b sin t, b cos t + a sin t),  t = p f.
// The frequency comes as a phase F, turns per position in units of 2^-64, so
// p * F modulo 2^64 (one integer multiply that wraps) is the angle's fraction of a turn,
// exact for every 32-bit position; its upper 32 bits, as a signed number, times
// pi / 2^31 is the angle in [-pi, pi), where cosf and sinf take their short
// path.  Products and sums round to fp32 one by one, then once to the type.
//
// Quantised cache rows: y = H_D(x) / 8 (H_D the D-point Hadamard transform in
// fp32 adds, strides 1, 2, 4, ...), scale = max|y| / top rounded up to bf16
// (top = 127 or 7), code = rint(y / scale).  The transform spreads a channel
// that stands out over the whole row, which is what lets one scale serve the
// row; and because H_D H_D = D, attention works on the rotated rows as they
// are (only q and the output are rotated).  Read back: H_D(codes) is a sum of
// integers below 2^24, exact in fp32 in any order, times scale * 8 / D.
//
// Bound by DRAM on long calls, by the launch on short ones (one token: 4.2 us).
// 16381 tokens of 32 query and 8 key heads of 128 in bf16: rotation of the 40
// heads 61 us (5540 GB/s), the same with keys and values written in 16 bits 67 us
// (6030 GB/s), in 8 and 4 bits 77 us (4800 and 4590 GB/s: the instructions of the
// transform count); keys and values alone, not rotated, 34 and 42 us.  So: a block
// takes one token, whose D/2 sines and cosines are computed once and stay in
// registers for all its query rows, of D/8 lanes each, a lane with both values of
// its pairs; keys and values have D/16 lanes a row, sums and differences two an
// instruction, a stage of the transform across lanes is a shuffle and a
// multiply-add by +-1, and codes come out of the low bits of a sum with 1.5 * 2^23.
// With D/8 lanes for keys and values too 81 us; four lanes a row need the fewest
// instructions, but 92 registers instead of 56, and the query rows that share the
// block want the occupancy: 100 us, and 98 to 125 with warps or blocks of their own
// for keys and values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "exl3_attn.h"

namespace exl3 {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeBlocks = 9;  // blocks an SM: 56 registers a thread (seven blocks of 72: 83 us for 79 below)
constexpr int kRopeBatch = 4;  // rows a lane group loads before it works on the first

__device__ __forceinline__ void unpack8(const uint4& w, bool bf16, float (&v)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8], bool bf16) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Two fp32 numbers an instruction.
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 mul2(const float2& a, const float2& b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
__device__ __forceinline__ void butterfly(float2& a, float2& b) {
  const float2 p = a;
  a = add2(p, b);
  b = fma2(b, twice(-1.0f), p);  // exact product: the difference, rounded once
}

__device__ __forceinline__ void unpack8(const uint4& w, bool bf16, float2* v) {
  float f[8];
  unpack8(w, bf16, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(f[2 * j], f[2 * j + 1]);
}
__device__ __forceinline__ uint4 pack8(const float2* v, bool bf16) {
  const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  return pack8(f, bf16);
}

// D-point Hadamard transform of a row held by D/16 neighbouring lanes, two
// chunks of eight consecutive values a lane: chunks l and l + D/16.  Strides in
// rising order (the sums round).
template <int D>
__device__ __forceinline__ void hadamard_lanes(float2 (&v)[8], int l) {
#pragma unroll
  for (int x = 0; x < 8; ++x) v[x] = make_float2(__fadd_rn(v[x].x, v[x].y), __fsub_rn(v[x].x, v[x].y));
#pragma unroll
  for (int s = 1; s < 4; s *= 2)
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (!(x & s)) butterfly(v[x], v[x + s]);
#pragma unroll
  for (int s = 1; s < D / 16; s *= 2) {
    const float2 sign = twice((l & s) != 0 ? -1.0f : 1.0f);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v[x].x, s), __shfl_xor_sync(0xffffffffu, v[x].y, s));
      v[x] = fma2(v[x], sign, o);  // exact product: the sum or the difference, rounded once
    }
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) butterfly(v[x], v[x + 4]);
}
// The same for a row held by four lanes, D/32 chunks of eight consecutive
// values a lane, of integers whose sums are exact: every bit of the place in a
// lane and of the lane is one stage, in any order.
template <int D>
__device__ __forceinline__ void hadamard_quads(float2 (&v)[D / 8], int l) {
  constexpr int C = D / 32;
#pragma unroll
  for (int x = 0; x < D / 8; ++x) v[x] = make_float2(__fadd_rn(v[x].x, v[x].y), __fsub_rn(v[x].x, v[x].y));
#pragma unroll
  for (int s = 1; s < 8; s *= 2)  // inside a chunk, then chunks 2 i and 2 i + 1
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
      if (!(x & s)) butterfly(v[x], v[x + s]);
#pragma unroll
  for (int s = 1; s < 4; s *= 2) {
    const float2 sign = twice((l & s) != 0 ? -1.0f : 1.0f);
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
      const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v[x].x, s), __shfl_xor_sync(0xffffffffu, v[x].y, s));
      v[x] = fma2(v[x], sign, o);
    }
  }
  if (C == 4) {
#pragma unroll
    for (int x = 0; x < D / 16; ++x) butterfly(v[x], v[x + D / 16]);
  }
}
// The larger magnitude, or NaN if either is.
__device__ __forceinline__ float max_mag(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(b)));
  return y;
}

// A row's values as hadamard_lanes takes them (all lanes of the warp come here)
// quantised into row `row` of a cache side; nothing is stored where `keep` is
// false.
template <int D>
__device__ __forceinline__ void quantise_row(float2 (&v)[8], int l, bool int8, uint8_t* dst, uint16_t* scales, int64_t row,
                                             bool keep) {
  hadamard_lanes<D>(v, l);
  float top = fabsf(v[0].x);
#pragma unroll
  for (int x = 0; x < 8; ++x) top = max_mag(max_mag(top, v[x].x), v[x].y);
#pragma unroll
  for (int s = 1; s < D / 16; s *= 2) top = max_mag(top, __shfl_xor_sync(0xffffffffu, top, s));
  const bool finite = top < __builtin_huge_valf();
  // y = v / 8: the eighth goes into the maximum and the reciprocal, exactly
  top *= 0.125f;
  float scale = __fmul_rn(top, int8 ? 1.0f / 127.0f : 1.0f / 7.0f);
  scale = __uint_as_float((__float_as_uint(scale) + 0xFFFFu) & 0xFFFF0000u);  // up, so that no code passes the top
  scale = fmaxf(scale, 7.888609052210118e-31f);                               // 2^-100: its reciprocal is finite
  if (top == 0.0f) scale = 1.0f;
  const float inv = __fdiv_rn(1.0f, scale) * 0.125f;
  // the product, rounded, plus 1.5 * 2^23 (and the offset): rounded to an integer in the low bits.  (One by one: a
  // product and a sum of pairs become one rounding, whatever they are told.)
  const float magic = int8 ? 12582912.0f + 128.0f : 12582912.0f + 8.0f;
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[2 * j] = __float_as_uint(__fadd_rn(__fmul_rn(v[4 * i + j].x, inv), magic));
      c[2 * j + 1] = __float_as_uint(__fadd_rn(__fmul_rn(v[4 * i + j].y, inv), magic));
    }
    lo[i] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    hi[i] = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
    if (!finite) lo[i] = hi[i] = int8 ? 0x80808080u : 0x08080808u;
  }
  if (!keep) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (int8) {
      *reinterpret_cast<uint2*>(dst + row * D + i * (D / 2) + 8 * l) = make_uint2(lo[i], hi[i]);
    } else {
      lo[i] &= 0x0F0F0F0Fu, hi[i] &= 0x0F0F0F0Fu;
      *reinterpret_cast<uint32_t*>(dst + row * (D / 2) + i * (D / 4) + 4 * l) =
          __byte_perm(lo[i] | lo[i] >> 4, hi[i] | hi[i] >> 4, 0x6420);
    }
  }
  // a row with a value that is not finite reads back as NaN
  if (l == 0) scales[row] = finite ? (uint16_t)(__float_as_uint(scale) >> 16) : (uint16_t)0x7FC0u;
}

// Rotation of the pair (a, b), products and sums rounded one by one.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float p = a, q = b;
  a = __fsub_rn(__fmul_rn(p, c), __fmul_rn(q, s));
  b = __fadd_rn(__fmul_rn(q, c), __fmul_rn(p, s));
}

// KV: there are keys and values
template <int D, bool KV>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_write_kernel(const RopeWriteArgs a, int units_per_block) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = kRopeThreads / LANES;
  constexpr int KLANES = D / 16;  // lanes of a key's or value's row, sixteen values each
  constexpr int KGROUPS = kRopeThreads / KLANES;
  __shared__ __align__(16) float cs[D / 2], sn[D / 2];
  const int64_t t = blockIdx.x;
  const int l = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  const bool bf16 = a.bf16 != 0;
  const int half = a.rope.rot_dim >> 1;
  const bool pairs = a.rope.interleaved != 0 || half == 0;  // a lane's eight values lie next to each other
  // where the row's values lie that this lane rotates: both of each pair
  const bool turns = 4 * l < half;
  const int at0 = !pairs && turns ? 4 * l : 8 * l;
  const int at1 = !pairs && turns ? half + 4 * l : 8 * l + 4;

  // this block's units: of x, GROUPS rows each, then of keys and values, KGROUPS rows each
  const int xu = (a.x_heads + GROUPS - 1) / GROUPS, ku = KV ? (2 * a.kv_heads + KGROUPS - 1) / KGROUPS : 0;
  const int u0 = blockIdx.y * units_per_block, u1 = min(xu + ku, u0 + units_per_block);

  const uint16_t* x = static_cast<const uint16_t*>(a.x.data) + t * a.x.token_stride;
  uint2 raw[kRopeBatch][2];
  auto load_x = [&](int u) {
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int r = (u + i) * GROUPS + group;
      raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
      if (u + i < min(xu, u1) && r < a.x_heads) {
        raw[i][0] = *reinterpret_cast<const uint2*>(x + (int64_t)r * a.x.head_stride + at0);
        raw[i][1] = *reinterpret_cast<const uint2*>(x + (int64_t)r * a.x.head_stride + at1);
      }
    }
  };
  load_x(u0);

  // where the keys and values go; nowhere for a negative or too large slot
  int64_t page = -1;
  int off = 0;
  if (KV) {
    const int64_t slot = a.slots[t];
    if (slot >= 0 && slot < (a.cache.num_pages << a.cache.page_shift)) {
      page = slot >> a.cache.page_shift;
      off = (int)(slot & ((1 << a.cache.page_shift) - 1));
    }
  }
  // the first keys and values are in flight too while the sines and cosines are computed
  const int ku0 = max(u0, xu), kl = threadIdx.x % KLANES;
  uint4 next[2];
  auto kv_row = [&](int u) { return (u - xu) * KGROUPS + (int)threadIdx.x / KLANES; };  // a key head, or kv_heads + a value head
  auto kv_src = [&](int r) {
    const bool isk = r < a.kv_heads;
    const HeadsView& src = isk ? a.k : a.v;
    return static_cast<const uint16_t*>(src.data) + t * src.token_stride + (int64_t)(isk ? r : r - a.kv_heads) * src.head_stride;
  };
  auto load_kv = [&](int u) {
    const int r = kv_row(u);
    next[0] = next[1] = make_uint4(0u, 0u, 0u, 0u);
    if (u >= u1 || r >= 2 * a.kv_heads) return;  // (the slot is still on its way)
    const uint16_t* src = kv_src(r);
    next[0] = *reinterpret_cast<const uint4*>(src + 8 * kl);
    next[1] = *reinterpret_cast<const uint4*>(src + D / 2 + 8 * kl);
  };
  if (KV) load_kv(ku0);

  if ((int)threadIdx.x < half) {
    const uint64_t turned = (uint64_t)(int64_t)a.rope.positions[t] * a.rope.phases[threadIdx.x];
    const float angle = __fmul_rn((float)(int32_t)(turned >> 32), 1.46291807926715968e-9f);  // pi / 2^31
    cs[threadIdx.x] = __fmul_rn(cosf(angle), a.rope.amplitude);
    sn[threadIdx.x] = __fmul_rn(sinf(angle), a.rope.amplitude);
  }
  __syncthreads();

  if (u0 < xu) {
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = turns ? cs[4 * l + j] : 1.0f, s[j] = turns ? sn[4 * l + j] : 0.0f;
    uint16_t* out = static_cast<uint16_t*>(a.out) + t * a.out_token_stride;
    for (int u = u0; u < min(xu, u1); u += kRopeBatch) {
      if (u > u0) load_x(u);
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i) {
        const int r = (u + i) * GROUPS + group;
        if (u + i >= min(xu, u1) || r >= a.x_heads) break;
        uint4 w = make_uint4(raw[i][0].x, raw[i][0].y, raw[i][1].x, raw[i][1].y);
        if (turns) {
          float v[8];
          unpack8(w, bf16, v);
          if (pairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) turn(v[2 * j], v[2 * j + 1], c[j], s[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) turn(v[j], v[4 + j], c[j], s[j]);
          }
          w = pack8(v, bf16);
        }
        *reinterpret_cast<uint2*>(out + (int64_t)r * a.out_head_stride + at0) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2*>(out + (int64_t)r * a.out_head_stride + at1) = make_uint2(w.z, w.w);
      }
    }
  }
  if constexpr (KV) {
    if (page < 0) return;  // alike in the whole block

    for (int u = ku0; u < u1; ++u) {
      uint4 w[2] = {next[0], next[1]};
      load_kv(u + 1);
      const int r = kv_row(u);
      const bool there = r < 2 * a.kv_heads, isk = r < a.kv_heads;
      if (isk && half > 0) {
        const int hl = half >> 3;  // chunks of one half
        const uint4 raw0 = w[0], raw1 = w[1];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ch = kl + KLANES * i;
          if (8 * ch >= 2 * half) continue;
          float2 v[4];
          unpack8(w[i], bf16, v);
          if (pairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) turn(v[j].x, v[j].y, cs[4 * ch + j], sn[4 * ch + j]);
          } else {
            // the other values of the pairs: this lane's own where the whole row turns, else read once more
            const bool upper = ch >= hl;
            const int f = 8 * (upper ? ch - hl : ch);
            float2 o[4];
            unpack8(hl == KLANES ? (i == 0 ? raw1 : raw0) : *reinterpret_cast<const uint4*>(kv_src(r) + 8 * (upper ? ch - hl : ch + hl)),
                    bf16, o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 c = *reinterpret_cast<const float2*>(cs + f + 2 * j);
              const float2 s = *reinterpret_cast<const float2*>(sn + f + 2 * j);
              // less a product is plus the product of the negated sine, to the bit
              v[j].x = __fadd_rn(__fmul_rn(v[j].x, c.x), __fmul_rn(o[j].x, upper ? s.x : -s.x));
              v[j].y = __fadd_rn(__fmul_rn(v[j].y, c.y), __fmul_rn(o[j].y, upper ? s.y : -s.y));
            }
          }
          w[i] = pack8(v, bf16);
        }
      }
      const int64_t row = there ? ((page * a.kv_heads + (isk ? r : r - a.kv_heads)) << a.cache.page_shift) + off : 0;
      uint8_t* dst = isk ? a.cache.k : a.cache.v;
      if (!kv_quantised(a.cache.format)) {
        if (there) {
          *reinterpret_cast<uint4*>(dst + row * (2 * D) + 16 * kl) = w[0];
          *reinterpret_cast<uint4*>(dst + row * (2 * D) + D + 16 * kl) = w[1];
        }
      } else {
        float2 v[8];
        unpack8(w[0], bf16, v);  // the row as its type holds it is what gets quantised
        unpack8(w[1], bf16, v + 4);
        quantise_row<D>(v, kl, a.cache.format == kKvInt8, dst, isk ? a.cache.k_scale : a.cache.v_scale, row, there);
      }
    }
  }
}

// Rows of whole tokens a block: keys, then values of each; four lanes a row,
// whose chunk i of lane l is chunk 4 i + l.  At 16381 tokens of 8 heads of 128
// 30 us in each format (4500 GB/s of 16-bit rows, 2830 of 4-bit ones): the chain
// slot, row, store of a block is what counts.  Sixteen lanes a row, as writing
// has them, took 40 (twice the shuffles and adds a row); two rows of four lanes
// in flight 32.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) kv_read_kernel(const KvReadArgs a, int tokens_per_block) {
  constexpr int C = D / 32;
  constexpr int GROUPS = kRopeThreads / 4;
  const int l = threadIdx.x & 3, group = threadIdx.x >> 2;
  const bool bf16 = a.bf16 != 0;
  const int kvh = a.cache.kv_heads;
  const int per = 2 * kvh;  // rows of a token
  const int64_t t0 = (int64_t)blockIdx.x * tokens_per_block;
  const int rows = (int)min((int64_t)tokens_per_block, a.tokens - t0) * per;
  const int64_t limit = a.cache.num_pages << a.cache.page_shift;
  const bool int8 = a.cache.format == kKvInt8, quant = kv_quantised(a.cache.format);
  for (int base = 0; base < rows; base += GROUPS) {
    const int r = base + group;
    const int tok = tokens_per_block == 1 ? 0 : r / per, which = r - tok * per;
    const bool isk = which < kvh;
    const int head = isk ? which : which - kvh;
    uint4 raw[C];
#pragma unroll
    for (int x = 0; x < C; ++x) raw[x] = make_uint4(0u, 0u, 0u, 0u);
    float scale = 0.0f;
    bool in = false;
    if (r < rows) {
      const int64_t slot = a.slots[t0 + tok];
      if (slot >= 0 && slot < limit) {
        in = true;
        const int64_t row = (((slot >> a.cache.page_shift) * kvh + head) << a.cache.page_shift) +
                            (slot & ((1 << a.cache.page_shift) - 1));
        const uint8_t* src = isk ? a.cache.k : a.cache.v;
#pragma unroll
        for (int x = 0; x < C; ++x) {
          const int ch = 4 * x + l;
          if (int8) {
            const uint2 c = *reinterpret_cast<const uint2*>(src + row * D + 8 * ch);
            raw[x].x = c.x;
            raw[x].y = c.y;
          } else if (quant) {
            raw[x].x = *reinterpret_cast<const uint32_t*>(src + row * (D / 2) + 4 * ch);
          } else {
            raw[x] = *reinterpret_cast<const uint4*>(src + row * (2 * D) + 16 * ch);
          }
        }
        if (quant) scale = __uint_as_float((uint32_t)(isk ? a.cache.k_scale : a.cache.v_scale)[row] << 16);
      }
    }
    if (quant) {
      // a code in the low byte of 2^23, less 2^23 and the offset
      float2 v[D / 8];
      const float2 less = twice(-8388608.0f - (int8 ? 128.0f : 8.0f));
#pragma unroll
      for (int x = 0; x < C; ++x) {
        auto code = [](uint32_t word, int byte) { return __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7540 + byte)); };
        const uint4& w = raw[x];
        if (int8) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            v[4 * x + j] = add2(make_float2(code(w.x, 2 * j), code(w.x, 2 * j + 1)), less);
            v[4 * x + 2 + j] = add2(make_float2(code(w.y, 2 * j), code(w.y, 2 * j + 1)), less);
          }
        } else {
          const uint32_t even = w.x & 0x0F0F0F0Fu, odd = w.x >> 4 & 0x0F0F0F0Fu;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * x + j] = add2(make_float2(code(even, j), code(odd, j)), less);
        }
      }
      hadamard_quads<D>(v, l);
      const float2 s = twice(__fmul_rn(scale, 8.0f / D));
#pragma unroll
      for (int x = 0; x < C; ++x) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * x + j] = mul2(v[4 * x + j], s);
        raw[x] = in ? pack8(v + 4 * x, bf16) : make_uint4(0u, 0u, 0u, 0u);
      }
    } else if ((a.cache.format == kKvBf16) != bf16) {
#pragma unroll
      for (int x = 0; x < C; ++x) {
        float2 v[4];
        unpack8(raw[x], a.cache.format == kKvBf16, v);
        raw[x] = pack8(v, bf16);
      }
    }
    if (r < rows) {
      uint16_t* out = static_cast<uint16_t*>(isk ? a.k : a.v) + ((t0 + tok) * kvh + head) * D;
#pragma unroll
      for (int x = 0; x < C; ++x) *reinterpret_cast<uint4*>(out + 8 * (4 * x + l)) = raw[x];
    }
  }
}

}  // namespace

cudaError_t launch_rope_write(const RopeWriteArgs& a, int head_dim, cudaStream_t stream) {
  const int groups = kRopeThreads / (head_dim / 8);
  const int units = (a.x_heads + groups - 1) / groups + (2 * a.kv_heads + 2 * groups - 1) / (2 * groups);
  // one block a token, or, while that leaves SMs idle, a token's rows over several blocks
  const int per = a.tokens >= 152 * 4 ? units : a.tokens >= 152 ? (units < kRopeBatch ? units : kRopeBatch) : 1;
  const dim3 grid((unsigned)a.tokens, (unsigned)((units + per - 1) / per));
  auto kernel = head_dim == 64 ? (a.kv_heads > 0 ? rope_write_kernel<64, true> : rope_write_kernel<64, false>)
                               : (a.kv_heads > 0 ? rope_write_kernel<128, true> : rope_write_kernel<128, false>);
  kernel<<<grid, kRopeThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t stream) {
  const int groups = kRopeThreads / 4;
  const int64_t per = 2 * a.cache.kv_heads;
  const int64_t tokens = per < groups ? groups / per : 1;  // one pass a block
  const unsigned blocks = (unsigned)((a.tokens + tokens - 1) / tokens);
  if (a.cache.head_dim == 64)
    kv_read_kernel<64><<<blocks, kRopeThreads, 0, stream>>>(a, (int)tokens);
  else
    kv_read_kernel<128><<<blocks, kRopeThreads, 0, stream>>>(a, (int)tokens);
  return cudaGetLastError();
}

}  // namespace exl3
