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
// Bound by DRAM on long calls, by the launch on short ones.  D/8 lanes hold a
// row (one 16-byte load each), a block one token: its D/2 sines and cosines are
// computed once and shared by all its heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "exl3_attn.h"

namespace exl3 {
namespace {

constexpr int kRopeThreads = 128;
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

// D-point Hadamard transform of a row held as eight consecutive values a lane
// by D/8 neighbouring lanes.
template <int D>
__device__ __forceinline__ void hadamard_lanes(float (&v)[8], int lane) {
#pragma unroll
  for (int s = 1; s < 8; s *= 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!(i & s)) {
        const float p = v[i], q = v[i + s];
        v[i] = p + q;
        v[i + s] = p - q;
      }
    }
  }
#pragma unroll
  for (int s = 1; s < D / 8; s *= 2) {
    const bool upper = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, v[i], s);
      v[i] = upper ? o - v[i] : v[i] + o;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeWriteArgs a, int rows_per_block) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = kRopeThreads / LANES;
  __shared__ __align__(16) float cs[D / 2], sn[D / 2];
  const int64_t t = blockIdx.x;
  const int l = threadIdx.x % LANES;
  const int group = threadIdx.x / LANES;
  const bool bf16 = a.bf16 != 0;
  const int half = a.rope.rot_dim >> 1;
  const int rows = a.x_heads + 2 * a.kv_heads;
  const int row0 = blockIdx.y * rows_per_block;
  const int row1 = min(rows, row0 + rows_per_block);

  // where the row's key or value goes; nowhere for a negative or too large slot
  int64_t page = -1;
  int off = 0;
  if (a.kv_heads > 0) {
    const int64_t slot = a.slots[t];
    if (slot >= 0 && slot < (a.cache.num_pages << a.cache.page_shift)) {
      page = slot >> a.cache.page_shift;
      off = (int)(slot & ((1 << a.cache.page_shift) - 1));
    }
  }

  bool table = half == 0;  // whether the block's sines and cosines are there
  for (int base = row0; base < row1; base += GROUPS * kRopeBatch) {
    uint4 raw[kRopeBatch];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int r = base + i * GROUPS + group;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < row1) {
        const bool isx = r < a.x_heads;
        const bool isk = r < a.x_heads + a.kv_heads;
        const HeadsView& src = isx ? a.x : isk ? a.k : a.v;
        const int h = isx ? r : isk ? r - a.x_heads : r - a.x_heads - a.kv_heads;
        raw[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src.data) + t * src.token_stride +
                                                 h * src.head_stride + 8 * l);
      }
    }
    if (!table) {
      // the loads above are in flight while these are computed
      if ((int)threadIdx.x < half) {
        const uint64_t turn = (uint64_t)(int64_t)a.rope.positions[t] * a.rope.phases[threadIdx.x];
        const float angle = __fmul_rn((float)(int32_t)(turn >> 32), 1.46291807926715968e-9f);  // pi / 2^31
        cs[threadIdx.x] = __fmul_rn(cosf(angle), a.rope.amplitude);
        sn[threadIdx.x] = __fmul_rn(sinf(angle), a.rope.amplitude);
      }
      __syncthreads();
      table = true;
    }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int r = base + i * GROUPS + group;
      if (base + i * GROUPS >= row1) break;  // alike in the whole block
      const bool there = r < row1;
      const bool isx = r < a.x_heads;
      const bool isk = !isx && r < a.x_heads + a.kv_heads;
      float v[8];
      unpack8(raw[i], bf16, v);
      if (half > 0) {
        // a key or query row's first 2 * half values turn
        const bool turns = (isx || isk) && 8 * l < 2 * half;
        if (a.rope.interleaved) {
          if (turns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float c = cs[4 * l + j], s = sn[4 * l + j];
              const float p = v[2 * j], q = v[2 * j + 1];
              v[2 * j] = __fsub_rn(__fmul_rn(p, c), __fmul_rn(q, s));
              v[2 * j + 1] = __fadd_rn(__fmul_rn(q, c), __fmul_rn(p, s));
            }
          }
        } else {
          const int hl = half >> 3;  // lanes of one half
          const bool upper = l >= hl;
          const int lane = threadIdx.x & 31;
          const int partner = turns ? (upper ? lane - hl : lane + hl) : lane;
          const int f = 8 * (upper ? l - hl : l);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float o = __shfl_sync(0xffffffffu, v[j], partner);
            if (turns) {
              const float c = cs[f + j], s = sn[f + j];
              v[j] = upper ? __fadd_rn(__fmul_rn(v[j], c), __fmul_rn(o, s))
                           : __fsub_rn(__fmul_rn(v[j], c), __fmul_rn(o, s));
            }
          }
        }
      }
      // a row that does not turn keeps its bits (a NaN's too)
      const uint4 packed = half > 0 && (isx || isk) ? pack8(v, bf16) : raw[i];
      if (there && isx) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + t * a.out_token_stride + r * a.out_head_stride +
                                  8 * l) = packed;
      }
      const bool keep = there && !isx && page >= 0;
      if (!__any_sync(0xffffffffu, keep)) continue;
      const int h = r - a.x_heads - (isk ? 0 : a.kv_heads);
      const int64_t row = keep ? ((page * a.kv_heads + h) << a.cache.page_shift) + off : 0;
      uint8_t* dst = isk ? a.cache.k : a.cache.v;
      if (!kv_quantised(a.cache.format)) {
        if (keep) *reinterpret_cast<uint4*>(dst + row * (2 * D) + 16 * l) = packed;
        continue;
      }
      unpack8(packed, bf16, v);  // the row as its type holds it is what gets quantised
      hadamard_lanes<D>(v, threadIdx.x);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = __fmul_rn(v[j], 0.125f);
        top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      }
#pragma unroll
      for (int s = 1; s < LANES; s *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
      const bool int8 = a.cache.format == kKvInt8;
      const float most = int8 ? 127.0f : 7.0f;
      float scale = __fmul_rn(__uint_as_float(top), int8 ? 1.0f / 127.0f : 1.0f / 7.0f);
      scale = __uint_as_float((__float_as_uint(scale) + 0xFFFFu) & 0xFFFF0000u);  // up, so that no code passes the top
      scale = fmaxf(scale, 7.888609052210118e-31f);                               // 2^-100: its reciprocal is finite
      if (top == 0u) scale = 1.0f;
      const bool finite = top < 0x7F800000u;
      const float inv = __fdiv_rn(1.0f, scale);
      uint32_t code[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = fminf(fmaxf(rintf(__fmul_rn(v[j], inv)), -most), most);
        code[j] = (uint32_t)((finite ? (int)c : 0) + (int8 ? 128 : 8));
      }
      if (keep) {
        if (int8) {
          uint2 w;
          w.x = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
          w.y = code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24;
          *reinterpret_cast<uint2*>(dst + row * D + 8 * l) = w;
        } else {
          uint32_t w = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) w |= code[j] << (4 * j);
          *reinterpret_cast<uint32_t*>(dst + row * (D / 2) + 4 * l) = w;
        }
        // a row with a value that is not finite reads back as NaN
        if (l == 0)
          (isk ? a.cache.k_scale : a.cache.v_scale)[row] =
              finite ? (uint16_t)(__float_as_uint(scale) >> 16) : (uint16_t)0x7FC0u;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) kv_read_kernel(const KvReadArgs a) {
  constexpr int LANES = D / 8;
  const int l = threadIdx.x % LANES;
  const bool bf16 = a.bf16 != 0;
  const int kvh = a.cache.kv_heads;
  const int per = 2 * kvh;  // rows of a token: its keys, then its values
  const int64_t rows = a.tokens * per;
  const int64_t groups = (int64_t)gridDim.x * (kRopeThreads / LANES);
  const int64_t limit = a.cache.num_pages << a.cache.page_shift;
  const int64_t first = (int64_t)blockIdx.x * (kRopeThreads / LANES);  // a whole block takes the same passes
  for (int64_t base = first; base < rows; base += groups * kRopeBatch) {
    uint4 raw[kRopeBatch];
    float scale[kRopeBatch];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int64_t r = base + i * groups + threadIdx.x / LANES;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      scale[i] = -1.0f;  // no row: zeros
      if (r < rows) {
        const int64_t t = r / per;
        const int w = (int)(r - t * per);
        const int64_t slot = a.slots[t];
        if (slot >= 0 && slot < limit) {
          const int h = w < kvh ? w : w - kvh;
          const int64_t row = (((slot >> a.cache.page_shift) * kvh + h) << a.cache.page_shift) +
                              (slot & ((1 << a.cache.page_shift) - 1));
          const uint8_t* src = w < kvh ? a.cache.k : a.cache.v;
          if (a.cache.format == kKvInt8) {
            const uint2 c = *reinterpret_cast<const uint2*>(src + row * D + 8 * l);
            raw[i].x = c.x;
            raw[i].y = c.y;
          } else if (a.cache.format == kKvInt4) {
            raw[i].x = *reinterpret_cast<const uint32_t*>(src + row * (D / 2) + 4 * l);
          } else {
            raw[i] = *reinterpret_cast<const uint4*>(src + row * (2 * D) + 16 * l);
          }
          scale[i] = 1.0f;
          if (kv_quantised(a.cache.format))
            scale[i] = __uint_as_float((uint32_t)(w < kvh ? a.cache.k_scale : a.cache.v_scale)[row] << 16);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (base + i * groups >= rows) break;  // alike in the whole block
      const int64_t r = base + i * groups + threadIdx.x / LANES;
      float v[8];
      const bool none = scale[i] == -1.0f;
      if (kv_quantised(a.cache.format)) {
        const bool int8 = a.cache.format == kKvInt8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t c = int8 ? ((j < 4 ? raw[i].x : raw[i].y) >> (8 * (j & 3))) & 255u : (raw[i].x >> (4 * j)) & 15u;
          v[j] = (float)((int)c - (int8 ? 128 : 8));
        }
        hadamard_lanes<D>(v, threadIdx.x);
        const float s = __fmul_rn(scale[i], 8.0f / D);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = none ? 0.0f : __fmul_rn(v[j], s);
      } else {
        unpack8(raw[i], a.cache.format == kKvBf16, v);
      }
      if (r < rows) {
        const int64_t t = r / per;
        const int w = (int)(r - t * per);
        const int h = w < kvh ? w : w - kvh;
        uint16_t* out = static_cast<uint16_t*>(w < kvh ? a.k : a.v);
        *reinterpret_cast<uint4*>(out + (t * kvh + h) * D + 8 * l) = pack8(v, bf16);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_write(const RopeWriteArgs& a, int head_dim, cudaStream_t stream) {
  const int groups = kRopeThreads / (head_dim / 8);
  const int rows = a.x_heads + 2 * a.kv_heads;
  // one block a token, or, while that leaves SMs idle, a token's rows over several blocks
  int per = groups * kRopeBatch;
  if (a.tokens >= 152 * 4) per = (rows + per - 1) / per * per;
  else if (a.tokens < 152) per = groups;
  const dim3 grid((unsigned)a.tokens, (unsigned)((rows + per - 1) / per));
  if (head_dim == 64)
    rope_write_kernel<64><<<grid, kRopeThreads, 0, stream>>>(a, per);
  else
    rope_write_kernel<128><<<grid, kRopeThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t stream) {
  const int groups = kRopeThreads / (a.cache.head_dim / 8);
  const int64_t rows = a.tokens * a.cache.kv_heads * 2;
  int64_t blocks = (rows + groups - 1) / groups;
  if (blocks > 152 * 16) blocks = (rows + groups * kRopeBatch - 1) / (groups * kRopeBatch);
  if (blocks > (1 << 30)) blocks = 1 << 30;
  if (a.cache.head_dim == 64)
    kv_read_kernel<64><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(a);
  else
    kv_read_kernel<128><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace exl3
