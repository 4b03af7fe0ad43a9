// exl3_attn.h -- internal: arguments and launchers of the rotary, cache and
// attention kernels (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/exl3.h"

namespace exl3 {

// Cache formats, numbered as exl3_kv_format_t.
enum KvFormat : int { kKvF16 = 0, kKvBf16 = 1, kKvInt8 = 2, kKvInt4 = 3 };
constexpr bool kv_quantised(int format) { return format >= kKvInt8; }
// Bytes of one cached row (one token, one head, key or value).
constexpr int kv_row_bytes(int format, int head_dim) {
  return format <= kKvBf16 ? 2 * head_dim : format == kKvInt8 ? head_dim : head_dim / 2;
}

// Heads of packed tokens: element (t, h, d) at data[t * token_stride + h * head_stride + d].
struct HeadsView {
  const void* data;
  int64_t token_stride, head_stride;
};

struct KvCache {
  uint8_t* k;
  uint8_t* v;
  uint16_t* k_scale;  // bf16, quantised formats only
  uint16_t* v_scale;
  int64_t num_pages;
  int page_shift;  // log2 of the page size
  int kv_heads, head_dim, format;
};

// Rotary positions; rot_dim 0: none.
struct RopeArgs {
  const uint64_t* phases;
  const int32_t* positions;
  int rot_dim, interleaved;
  float amplitude;
};

// Rotary rows to `out` (heads [0, rope_heads) of the call), then the key and
// value rows into the cache (kv_heads of each; 0 for a call without a cache).
struct RopeWriteArgs {
  HeadsView x;  // rows that are rotated into out
  void* out;
  int64_t out_token_stride, out_head_stride;
  int x_heads;
  HeadsView k, v;
  const int64_t* slots;
  KvCache cache;
  int kv_heads;
  int64_t tokens;
  RopeArgs rope;
  int bf16;
};
cudaError_t launch_rope_write(const RopeWriteArgs& a, int head_dim, cudaStream_t stream);

struct KvReadArgs {
  KvCache cache;
  const int64_t* slots;
  int64_t tokens;
  void* k;
  void* v;
  int bf16;  // type of k and v
};
cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t stream);

struct AttnArgs {
  HeadsView q, k, v;  // k, v: prompt attention only
  void* out;
  int64_t out_token_stride, out_head_stride;
  KvCache cache;          // paged attention only
  const int32_t* table;   // [batch][table_width] page ids
  int table_width;
  const int32_t* cu_q;    // [batch + 1]
  const int32_t* kv_lens; // [batch]; prompt attention: nullptr (the query lengths)
  int64_t total_q;
  int batch, heads, kv_heads, head_dim;
  int max_q;
  int window;             // 0: none
  float scale_log2;       // softmax scale * log2(e)
  int bf16;               // type of q and out
  int splits;             // parts of each item's keys (tile kernel)
  int tile_tokens;        // query tokens of a row tile (tile kernel)
  int ctas;               // grid of the token kernel
  float* part_o;
  float2* part_ml;
};
// Rows (query tokens x heads of a group) one item of the token kernel holds.
constexpr int kTokenRows = 16;
// CTAs of the token kernel an SM holds, by the rows it is compiled for (8 or 16).
constexpr int token_ctas_per_sm(int rows) { return rows <= 8 ? 3 : 2; }
// Keys per scheduling unit of the token kernel.
constexpr int kTokenUnit = 64;
// fp16 operands of the quantised formats are held in units of a power of two near their largest value.  Exponent field of
// the power at or below x, well inside fp32's range; 1's for a 0 and for what is not finite.
__device__ __forceinline__ uint32_t unit_exponent(float x) {
  const uint32_t e = __float_as_uint(x) >> 23 & 255u;
  return x == 0.0f || e == 255u ? 127u : e < 24u ? 24u : e > 230u ? 230u : e;
}
__device__ __forceinline__ float power(uint32_t e) { return __uint_as_float(e << 23); }  // 2^(e - 127)
// Few query rows a sequence (max_q * group <= kTokenRows) over a paged cache.
cudaError_t launch_attn_token(const AttnArgs& a, cudaStream_t stream);
// Rows of a row tile of the tile kernel: it holds kTileTokenRows / group whole query tokens.
constexpr int kTileTokenRows = 128;
// Query rows in row tiles, prompt (k, v) or paged.
cudaError_t launch_attn_tile(const AttnArgs& a, bool paged, cudaStream_t stream);
// Lets KERNEL use `bytes` of dynamic shared memory and, with regs > 0, checks that it was built for `regs` registers a
// thread: asked of the runtime once a kernel and device.
template <auto* KERNEL>
cudaError_t allow_smem(int bytes, int regs = 0) {
  static std::atomic<uint64_t> done{0};  // bit: device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1u)) return cudaSuccess;
  if (regs > 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, KERNEL);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != regs) return cudaErrorInvalidConfiguration;
  }
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return e;
}
// A CUDA result as a status; keeps an error's text for exl3_last_error.
exl3_status_t api_status(cudaError_t e, const char* where);
// Wait-timeout flag of the tile kernel's translation unit.
cudaError_t take_device_error_attn(uint32_t* flags);

}  // namespace exl3
