// exl3_attn_api.cu -- the rotary, cache and attention calls of include/exl3.h:
// host-side validation, the split policy and dispatch to the kernels.
#include <math.h>

#include "exl3_attn.h"

namespace {

constexpr int64_t kSms = 152;

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(int d) { return d == EXL3_F16 || d == EXL3_BF16; }
bool valid_rows(int64_t n) { return n >= 0 && n <= EXL3_MAX_ROWS; }
bool valid_strides(int64_t token, int64_t head) {
  constexpr int64_t kMost = int64_t(1) << 32;  // byte strides stay below what a tensor map takes
  return token > 0 && head > 0 && token % 8 == 0 && head % 8 == 0 && token < kMost && head < kMost;
}
bool valid_heads(const exl3_heads_t* h) {
  return h != nullptr && aligned16(h->data) && valid_strides(h->token_stride, h->head_stride);
}
// An output of rows like x's: aligned, and where it is x itself, element by element.
bool valid_out(const exl3_heads_t* x, const void* out, int64_t token, int64_t head) {
  return aligned16(out) && (out != x->data || (token == x->token_stride && head == x->head_stride));
}
// No sequence is longer than 2^30 keys, so a window of that size is none; the kernels subtract smaller ones from positions,
// which may be negative, in 32 bits.
int kernel_window(int32_t window) { return window >= (1 << 30) ? 0 : window; }
// A group's query heads are rows of one tile.
bool valid_head_counts(int32_t q_heads, int32_t kv_heads) {
  return kv_heads >= 1 && q_heads >= 1 && q_heads % kv_heads == 0 && q_heads / kv_heads <= 128 && q_heads <= 65536;
}
exl3_status_t check_head_dim(int32_t d) {
  if (d < 1) return EXL3_EINVAL;
  return d == 64 || d == 128 ? EXL3_OK : EXL3_EUNSUPPORTED;
}
exl3::HeadsView view(const exl3_heads_t* h) { return {h->data, h->token_stride, h->head_stride}; }

exl3_status_t check_rope(const exl3_rope_t* r, int32_t head_dim, int64_t tokens, exl3::RopeArgs* out) {
  if (r == nullptr || r->rot_dim < 16 || r->rot_dim % 16 != 0 || r->rot_dim > head_dim) return EXL3_EINVAL;
  if (r->layout != EXL3_ROPE_HALF && r->layout != EXL3_ROPE_INTERLEAVED) return EXL3_EINVAL;
  if (!isfinite(r->amplitude)) return EXL3_EINVAL;
  if (r->phases == nullptr || (reinterpret_cast<uintptr_t>(r->phases) & 7u) != 0) return EXL3_EINVAL;
  if (tokens > 0 && (r->positions == nullptr || (reinterpret_cast<uintptr_t>(r->positions) & 3u) != 0)) return EXL3_EINVAL;
  *out = {r->phases, r->positions, r->rot_dim, r->layout == EXL3_ROPE_INTERLEAVED ? 1 : 0, r->amplitude};
  return EXL3_OK;
}

exl3_status_t check_cache(const exl3_kv_cache_t* c, exl3::KvCache* out) {
  if (c == nullptr || c->format < EXL3_KV_F16 || c->format > EXL3_KV_INT4) return EXL3_EINVAL;
  if (c->kv_heads < 1 || c->kv_heads > 65536 || c->num_pages < 1 || c->num_pages >= (int64_t(1) << 31)) return EXL3_EINVAL;
  int shift = 4;
  while (shift < 8 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size) return EXL3_EINVAL;
  const exl3_status_t st = check_head_dim(c->head_dim);
  if (st != EXL3_OK) return st;
  // cache rows (and one past the last) are coordinates of a tensor map
  if (((c->num_pages * c->kv_heads) << shift) >= (int64_t(1) << 31)) return EXL3_EINVAL;
  if (!aligned16(c->k) || !aligned16(c->v)) return EXL3_EINVAL;
  if (exl3::kv_quantised(c->format) && (!aligned16(c->k_scale) || !aligned16(c->v_scale))) return EXL3_EINVAL;
  *out = {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale, c->num_pages,
          shift, c->kv_heads, c->head_dim, (int)c->format};
  return EXL3_OK;
}
// A 16-bit cache holds rows of one type only.
bool format_fits(int format, exl3_dtype_t dtype) {
  return exl3::kv_quantised(format) || (format == EXL3_KV_BF16) == (dtype == EXL3_BF16);
}

// How a paged call is split: by the token kernel (few rows a sequence) over
// equal ranges of all keys, else by row tiles and parts of their keys.
struct PagedPlan {
  bool token;
  int ctas, splits;
  size_t o_bytes, ml_bytes;
};
PagedPlan paged_plan(int64_t total_q, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_q,
                     int64_t max_kv, int64_t window) {
  PagedPlan p = {};
  const int64_t group = q_heads / kv_heads;
  p.splits = 1;
  p.token = max_q * group <= exl3::kTokenRows;
  if (p.token) {
    // as many CTAs as the SMs hold, but at least two units of keys each
    const int64_t pairs = batch * kv_heads * ((max_kv + 2 * exl3::kTokenUnit - 1) / (2 * exl3::kTokenUnit) + 1);
    const int64_t most = kSms * exl3::token_ctas_per_sm((int)(max_q * group));
    p.ctas = (int)(pairs < most ? pairs : most);
    p.o_bytes = (size_t)2 * p.ctas * exl3::kTokenRows * head_dim * sizeof(float);
    p.ml_bytes = (size_t)2 * p.ctas * exl3::kTokenRows * 2 * sizeof(float);
    return p;
  }
  // Row tiles, two an item.  The keys of each item may go to several CTAs: the number of parts is the one that a simple
  // model of the time likes best, waves of items, each as long as its blocks of 64 keys (about 0.85 us each) and the
  // beginning and end of an item (about 4 us), and what the parts cost to write and join.  512 tokens of 32 heads over
  // 32768 keys of 8: 232, 234, 218 and 230 us in 2, 4, 7 and 9 parts, 230, 238, 217 and 232 by the model.
  const int64_t per = 2 * (exl3::kTileTokenRows / group);
  const int64_t tiles = batch == 1 ? (total_q + per - 1) / per : total_q / per + (total_q < batch ? total_q : batch);
  const int64_t items = tiles * kv_heads;
  const int64_t seen = window > 0 && window + per < max_kv ? window + per : max_kv;  // keys of an item
  const double blocks = (double)(seen > 64 ? seen : 64) / 64.0;
  double best = 0.0;
  int64_t splits = 1;
  for (int64_t s = 1; s <= 16 && blocks / s >= 8.0 && (s == 1 || items <= kSms); ++s) {
    const double waves = (double)((items * s + kSms - 1) / kSms);
    const double join = s > 1 ? 4.0 + (double)s * total_q * q_heads * head_dim * 8.0 / 8.0e6 : 0.0;
    const double us = waves * (blocks / s * 0.85 + 4.0) + join;
    if (s == 1 || us < 0.97 * best) {
      best = us;
      splits = s;
    }
  }
  if (splits > 1) {
    p.splits = (int)splits;
    p.o_bytes = (size_t)splits * total_q * q_heads * head_dim * sizeof(float);
    p.ml_bytes = (size_t)splits * total_q * q_heads * 2 * sizeof(float);
  }
  return p;
}

}  // namespace

extern "C" {

exl3_status_t exl3_rope_phases(int32_t rot_dim, double base, exl3_rope_scaling_t scaling, double factor, double fast,
                               double slow, double original_len, uint64_t* phases, float* amplitude) {
  if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !isfinite(base) || phases == nullptr || amplitude == nullptr) return EXL3_EINVAL;
  if (scaling < EXL3_ROPE_PLAIN || scaling > EXL3_ROPE_YARN) return EXL3_EINVAL;
  if (scaling != EXL3_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return EXL3_EINVAL;
  if (scaling == EXL3_ROPE_NTK && rot_dim < 4) return EXL3_EINVAL;
  if (scaling == EXL3_ROPE_YARN && (!(slow > 0.0) || !(fast > slow) || !isfinite(fast) || !(original_len > 0.0) || !isfinite(original_len))) return EXL3_EINVAL;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (scaling == EXL3_ROPE_NTK) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == EXL3_ROPE_LINEAR) f /= factor;
    if (scaling == EXL3_ROPE_YARN) {
      const double turns = original_len * f / kTwoPi;
      double g = (turns - slow) / (fast - slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f *= g + (1.0 - g) / factor;
    }
    phases[i] = (uint64_t)(f / kTwoPi * 18446744073709551616.0);  // f <= 1: below 2^62
  }
  *amplitude = scaling == EXL3_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return EXL3_OK;
}

exl3_status_t exl3_rope(const exl3_heads_t* x, exl3_dtype_t dtype, int64_t tokens, int32_t heads, int32_t head_dim,
                        const exl3_rope_t* rope, void* out, int64_t out_token_stride, int64_t out_head_stride,
                        void* stream) {
  if (!valid_rows(tokens) || heads < 1 || heads > 65536 || !valid_dtype(dtype)) return EXL3_EINVAL;
  exl3_status_t st = check_head_dim(head_dim);
  if (st != EXL3_OK) return st;
  exl3::RopeWriteArgs a = {};
  st = check_rope(rope, head_dim, tokens, &a.rope);
  if (st != EXL3_OK) return st;
  if (!valid_strides(out_token_stride, out_head_stride)) return EXL3_EINVAL;
  if (tokens == 0) return EXL3_OK;
  if (!valid_heads(x) || !valid_out(x, out, out_token_stride, out_head_stride)) return EXL3_EINVAL;
  a.x = view(x);
  a.x_heads = heads;
  a.out = out;
  a.out_token_stride = out_token_stride;
  a.out_head_stride = out_head_stride;
  a.tokens = tokens;
  a.bf16 = dtype == EXL3_BF16;
  return exl3::api_status(exl3::launch_rope_write(a, head_dim, static_cast<cudaStream_t>(stream)), "exl3_rope");
}

exl3_status_t exl3_kv_write(const exl3_kv_cache_t* cache, const exl3_heads_t* k, const exl3_heads_t* v,
                            exl3_dtype_t dtype, int64_t tokens, const int64_t* slots, const exl3_rope_t* rope,
                            const exl3_heads_t* q, int32_t q_heads, void* q_out, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, void* stream) {
  if (!valid_rows(tokens) || !valid_dtype(dtype) || q_heads < 0 || q_heads > 65536) return EXL3_EINVAL;
  exl3::RopeWriteArgs a = {};
  exl3_status_t st = check_cache(cache, &a.cache);
  if (st != EXL3_OK) return st;
  if (!format_fits(a.cache.format, dtype)) return EXL3_EINVAL;
  if (rope != nullptr) {
    st = check_rope(rope, a.cache.head_dim, tokens, &a.rope);
    if (st != EXL3_OK) return st;
  } else if (q_heads != 0) {
    return EXL3_EINVAL;
  }
  if (q_heads > 0 && !valid_strides(q_out_token_stride, q_out_head_stride)) return EXL3_EINVAL;
  if (tokens == 0) return EXL3_OK;
  if (!valid_heads(k) || !valid_heads(v)) return EXL3_EINVAL;
  if (slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return EXL3_EINVAL;
  if (q_heads > 0) {
    if (!valid_heads(q) || !valid_out(q, q_out, q_out_token_stride, q_out_head_stride)) return EXL3_EINVAL;
    a.x = view(q);
    a.out = q_out;
    a.out_token_stride = q_out_token_stride;
    a.out_head_stride = q_out_head_stride;
  }
  a.x_heads = q_heads;
  a.k = view(k);
  a.v = view(v);
  a.slots = slots;
  a.kv_heads = a.cache.kv_heads;
  a.tokens = tokens;
  a.bf16 = dtype == EXL3_BF16;
  return exl3::api_status(exl3::launch_rope_write(a, a.cache.head_dim, static_cast<cudaStream_t>(stream)), "exl3_kv_write");
}

exl3_status_t exl3_kv_read(const exl3_kv_cache_t* cache, const int64_t* slots, int64_t tokens, exl3_dtype_t dtype,
                           void* k, void* v, void* stream) {
  if (!valid_rows(tokens) || !valid_dtype(dtype)) return EXL3_EINVAL;
  exl3::KvReadArgs a = {};
  const exl3_status_t st = check_cache(cache, &a.cache);
  if (st != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  if (slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0 || !aligned16(k) || !aligned16(v)) return EXL3_EINVAL;
  a.slots = slots;
  a.tokens = tokens;
  a.k = k;
  a.v = v;
  a.bf16 = dtype == EXL3_BF16;
  return exl3::api_status(exl3::launch_kv_read(a, static_cast<cudaStream_t>(stream)), "exl3_kv_read");
}

exl3_status_t exl3_attention_prompt(const exl3_heads_t* q, const exl3_heads_t* k, const exl3_heads_t* v,
                                    exl3_dtype_t dtype, int64_t total, int32_t q_heads, int32_t kv_heads,
                                    int32_t head_dim, const int32_t* cu_seqlens, int32_t batch, int32_t window,
                                    float scale, void* out, int64_t out_token_stride, int64_t out_head_stride,
                                    void* stream) {
  if (!valid_rows(total) || !valid_rows(batch) || !valid_dtype(dtype) || !valid_head_counts(q_heads, kv_heads)) return EXL3_EINVAL;
  const exl3_status_t st = check_head_dim(head_dim);
  if (st != EXL3_OK) return st;
  if (window < 0 || !(scale > 0.0f) || !isfinite(scale) || !valid_strides(out_token_stride, out_head_stride)) return EXL3_EINVAL;
  if (total == 0 || batch == 0) return EXL3_OK;
  if (!valid_heads(q) || !valid_heads(k) || !valid_heads(v) || !valid_out(q, out, out_token_stride, out_head_stride)) return EXL3_EINVAL;
  if (cu_seqlens == nullptr || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return EXL3_EINVAL;
  exl3::AttnArgs a = {};
  a.q = view(q);
  a.k = view(k);
  a.v = view(v);
  a.out = out;
  a.out_token_stride = out_token_stride;
  a.out_head_stride = out_head_stride;
  a.cu_q = cu_seqlens;
  a.total_q = total;
  a.batch = batch;
  a.heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.window = kernel_window(window);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.bf16 = dtype == EXL3_BF16;
  a.splits = 1;
  a.tile_tokens = exl3::kTileTokenRows / (q_heads / kv_heads);
  return exl3::api_status(exl3::launch_attn_tile(a, false, static_cast<cudaStream_t>(stream)), "exl3_attention_prompt");
}

size_t exl3_attention_paged_workspace_bytes(int64_t total_q, int32_t batch, int32_t q_heads, int32_t kv_heads,
                                            int32_t head_dim, int32_t max_q, int32_t max_kv, int32_t window) {
  if (!valid_rows(total_q) || !valid_rows(batch) || !valid_head_counts(q_heads, kv_heads)) return 0;
  if (check_head_dim(head_dim) != EXL3_OK || max_q < 1 || max_kv < 0 || window < 0 || total_q == 0 || batch == 0) return 0;
  const PagedPlan p = paged_plan(total_q, batch, q_heads, kv_heads, head_dim, max_q, max_kv, window);
  return p.o_bytes + p.ml_bytes;
}

exl3_status_t exl3_attention_paged(const exl3_heads_t* q, exl3_dtype_t dtype, int64_t total_q, int32_t q_heads,
                                   const exl3_kv_cache_t* cache, const int32_t* block_table, int32_t table_width,
                                   const int32_t* cu_q, const int32_t* kv_lens, int32_t batch, int32_t max_q,
                                   int32_t max_kv, int32_t window, float scale, void* out, int64_t out_token_stride,
                                   int64_t out_head_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_rows(total_q) || !valid_rows(batch) || !valid_dtype(dtype)) return EXL3_EINVAL;
  exl3::AttnArgs a = {};
  const exl3_status_t st = check_cache(cache, &a.cache);
  if (st != EXL3_OK) return st;
  if (!valid_head_counts(q_heads, a.cache.kv_heads) || !format_fits(a.cache.format, dtype)) return EXL3_EINVAL;
  if (table_width < 1 || ((int64_t)table_width << a.cache.page_shift) > (int64_t(1) << 30)) return EXL3_EINVAL;
  if (max_q < 1 || max_kv < 0 || window < 0 || !(scale > 0.0f) || !isfinite(scale)) return EXL3_EINVAL;
  if (!valid_strides(out_token_stride, out_head_stride)) return EXL3_EINVAL;
  if (total_q == 0 || batch == 0) return EXL3_OK;
  if (!valid_heads(q) || !valid_out(q, out, out_token_stride, out_head_stride)) return EXL3_EINVAL;
  const void* ints[3] = {block_table, cu_q, kv_lens};
  for (const void* p : ints)
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0) return EXL3_EINVAL;
  const PagedPlan plan = paged_plan(total_q, batch, q_heads, a.cache.kv_heads, a.cache.head_dim, max_q, max_kv, window);
  if (plan.token && (int64_t)batch * a.cache.kv_heads > INT32_MAX) return EXL3_EUNSUPPORTED;  // blocks of the join
  if (plan.o_bytes > 0 && !aligned16(workspace)) return EXL3_EINVAL;
  if (workspace_bytes < plan.o_bytes + plan.ml_bytes) return EXL3_EWORKSPACE;
  a.q = view(q);
  a.out = out;
  a.out_token_stride = out_token_stride;
  a.out_head_stride = out_head_stride;
  a.table = block_table;
  a.table_width = table_width;
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.total_q = total_q;
  a.batch = batch;
  a.heads = q_heads;
  a.kv_heads = a.cache.kv_heads;
  a.head_dim = a.cache.head_dim;
  a.max_q = max_q;
  a.window = kernel_window(window);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.bf16 = dtype == EXL3_BF16;
  a.splits = plan.splits;
  a.tile_tokens = exl3::kTileTokenRows / (q_heads / a.kv_heads);
  a.ctas = plan.ctas;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + plan.o_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return exl3::api_status(plan.token ? exl3::launch_attn_token(a, s) : exl3::launch_attn_tile(a, true, s), "exl3_attention_paged");
}

}  // extern "C"
