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
  *out = {r->phases, r->positions, r->rot_dim, r->layout == EXL3_ROPE_INTERLEAVED ? 1 : 0, r->amplitude, nullptr, 1};
  return EXL3_OK;
}
// Adds the axes of a checked rotation's pairs; null: the positions have one row.
exl3_status_t check_axes(const exl3_rope_axes_t* axes, exl3::RopeArgs* out) {
  if (axes == nullptr) return EXL3_OK;
  if (axes->axes == nullptr || axes->num_axes < 1 || axes->num_axes > 255) return EXL3_EINVAL;
  out->axes = axes->axes;
  out->num_axes = axes->num_axes;
  return EXL3_OK;
}
exl3_status_t check_norm(const exl3_head_norm_t* n, exl3::HeadNorm* out) {
  if (n == nullptr) return EXL3_OK;
  if (!aligned16(n->weight) || n->head_stride < 0 || n->head_stride % 8 != 0 || n->head_stride > (int64_t(1) << 32)) return EXL3_EINVAL;
  if (!(n->eps >= 1.1754944e-38f) || !isfinite(n->eps)) return EXL3_EINVAL;  // a row of zeros stays one
  *out = {static_cast<const uint16_t*>(n->weight), n->head_stride, n->eps};
  return EXL3_OK;
}
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// log2 of a page size that the cache has, or -1.
int page_shift(int32_t page_size) {
  for (int shift = 4; shift <= 8; ++shift)
    if ((1 << shift) == page_size) return shift;
  return -1;
}
exl3_status_t check_tables(const exl3_kv_tables_t* t, exl3::KvTables* out) {
  if (t == nullptr || !valid_rows(t->batch) || t->table_width < 1 || t->capacity < 1) return EXL3_EINVAL;
  const int shift = page_shift(t->page_size);
  if (shift < 0 || ((int64_t)t->table_width << shift) > (int64_t(1) << 30)) return EXL3_EINVAL;
  if (t->capacity >= (1 << 30)) return EXL3_EINVAL;  // where sums of pages saturate: one that has is above every stack
  if (!aligned4(t->free_pages) || !aligned4(t->free_count)) return EXL3_EINVAL;
  if (t->batch > 0 && (!aligned4(t->block_table) || !aligned4(t->kv_lens) || !aligned4(t->held))) return EXL3_EINVAL;
  *out = {t->block_table, t->kv_lens, t->held, t->free_pages, t->free_count, t->batch, t->table_width, shift, t->capacity};
  return EXL3_OK;
}

exl3_status_t check_cache(const exl3_kv_cache_t* c, exl3::KvCache* out) {
  if (c == nullptr || c->format < EXL3_KV_F16 || c->format > EXL3_KV_INT4) return EXL3_EINVAL;
  if (c->kv_heads < 1 || c->kv_heads > 65536 || c->num_pages < 1 || c->num_pages >= (int64_t(1) << 31)) return EXL3_EINVAL;
  const int shift = page_shift(c->page_size);
  if (shift < 0) return EXL3_EINVAL;
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

// The keys of each item of row tiles may go to several CTAs: the number of parts is the one that a simple model of the
// time likes best, waves of items, each as long as its blocks of 64 keys (about 0.85 us each) and the beginning and end
// of an item (about 4 us), and what the parts cost to write and join.  512 tokens of 32 heads over 32768 keys of 8: 232,
// 234, 218 and 230 us in 2, 4, 7 and 9 parts, 230, 238, 217 and 232 by the model.
int64_t item_parts(int64_t items, int64_t keys, int64_t values) {
  const double blocks = (double)(keys > 64 ? keys : 64) / 64.0;
  double best = 0.0;
  int64_t parts = 1;
  for (int64_t s = 1; s <= 16 && blocks / s >= 8.0 && (s == 1 || items <= kSms); ++s) {
    const double waves = (double)((items * s + kSms - 1) / kSms);
    const double join = s > 1 ? 4.0 + (double)s * values * 8.0 / 8.0e6 : 0.0;
    const double us = waves * (blocks / s * 0.85 + 4.0) + join;
    if (s == 1 || us < 0.97 * best) {
      best = us;
      parts = s;
    }
  }
  return parts;
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
  // row tiles, two an item
  const int64_t per = 2 * (exl3::kTileTokenRows / group);
  const int64_t tiles = batch == 1 ? (total_q + per - 1) / per : total_q / per + (total_q < batch ? total_q : batch);
  const int64_t items = tiles * kv_heads;
  const int64_t seen = window > 0 && window + per < max_kv ? window + per : max_kv;  // keys of an item
  const int64_t splits = item_parts(items, seen, total_q * q_heads * head_dim);
  if (splits > 1) {
    p.splits = (int)splits;
    p.o_bytes = (size_t)splits * total_q * q_heads * head_dim * sizeof(float);
    p.ml_bytes = (size_t)splits * total_q * q_heads * 2 * sizeof(float);
  }
  return p;
}

// How a call behind shared prefixes is split: the prefixes' row tiles into CTAs (how many each gets is for the GPU to say,
// which knows the lengths), then the sequences' own keys as in a paged call.
struct SharedPlan {
  bool token;
  int ctas, prefix_ctas, splits;
  size_t at[11];  // where in the workspace each array begins, and the end
};
SharedPlan shared_plan(int64_t total_q, int64_t batch, int64_t groups, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                       int64_t max_q, int64_t max_kv) {
  SharedPlan p = {};
  const int64_t group = q_heads / kv_heads, per = 2 * (exl3::kTileTokenRows / group), rows = total_q * q_heads;
  p.token = max_q * group <= exl3::kTokenRows;
  // an item for each row tile, and room for parts: one wave of CTAs, or where the row tiles alone are more than that
  // two more, which even out the last
  const int64_t tiles = exl3::shared_tiles(total_q, groups, per) * kv_heads;
  p.prefix_ctas = (int)(tiles + (tiles < kSms ? kSms : 2 * kSms));
  int64_t cut = 0;
  if (p.token) {
    const PagedPlan own = paged_plan(total_q, batch, q_heads, kv_heads, head_dim, max_q, max_kv, 0);
    p.ctas = own.ctas;
    cut = 2 * (int64_t)own.ctas * exl3::kTokenRows;
  } else {
    // room for the parts of sequences that share nothing and are as long as any; of how many parts each is the GPU says
    p.splits = (int)item_parts(exl3::shared_tiles(total_q, batch, per) * kv_heads, max_kv > max_q ? max_kv : max_q, rows * head_dim);
  }
  const int64_t own = p.token ? rows : p.splits * rows, prefix = (int64_t)p.prefix_ctas * exl3::kPrefixRows;
  const int64_t bytes[10] = {prefix * head_dim * 4, prefix * 8, own * head_dim * 4, own * 8, cut * head_dim * 4, cut * 8,
                             groups * (int64_t)sizeof(exl3::SharedGroup), batch * 8, p.token ? (batch + 1) * 8 : 0, 16};
  for (int i = 0; i < 10; ++i) p.at[i + 1] = p.at[i] + (size_t)((bytes[i] + 15) / 16 * 16);
  return p;
}

// Row tiles in up to 16 parts are CTAs of one grid, and counted in 32 bits.
bool shared_fits(int64_t total_q, int64_t q_heads) { return total_q * q_heads * 16 <= INT32_MAX; }

// Whether sharing pays, for groups that hold `sharers` of the call's sequences: what the prefixes take when every sequence
// reads them for itself, less what they take when they are read once, against what the call has in addition (two launches,
// the lengths, the join).  Each time is a sum of SM time by measured rates, so the sides are those of the sizes at hand: how
// many groups, how long, how wide.  All prefixes count as the longest, and sequences and groups as equally large.
//   Row tiles take `joint` or `full` us for 64 keys, by whether the rows fill one tile of 128, and `fixed` us an item.  Many
// more rows than an item holds leave the last item of each list half empty, or a little more.
//   Few rows go through the token kernel: 34 keys and key heads a ns (128 values; 24 where a key head has more than 8
// rows), or DRAM, which gives a prefix to every sequence where those of the groups do not stay in L2 together.  Its
// join looks through all sequences for each of them.  The lengths take 0.17 us a group and 0.04 a sequence.
//   us of a layer by the paged call and shared, layers in turn whose caches are larger than L2 together; 32 and 8 heads of
// 128, 16 bits but where it says codes:
//     single tokens of one group: 8 sequences behind 8192 keys 27 and 28 (codes 27 and 33), 16 behind 4096 28 and 30 (29 and
//       35), 16 behind 8192 44 and 32 (45 and 37), 32 behind 1024 25 and 24, 64 behind 512 33 and 28
//     pairs: 16 behind 4096 82 and 67 (codes 53 and 83), 64 behind 4096 353 and 233 (203 and 290), 250 behind 512 401 and
//       320 (335 and 354); 64 groups of four behind 512 160 and 122 (135 and 131)
//     2, 8 and 32 of 62 to 64 behind 8192, the others alone: 102 and 117, 109 and 116, 108 and 81
//     8 tokens each (32 rows): 4 sequences behind 4096 21 and 24, 8 behind 4096 30 and 24, 40 behind 1024 50 and 41
//     30 tokens each (120 rows): 4 behind 2048 20 and 29, 8 behind 4096 42 and 37, 16 behind 8192 72 and 79 (codes 120
//       and 104)
//     chunks of about 100 tokens, 16 sequences: behind 4000 119 and 140, 8000 213 and 192, 16000 408 and 349; of about 1500,
//       2 sequences: behind 8000 341 and 355, 16000 640 and 666, 32000 1250 and 1296 (waves of items move single sizes by
//       tenths either way, which no sum of times sees)
// Over 2550 sizes, two thirds of them drawn, the side chosen takes 1.6% more than the better one on average (always the
// paged call: 34%); where it is the shared one, 29% more at the most, and more than a tenth at 34 sizes.
// Rows of fp16 over codes, where the token kernel holds the rotated q in two terms and the row tiles in one, stay with the
// former: 17 tokens of 48 heads behind 7791 8-bit keys would have 0.0004 of the result's norm in place of 0.0002.
bool worth_sharing(int64_t total_q, int64_t batch, int64_t sharers, int64_t groups, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                   int format, bool bf16, int64_t max_q, int64_t max_prefix) {
  if (max_prefix == EXL3_SHARE_ALWAYS) return groups > 0;
  if (groups == 0 || sharers <= groups || max_prefix < exl3::kLeastPrefix || !shared_fits(total_q, q_heads)) return false;
  const bool quant = exl3::kv_quantised(format);
  const int64_t each = max_q * (q_heads / kv_heads);
  const bool token = each <= exl3::kTokenRows;
  if (token && quant && !bf16) return false;
  const double wide = head_dim / 128.0, blocks = max_prefix / 64.0 * wide;
  const double joint = quant ? 0.82 : 0.72, full = 0.9, fixed = token ? 14.0 : quant ? 6.0 : 5.0;
  // of row tiles over the prefix, `lists` times `rows` rows
  auto items = [&](double lists, double rows) { return (rows <= 256.0 ? lists : lists * (rows / 256.0 + 0.55)) * kv_heads / kSms; };
  auto tiles = [&](double lists, double rows) { return items(lists, rows) * (fixed + blocks * (rows <= 128.0 ? joint : full)); };
  const double own = (double)total_q * (q_heads / kv_heads) / batch, all = own * sharers / groups;  // rows of a sequence and of a group
  const bool some = sharers < batch;
  double alone, together, more = 0.17 * groups + 0.04 * batch;
  if (token) {
    const double bytes = (double)max_prefix * kv_heads * 2 * exl3::kv_row_bytes(format, (int)head_dim);
    auto dram = [&](double times) { return times * bytes / 6.8e6; };
    alone = fmax((double)sharers * max_prefix * kv_heads * wide / (each <= 8 ? 34e3 : 24e3), dram(groups * bytes > 80e6 ? sharers : groups)) +
            0.0008 * batch * batch * (q_heads * max_q / 32.0);
    together = fmax(tiles(groups, all), dram(groups));
    more += total_q * q_heads <= 4 * kSms ? 16.0 : some ? 13.0 : quant ? 9.0 : 7.0;
  } else {
    // (the sequences' own keys are items of their own, and every row has parts to be joined)
    alone = tiles(sharers, own);
    together = tiles(groups, all);
    more += (quant ? 4.0 : 7.5) + (some ? 7.5 : 0.0) + 6.5 * items(batch, own) + 0.0115 * total_q * q_heads / 32.0 * wide;
  }
  return alone - together > more;
}

// Checks of a paged call and what the kernels take of it, but for the split; an empty call is not filled in.
exl3_status_t paged_args(const exl3_heads_t* q, exl3_dtype_t dtype, int64_t total_q, int32_t q_heads, const exl3_kv_cache_t* cache,
                         const int32_t* block_table, int32_t table_width, const int32_t* cu_q, const int32_t* kv_lens, int32_t batch,
                         int32_t max_q, int32_t max_kv, int32_t window, float scale, void* out, int64_t out_token_stride,
                         int64_t out_head_stride, exl3::AttnArgs* args) {
  exl3::AttnArgs& a = *args;
  if (!valid_rows(total_q) || !valid_rows(batch) || !valid_dtype(dtype)) return EXL3_EINVAL;
  const exl3_status_t st = check_cache(cache, &a.cache);
  if (st != EXL3_OK) return st;
  if (!valid_head_counts(q_heads, a.cache.kv_heads) || !format_fits(a.cache.format, dtype)) return EXL3_EINVAL;
  if (table_width < 1 || ((int64_t)table_width << a.cache.page_shift) > (int64_t(1) << 30)) return EXL3_EINVAL;
  if (max_q < 1 || max_kv < 0 || window < 0 || !(scale > 0.0f) || !isfinite(scale)) return EXL3_EINVAL;
  if (!valid_strides(out_token_stride, out_head_stride)) return EXL3_EINVAL;
  if (total_q == 0 || batch == 0) return EXL3_OK;
  if (!valid_heads(q) || !valid_out(q, out, out_token_stride, out_head_stride)) return EXL3_EINVAL;
  if (!aligned4(block_table) || !aligned4(cu_q) || !aligned4(kv_lens)) return EXL3_EINVAL;
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
  a.tile_tokens = exl3::kTileTokenRows / (q_heads / a.kv_heads);
  return EXL3_OK;
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
  return exl3_norm_rope(x, dtype, tokens, heads, head_dim, nullptr, rope, nullptr, out, out_token_stride, out_head_stride, stream);
}

exl3_status_t exl3_norm_rope(const exl3_heads_t* x, exl3_dtype_t dtype, int64_t tokens, int32_t heads, int32_t head_dim,
                             const exl3_head_norm_t* norm, const exl3_rope_t* rope, const exl3_rope_axes_t* axes, void* out,
                             int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  if (!valid_rows(tokens) || heads < 1 || heads > 65536 || !valid_dtype(dtype)) return EXL3_EINVAL;
  exl3_status_t st = check_head_dim(head_dim);
  if (st != EXL3_OK) return st;
  exl3::RopeWriteArgs a = {};
  st = check_norm(norm, &a.x_norm);
  if (st != EXL3_OK) return st;
  if (rope != nullptr || norm == nullptr) {
    st = check_rope(rope, head_dim, tokens, &a.rope);
    if (st == EXL3_OK) st = check_axes(axes, &a.rope);
    if (st != EXL3_OK) return st;
  } else if (axes != nullptr) {
    return EXL3_EINVAL;
  }
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
  return exl3::api_status(exl3::launch_rope_write(a, head_dim, static_cast<cudaStream_t>(stream)), norm != nullptr ? "exl3_norm_rope" : "exl3_rope");
}

exl3_status_t exl3_kv_write(const exl3_kv_cache_t* cache, const exl3_heads_t* k, const exl3_heads_t* v,
                            exl3_dtype_t dtype, int64_t tokens, const int64_t* slots, const exl3_rope_t* rope,
                            const exl3_heads_t* q, int32_t q_heads, void* q_out, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, void* stream) {
  return exl3_norm_kv_write(cache, k, v, dtype, tokens, slots, nullptr, nullptr, rope, nullptr, q, q_heads, q_out,
                            q_out_token_stride, q_out_head_stride, stream);
}

exl3_status_t exl3_norm_kv_write(const exl3_kv_cache_t* cache, const exl3_heads_t* k, const exl3_heads_t* v,
                                 exl3_dtype_t dtype, int64_t tokens, const int64_t* slots,
                                 const exl3_head_norm_t* q_norm, const exl3_head_norm_t* k_norm,
                                 const exl3_rope_t* rope, const exl3_rope_axes_t* axes, const exl3_heads_t* q,
                                 int32_t q_heads, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                                 void* stream) {
  if (!valid_rows(tokens) || !valid_dtype(dtype) || q_heads < 0 || q_heads > 65536) return EXL3_EINVAL;
  exl3::RopeWriteArgs a = {};
  exl3_status_t st = check_cache(cache, &a.cache);
  if (st != EXL3_OK) return st;
  if (!format_fits(a.cache.format, dtype)) return EXL3_EINVAL;
  st = check_norm(k_norm, &a.k_norm);
  if (st == EXL3_OK) st = check_norm(q_norm, &a.x_norm);
  if (st != EXL3_OK) return st;
  if (rope != nullptr) {
    st = check_rope(rope, a.cache.head_dim, tokens, &a.rope);
    if (st == EXL3_OK) st = check_axes(axes, &a.rope);
    if (st != EXL3_OK) return st;
  } else if ((q_heads != 0 && q_norm == nullptr) || axes != nullptr) {
    return EXL3_EINVAL;
  }
  if (q_norm != nullptr && q_heads == 0) return EXL3_EINVAL;
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

exl3_status_t exl3_kv_plan(const exl3_kv_tables_t* tables, const int32_t* new_lens, int64_t total, int32_t* kv_lens_out,
                           int32_t* held_out, int32_t* free_count_out, int32_t* cu_q, int32_t* positions, int64_t* slots,
                           uint8_t* granted, void* stream) {
  exl3::KvPlanArgs a = {};
  const exl3_status_t st = check_tables(tables, &a.t);
  if (st != EXL3_OK) return st;
  if (!valid_rows(total) || !aligned4(cu_q) || !aligned4(free_count_out)) return EXL3_EINVAL;
  if (a.t.batch > 0 && (!aligned4(new_lens) || !aligned4(kv_lens_out) || !aligned4(held_out) || granted == nullptr)) return EXL3_EINVAL;
  if (total > 0 && (!aligned4(positions) || slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)) return EXL3_EINVAL;
  a.new_lens = new_lens;
  a.total = total;
  a.kv_lens_out = kv_lens_out;
  a.held_out = held_out;
  a.free_count_out = free_count_out;
  a.cu_q = cu_q;
  a.positions = positions;
  a.slots = slots;
  a.granted = granted;
  return exl3::api_status(exl3::launch_kv_plan(a, static_cast<cudaStream_t>(stream)), "exl3_kv_plan");
}

exl3_status_t exl3_kv_release(const exl3_kv_tables_t* tables, const uint8_t* ended, const int32_t* shared,
                              int32_t* kv_lens_out, int32_t* held_out, int32_t* free_count_out, void* stream) {
  exl3::KvReleaseArgs a = {};
  const exl3_status_t st = check_tables(tables, &a.t);
  if (st != EXL3_OK) return st;
  if (!aligned4(free_count_out) || (reinterpret_cast<uintptr_t>(shared) & 3u) != 0) return EXL3_EINVAL;
  if (a.t.batch > 0 && (ended == nullptr || !aligned4(kv_lens_out) || !aligned4(held_out))) return EXL3_EINVAL;
  a.ended = ended;
  a.shared = shared;
  a.kv_lens_out = kv_lens_out;
  a.held_out = held_out;
  a.free_count_out = free_count_out;
  return exl3::api_status(exl3::launch_kv_release(a, static_cast<cudaStream_t>(stream)), "exl3_kv_release");
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
  exl3::AttnArgs a = {};
  const exl3_status_t st = paged_args(q, dtype, total_q, q_heads, cache, block_table, table_width, cu_q, kv_lens, batch, max_q, max_kv,
                                      window, scale, out, out_token_stride, out_head_stride, &a);
  if (st != EXL3_OK || total_q == 0 || batch == 0) return st;
  const PagedPlan plan = paged_plan(total_q, batch, q_heads, a.kv_heads, a.head_dim, max_q, max_kv, window);
  if (plan.token && (int64_t)batch * a.kv_heads > INT32_MAX) return EXL3_EUNSUPPORTED;  // blocks of the join
  if (plan.o_bytes > 0 && !aligned16(workspace)) return EXL3_EINVAL;
  if (workspace_bytes < plan.o_bytes + plan.ml_bytes) return EXL3_EWORKSPACE;
  a.splits = plan.splits;
  a.ctas = plan.ctas;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + plan.o_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return exl3::api_status(plan.token ? exl3::launch_attn_token(a, s) : exl3::launch_attn_tile(a, true, s), "exl3_attention_paged");
}

size_t exl3_attention_shared_workspace_bytes(int64_t total_q, int32_t batch, int32_t groups, int32_t q_heads,
                                             int32_t kv_heads, int32_t head_dim, exl3_dtype_t dtype,
                                             exl3_kv_format_t format, int32_t max_q, int32_t max_kv, int32_t max_prefix) {
  if (!valid_rows(total_q) || !valid_rows(batch) || !valid_rows(groups) || !valid_head_counts(q_heads, kv_heads)) return 0;
  if (check_head_dim(head_dim) != EXL3_OK || max_q < 1 || max_kv < 0 || max_prefix < 0 || total_q == 0 || batch == 0) return 0;
  if (!worth_sharing(total_q, batch, batch, groups, q_heads, kv_heads, head_dim, format, dtype == EXL3_BF16, max_q, max_prefix))
    return exl3_attention_paged_workspace_bytes(total_q, batch, q_heads, kv_heads, head_dim, max_q, max_kv, 0);
  return shared_plan(total_q, batch, groups, q_heads, kv_heads, head_dim, max_q, max_kv).at[10];
}

int32_t exl3_attention_shared_pays(int64_t total_q, int32_t batch, int32_t sharers, int32_t groups, int32_t q_heads,
                                   int32_t kv_heads, int32_t head_dim, exl3_dtype_t dtype, exl3_kv_format_t format,
                                   int32_t max_q, int32_t max_prefix) {
  if (!valid_rows(total_q) || !valid_rows(batch) || !valid_rows(groups) || !valid_head_counts(q_heads, kv_heads)) return 0;
  if (check_head_dim(head_dim) != EXL3_OK || max_q < 1 || max_prefix < 0 || total_q == 0 || batch == 0 || sharers < 0 || sharers > batch) return 0;
  return worth_sharing(total_q, batch, sharers, groups, q_heads, kv_heads, head_dim, format, dtype == EXL3_BF16, max_q, max_prefix) ? 1 : 0;
}

exl3_status_t exl3_attention_shared(const exl3_heads_t* q, exl3_dtype_t dtype, int64_t total_q, int32_t q_heads,
                                    const exl3_kv_cache_t* cache, const int32_t* block_table, int32_t table_width,
                                    const int32_t* cu_q, const int32_t* kv_lens, int32_t batch, const int32_t* cu_groups,
                                    const int32_t* prefix_lens, int32_t groups, int32_t max_q, int32_t max_kv,
                                    int32_t max_prefix, float scale, void* out, int64_t out_token_stride,
                                    int64_t out_head_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_rows(groups) || max_prefix < 0) return EXL3_EINVAL;
  if (groups > 0 && total_q != 0 && batch != 0 && (!aligned4(cu_groups) || !aligned4(prefix_lens))) return EXL3_EINVAL;
  exl3::AttnArgs a = {};
  const exl3_status_t st = paged_args(q, dtype, total_q, q_heads, cache, block_table, table_width, cu_q, kv_lens, batch, max_q, max_kv, 0,
                                      scale, out, out_token_stride, out_head_stride, &a);
  if (st != EXL3_OK || total_q == 0 || batch == 0) return st;
  if (!worth_sharing(total_q, batch, batch, groups, q_heads, a.kv_heads, a.head_dim, a.cache.format, dtype == EXL3_BF16, max_q, max_prefix))
    return exl3_attention_paged(q, dtype, total_q, q_heads, cache, block_table, table_width, cu_q, kv_lens, batch, max_q, max_kv, 0,
                                scale, out, out_token_stride, out_head_stride, workspace, workspace_bytes, stream);
  if (!shared_fits(total_q, q_heads)) return EXL3_EUNSUPPORTED;
  const SharedPlan plan = shared_plan(total_q, batch, groups, q_heads, a.kv_heads, a.head_dim, max_q, max_kv);
  if (!aligned16(workspace)) return EXL3_EINVAL;
  if (workspace_bytes < plan.at[10]) return EXL3_EWORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.groups = groups;
  a.prefix_ctas = plan.prefix_ctas;
  a.splits = plan.splits;
  a.ctas = plan.ctas;
  a.prefix_o = reinterpret_cast<float*>(w + plan.at[0]);
  a.prefix_ml = reinterpret_cast<float2*>(w + plan.at[1]);
  a.own_o = reinterpret_cast<float*>(w + plan.at[2]);
  a.own_ml = reinterpret_cast<float2*>(w + plan.at[3]);
  a.cut_o = reinterpret_cast<float*>(w + plan.at[4]);
  a.cut_ml = reinterpret_cast<float2*>(w + plan.at[5]);
  a.group = reinterpret_cast<const exl3::SharedGroup*>(w + plan.at[6]);
  a.seq = reinterpret_cast<const int2*>(w + plan.at[7]);
  a.units = reinterpret_cast<const int64_t*>(w + plan.at[8]);
  a.counts = reinterpret_cast<const int4*>(w + plan.at[9]);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = exl3::launch_shared_prep(a, cu_groups, prefix_lens, plan.token, s);
  if (e == cudaSuccess) e = exl3::launch_attn_tile_shared(a, !plan.token, s);
  if (e == cudaSuccess && plan.token) e = exl3::launch_attn_token_shared(a, s);
  if (e == cudaSuccess) e = exl3::launch_shared_join(a, plan.token, s);
  return exl3::api_status(e, "exl3_attention_shared");
}

}  // extern "C"
