// exl3_attn_seq.cuh -- what the token kernel and the joins of its parts make of a
// sequence.
#pragma once

#include "exl3_attn.h"

namespace exl3 {
namespace {

// What an item's beginning and end cost, in units of keys (for the cuts).
constexpr int kItemUnits = 4;

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
// SHARED: the keys before a.seq[b].x are not its own.
template <bool SHARED>
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  Seq s;
  const int64_t c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
  s.q0 = c0 < 0 ? 0 : c0 > a.total_q ? a.total_q : c0;
  const int64_t n = (c1 > a.total_q ? a.total_q : c1) - s.q0;
  s.q_len = n < 0 ? 0 : n > a.max_q ? a.max_q : (int)n;
  const int64_t room = (int64_t)a.table_width << a.cache.page_shift;
  const int64_t kl = a.kv_lens[b];
  s.kv_len = (int)(kl < 0 ? 0 : kl > room ? room : kl);
  const int64_t first = SHARED ? __ldcg(&a.seq[b].x) : a.window > 0 ? (int64_t)s.kv_len - s.q_len - a.window + 1 : 0;
  s.first = first > 0 ? (int)first : 0;
  s.lo = s.first / kTokenUnit * kTokenUnit;
  // a sequence without keys still has a unit: its rows are zeros
  const int u = (s.kv_len - s.lo + kTokenUnit - 1) / kTokenUnit;
  s.units = s.q_len == 0 ? 0 : u < 1 ? 1 : u;
  return s;
}

// Parts of a sequence's own keys in row tiles behind shared prefixes, `unit` blocks of 64 at the most.
__device__ __forceinline__ int shared_own_parts(const AttnArgs& a, int b, int unit) {
  if (a.splits <= 1) return 1;
  const int keys = max(0, min(a.kv_lens[b], a.table_width << a.cache.page_shift)) - __ldcg(&a.seq[b].x);
  return max(1, ((max(0, keys) + 63) / 64 + unit - 1) / unit);
}

}  // namespace
}  // namespace exl3
