// The 4-bit paged cache and the ragged batch that its kernels work on.
#pragma once

#include <type_traits>

#include "launch.h"
#include "u4_common.h"

namespace qlora {

// What the caller's device arrays say about a sequence is checked here, on
// the device, since the host cannot see it: rows outside [0, T), lengths
// past the block table and pages outside the pool never become addresses.
struct Kv4Seq {
  int64_t row0;  // first of its rows
  int64_t n;     // rows (0 for a sequence without)
  int64_t pos0;  // position of row0 in the sequence
  int64_t len;   // tokens of the sequence, its new ones among them
};
__host__ __device__ __forceinline__ Kv4Seq kv4_seq(const Kv4BatchArg& bt, int b) {
  const int64_t first = bt.cu_q[b], last = bt.cu_q[b + 1];
  Kv4Seq q;
  q.row0 = first;
  q.len = bt.seq_lens[b];
  q.pos0 = q.len - (last - first);
  // a start before row 0 or behind the end leaves nothing; rows past T are
  // left out
  q.n = (last < bt.rows ? last : bt.rows) - first;
  if (first < 0 || q.n < 0) q.n = 0;
  if (q.n > bt.max_q) q.n = bt.max_q;
  return q;
}

// The keys of a tile of query rows: [lo, hi) inside the block table, lo a
// multiple of kKv4Step, cut into n chunks of `chunk` keys.
constexpr int kKv4Step = 32;
struct Span {
  int lo, hi, chunk, n;
  int i0, i1;  // first and last query token of the tile
  // Chunk s < n (or 0).  lo, hi and chunk may each be 2^30 and a little more,
  // so only differences are compared.
  __host__ __device__ int begin(int s) const { return lo + s * chunk; }
  __host__ __device__ int end(int s) const {
    return hi - begin(s) < chunk ? hi : begin(s) + chunk;
  }
};
__host__ __device__ __forceinline__ Span kv4_span(const Kv4Seq& sq, const Kv4AttnArg& a, int group,
                                                  int r0, int tile, int chunk, int splits) {
  Span s;
  const int last = (int)sq.n * group - 1, end = r0 + tile - 1;
  s.i0 = r0 / group;
  s.i1 = (end < last ? end : last) / group;
  // the table's last key bounds what can be read
  int64_t hi = sq.len < a.table_keys ? sq.len : a.table_keys, lo = 0;
  if (a.causal && sq.pos0 + s.i1 + 1 < hi) hi = sq.pos0 + s.i1 + 1;
  if (a.window > 0 && sq.pos0 + s.i0 - a.window + 1 > 0) lo = sq.pos0 + s.i0 - a.window + 1;
  // A length far past the table puts a window behind it, up to 2^31: no keys
  // then, and no such number into the walk.
  if (lo >= hi) lo = hi = 0;
  s.hi = (int)hi;
  s.lo = (int)(lo & ~(int64_t)(kKv4Step - 1));
  const int keys = s.hi - s.lo;
  // a sequence longer than the call was planned for takes larger chunks
  const int need = (keys + splits - 1) / splits, whole = (need + kKv4Step - 1) / kKv4Step * kKv4Step;
  s.chunk = chunk > whole ? chunk : whole;
  s.n = keys > 0 ? (keys - 1) / s.chunk + 1 : 0;
  return s;
}

// Token slot (page, head, row of the page) of position pos >= 0, or -1
// where the table or the pool has no such page.
__device__ __forceinline__ int64_t kv4_slot(const Kv4CacheArg& c, const Kv4BatchArg& bt, int b,
                                            int64_t pos, int h) {
  const int64_t e = pos >> c.page_log2;
  if (e >= bt.table_width) return -1;
  const int64_t page = bt.block_table[(int64_t)b * bt.table_width + e];
  if (page < 0 || page >= c.pages) return -1;
  return ((page * c.kv_heads + h) << c.page_log2) + (pos & ((1 << c.page_log2) - 1));
}

}  // namespace qlora
