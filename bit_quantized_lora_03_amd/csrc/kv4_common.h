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
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4BatchArg& bt, int b) {
  const int64_t first = bt.cu_q[b], last = bt.cu_q[b + 1];
  Kv4Seq q;
  q.row0 = first;
  q.len = bt.seq_lens[b];
  q.pos0 = q.len - (last - first);
  // a start before row 0 leaves nothing; rows past T are left out
  q.n = first < 0 ? 0 : (last < bt.rows ? last : bt.rows) - first;
  if (q.n > bt.max_q) q.n = bt.max_q;
  return q;
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
