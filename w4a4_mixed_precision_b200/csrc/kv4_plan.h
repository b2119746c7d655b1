// kv4_plan.h -- index arithmetic of the paged INT4 KV cache: pages, sequences,
// query rows and the division of the attention's work. Plain C++ that both the
// kernels and a host compiler take, so that it is tested without a GPU.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define KV4_HD __host__ __device__ __forceinline__
#else
#define KV4_HD inline
#endif

namespace atomk {

// Division of 0 <= n < 2^31 by a fixed 1 <= d < 2^31: with s = ceil(log2 d) and
// m = ceil(2^(31+s) / d) < 2^32, floor(n / d) = (n * m) >> (31 + s), because
// m * d exceeds 2^(31+s) by less than d <= 2^s and n < 2^31.
struct Kv4Div {
  uint32_t m, shift;
};

inline Kv4Div kv4_div_by(int64_t d) {
  uint32_t s = 0;
  while ((int64_t(1) << s) < d) ++s;
  const uint64_t p = uint64_t(1) << (31 + s);
  return Kv4Div{static_cast<uint32_t>((p + static_cast<uint64_t>(d) - 1) / static_cast<uint64_t>(d)),
                31 + s};
}

KV4_HD int kv4_div(int n, const Kv4Div &d) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * d.m) >> d.shift);
}

// A cache's geometry. Vectors (one token of one head) are addressed by number:
// vector v has its 64 bytes of codes at 64 v and its scale at v.
struct Kv4Geom {
  int page_stride, token_stride, head_stride;   // in vectors
  int pages, page_size, heads;
  Kv4Div by_page;
};

// Positions and rows are 32-bit, and stay so far below 2^31 that loops may step
// past them.
constexpr int kKv4MaxPositions = 1 << 30;
inline int kv4_capacity(int64_t max_pages, int64_t page_size) {
  return max_pages > kKv4MaxPositions / page_size ? kKv4MaxPositions
                                                  : static_cast<int>(max_pages * page_size);
}

// The sequences of a call; `capacity` is what kv4_capacity says.
struct Kv4Seqs {
  const int32_t *table;    // [batch][table_stride], pages of each sequence
  int64_t table_stride;
  const int32_t *kv_lens;  // [batch]
  const int32_t *cu_q;     // [batch + 1]
  int batch, rows, capacity;
};

// One sequence: rows [q0, q0 + qn) of the call are its new tokens, the last
// qn of its `len` cached positions. `ok` is false (and qn = len = 0) where the
// arrays on the device contradict the call's sizes; such a sequence is skipped.
struct Kv4Seq {
  int q0, qn, len;
  bool ok;
};

KV4_HD Kv4Seq kv4_seq_of(int q0, int q1, int len, int rows, int capacity) {
  Kv4Seq s{q0, q1 - q0, len, true};
  if (q0 < 0 || q1 < q0 || q1 > rows || len < 0 || len > capacity) s = Kv4Seq{0, 0, 0, false};
  return s;
}

// Vector number of (page, slot, head), or -1 for a page outside the cache.
KV4_HD int64_t kv4_vector(const Kv4Geom &c, int page, int slot, int head) {
  if (page < 0 || page >= c.pages) return -1;
  return static_cast<int64_t>(page) * c.page_stride + static_cast<int64_t>(slot) * c.token_stride +
         static_cast<int64_t>(head) * c.head_stride;
}

// Cached positions a query may see: all, or (causal) those up to its own.
KV4_HD int kv4_limit(const Kv4Seq &s, int qi, bool causal) {
  const int64_t lim = causal ? static_cast<int64_t>(s.len) - s.qn + qi + 1 : s.len;
  return lim < 0 ? 0 : (lim > s.len ? s.len : static_cast<int>(lim));
}

// The attention's work. The new tokens of a sequence and the `group` query
// heads that share a KV head form qn * group query rows (row = qi * group + g),
// cut into tiles of `tile` rows; a tile's cached positions are cut into units
// of kKv4Unit. In the order sequence, head, tile, unit the units of a call form
// one line, of which part i of n gets [i * total / n, (i + 1) * total / n).
constexpr int kKv4Unit = 256;

KV4_HD int kv4_tiles(const Kv4Seq &s, int group, int tile) {
  return static_cast<int>((static_cast<int64_t>(s.qn) * group + tile - 1) / tile);
}
// A tile of a sequence with nothing cached still is one unit: its outputs are
// written.
KV4_HD int kv4_units(int len) { return len == 0 ? 1 : (len - 1) / kKv4Unit + 1; }

// (= floor(i * total / parts), without the long product)
KV4_HD int64_t kv4_part_begin(int64_t total, int parts, int i) {
  return total / parts * i + total % parts * i / parts;
}
// How many parts to divide the line among `ctas` CTAs into: all, or where fewer
// tiles than CTAs have at least a tenth of a CTA's slack, as many as give every
// tile the same number. Tiles of one length then begin and end at part
// boundaries, and the heads of a sequence are at the same positions at the same
// time: in a token-major cache they share 128-byte lines (2 x 131072 tokens, 8
// heads: 568 -> 288 MB read).
KV4_HD int kv4_parts(int64_t total, int64_t tiles, int ctas) {
  if (total < ctas) return static_cast<int>(total);
  if (tiles < 1 || tiles >= ctas) return ctas;
  const int even = static_cast<int>(ctas / tiles * tiles);
  return even >= ctas - ctas / 10 ? even : ctas;
}
// The part that holds place `at` of the line: the largest i with
// i * total / parts < at + 1.
KV4_HD int kv4_part_of(int64_t total, int parts, int64_t at) {
  return static_cast<int>(((at + 1) * parts - 1) / total);
}

// Largest number of query rows of a KV head that goes to the decode kernel where
// a call has `pairs` (sequence, KV head) pairs with up to `max_rows` of them; more
// go to the prompt kernel.
// The decode kernel reads the cache once per 16 rows and divides that evenly over
// the GPU: 44 us per million tokens, pair and 16 rows. The prompt kernel reads it
// once per 256 rows, with one CTA an SM and a CTA a pair and 256 rows: 22 us per
// thousand tokens for each round of CTAs. (Both measured, us: 16 sequences of 3000
// tokens, 8 heads, 32 rows 46 and 74, 64 rows 77 and 76, 128 rows 141 and 76; one
// sequence, 512 rows 46 and 73; four of 20000, 128 rows 204 and 410, 256 rows 391
// and 412, 512 rows 766 and 413. Neither divides the cached tokens of many rows:
// with one KV head, 8 query heads and 1024 new tokens behind 32768 both are far
// from the tensor cores' 83 us, 634 and 676.)
inline int64_t kv4_few_rows(int64_t pairs, int64_t max_rows, int sms) {
  if (pairs > int64_t(1) << 40) pairs = int64_t(1) << 40;   // (the products stay in 64 bits)
  int64_t rows = 16;
  for (; rows < max_rows && rows < 4096; rows += 16) {
    const int64_t rounds = (pairs * ((rows + 16 + 255) / 256) + sms - 1) / sms;
    if (pairs * ((rows + 16) / 16) >= 500 * rounds) break;
  }
  return rows;
}
// The copies of an item's two query tiles, each into a buffer of its own as soon
// as that is empty. started[w]: copies into buffer w so far; each completes one
// phase of the buffer's barrier. False: a wait gave up, with what was started
// before it still under way.
template <class Wait, class Start>
KV4_HD bool kv4_start_queries(uint32_t (&started)[2], const Wait &wait_empty, const Start &start) {
  for (int w = 0; w < 2; ++w) {
    if (!wait_empty(w, (started[w] & 1) ^ 1u)) return false;
    start(w);
    ++started[w];
  }
  return true;
}
// Waits until none of them is under way.
template <class Wait>
KV4_HD void kv4_drain_queries(const uint32_t (&started)[2], const Wait &wait_full) {
  for (int w = 0; w < 2; ++w)
    if (started[w] > 0) wait_full(w, (started[w] - 1) & 1);
}

// Sort key of an accumulated weight: larger weights have larger keys, the two
// zeros the same, NaN the smallest.
KV4_HD uint32_t kv4_weight_key(uint32_t bits) {
  if ((bits & 0x7FFFFFFFu) > 0x7F800000u) return 0;
  if ((bits & 0x7FFFFFFFu) == 0) bits = 0;
  return (bits & 0x80000000u) != 0 ? ~bits : bits | 0x80000000u;
}

}  // namespace atomk
