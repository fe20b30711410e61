// Index arithmetic of the paged int8 cache and of the batch that is written
// into it or attends over it.  Plain functions without device code, so that
// the host (argument checks, tests) and the kernels share them.
//
// A batch is `batch` sequences.  Sequence b has q_len = q_start[b + 1] -
// q_start[b] new tokens, which are the last of the kv_len[b] tokens that the
// cache holds of it; new token j sits at position kv_len - q_len + j.
// Position t of a sequence is place t % page of page table[b][t / page].
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define W4A8_HD __host__ __device__ __forceinline__
#else
#define W4A8_HD inline
#endif

namespace w4a8 {

constexpr int64_t kKvMaxTokens = int64_t(1) << 30;  // that a block table has places for, a sequence

struct KvSeq {
  int start;    // row of its first new token
  int q_len;    // new tokens
  int kv_len;   // tokens in the cache, the new ones among them
  bool bad;     // the batch's numbers do not fit together: nothing is done for it
};

// What a sequence's numbers say, or an empty, bad sequence where they leave
// the buffers: rows outside [0, tokens], more new tokens than the cache
// holds, or a length past the block table.
W4A8_HD KvSeq kv_seq(int start, int end, int kv_len, int64_t tokens, int64_t table_tokens) {
  KvSeq s;
  s.bad = start < 0 || end < start || int64_t(end) > tokens || kv_len < 0 || end - start > kv_len ||
          int64_t(kv_len) > table_tokens;
  s.start = s.bad ? 0 : start;
  s.q_len = s.bad ? 0 : end - start;
  s.kv_len = s.bad ? 0 : kv_len;
  return s;
}

// Pages that a sequence's new tokens lie in: [kv_first_page, + kv_touched).
W4A8_HD int kv_first_page(const KvSeq& s, int page_shift) { return (s.kv_len - s.q_len) >> page_shift; }
W4A8_HD int kv_touched(const KvSeq& s, int page_shift) {
  return s.q_len == 0 ? 0 : ((s.kv_len - 1) >> page_shift) - kv_first_page(s, page_shift) + 1;
}

// An upper bound of the touched pages of a batch that only needs host
// numbers: n new tokens lie in at most (n - 2) / page + 2 <= n / page + 2
// pages of a sequence (n of them where that is fewer).
W4A8_HD int64_t kv_touched_bound(int64_t tokens, int64_t batch, int page) {
  const int64_t a = tokens / page + 2 * batch;
  return a < tokens ? a : tokens;
}

// Keys that a row tile sees: of the new tokens j0 .. j1 (inclusive) the
// first one's window starts the range and the last one's position ends it.
struct KvRange {
  int lo, hi;  // [lo, hi)
};
W4A8_HD KvRange kv_range(const KvSeq& s, int j0, int j1, int window) {
  KvRange r;
  const int p0 = s.kv_len - s.q_len + j0;
  r.hi = s.kv_len - s.q_len + j1 + 1;
  r.lo = (window > 0 && p0 - window + 1 > 0) ? p0 - window + 1 : 0;
  return r;
}

// The first key of the pages that a range sees.  The kernels' first tile may
// start before it, in pages that the window has passed and the caller may
// have given to another sequence: their table entries are not read.
W4A8_HD int kv_first_key(const KvRange& r, int page_shift) { return (r.lo >> page_shift) << page_shift; }

// Whether the tensor-memory attention kernel takes a batch's sequences of many
// rows, by both kernels' estimated times in ns (whole numbers, so that the two
// kernels, which each ask, agree).  `units` are its row tiles times key heads,
// row_keys the sum of rows * (keys + 512) times key heads, most_keys the longest
// range.  The streaming kernel does 140 TFLOP/s after 8 us and spends on each
// row tile what 512 more keys would cost; the other one takes rate ns for 64 keys
// of a unit after its base, with units in waves of one to an SM, or up to four
// parts of each.  Measured, streaming / tensor-memory, us: 130 new tokens of
// 32/8 heads of 128 on 230 keys 14 / 28, 260 of 8/2 on 6000 keys 53 / 58, 500
// of 8/2 on 6000 90 / 58, 260 of 12/1 heads of 256 on 6000 133 / 70.
// All of them without a window: under one, both estimates take the sequence's
// whole range of keys for each row's and each tile's, and are too long.
constexpr int kKpMaxParts = 4;
W4A8_HD bool kv_tiles_pay(int64_t units, int64_t row_keys, int64_t most_keys, int D, int sms) {
  if (units == 0) return false;
  const int64_t base = D == 64 ? 20000 : D == 128 ? 27000 : 33000, rate = D == 64 ? 1150 : D == 128 ? 1400 : 1500;
  const int64_t parts = units * kKpMaxParts <= sms ? kKpMaxParts : units < sms ? sms / units : 1;
  const int64_t waves = (units * parts + sms - 1) / sms;
  // (divided first: rows * heads of a q that fits in memory, times 2^30 keys and D, would pass 64 bits)
  return 8000 + row_keys / 35000 * D > base + rate * ((most_keys + 63) / 64) * waves / parts;
}

// What a sequence adds to that estimate: nothing below kKpMinRows rows (new
// tokens x query heads of a key head), which the streaming kernel keeps.
constexpr int kKpMinRows = 128;
W4A8_HD constexpr int kp_rows(int D) { return D <= 128 ? 256 : 128; }  // of a row tile
struct KvTiles {  // of a sequence that has any (kv_has_tiles)
  int tiles, keys;
  int64_t row_keys;
};
W4A8_HD bool kv_has_tiles(const KvSeq& s, int group) { return s.q_len * group >= kKpMinRows; }
W4A8_HD KvTiles kv_tiles_of(const KvSeq& s, int group, int window, int tile_rows) {
  const int rows = s.q_len * group;
  const KvRange r = kv_range(s, 0, s.q_len - 1, window);
  return KvTiles{(rows + tile_rows - 1) / tile_rows, r.hi - r.lo, int64_t(rows) * (r.hi - r.lo + 512)};
}

// The host knows only the batch's totals and the block table's width: it
// launches the tensor-memory kernel too where that would pay at the table's
// width, and the average sequence has rows for it or the total is so large
// that a few of many sequences may (a launch that finds nothing to do costs
// 5 us).
constexpr int64_t kKpMinCtas = 4, kKpSureCtas = 32;
inline int64_t kv_min(int64_t a, int64_t b) { return a < b ? a : b; }
// Tiles of that many rows that the batch may have, for each key head.
inline int64_t kp_tiles_bound(int64_t rows, int64_t batch, int tile_rows) {
  return rows / tile_rows + kv_min(batch, rows / kKpMinRows);
}
inline bool kv_tiles_may_pay(int64_t tokens, int64_t batch, int group, int kv_heads, int64_t capacity, int window, int D,
                             int sms) {
  const int64_t rows = tokens * group, bound = kp_tiles_bound(rows, batch, 256) * kv_heads;
  const int64_t keys = window > 0 ? kv_min(capacity, int64_t(window) + tokens) : capacity;
  return bound >= kKpMinCtas && (bound >= kKpSureCtas || rows >= kKpMinRows * batch) &&
         kv_tiles_pay(kp_tiles_bound(rows, batch, kp_rows(D)) * kv_heads, rows * (keys + 512) * kv_heads, keys, D, sms);
}

// The streaming kernel's items over its CTAs: a CTA's share of `total` items
// among the first `ctas` = min(CTAs, total) CTAs, and the CTA of an item.
W4A8_HD long long ka_first_item(long long c, long long total, long long ctas) { return total * c / ctas; }
W4A8_HD int ka_item_cta(long long i, long long total, long long ctas) {
  return int(((i + 1) * ctas + total - 1) / total - 1);
}

}  // namespace w4a8
