// Attention of new tokens over the int8 paged cache, streaming kernel.
//
//   o_i = sum_j P'_ij c_j / sum_j (P'_ij / vs_j),
//   P'_ij = 2^(t_ij - z_i),  t_ij = (q_i . k_j) ks_j scale log2(e) + log2(vs_j)
//
// over the positions j <= i of the sequence (and j > i - window), which is
// softmax(scale q_i . K_j) V_j with K_j = ks_j k_j, V_j = vs_j c_j: k_j, c_j are
// the int8 codes, ks_j, vs_j their pages' scales.  The codes are exact in
// fp16, so both products run on fp16 operands with fp32 accumulation.
//   * q is taken to fp16 with a power of two per row (ka_row_power): exact for
//     values down to 2^-30 of the row's largest, since bf16 has fewer significant
//     bits; smaller ones are off by at most 2^-38 of the largest.
//   * P' is taken to fp16.  z_i is the running maximum of t_ij less 15: page
//     scales of one head may be far apart, and the largest p need not carry
//     the largest share of the result, so the reference is the share; what
//     fp16 drops is below 2^-39 of the largest one.
//   * the sum of p comes from P' before its rounding, in fp32, a page's worth
//     at a time (times 1 / vs).
//
// The cache is read once, so at decode sizes its bytes bound the kernel
// (6.5 TB/s: 23 bytes a clock and SM, against which the fp16 expansion of
// the codes costs about one instruction per byte and 32 lanes).  The codes
// are the first operand of both products (16 keys, or 16 columns of V, to an
// MMA) and the rows the second, so a row tile is one block of 8 rows, the
// query heads of a key head in a decode step, or two (16 rows: larger groups,
// or several new tokens, whose expansions are then shared; the rule is
// ka_few_rows).  Rows as the first operand, always 16, took 217 / 70.6 us
// where 8 take 179 / 56.7 (48 sequences of up to 16384 keys, 32/8 heads of
// 128 / one of 131072, 24/4 heads of 256): twice the MMAs and scores, half of
// them for rows that are not there.  The scores' fragment is transposed in
// registers between the products.
//
// Work is a list of items of a TK-key tile per warp,
// [sequence][key head][row tile][item], of which every CTA takes an equal
// contiguous share (one CTA per SM), so ragged batches and single long
// contexts fill the GPU alike.  Each warp keeps its own running maximum, sum
// and accumulator over its keys; warps join through shared memory at the end
// of a row tile, CTAs that share a row tile through partial results that the
// last of them to arrive adds in CTA order (the result does not depend on
// the order of arrival).
//
// Each warp feeds itself: a ring of TMA tiles, refilled by its own lanes as
// soon as it has used a tile, with the page ids and scales of its next tiles
// held one to a lane and fetched a batch ahead.  (A producer warp with a lane
// per consumer ran those lanes' divergent steps one after the other, about
// 1000 clocks a tile: 123 us for 131072 keys of 24/4 heads of 256, against
// the 41 us that the bytes take.)  The next row tile's first loads go out
// before this one is joined.
//
// K fragments are 16-byte reads of a token's codes in the order d = 64 c +
// 16 t + 4 s + e (q's fragments use the same order); V fragments come from
// ldmatrix.trans on code pairs, whose even and odd codes make two output
// tiles.  Tokens of an 8-token group are taken in the order tau, which keeps
// the swizzled K reads free of bank conflicts.
//
// Eight warps of three stages: twelve of two hide no more latency (220 us
// for the batch above, at 216, both with rows as the first operand).  Of the
// bytes' time the batch now takes 1.09 and the long context 1.36: 6.0 and 4.8
// TB/s.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kv_cache.cuh"
#include "kv_index.h"
#include "qk_rope.cuh"

namespace w4a8 {

constexpr float kKvLeastScale = 0x1p-80f;  // V scales below count as 0 (in the sum of p, as this)
constexpr int kKaMaxRows = 16;                   // rows of a tile: 8 or 16
constexpr int kKaTileBytes = 4096;               // one warp's K (or V) tile
constexpr int kKaMaxCtas = 160;

// NR: blocks of 8 rows (1 or 2) in a row tile.
template <int D, int NR>
struct KaCfg {
  static constexpr int TK = kKaTileBytes / D;  // keys of a warp's tile: 64, 32, 16
  static constexpr int KG = TK / 16;           // groups of 16 keys
  static constexpr int R = 8 * NR;
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = 3;
  static constexpr int kItem = kWarps * TK;  // keys of an item
  static constexpr int kSteps = D / 16;
  static constexpr bool kQRegs = D * NR <= 256;  // q fragments in registers
  static constexpr int kBatch = 32 / KG;       // tiles whose page ids a warp holds
  static constexpr uint32_t kRowBytes = D < 128 ? D : 128;  // bytes of a row in a TMA box
  static constexpr int kColBlocks = D / int(kRowBytes);
  static constexpr uint32_t kRing = kWarps * kStages * 2 * kKaTileBytes;
  // joining the warps: TPR threads a row, two columns each; the rows of the buffer are 4 words apart in banks
  static constexpr int TPR = kThreads / R, kJoinCols = 2 * TPR, kJoinStride = kJoinCols + 4;
  static constexpr uint32_t kJoin = kWarps * R * kJoinStride * 4;  // kJoinCols columns of every warp; the CTAs' weights
  static_assert(R * kKaMaxCtas * 4 <= kJoin, "weights of a row tile's CTAs");
  static constexpr uint32_t kQ = R * D * 2;
  static constexpr size_t kSmem = 1024 + kRing + kJoin + kQ + 4096;
  static constexpr int kSlotFloats = R * D + 2 * R;
};

struct KaParams {
  HeadRows q, out;
  KvCacheParams cache;
  KvBatchParams batch;
  float scale_log2;  // softmax scale times log2(e)
  int window;
  int group;         // query heads of a key head
  int box_shift;     // log2 of a TMA box's rows
  int both;          // the tensor-memory kernel is launched as well
  int sms;
  float* part;       // [CTA][2][kSlotFloats]; the tensor-memory kernel's parts before that
  unsigned* counters;  // [kKaMaxCtas] by CTA, then the tensor-memory kernel's, by split unit
  unsigned* err;
};

constexpr int kKaMaxWarps = 8, kKaMaxStages = 3;
struct KaShared {
  uint64_t full[kKaMaxWarps][kKaMaxStages];
  float scales[kKaMaxWarps][kKaMaxStages][3][4];  // ks, log2(vs), 1 / vs of each group of 16 keys
  float warp_z[kKaMaxWarps][kKaMaxRows];
  float warp_l[kKaMaxWarps][kKaMaxRows];
  float row_factor[kKaMaxRows];
  long long base;   // first item of sequence b0
  long long total;  // items of the batch
  int b0, small_only;
  int last;         // this CTA joins the row tile's partial results
  volatile int abort;
};

__device__ __forceinline__ bool ka_wait(uint64_t* bar, uint32_t parity, KaShared* sh, unsigned* err) {
  for (uint32_t i = 0; i < (1u << 20); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 1023u && sh->abort) return false;
  }
  sh->abort = 1;
  record_error(err, kErrTimeout);
  return false;
}

// Units (row tiles times key heads) of the batch that the tensor-memory kernel
// (kv_prefill.cuh) takes: those of the sequences of at least kKpMinRows rows,
// where that pays (kv_tiles_pay).  0 where the streaming kernel takes all.
template <int D>
__device__ __forceinline__ int kp_units(const KaParams& p) {  // whole warp
  const int lane = threadIdx.x & 31;
  int units = 0, most = 0;
  long long work = 0;
  for (int b0 = 0; b0 < p.batch.batch; b0 += 32) {
    if (b0 + lane < p.batch.batch) {
      const KvSeq s = kv_load_seq(p.batch, b0 + lane, p.cache.page_shift);
      if (kv_has_tiles(s, p.group)) {
        const KvTiles t = kv_tiles_of(s, p.group, p.window, kp_rows(D));
        units += t.tiles;
        work += t.row_keys;
        most = max(most, t.keys);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    units += __shfl_xor_sync(0xffffffffu, units, off);
    work += __shfl_xor_sync(0xffffffffu, work, off);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
  }
  const int heads = p.cache.kv_heads;
  return kv_tiles_pay((long long)units * heads, work * heads, most, D, p.sms) ? units * heads : 0;
}

// Row tiles of a sequence, and items of each (the same for all of them: a
// tile skips the keys outside its own range).
template <int D, int NR>
__device__ __forceinline__ void ka_counts(const KvSeq& s, const KaParams& p, bool small_only, int& tiles, int& items) {
  const KvRange r = kv_range(s, 0, s.q_len - 1, p.window);
  using C = KaCfg<D, NR>;
  const int lo = r.lo & ~(C::TK - 1);
  tiles = (s.q_len * p.group + C::R - 1) / C::R;
  items = s.q_len == 0 ? 0 : (s.kv_len - lo + C::kItem - 1) / C::kItem;
  if (small_only && s.q_len * p.group >= kKpMinRows) tiles = items = 0;
}

// The row tile at the front of a CTA's range.
struct KaSeg {
  KvSeq s;
  int b, head, tile;
  int item0, item1, items;  // of the tile's `items`, this CTA has [item0, item1)
  long long start;          // first item of the tile in the batch
  int key0;                 // first key of its item 0
  KvRange range;
};

template <int D, int NR>
struct KaWalk {
  using C = KaCfg<D, NR>;
  long long pos, end, base;
  int b, tiles, items;
  bool small_only;
  KvSeq s;
  __device__ __forceinline__ void load(const KaParams& p) {
    s = kv_load_seq(p.batch, b, p.cache.page_shift);
    ka_counts<D, NR>(s, p, small_only, tiles, items);
  }
  __device__ __forceinline__ bool next(const KaParams& p, KaSeg& g) {
    if (pos >= end) return false;
    while (pos >= base + (long long)p.cache.kv_heads * tiles * items) {
      base += (long long)p.cache.kv_heads * tiles * items;
      ++b;
      load(p);
    }
    const long long local = pos - base;
    const long long unit = local / items;
    g.s = s;
    g.b = b;
    g.items = items;
    g.item0 = int(local - unit * items);
    g.head = int(unit / tiles);
    g.tile = int(unit - (long long)g.head * tiles);
    g.start = base + unit * items;
    const long long left = end - pos;
    g.item1 = left < items - g.item0 ? g.item0 + int(left) : items;
    g.key0 = kv_range(s, 0, s.q_len - 1, p.window).lo & ~(C::TK - 1);
    const int j0 = g.tile * C::R / p.group;
    const int last_row = min(s.q_len * p.group, (g.tile + 1) * C::R) - 1;
    g.range = kv_range(s, j0, last_row / p.group, p.window);
    pos += g.item1 - g.item0;
    return true;
  }
};

__device__ __forceinline__ void ka_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two int8 codes (already xor 0x80: code + 128) as fp16: the byte under the
// high byte 0x64 is 1024 + code + 128, less 1152 (exact).
__device__ __forceinline__ uint32_t ka_codes(uint32_t biased, uint32_t sel) {
  const uint32_t w = prmt(biased, 0x64646464u, sel);
  const uint32_t off = 0x64806480u;
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&off));
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The power of two e that takes a row of q to fp16: its largest value lands in [2^13, 2^14), for any finite value (-114
// at 2^127; at the small end 126, as 2^-e must be a normal number too: values below 2^-113 land below 2^13).
__device__ __forceinline__ int ka_row_power(float top) { return min(126, 127 + 13 - int(__float_as_uint(top) >> 23)); }

template <int D>
__device__ __forceinline__ uint32_t ka_tau(uint32_t i) {
  return D < 128 ? i : (i >> 1) | ((i & 1u) << 2);
}
// Byte offset of 16-byte chunk c of row r in a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t ka_at(uint32_t r, uint32_t c) {
  if constexpr (D < 128) return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
  return (c >> 3) * uint32_t(kKaTileBytes / D * 128) + r * 128u + (((c & 7u) ^ (r & 7u)) << 4);
}

// Transpose of an 8 x 8 matrix of 16-bit values held as a fragment (row lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t ka_transpose(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

template <int D, int NR>
__global__ void __launch_bounds__(KaCfg<D, NR>::kThreads, 1)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const KaParams p) {
  using C = KaCfg<D, NR>;
  extern __shared__ __align__(1024) uint8_t ka_smem[];
  const uint32_t ring = (smem_u32(ka_smem) + 1023u) & ~1023u;
  uint8_t* after = ka_smem + (ring - smem_u32(ka_smem)) + C::kRing;
  float* join = reinterpret_cast<float*>(after);
  uint32_t* qf = reinterpret_cast<uint32_t*>(after + C::kJoin);  // [step][lane][4]
  KaShared* sh = reinterpret_cast<KaShared*>(after + C::kJoin + C::kQ);
  static_assert(sizeof(KaShared) <= 4096, "shared block");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();
  if (threadIdx.x == 0) {
    for (int w = 0; w < C::kWarps; ++w)
      for (int s = 0; s < C::kStages; ++s) {
        mbar_init(&sh->full[w][s], 1);
      }
    sh->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    // The batch's items, then the sequence that holds this CTA's first one.
    const bool small_only = p.both && kp_units<D>(p) > 0;
    long long total = 0;
    for (int b0 = 0; b0 < p.batch.batch; b0 += 32) {
      int tiles = 0, items = 0;
      if (b0 + lane < p.batch.batch) {
        const KvSeq s = kv_load_seq(p.batch, b0 + lane, p.cache.page_shift);
        if (s.bad) record_error(p.err, kErrInput);
        ka_counts<D, NR>(s, p, small_only, tiles, items);
      }
      total += (long long)p.cache.kv_heads * tiles * items;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    const long long ctas = total < gridDim.x ? total : gridDim.x;
    const long long i0 = int(blockIdx.x) < ctas ? ka_first_item(blockIdx.x, total, ctas) : total;
    long long before = 0, base = 0;
    int at = -1;
    for (int b0 = 0; b0 < p.batch.batch && at < 0 && i0 < total; b0 += 32) {
      int tiles = 0, items = 0;
      if (b0 + lane < p.batch.batch)
        ka_counts<D, NR>(kv_load_seq(p.batch, b0 + lane, p.cache.page_shift), p, small_only, tiles, items);
      const long long own = (long long)p.cache.kv_heads * tiles * items;
      long long sum = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + sum > i0);
      if (past) {
        const int l = __ffs(past) - 1;
        at = b0 + l;
        base = before + __shfl_sync(0xffffffffu, sum - own, l);
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      sh->total = total;
      sh->b0 = at;
      sh->base = base;
      sh->small_only = small_only;
    }
  }
  __syncthreads();
  const long long total = sh->total;
  const long long ctas = total < gridDim.x ? total : gridDim.x;
  if (int(blockIdx.x) >= ctas) return;
  const long long i0 = ka_first_item(blockIdx.x, total, ctas);
  KaWalk<D, NR> walk;
  walk.pos = i0;
  walk.end = ka_first_item(blockIdx.x + 1, total, ctas);
  walk.base = sh->base;
  walk.b = sh->b0;
  walk.small_only = sh->small_only;
  walk.load(p);

  // -------------------------------------------------- the warp's feed
  // Tiles of a row tile that this warp takes: items [fi, fend) with a key in range.  Lane l holds the page id and
  // scales of key group l % KG of tile fbase + l / KG; the batch after it is on its way.
  const int per = 1 << (p.box_shift - 4);  // key groups of a TMA box
  const int fgroup = lane % C::KG, ftile = lane / C::KG;
  int fi = 0, fend = 0, fbase = 0, fstage = 0, fid = -1, nraw = -1;
  float fks = 0.f, fvs = 0.f;
  KaSeg fseg{};
  auto group_key = [&](int item) { return fseg.key0 + (item * C::kWarps + warp) * C::TK + 16 * fgroup; };
  auto fetch_raw = [&](int base) {
    const int item = base + ftile;
    return item < fend && group_key(item) >= fseg.range.lo && group_key(item) < fseg.range.hi
               ? __ldg(p.batch.table + (long long)fseg.b * p.batch.table_stride + (group_key(item) >> p.cache.page_shift))
               : -1;
  };
  auto take_batch = [&](int base) {  // nraw, fetched for `base`, becomes the batch at hand
    fid = nraw;
    if (fid >= p.cache.pages ||
        (fid < 0 && base + ftile < fend && group_key(base + ftile) >= fseg.range.lo && group_key(base + ftile) < fseg.range.hi)) {
      record_error(p.err, kErrInput);
      fid = -1;
    }
    fbase = base;
    const long long at = (long long)max(fid, 0) * p.cache.kv_heads + fseg.head;
    fks = __ldg(p.cache.scales[0] + at);
    fvs = __ldg(p.cache.scales[1] + at);
    nraw = fetch_raw(base + C::kBatch);
  };
  // Loads of tile fi into the next stage (its scales beside it).
  auto issue = [&]() {
    if (fi == fbase + C::kBatch) take_batch(fi);
    const bool mine = fi == fbase + ftile;
    const bool box = mine && fid >= 0 && fgroup % per == 0;
    const unsigned boxes = __popc(__ballot_sync(0xffffffffu, box));
    uint64_t* bar = &sh->full[warp][fstage];
    if (lane == 0) mbar_arrive_expect_tx(bar, boxes * 2u * (uint32_t(D) << p.box_shift));
    __syncwarp();
    if (box) {
      const uint32_t kt = ring + uint32_t((warp * C::kStages + fstage) * 2) * kKaTileBytes + uint32_t(16 * fgroup) * C::kRowBytes;
      const int row = int((((long long)fid * p.cache.kv_heads + fseg.head) << p.cache.page_shift) +
                          (group_key(fi) & ((1 << p.cache.page_shift) - 1)));
#pragma unroll
      for (int cb = 0; cb < C::kColBlocks; ++cb) {
        tma_load_2d(kt + uint32_t(cb) * C::TK * 128u, &tmap_k, bar, cb * 128, row);
        tma_load_2d(kt + kKaTileBytes + uint32_t(cb) * C::TK * 128u, &tmap_v, bar, cb * 128, row);
      }
    }
    if (mine) {
      const float vs = fid >= 0 ? fmaxf(fvs, kKvLeastScale) : kKvLeastScale;
      sh->scales[warp][fstage][0][fgroup] = fid >= 0 ? fks : 0.f;
      sh->scales[warp][fstage][1][fgroup] = __log2f(vs);
      sh->scales[warp][fstage][2][fgroup] = __fdividef(1.f, vs);
    }
    __syncwarp();
    ++fi;
    if (++fstage == C::kStages) fstage = 0;
  };
  // The first loads of a row tile; its tiles are [nfirst, fend).
  int nfirst = 0;
  auto start = [&](const KaSeg& s) {
    fseg = s;
    // items with key < hi, and key + TK > lo (key0 is at most TK - 1 below the lowest lo of the sequence)
    const int first = s.range.lo - s.key0 - warp * C::TK;
    fi = max(s.item0, first > 0 ? first / C::kItem + (first % C::kItem >= C::TK ? 1 : 0) : 0);
    fend = min(s.item1, (s.range.hi - s.key0 - warp * C::TK + C::kItem - 1) / C::kItem);
    nfirst = fi;
    fseg.range.lo = kv_first_key(fseg.range, p.cache.page_shift);  // (what the feed looks up starts there)
    nraw = fetch_raw(fi);
    if (fi < fend) take_batch(fi);
    for (int n = 0; n < C::kStages && fi < fend; ++n) issue();
  };

  // -------------------------------------------------- row tiles
  const int g = lane >> 2, t = lane & 3;
  const int tid = threadIdx.x;
  bool ok = true;  // every warp goes through every barrier below, even after a wait that gave up
  int stage = 0;
  uint32_t phase = 0;
  KaSeg seg, nxt;
  bool have = walk.next(p, seg);
  if (have) start(seg);
  while (have) {
    const int c_first_item = nfirst, c_end_item = fend;
    // ---- q rows of the tile into fragments: half a warp per row
    const int rows = seg.s.q_len * p.group;
    if (warp < C::R / 2) {
      const int r = 2 * warp + (lane >> 4), l16 = lane & 15;
      const int row = seg.tile * C::R + r;
      float v[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) v[i] = 0.f;
      if (row < rows) {
        const int j = row / p.group, h = seg.head * p.group + row - j * p.group;
        const uint16_t* src = p.q.data + (long long)(seg.s.start + j) * p.q.token + h * p.q.head + l16 * (D / 16);
#pragma unroll
        for (int i = 0; i < D / 16; i += 4) {
          const uint2 raw = __ldcg(reinterpret_cast<const uint2*>(src + i));
          v[i] = __uint_as_float(raw.x << 16);
          v[i + 1] = __uint_as_float(raw.x & 0xFFFF0000u);
          v[i + 2] = __uint_as_float(raw.y << 16);
          v[i + 3] = __uint_as_float(raw.y & 0xFFFF0000u);
        }
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const int e = ka_row_power(top);
      // (a negative scale goes into q, so that larger products stay larger scores)
      const float up = copysignf(__uint_as_float(uint32_t(127 + e) << 23), p.scale_log2);
      if (l16 == 0) sh->row_factor[r] = __uint_as_float(uint32_t(127 - e) << 23) * fabsf(p.scale_log2);
#pragma unroll
      for (int i = 0; i < D / 16; i += 2) {
        const int d = l16 * (D / 16) + i;
        const int step = (d >> 6) * 4 + ((d >> 2) & 3), ln = (r & 7) * 4 + ((d >> 4) & 3);
        const int reg = ((d & 2) ? NR : 0) + (r >> 3);
        const __half2 h = __floats2half2_rn(v[i] * up, v[i + 1] * up);
        qf[(step * 32 + ln) * (2 * NR) + reg] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    __syncthreads();
    auto q_frag = [&](int step, uint32_t (&f)[2 * NR]) {  // b0 of every row block, then b1
      if constexpr (NR == 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(qf + (step * 32 + lane) * 4);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(qf + (step * 32 + lane) * 2);
        f[0] = v.x, f[1] = v.y;
      }
    };
    uint32_t qr[C::kQRegs ? C::kSteps : 1][2 * NR];
    if constexpr (C::kQRegs) {
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s) q_frag(s, qr[s]);
    }
    // this lane's rows: 8 n + 2 t + e
    float f[NR][2];
    int lim[NR][2], low[NR][2];  // the last key a row sees, and the first
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e, row = min(seg.tile * C::R + r, rows - 1);
        f[n][e] = sh->row_factor[r];
        lim[n][e] = seg.s.kv_len - seg.s.q_len + row / p.group;
        low[n][e] = p.window > 0 ? lim[n][e] - p.window + 1 : 0;
      }
    const int lim_min = seg.s.kv_len - seg.s.q_len + seg.tile * C::R / p.group;
    const int low_max = p.window > 0 ? seg.range.hi - p.window : 0;

    float o[D / 16][NR][4];  // (even d, row e = 0), (even, 1), (odd, 0), (odd, 1) of 16 columns
    float z[NR][2], l[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
      z[n][0] = z[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    for (int item = c_first_item; item < c_end_item; ++item) {
      const int key = seg.key0 + (item * C::kWarps + warp) * C::TK;
      if (ok) ok = __all_sync(0xffffffffu, ka_wait(&sh->full[warp][stage], phase, sh, p.err));
      if (!ok) break;
      const uint32_t kt = ring + uint32_t((warp * C::kStages + stage) * 2) * kKaTileBytes, vt = kt + kKaTileBytes;
      // ---- scores: keys 16 kb + tau(g) and 16 kb + 8 + tau(g) of every row
      float s[C::KG][NR][4];
#pragma unroll
      for (int kb = 0; kb < C::KG; ++kb)
#pragma unroll
        for (int n = 0; n < NR; ++n) s[kb][n][0] = s[kb][n][1] = s[kb][n][2] = s[kb][n][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t qs[4][2 * NR];
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          if constexpr (C::kQRegs) {
#pragma unroll
            for (int i = 0; i < 2 * NR; ++i) qs[st][i] = qr[4 * c + st][i];
          } else {
            q_frag(4 * c + st, qs[st]);
          }
        }
#pragma unroll
        for (int kb = 0; kb < C::KG; ++kb) {
          uint32_t w[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[h][0]), "=r"(w[h][1]), "=r"(w[h][2]), "=r"(w[h][3])
                         : "r"(kt + ka_at<D>(uint32_t(16 * kb + 8 * h) + ka_tau<D>(g), uint32_t(4 * c + t))));
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint32_t x = w[0][st] ^ 0x80808080u, y = w[1][st] ^ 0x80808080u;
            const uint32_t a[4] = {ka_codes(x, 0x4140u), ka_codes(y, 0x4140u), ka_codes(x, 0x4342u), ka_codes(y, 0x4342u)};
#pragma unroll
            for (int n = 0; n < NR; ++n) ka_mma(s[kb][n], a, qs[st][n], qs[st][NR + n]);
          }
        }
      }
      // ---- the rows' references
      const float* ks = sh->scales[warp][stage][0];
      const float* lv = sh->scales[warp][stage][1];
      const float* iv = sh->scales[warp][stage][2];
      const bool edge = key + C::TK - 1 > lim_min || key < low_max;
      if (edge) {
#pragma unroll
        for (int kb = 0; kb < C::KG; ++kb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = key + 16 * kb + 8 * h + int(ka_tau<D>(g));
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (at > lim[n][e] || at < low[n][e]) s[kb][n][2 * h + e] = -INFINITY;
          }
      }
      float x[NR][2];
      bool more_z = false;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[n][e] = -INFINITY;
#pragma unroll
          for (int kb = 0; kb < C::KG; ++kb)
            // (fmaxf drops the NaN of a wholly masked group under a K scale of 0)
            x[n][e] = fmaxf(x[n][e], fmaf(fmaxf(s[kb][n][e], s[kb][n][2 + e]), f[n][e] * ks[kb], lv[kb]));
          // (rounded up: no t of the tile is more than 15 above z, however large the scores are)
          x[n][e] = __fadd_ru(x[n][e], -15.f);
          more_z |= x[n][e] > z[n][e];
        }
      if (__any_sync(0xffffffffu, more_z)) {  // (a row's keys are spread over 8 lanes)
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) x[n][e] = fmaxf(x[n][e], __shfl_xor_sync(0xffffffffu, x[n][e], off));
            const float nz = fmaxf(z[n][e], x[n][e]);
            const float grow = z[n][e] == -INFINITY ? 0.f : ex2(z[n][e] - nz);
            l[n][e] *= grow;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[i][n][e] *= grow;
              o[i][n][2 + e] *= grow;
            }
            z[n][e] = nz;
          }
      }
      // ---- P', the sum of p, and the product with V
#pragma unroll
      for (int kb = 0; kb < C::KG; ++kb) {
        const float w = iv[kb];
        uint32_t b[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float kf = f[n][e] * ks[kb], ref = z[n][e] == -INFINITY ? 0.f : z[n][e];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float sc = s[kb][n][2 * h + e];
              // (t rounded as it is in z: in one multiply-add with z they would differ by what t's rounding lost)
              pr[2 * h + e] = ex2(fmaf(sc, kf, lv[kb]) - ref);
              if (edge && sc == -INFINITY) pr[2 * h + e] = 0.f;  // (a masked score times a K scale of 0 is no zero)
            }
            l[n][e] = fmaf(pr[e] + pr[2 + e], w, l[n][e]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __half2 hh = __floats2half2_rn(pr[2 * h], pr[2 * h + 1]);
            b[n][h] = ka_transpose(*reinterpret_cast<const uint32_t*>(&hh));
            if (w >= 1.f / kKvLeastScale) b[n][h] = 0u;  // a page without a V scale: its values are zeros
          }
        }
        const uint32_t vrow = uint32_t(16 * kb + ((lane >> 3) & 1) * 8) + ka_tau<D>(lane & 7);
#pragma unroll
        for (int c2 = 0; c2 < D / 32; ++c2) {
          uint32_t r[4];
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                       : "r"(vt + ka_at<D>(vrow, uint32_t(2 * c2 + (lane >> 4)))));
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] ^= 0x80808080u;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t a[4] = {ka_codes(r[2 * hf], 0x4240u), ka_codes(r[2 * hf], 0x4341u),
                                   ka_codes(r[2 * hf + 1], 0x4240u), ka_codes(r[2 * hf + 1], 0x4341u)};
#pragma unroll
            for (int n = 0; n < NR; ++n) ka_mma(o[2 * c2 + hf][n], a, b[n][0], b[n][1]);
          }
        }
      }
      __syncwarp();  // every lane has used the tile: its stage takes the next one
      if (fi < fend) issue();
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
    }

    // ---- the next row tile's loads go out, then join the warps
    const bool more = walk.next(p, nxt);
    if (!more) pdl_launch_dependents();  // (late: the next kernel's bounded waits must not last as long as this one)
    if (more && ok) start(nxt);
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
        if (g == 0) {
          sh->warp_z[warp][8 * n + 2 * t + e] = z[n][e];
          sh->warp_l[warp][8 * n + 2 * t + e] = l[n][e];
        }
      }
    __syncthreads();
    float wt[NR][2];  // of this warp's sums
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, sh->warp_z[w][8 * n + 2 * t + e]);
        wt[n][e] = z[n][e] == -INFINITY ? 0.f : ex2(z[n][e] - top);
      }
    // this thread's place in the joined tile: row jr, columns 2 jc, 2 jc + 1 of each kJoinCols
    const int jr = tid / C::TPR, jc = tid % C::TPR;
    float jz = -INFINITY, jl = 0.f;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) jz = fmaxf(jz, sh->warp_z[w][jr]);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w)
      if (sh->warp_z[w][jr] != -INFINITY) jl += sh->warp_l[w][jr] * ex2(sh->warp_z[w][jr] - jz);
    const bool whole = seg.item0 == 0 && seg.item1 == seg.items;
    const int slot = int(blockIdx.x) * 2 + (i0 >= seg.start ? 0 : 1);
    float* part = p.part + (size_t)slot * C::kSlotFloats;
    const int row = seg.tile * C::R + jr;
    const int oj = row / p.group, oh = seg.head * p.group + row - oj * p.group;
    uint16_t* dst = p.out.data + (long long)(seg.s.start + oj) * p.out.token + oh * p.out.head;
    const float norm = jl > 0.f ? __fdiv_rn(1.f, jl) : 0.f;
    constexpr int kCols = C::kJoinCols < D ? C::kJoinCols : D;
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += kCols) {
      float* mine = join + warp * (C::R * C::kJoinStride);
#pragma unroll
      for (int i = 0; i < kCols / 16; ++i)
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float(&v)[4] = o[c0 / 16 + i][n];
            *reinterpret_cast<float2*>(mine + (8 * n + 2 * t + e) * C::kJoinStride + 16 * i + 2 * g) =
                make_float2(v[e] * wt[n][e], v[2 + e] * wt[n][e]);
          }
      __syncthreads();
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(join + (w * C::R + jr) * C::kJoinStride + 2 * jc);
        x += v.x;
        y += v.y;
      }
      if (!whole) {
        *reinterpret_cast<float2*>(part + jr * D + c0 + 2 * jc) = make_float2(x, y);
      } else if (row < rows && ok) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x * norm, y * norm);
        *reinterpret_cast<__nv_bfloat162*>(dst + c0 + 2 * jc) = b;
      }
      __syncthreads();
    }
    if (!whole) {
      if (jc == 0) {
        part[C::R * D + jr] = jz;
        part[C::R * D + C::R + jr] = jl;
      }
      const int c_first = ka_item_cta(seg.start, total, ctas), c_last = ka_item_cta(seg.start + seg.items - 1, total, ctas);
      __threadfence();
      __syncthreads();
      if (tid == 0) sh->last = atomicAdd(p.counters + c_first, 1u) == unsigned(c_last - c_first);
      __syncthreads();
      if (sh->last) {
        __threadfence();
        // Slot of CTA c: its first row tile's, but for the CTA in which the tile starts behind another one.  A row's
        // threads take the CTAs' maxima and sums, one each at a time, and leave the CTAs' weights in shared memory; the
        // accumulators then come in eight at a time (one at a time waits a round trip to L2 for each).
        const int n_cta = c_last - c_first + 1;
        const float* slot0 = p.part + (size_t)(c_first * 2 + (ka_first_item(c_first, total, ctas) >= seg.start ? 0 : 1)) * C::kSlotFloats;
        auto slot_of = [&](int c) {
          return c == 0 ? slot0 : p.part + (size_t)((c_first + c) * 2) * C::kSlotFloats;
        };
        float* weight = join + jr * kKaMaxCtas;
        float top = -INFINITY, sum = 0.f;
        for (int c = jc; c < n_cta; c += C::TPR) {
          const float* m = slot_of(c) + C::R * D + jr;
          const float cz = __ldcg(m), cl = __ldcg(m + C::R);
          const float nt = fmaxf(top, cz);
          if (nt > -INFINITY) sum = sum * ex2(top - nt) + (cz > -INFINITY ? cl * ex2(cz - nt) : 0.f);
          top = nt;
          weight[c] = cz;
        }
#pragma unroll
        for (int off = 1; off < C::TPR; off <<= 1) {
          const float ot = __shfl_xor_sync(0xffffffffu, top, off), os = __shfl_xor_sync(0xffffffffu, sum, off);
          const float nt = fmaxf(top, ot);
          if (nt > -INFINITY) sum = sum * ex2(top - nt) + os * ex2(ot - nt);
          top = nt;
        }
        for (int c = jc; c < n_cta; c += C::TPR) weight[c] = weight[c] == -INFINITY ? 0.f : ex2(weight[c] - top);
        __syncwarp();
        constexpr int VW = D / C::TPR < 4 ? D / C::TPR : 4, NV = D / C::TPR / VW;  // columns VW jc .. of each VW TPR
        float acc[NV][VW];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < VW; ++k) acc[i][k] = 0.f;
        constexpr int kAhead = D / C::TPR <= 8 ? 8 : 4;
        for (int c0 = 0; c0 < n_cta; c0 += kAhead) {
          float v[kAhead][NV][VW];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const float* src = slot_of(min(c0 + u, n_cta - 1)) + jr * D + jc * VW;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              if constexpr (VW == 4) {
                const float4 q = __ldcg(reinterpret_cast<const float4*>(src + i * VW * C::TPR));
                v[u][i][0] = q.x, v[u][i][1] = q.y, v[u][i][2] = q.z, v[u][i][3] = q.w;
              } else {
                const float2 q = __ldcg(reinterpret_cast<const float2*>(src + i * VW * C::TPR));
                v[u][i][0] = q.x, v[u][i][1] = q.y;
              }
            }
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const float f = c0 + u < n_cta ? weight[c0 + u] : 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int k = 0; k < VW; ++k) acc[i][k] += f * v[u][i][k];
          }
        }
        const float n = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
        if (row < rows) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < VW; k += 2)
              *reinterpret_cast<__nv_bfloat162*>(dst + i * VW * C::TPR + jc * VW + k) =
                  __floats2bfloat162_rn(acc[i][k] * n, acc[i][k + 1] * n);
        }
        if (tid == 0) p.counters[c_first] = 0u;  // ready for the next launch on this workspace
      }
    }
    __syncthreads();  // q fragments, warp_z, warp_l and the join buffer are free again
    seg = nxt;
    have = more;
  }
  if (sh->abort) {
    // let the copies in flight land before the CTA exits (bounded: 50 us)
    unsigned long long ta, tb;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(ta));
    do {
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(tb));
    } while (tb - ta < 50000ull);
  }
}

}  // namespace w4a8
