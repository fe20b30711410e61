// Attention of new tokens over the int8 paged cache, streaming kernel.
//
//   o_i = sum_j P'_ij c_j / sum_j (P'_ij / vs_j),
//   P'_ij = 2^(t_ij - z_i),  t_ij = (q_i . k_j) ks_j scale log2(e) + log2(vs_j)
//
// over the positions j <= i of the sequence (and j > i - window), which is
// softmax(scale q_i . K_j) V_j with K_j = ks_j k_j, V_j = vs_j c_j: k_j, c_j are
// the int8 codes, ks_j, vs_j their pages' scales.  The codes are exact in
// fp16, so both products run on fp16 operands with fp32 accumulation.
//   * q is taken to fp16 with a power of two per row (exact: bf16 has fewer
//     significant bits, the power keeps its range).
//   * P' is taken to fp16.  z_i is the running maximum of t_ij less 15: page
//     scales of one head may be far apart, and the largest p need not carry
//     the largest share of the result, so the reference is the share; what
//     fp16 drops is below 2^-39 of the largest one.
//   * the sum of p comes from P' before its rounding, in fp32, a page's worth
//     at a time (times 1 / vs).
//
// The cache is read once, so at decode sizes its bytes bound the kernel
// (6.5 TB/s: 23 bytes a clock and SM, against which the fp16 expansion of
// the codes costs about one instruction per byte and 32 lanes).  A row tile
// is 16 rows, the query heads of one key head (and neighbouring new tokens,
// if the group is smaller); work is a list of items of a TK-key tile per
// warp,
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
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kv_cache.cuh"
#include "kv_index.h"
#include "qk_rope.cuh"

namespace w4a8 {

constexpr float kKvLeastScale = 0x1p-80f;  // V scales below count as 0 (in the sum of p, as this)
constexpr int kKaRows = 16;
constexpr int kKaTileBytes = 4096;               // one warp's K (or V) tile
constexpr int kKaMaxCtas = 160;

template <int D>
struct KaCfg {
  static constexpr int TK = kKaTileBytes / D;  // keys of a warp's tile: 64, 32, 16
  static constexpr int KG = TK / 16;           // groups of 16 keys
  // 12 warps with 168 registers hide latencies better than 8 with 250 (the kernel is bound by its dependent
  // instructions, not by memory); heads of 256 need the registers for their accumulator.
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = 3;
  static constexpr int kItem = kWarps * TK;  // keys of an item
  static constexpr int kSteps = D / 16;
  static constexpr bool kQRegs = D <= 128;     // q fragments in registers
  static constexpr int kBatch = 32 / KG;       // tiles whose page ids a warp holds
  static constexpr uint32_t kRowBytes = D < 128 ? D : 128;  // bytes of a row in a TMA box
  static constexpr int kColBlocks = D / int(kRowBytes);
  static constexpr uint32_t kRing = kWarps * kStages * 2 * kKaTileBytes;
  static constexpr uint32_t kJoin = kWarps * kKaRows * 32 * 4;  // 32 columns of every warp; the CTAs' weights
  static_assert(kKaRows * kKaMaxCtas * 4 <= kJoin, "weights of a row tile's CTAs");
  static constexpr uint32_t kQ = kKaRows * D * 2;
  static constexpr size_t kSmem = 1024 + kRing + kJoin + kQ + 4096;
  static constexpr int kSlotFloats = kKaRows * D + 2 * kKaRows;
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
  float* part;       // [CTA][2][kSlotFloats]
  unsigned* counters;  // [CTA]
  unsigned* err;
};

constexpr int kKaMaxWarps = 12, kKaMaxStages = 3;
struct KaShared {
  uint64_t full[kKaMaxWarps][kKaMaxStages];
  float scales[kKaMaxWarps][kKaMaxStages][3][4];  // ks, log2(vs), 1 / vs of each group of 16 keys
  float warp_z[kKaMaxWarps][kKaRows];
  float warp_l[kKaMaxWarps][kKaRows];
  float row_factor[kKaRows];
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

// A CTA's share of `total` items among the first min(ctas, total) CTAs.
W4A8_HD long long ka_first_item(long long c, long long total, long long ctas) { return total * c / ctas; }
W4A8_HD int ka_item_cta(long long i, long long total, long long ctas) {
  return int(((i + 1) * ctas + total - 1) / total - 1);
}

// A sequence of at least kKpMinRows rows (new tokens x query heads of a key
// head) is left to the tensor-memory kernel (kv_prefill.cuh) when the batch
// has enough such tiles of 256 rows to occupy the SMs, which that kernel
// does not split along the keys: it then does about 4.5 TFLOP/s a CTA
// against 140 for this whole kernel.
constexpr int kKpMinRows = 128;
constexpr int kKpMinCtas = 32;
__device__ __forceinline__ bool kp_takes_big(const KaParams& p) {  // whole warp
  const int lane = threadIdx.x & 31;
  long long ctas = 0;
  for (int b0 = 0; b0 < p.batch.batch; b0 += 32) {
    if (b0 + lane < p.batch.batch) {
      const long long rows = (long long)kv_load_seq(p.batch, b0 + lane, p.cache.page_shift).q_len * p.group;
      if (rows >= kKpMinRows) ctas += (rows + 255) / 256 * p.cache.kv_heads;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ctas += __shfl_xor_sync(0xffffffffu, ctas, off);
  return ctas >= kKpMinCtas;
}

// Row tiles of a sequence, and items of each (the same for all of them: a
// tile skips the keys outside its own range).
template <int D>
__device__ __forceinline__ void ka_counts(const KvSeq& s, const KaParams& p, bool small_only, int& tiles, int& items) {
  const KvRange r = kv_range(s, 0, s.q_len - 1, p.window);
  const int lo = r.lo & ~(KaCfg<D>::TK - 1);
  tiles = (s.q_len * p.group + kKaRows - 1) / kKaRows;
  items = s.q_len == 0 ? 0 : (s.kv_len - lo + KaCfg<D>::kItem - 1) / KaCfg<D>::kItem;
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

template <int D>
struct KaWalk {
  long long pos, end, base;
  int b, tiles, items;
  bool small_only;
  KvSeq s;
  __device__ __forceinline__ void load(const KaParams& p) {
    s = kv_load_seq(p.batch, b, p.cache.page_shift);
    ka_counts<D>(s, p, small_only, tiles, items);
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
    g.key0 = kv_range(s, 0, s.q_len - 1, p.window).lo & ~(KaCfg<D>::TK - 1);
    const int j0 = g.tile * kKaRows / p.group;
    const int last_row = min(s.q_len * p.group, (g.tile + 1) * kKaRows) - 1;
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

template <int D>
__device__ __forceinline__ uint32_t ka_tau(uint32_t i) {
  return D < 128 ? i : (i >> 1) | ((i & 1u) << 2);
}
// Byte offset of 16-byte chunk c of row r in a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t ka_at(uint32_t r, uint32_t c) {
  if constexpr (D < 128) return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
  return (c >> 3) * uint32_t(KaCfg<D>::TK * 128) + r * 128u + (((c & 7u) ^ (r & 7u)) << 4);
}

template <int D>
__global__ void __launch_bounds__(KaCfg<D>::kThreads, 1)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const KaParams p) {
  using C = KaCfg<D>;
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
    const bool small_only = p.both && kp_takes_big(p);
    long long total = 0;
    for (int b0 = 0; b0 < p.batch.batch; b0 += 32) {
      int tiles = 0, items = 0;
      if (b0 + lane < p.batch.batch) {
        const KvSeq s = kv_load_seq(p.batch, b0 + lane, p.cache.page_shift);
        if (s.bad) record_error(p.err, kErrInput);
        ka_counts<D>(s, p, small_only, tiles, items);
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
        ka_counts<D>(kv_load_seq(p.batch, b0 + lane, p.cache.page_shift), p, small_only, tiles, items);
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
  KaWalk<D> walk;
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
    return item < fend && group_key(item) < fseg.range.hi
               ? __ldg(p.batch.table + (long long)fseg.b * p.batch.table_stride + (group_key(item) >> p.cache.page_shift))
               : -1;
  };
  auto take_batch = [&](int base) {  // nraw, fetched for `base`, becomes the batch at hand
    fid = nraw;
    if (fid >= p.cache.pages || (fid < 0 && base + ftile < fend && group_key(base + ftile) < fseg.range.hi)) {
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
    if (warp < kKaRows / 2) {
      const int r = 2 * warp + (lane >> 4), l16 = lane & 15;
      const int row = seg.tile * kKaRows + r;
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
      // the row's power of two: its largest value lands in [2^13, 2^14)
      const int e = min(100, max(-100, 127 + 13 - int(__float_as_uint(top) >> 23)));
      // (a negative scale goes into q, so that larger products stay larger scores)
      const float up = copysignf(__uint_as_float(uint32_t(127 + e) << 23), p.scale_log2);
      if (l16 == 0) sh->row_factor[r] = __uint_as_float(uint32_t(127 - e) << 23) * fabsf(p.scale_log2);
#pragma unroll
      for (int i = 0; i < D / 16; i += 2) {
        const int d = l16 * (D / 16) + i;
        const int step = (d >> 6) * 4 + ((d >> 2) & 3), ln = (r & 7) * 4 + ((d >> 4) & 3);
        const int reg = ((d & 2) ? 2 : 0) + (r >> 3);
        const __half2 h = __floats2half2_rn(v[i] * up, v[i + 1] * up);
        qf[(step * 32 + ln) * 4 + reg] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    __syncthreads();
    uint32_t qr[C::kQRegs ? C::kSteps : 1][4];
    if constexpr (C::kQRegs) {
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s) {
        const uint4 f = *reinterpret_cast<const uint4*>(qf + (s * 32 + lane) * 4);
        qr[s][0] = f.x, qr[s][1] = f.y, qr[s][2] = f.z, qr[s][3] = f.w;
      }
    }
    const float f0 = sh->row_factor[g], f1 = sh->row_factor[g + 8];
    int lim[2], low[2];  // the last key a row sees, and the first
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = min(seg.tile * kKaRows + g + 8 * i, rows - 1);
      lim[i] = seg.s.kv_len - seg.s.q_len + row / p.group;
      low[i] = p.window > 0 ? lim[i] - p.window + 1 : 0;
    }
    const int lim_min = seg.s.kv_len - seg.s.q_len + seg.tile * kKaRows / p.group;
    const int low_max = p.window > 0 ? seg.range.hi - p.window : 0;

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float z0 = -INFINITY, z1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int item = c_first_item; item < c_end_item; ++item) {
      const int key = seg.key0 + (item * C::kWarps + warp) * C::TK;
      if (ok) ok = __all_sync(0xffffffffu, ka_wait(&sh->full[warp][stage], phase, sh, p.err));
      if (!ok) break;
      const uint32_t kt = ring + uint32_t((warp * C::kStages + stage) * 2) * kKaTileBytes, vt = kt + kKaTileBytes;
      // ---- scores
      float s[C::TK / 8][4];
#pragma unroll
      for (int j = 0; j < C::TK / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t qs[4][4];
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          if constexpr (C::kQRegs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) qs[st][i] = qr[4 * c + st][i];
          } else {
            const uint4 f = *reinterpret_cast<const uint4*>(qf + ((4 * c + st) * 32 + lane) * 4);
            qs[st][0] = f.x, qs[st][1] = f.y, qs[st][2] = f.z, qs[st][3] = f.w;
          }
        }
#pragma unroll
        for (int j = 0; j < C::TK / 8; ++j) {
          uint32_t w[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(kt + ka_at<D>(uint32_t(8 * j) + ka_tau<D>(g), uint32_t(4 * c + t))));
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint32_t x = w[st] ^ 0x80808080u;
            ka_mma(s[j], qs[st], ka_codes(x, 0x4140u), ka_codes(x, 0x4342u));
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
        for (int j = 0; j < C::TK / 8; ++j) {
          const int ka = key + 8 * j + int(ka_tau<D>(2 * t)), kc = key + 8 * j + int(ka_tau<D>(2 * t + 1));
          if (ka > lim[0] || ka < low[0]) s[j][0] = -INFINITY;
          if (kc > lim[0] || kc < low[0]) s[j][1] = -INFINITY;
          if (ka > lim[1] || ka < low[1]) s[j][2] = -INFINITY;
          if (kc > lim[1] || kc < low[1]) s[j][3] = -INFINITY;
        }
      }
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < C::KG; ++kb) {
        const float g0 = fmaxf(fmaxf(s[2 * kb][0], s[2 * kb][1]), fmaxf(s[2 * kb + 1][0], s[2 * kb + 1][1]));
        const float g1 = fmaxf(fmaxf(s[2 * kb][2], s[2 * kb][3]), fmaxf(s[2 * kb + 1][2], s[2 * kb + 1][3]));
        const float k = ks[kb], off = lv[kb] - 15.f;
        // (fmaxf drops the NaN of a wholly masked group under a K scale of 0)
        x0 = fmaxf(x0, fmaf(g0, f0 * k, off));
        x1 = fmaxf(x1, fmaf(g1, f1 * k, off));
      }
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
      }
      if (__any_sync(0xffffffffu, x0 > z0 || x1 > z1)) {
        const float n0 = fmaxf(z0, x0), n1 = fmaxf(z1, x1);
        const float r0 = z0 == -INFINITY ? 0.f : ex2(z0 - n0), r1 = z1 == -INFINITY ? 0.f : ex2(z1 - n1);
        l0 *= r0;
        l1 *= r1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= r0;
          o[i][1] *= r0;
          o[i][2] *= r1;
          o[i][3] *= r1;
        }
        z0 = n0;
        z1 = n1;
      }
      const float u0 = z0 == -INFINITY ? 0.f : z0, u1 = z1 == -INFINITY ? 0.f : z1;
      // ---- P', the sum of p, and the product with V
#pragma unroll
      for (int kb = 0; kb < C::KG; ++kb) {
        const float k0 = f0 * ks[kb], k1 = f1 * ks[kb], o0 = lv[kb] - u0, o1 = lv[kb] - u1, w = iv[kb];
        uint32_t a[4];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* x = s[2 * kb + i];
          float p0 = ex2(fmaf(x[0], k0, o0)), p1 = ex2(fmaf(x[1], k0, o0));
          float p2 = ex2(fmaf(x[2], k1, o1)), p3 = ex2(fmaf(x[3], k1, o1));
          if (edge) {  // (a masked score times a K scale of 0 is no zero)
            p0 = x[0] == -INFINITY ? 0.f : p0;
            p1 = x[1] == -INFINITY ? 0.f : p1;
            p2 = x[2] == -INFINITY ? 0.f : p2;
            p3 = x[3] == -INFINITY ? 0.f : p3;
          }
          s0 += p0 + p1;
          s1 += p2 + p3;
          const __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
          a[2 * i] = *reinterpret_cast<const uint32_t*>(&h0);
          a[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h1);
        }
        l0 = fmaf(s0, w, l0);
        l1 = fmaf(s1, w, l1);
        if (w >= 1.f / kKvLeastScale) a[0] = a[1] = a[2] = a[3] = 0u;  // a page without a V scale: its values are zeros
        const uint32_t vrow = uint32_t(16 * kb + ((lane >> 3) & 1) * 8) + ka_tau<D>(lane & 7);
#pragma unroll
        for (int c2 = 0; c2 < D / 32; ++c2) {
          uint32_t r[4];
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                       : "r"(vt + ka_at<D>(vrow, uint32_t(2 * c2 + (lane >> 4)))));
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] ^= 0x80808080u;
          ka_mma(o[4 * c2], a, ka_codes(r[0], 0x4240u), ka_codes(r[1], 0x4240u));
          ka_mma(o[4 * c2 + 1], a, ka_codes(r[0], 0x4341u), ka_codes(r[1], 0x4341u));
          ka_mma(o[4 * c2 + 2], a, ka_codes(r[2], 0x4240u), ka_codes(r[3], 0x4240u));
          ka_mma(o[4 * c2 + 3], a, ka_codes(r[2], 0x4341u), ka_codes(r[3], 0x4341u));
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
    for (int off = 1; off < 4; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (t == 0) {
      sh->warp_z[warp][g] = z0;
      sh->warp_z[warp][g + 8] = z1;
      sh->warp_l[warp][g] = l0;
      sh->warp_l[warp][g + 8] = l1;
    }
    __syncthreads();
    float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      top0 = fmaxf(top0, sh->warp_z[w][g]);
      top1 = fmaxf(top1, sh->warp_z[w][g + 8]);
    }
    const float w0 = z0 == -INFINITY ? 0.f : ex2(z0 - top0), w1 = z1 == -INFINITY ? 0.f : ex2(z1 - top1);
    // this thread's place in the joined tile: row jr, columns 2 jc, 2 jc + 1 of each 32 (threads past 256 have none)
    const int jr = (tid >> 4) & 15, jc = tid & 15;
    const bool joins = tid < 256;
    float jz = -INFINITY, jl = 0.f;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) jz = fmaxf(jz, sh->warp_z[w][jr]);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w)
      if (sh->warp_z[w][jr] != -INFINITY) jl += sh->warp_l[w][jr] * ex2(sh->warp_z[w][jr] - jz);
    const bool whole = seg.item0 == 0 && seg.item1 == seg.items;
    const int slot = int(blockIdx.x) * 2 + (i0 >= seg.start ? 0 : 1);
    float* part = p.part + (size_t)slot * C::kSlotFloats;
    const int row = seg.tile * kKaRows + jr;
    const int oj = row / p.group, oh = seg.head * p.group + row - oj * p.group;
    uint16_t* dst = p.out.data + (long long)(seg.s.start + oj) * p.out.token + oh * p.out.head;
    const float norm = jl > 0.f ? __fdiv_rn(1.f, jl) : 0.f;
#pragma unroll
    for (int c2 = 0; c2 < D / 32; ++c2) {
      float* mine = join + warp * (kKaRows * 32);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float(&e)[4] = o[4 * c2 + 2 * hf];
        const float(&d)[4] = o[4 * c2 + 2 * hf + 1];
        *reinterpret_cast<float4*>(mine + g * 32 + 16 * hf + 4 * t) =
            make_float4(e[0] * w0, d[0] * w0, e[1] * w0, d[1] * w0);
        *reinterpret_cast<float4*>(mine + (g + 8) * 32 + 16 * hf + 4 * t) =
            make_float4(e[2] * w1, d[2] * w1, e[3] * w1, d[3] * w1);
      }
      __syncthreads();
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(join + w * (kKaRows * 32) + jr * 32 + 2 * jc);
        x += v.x;
        y += v.y;
      }
      if (!joins) {
      } else if (!whole) {
        *reinterpret_cast<float2*>(part + jr * D + 32 * c2 + 2 * jc) = make_float2(x, y);
      } else if (row < rows && ok) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x * norm, y * norm);
        *reinterpret_cast<__nv_bfloat162*>(dst + 32 * c2 + 2 * jc) = b;
      }
      __syncthreads();
    }
    if (!whole) {
      if (joins && jc == 0) {
        part[kKaRows * D + jr] = jz;
        part[kKaRows * D + kKaRows + jr] = jl;
      }
      const int c_first = ka_item_cta(seg.start, total, ctas), c_last = ka_item_cta(seg.start + seg.items - 1, total, ctas);
      __threadfence();
      __syncthreads();
      if (tid == 0) sh->last = atomicAdd(p.counters + c_first, 1u) == unsigned(c_last - c_first);
      __syncthreads();
      if (sh->last && joins) {
        __threadfence();
        // Slot of CTA c: its first row tile's, but for the CTA in which the tile starts behind another one.  A row's
        // 16 threads take the CTAs' maxima and sums 16 at a time, and leave the CTAs' weights in shared memory; the
        // accumulators then come in eight at a time (one at a time waits a round trip to L2 for each).
        const int n_cta = c_last - c_first + 1;
        const float* slot0 = p.part + (size_t)(c_first * 2 + (ka_first_item(c_first, total, ctas) >= seg.start ? 0 : 1)) * C::kSlotFloats;
        auto slot_of = [&](int c) {
          return c == 0 ? slot0 : p.part + (size_t)((c_first + c) * 2) * C::kSlotFloats;
        };
        float* weight = join + jr * kKaMaxCtas;
        float top = -INFINITY, sum = 0.f;
        for (int c = jc; c < n_cta; c += 16) {
          const float* m = slot_of(c) + kKaRows * D + jr;
          const float cz = __ldcg(m), cl = __ldcg(m + kKaRows);
          const float nt = fmaxf(top, cz);
          if (nt > -INFINITY) sum = sum * ex2(top - nt) + (cz > -INFINITY ? cl * ex2(cz - nt) : 0.f);
          top = nt;
          weight[c] = cz;
        }
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) {
          const float ot = __shfl_xor_sync(0xffffffffu, top, off), os = __shfl_xor_sync(0xffffffffu, sum, off);
          const float nt = fmaxf(top, ot);
          if (nt > -INFINITY) sum = sum * ex2(top - nt) + os * ex2(ot - nt);
          top = nt;
        }
        for (int c = jc; c < n_cta; c += 16) weight[c] = weight[c] == -INFINITY ? 0.f : ex2(weight[c] - top);
        __syncwarp();
        float acc[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) acc[i] = 0.f;
        constexpr int kAhead = D <= 128 ? 8 : 4;
        for (int c0 = 0; c0 < n_cta; c0 += kAhead) {
          float4 v[kAhead][D / 64];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const float* src = slot_of(min(c0 + u, n_cta - 1)) + jr * D + jc * 4;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) v[u][i] = __ldcg(reinterpret_cast<const float4*>(src + i * 64));
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const float f = c0 + u < n_cta ? weight[c0 + u] : 0.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              acc[4 * i] += f * v[u][i].x;
              acc[4 * i + 1] += f * v[u][i].y;
              acc[4 * i + 2] += f * v[u][i].z;
              acc[4 * i + 3] += f * v[u][i].w;
            }
          }
        }
        const float n = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
        if (row < rows) {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(acc[4 * i] * n, acc[4 * i + 1] * n);
            const __nv_bfloat162 y = __floats2bfloat162_rn(acc[4 * i + 2] * n, acc[4 * i + 3] * n);
            *reinterpret_cast<uint2*>(dst + jc * 4 + i * 64) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
          }
        }
        if (tid == 0) p.counters[c_first] = 0u;  // ready for the next launch on this workspace
      }
    }
    __syncthreads();  // q fragments, warp_m and the join buffer are free again
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
