// The int8 paged cache: writing new tokens into it and reading pages back.
//
// codes  int8 [pages][kv_heads][page][D], scales fp32 [pages][kv_heads], one
// set for K and one for V.  Value = code * scale of its (page, head).
//
// Update of one (page, head) with new rows at places [first, first + n):
//   need = max |row value| / 127
//   s'   = max(s, need), where s = 0 if the page starts with these rows
//   codes of the places before `first`: rint(c * (s / s')) if s' > s
//   new codes: clamp(rint(v / s'), -127, 127)
// Places behind the new rows are left as they are.
//
// K rows are normed and rotated on the way (qk_rope.cuh) and quantised from
// fp32, so they are rounded once.  One CTA per (touched page, head, K or V);
// more CTAs of the same launch norm and rotate q, so a decode step's work
// between the projection and the attention is this one launch.
#pragma once

#include "act.cuh"
#include "common.cuh"
#include "int8_quant.cuh"
#include "kv_index.h"
#include "qk_rope.cuh"

namespace w4a8 {

struct KvCacheParams {
  int8_t* codes[2];   // K, V
  float* scales[2];
  long long pages;
  int kv_heads, page_shift, D;
};

struct KvBatchParams {
  const int* table;      // [batch][table_stride]
  long long table_stride;
  const int* q_start;    // [batch + 1]
  const int* kv_len;     // [batch]
  int batch;
  int tokens;
};

__device__ __forceinline__ KvSeq kv_load_seq(const KvBatchParams& b, int i, int page_shift) {
  return kv_seq(__ldg(b.q_start + i), __ldg(b.q_start + i + 1), __ldg(b.kv_len + i), b.tokens,
                b.table_stride << page_shift);
}

// Which touched page of which sequence unit u is (whole warp; the same
// answer in every lane): sequences are scanned 32 at a time.  False past the
// last one.
__device__ __forceinline__ bool kv_find_page(const KvBatchParams& b, int page_shift, int u, int& seq, int& nth,
                                             KvSeq& s, unsigned* err) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b0 = 0; b0 < b.batch; b0 += 32) {
    KvSeq mine{0, 0, 0, false};
    if (b0 + lane < b.batch) mine = kv_load_seq(b, b0 + lane, page_shift);
    if (mine.bad && err) record_error(err, kErrInput);
    int sum = kv_touched(mine, page_shift);
    const int own = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > u);
    if (past) {
      const int l = __ffs(past) - 1;
      seq = b0 + l;
      nth = u - (before + __shfl_sync(0xffffffffu, sum - own, l));
      s.start = __shfl_sync(0xffffffffu, mine.start, l);
      s.q_len = __shfl_sync(0xffffffffu, mine.q_len, l);
      s.kv_len = __shfl_sync(0xffffffffu, mine.kv_len, l);
      s.bad = false;
      return true;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

// Position in its sequence of new token `row` (whole warp); -1 if it belongs
// to none (rows behind the last sequence, or a bad sequence).
__device__ __forceinline__ int kv_find_position(const KvBatchParams& b, int page_shift, int row) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < b.batch; b0 += 32) {
    KvSeq s{0, 0, 0, false};
    if (b0 + lane < b.batch) s = kv_load_seq(b, b0 + lane, page_shift);
    const unsigned in = __ballot_sync(0xffffffffu, row >= s.start && row < s.start + s.q_len);
    if (in) return __shfl_sync(0xffffffffu, s.kv_len - s.q_len + (row - s.start), __ffs(in) - 1);
  }
  return -1;
}

struct KvUpdateParams {
  QkParams qk;          // q, k (k_out unused), norm weights, rotation; positions may be NULL (the cache's)
  HeadRows v;
  KvCacheParams cache;
  KvBatchParams batch;
  int page_ctas;        // units * kv_heads * 2
  int stride;           // every so many CTAs one takes a page, as far as there are any; the others take q
  int q_parts;          // warps that share a token's heads
  int rest_cta;         // the CTA that looks at the sequences behind the 32nd, or -1
  unsigned* err;
};

template <int THREADS>
__device__ __forceinline__ float block_max(float v, float* warp_max) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_max[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) v = fmaxf(v, warp_max[i]);
  return v;
}

__device__ __forceinline__ uint2 quant8(const float (&v)[8], const QuantScale& qs) {
  const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
  return qs.fast ? make_uint2(q8_code4<true>(a, qs), q8_code4<true>(b, qs))
                 : make_uint2(q8_code4<false>(a, qs), q8_code4<false>(b, qs));
}

__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = int(int8_t(w >> (8 * i)));
    out |= (uint32_t(int(rintf(float(c) * ratio))) & 0xFFu) << (8 * i);
  }
  return out;
}

// q's CTAs lie between the pages', which wait more than they compute (3354
// tokens of 24/4 heads of 256 in three sequences: 30.9 us, 32.3 one after the
// other; the pages alone 15.2, q alone 17.0).
// THREADS: 256, or 64 where a page gets a token or two (a decode step: the
// CTAs of 64 sequences x 8 heads are then all resident at once).
// Three (or twelve) CTAs an SM cap the registers at 80, of which the pages'
// path spills 188 to 204 bytes a thread (its four rows of angles and values);
// the cap holds for q's path too.  That the two together take nearly the sum
// of their own times is in part this.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 768 / THREADS) kv_update_kernel(const KvUpdateParams p) {
  constexpr int LPH = D / 8, RPP = THREADS / LPH;  // rows per pass
  constexpr int kAhead = 4;                        // passes of a chunk
  __shared__ float warp_max[THREADS / 32];
  pdl_launch_dependents();  // (the next kernel waits for this one, and this one for the last)
  pdl_wait();
  const int g = threadIdx.x / LPH, sub = threadIdx.x & (LPH - 1);
  const int ps = p.cache.page_shift;
  if (int(blockIdx.x) == p.rest_cta) {
    // The pages' search ends at the group of 32 sequences that holds its page, and reports what it sees.  Batches of more
    // have one CTA that looks at the rest, so that a bad sequence is reported wherever it stands.
#pragma unroll 1
    for (int b = 32 + threadIdx.x; b < p.batch.batch; b += THREADS)
      if (kv_load_seq(p.batch, b, ps).bad) record_error(p.err, kErrInput);
    return;
  }
  const int turn_at = int(blockIdx.x) / p.stride;
  if (turn_at >= p.page_ctas || int(blockIdx.x) != turn_at * p.stride) {
    // ------------------------------------------------ q: a warp per share of a token's heads
    const int nth_q = int(blockIdx.x) - min(p.page_ctas, turn_at + 1);
    const long long unit = ((long long)nth_q * THREADS + threadIdx.x) >> 5;
    const int token = int(unit / p.q_parts), part = int(unit - (long long)token * p.q_parts);
    if (token >= p.batch.tokens) return;
    const int at = kv_find_position(p.batch, ps, token);
    if (at < 0) return;
    QkParams qk = p.qk;
    qk.k.data = nullptr;
    qk_token<D>(qk, token, qk.positions ? __ldg(qk.positions + token) : at, part, p.q_parts);
    return;
  }
  // -------------------------------------------------- a page of a head, K or V
  const int kind = turn_at & 1;
  const int head = (turn_at >> 1) % p.cache.kv_heads;
  const int unit = (turn_at >> 1) / p.cache.kv_heads;
  int seq, nth;
  KvSeq s;
  if (!kv_find_page(p.batch, ps, unit, seq, nth, s, p.err)) return;
  const int page = 1 << ps;
  const int pi = kv_first_page(s, ps) + nth;                       // page of the sequence
  const int j0 = max(0, (pi << ps) - (s.kv_len - s.q_len));        // its first new token here
  const int first = s.kv_len - s.q_len + j0 - (pi << ps);          // and that token's place
  const int n = min(s.q_len - j0, page - first);
  const int id = __ldg(p.batch.table + (long long)seq * p.batch.table_stride + pi);
  if (id < 0 || id >= p.cache.pages) {
    if (threadIdx.x == 0) record_error(p.err, kErrInput);
    return;
  }
  const HeadRows& src = kind ? p.v : p.qk.k;
  const float* weight = kind ? nullptr : p.qk.k_weight;
  const Head8 w = head_weight(weight, sub);
  float* scale = p.cache.scales[kind] + (long long)id * p.cache.kv_heads + head;
  const float old = first == 0 ? 0.f : __ldcg(scale);
  const bool turn = kind == 0 && p.qk.rope.inv_freq;
  // A chunk of rows, kAhead passes: their loads go out together, then norm and rotation.  The values stay in
  // registers; where the rows are more than one chunk, the chunks are made again once the scale is known.
  Head8 v[kAhead];
  auto chunk = [&](int r0) {
    uint4 raw[kAhead];
    int pos[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int r = r0 + a * RPP + g;
      const long long token = s.start + j0 + r;
      raw[a] = r < n ? __ldcg(reinterpret_cast<const uint4*>(src.data + token * src.token + head * src.head) + sub)
                     : make_uint4(0u, 0u, 0u, 0u);
      pos[a] = turn && p.qk.positions && r < n ? __ldg(p.qk.positions + token) : s.kv_len - s.q_len + j0 + r;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (r0 + a * RPP >= n) break;  // (the same for all lanes: the norm and the rotation shuffle)
      v[a] = head_unpack(raw[a]);
      if (weight) head_norm<LPH>(v[a], w, p.qk.eps);
      if (turn) head_rope(v[a], p.qk.rope.interleaved, head_turn<LPH>(p.qk.rope, sub, pos[a]));
    }
  };
  float amax = 0.f;
  for (int r0 = 0; r0 < n; r0 += kAhead * RPP) {
    chunk(r0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (r0 + a * RPP + g < n) {
        float x[8];
        head_values(v[a], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
      }
    }
  }
  const float need = quant_scale(block_max<THREADS>(amax, warp_max));
  const float now = fmaxf(old, need);
  int8_t* codes = p.cache.codes[kind] + (((long long)id * p.cache.kv_heads + head) << ps) * D;
  if (first > 0 && now > old) {
    const float ratio = __fdiv_rn(old, now);
    for (int i = threadIdx.x * 16; i < first * D; i += THREADS * 16) {
      uint4 c = *reinterpret_cast<uint4*>(codes + i);
      c.x = recode4(c.x, ratio);
      c.y = recode4(c.y, ratio);
      c.z = recode4(c.z, ratio);
      c.w = recode4(c.w, ratio);
      *reinterpret_cast<uint4*>(codes + i) = c;
    }
  }
  const QuantScale qs = quant_prepare(now);
  for (int r0 = 0; r0 < n; r0 += kAhead * RPP) {
    if (n > kAhead * RPP) chunk(r0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int r = r0 + a * RPP + g;
      if (r < n) {
        float x[8];
        head_values(v[a], x);
        *reinterpret_cast<uint2*>(codes + (first + r) * D + 8 * sub) = quant8(x, qs);
      }
    }
  }
  if (threadIdx.x == 0) *scale = now;  // (every thread read the old one before block_max's barrier)
}

// Pages back to bf16: values code * scale of both kinds, [n][kv_heads][page][D].
// A CTA takes 4096 codes of one (page, head) of one kind (or the whole of a
// smaller one), a thread two groups of 8, so that a warp's loads and stores
// are whole runs of 256 and 512 bytes: 107 pages of 32 tokens, 4 heads of 256,
// take 4.2 us (5.1 with 16 codes on end to a thread, 6.3 with 32), of which the
// 21 MB are 3.2; the rest is the chain id -> codes -> values.
constexpr int kDqThreads = 256;
__global__ void __launch_bounds__(kDqThreads) kv_dequant_kernel(KvCacheParams c, const int* __restrict__ ids, int n,
                                                                uint16_t* __restrict__ k_out,
                                                                uint16_t* __restrict__ v_out, unsigned* err) {
  pdl_launch_dependents();  // (the next kernel waits for this one, and this one for the last)
  pdl_wait();
  const int slab = c.D << c.page_shift;  // codes of a (page, head), a multiple of 1024
  const int parts = (slab + 16 * kDqThreads - 1) / (16 * kDqThreads);
  const long long unit = blockIdx.x / parts;  // (kind, nth, head)
  const int first = (int(blockIdx.x) - int(unit) * parts) * 16 * kDqThreads + threadIdx.x * 8;
  if (first >= slab) return;
  const long long row = unit / c.kv_heads;
  const int head = int(unit - row * c.kv_heads), kind = row >= n;
  const long long nth = kind ? row - n : row;
  const int id = __ldg(ids + nth);
  constexpr int kHalf = 8 * kDqThreads;  // a thread's two groups of 8 codes are this far apart
  const bool two = first + kHalf < slab;
  uint2 w[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
  float s = 0.f;
  if (id >= 0 && id < c.pages) {
    const long long at_head = (long long)id * c.kv_heads + head;
    const int8_t* codes = (kind ? c.codes[1] : c.codes[0]) + at_head * slab + first;
    w[0] = __ldcg(reinterpret_cast<const uint2*>(codes));
    if (two) w[1] = __ldcg(reinterpret_cast<const uint2*>(codes + kHalf));
    s = __ldcg((kind ? c.scales[1] : c.scales[0]) + at_head);
  } else {
    record_error(err, kErrInput);
  }
  uint16_t* out = (kind ? v_out : k_out) + (nth * c.kv_heads + head) * slab + first;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t ws[2] = {w[h].x ^ 0x80808080u, w[h].y ^ 0x80808080u};
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // code + 128 under the exponent of 2^23, less 2^23 + 128 (exact; an integer conversion runs at an eighth the rate)
      const uint32_t bits = prmt(ws[j >> 2], 0x4B000000u, 0x7540u + (j & 3));
      v[j] = (__uint_as_float(bits) - 8388736.f) * s;
    }
    if (h == 0 || two) *reinterpret_cast<uint4*>(out + h * kHalf) = float_to_bf16x8(v);
  }
}

}  // namespace w4a8
