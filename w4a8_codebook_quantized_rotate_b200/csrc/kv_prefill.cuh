// Attention of many new tokens over the int8 paged cache, on the 5th
// generation tensor cores.  Same mathematics as kv_attn.cuh:
//
//   o_i = sum_j P'_ij c_j / sum_j (P'_ij / vs_j),
//   P'_ij = 2^(t_ij - z_i),  t_ij = q_i . k_j ks_j scale log2(e) + log2(vs_j)
//
// with integer codes k_j, c_j (exact in fp16) and z_i the running maximum of
// t_ij less 7, kept until t grows by more than 8 (so P' stays in fp16's range
// and the accumulator is rescaled a few times a row, not every tile).
//
// A CTA takes 256 rows of one key head (the query heads of the group,
// neighbouring new tokens) as two tiles of 128, TMEM's lanes (heads of 256:
// one tile), and walks the keys in tiles of 64.  Roles:
//   * 4 converter warps expand K and V codes to fp16 in 128-byte-swizzled
//     shared memory, a ring of stages each, with the loads of the next tile
//     in registers.  Expanding once per 256 rows is what makes the expansion
//     cheap: its shared-memory writes are a third of the MMAs' reads.
//   * one thread issues the MMAs of S = Q K^T from shared memory, another those
//     of O += P' V with P' in TMEM (fp16, in S's place) and V as it lies
//     ([key][d], the operand's MN-major order), O in TMEM.  (One thread for
//     both could not issue them fast enough: 2500 clocks per 256 x 64 scores
//     of heads of 128, against 1300 that the MMAs take.)
//   * a softmax warpgroup per row tile, a thread per row: maximum over the
//     row's scores, then P' back to TMEM.
// Every row tile has two score buffers: the scores of the next key tile are
// made while the softmax of this one runs, so the softmax warps, which bound
// the kernel, do not wait for the MMAs.
// The CTAs that are left over after whole waves of one CTA an SM are split
// along their keys where that fills the SMs better (a rest of at most half a
// wave, in up to four parts); the parts' O, maxima and sums meet in the
// workspace, where the last one to arrive adds them in their order (two
// sequences of up to 2048 new tokens on up to 8192, 32/8 heads of 128, in a
// captured stream: 492 us, 530 unsplit; 478 with the softmax's sums and
// exponents' arguments two to an instruction and its maxima over three).
// Slower at that size: P' in buffers of its own, so that the scores wait only
// for the softmax (493), and tiles of 128 keys with one buffer of scores (651,
// the scores read twice).  Without its exponentials, its expansion or its
// loads the kernel takes 440 to 455, so none of them alone bounds it: the
// hand-offs between the roles do, about 150 clocks each.
// Bounds: per 256 x 128 (rows x keys) and D = 128 the MMAs take 2048 clocks
// of an SM (2560 with the operand reads of 64-key tiles), its exponentials (16
// a clock) 2048, so the softmax keeps to about four other instructions a
// score: scores are scaled in the exponent's multiply-add, and the sum of p
// comes from P' per page (sum of P' / vs).
#pragma once

#include "common.cuh"
#include "gemm_tc.cuh"
#include "kv_attn.cuh"
#include "kv_cache.cuh"

namespace w4a8 {

constexpr int kKpConvWarps = 4;

template <int D>
struct KpCfg {
  static constexpr int kTiles = D <= 128 ? 2 : 1;        // row tiles of a CTA
  static constexpr int TK = 64;                          // keys of a tile
  static constexpr int kStages = D <= 128 ? 4 : 2;       // of K, and of V
  static constexpr int KG = TK / 16;                     // key groups (one page each)
  static constexpr int kRows = kp_rows(D);
  static_assert(kRows == 128 * kTiles, "TMEM lanes");
  static constexpr int kSoftWarps = 4 * kTiles;
  static constexpr int kThreads = 32 * (kSoftWarps + kKpConvWarps + 2);  // softmax, converters, two MMA warps
  static constexpr uint32_t kQ = 128 * D * 2;            // a tile of q, fp16
  static constexpr uint32_t kKV = TK * D * 2;            // a stage of K or V, fp16
  static constexpr size_t kSmem = 1024 + kTiles * kQ + 2 * kStages * kKV + 1024;
  static constexpr uint32_t kSCols = TK;                 // fp32 scores; P' takes the first half
  static constexpr uint32_t kOCol = 2 * kTiles * kSCols; // two score buffers a tile, then O of each tile
  static_assert(kOCol + kTiles * D <= 512, "TMEM");
  // kind::f16: fp16 A and B, fp32 D, M = 128
  static constexpr uint32_t kIdescQK = (1u << 4) | (uint32_t(TK >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (8u << 24);  // B MN-major
};

struct KpShared {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t q_full;
  uint64_t s_full[4], p_full[4];  // [2 tile + buffer]
  uint64_t pv_done[4];            // [2 tile + buffer]: one each, as the scores may be two products behind
  uint64_t drain;
  float ks[8][4], lv[8][4], iv[8][4];  // ks, log2(vs), 1 / vs of a tile's key groups (ring of 8 tiles)
  uint32_t tmem_base;
  int found, last;
  int b, tile, head;
  int slot, part, parts;  // of a split unit's parts this CTA is `part`
  volatile int abort;
};

__device__ __forceinline__ bool kp_wait(uint64_t* bar, uint32_t parity, KpShared* sh, unsigned* err) {
  for (uint32_t i = 0; i < (1u << 20); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 1023u && sh->abort) return false;
  }
  sh->abort = 1;
  record_error(err, kErrTimeout);
  return false;
}

// A warp's wait: lane 0 polls (32 lanes polling one word take the shared
// memory's time from the MMAs), the others learn the outcome.
__device__ __forceinline__ bool kp_wait_warp(uint64_t* bar, uint32_t parity, KpShared* sh, unsigned* err) {
  const int ok = (threadIdx.x & 31) == 0 ? int(kp_wait(bar, parity, sh, err)) : 0;
  __syncwarp();
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// D[tmem] (+)= A[smem desc] * B[smem desc], kind::f16.
__device__ __forceinline__ void tc_mma_ss_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// MN-major operand with 128-byte swizzling: rows (k) of 64 values, 8-row
// groups 1024 bytes apart (SBO), 64-value blocks `lbo` bytes apart.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t smem_addr, uint32_t lbo) {
  return uint64_t((smem_addr >> 4) & 0x3FFFu) | (uint64_t(lbo >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// The row tile (of kRows rows) that unit u is; the tiles of a sequence are
// taken from its last, whose range of keys is longest.  False past the last
// one.
template <int D>
__device__ __forceinline__ bool kp_find(const KaParams& p, int u, int& seq, int& tile) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b0 = 0; b0 < p.batch.batch; b0 += 32) {
    KvSeq s{0, 0, 0, false};
    if (b0 + lane < p.batch.batch) s = kv_load_seq(p.batch, b0 + lane, p.cache.page_shift);
    const int rows = s.q_len * p.group;
    const int own = rows < kKpMinRows ? 0 : (rows + KpCfg<D>::kRows - 1) / KpCfg<D>::kRows;
    int sum = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > u);
    if (past) {
      const int l = __ffs(past) - 1;
      seq = b0 + l;
      tile = __shfl_sync(0xffffffffu, before + sum, l) - 1 - u;
      return true;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

template <int D>
__global__ void __launch_bounds__(KpCfg<D>::kThreads, 1) kv_prefill_kernel(const KaParams p) {
  using C = KpCfg<D>;
  extern __shared__ __align__(1024) uint8_t kp_smem[];
  const uint32_t q0 = (smem_u32(kp_smem) + 1023u) & ~1023u;
  const uint32_t k0 = q0 + C::kTiles * C::kQ, v0 = k0 + C::kStages * C::kKV;
  KpShared* sh = reinterpret_cast<KpShared*>(kp_smem + (v0 + C::kStages * C::kKV - smem_u32(kp_smem)));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh->k_full[i], kKpConvWarps);
      mbar_init(&sh->v_full[i], kKpConvWarps);
      mbar_init(&sh->k_empty[i], 1);
      mbar_init(&sh->v_empty[i], 1);
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->pv_done[i], 1);
      mbar_init(&sh->p_full[i], 4);
    }
    mbar_init(&sh->q_full, C::kSoftWarps);
    mbar_init(&sh->drain, 2);
    sh->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    const int units = kp_units<D>(p), rest = units % p.sms, whole = units - rest;
    // 1 where the rest is more than half a wave (or where sequences share rows, and so have more units than CTAs)
    const int parts = rest > 0 && units <= int(gridDim.x) - p.sms ? min(kKpMaxParts, p.sms / rest) : 1;
    const int over = int(blockIdx.x) - whole;                          // place among the parts of the rest
    const int nth = over < 0 ? int(blockIdx.x) : whole + over / parts;
    int b = 0, tile = 0;
    const bool found = nth < units && kp_find<D>(p, nth / p.cache.kv_heads, b, tile);
    if (lane == 0) {
      sh->found = found, sh->b = b, sh->tile = tile, sh->head = nth % p.cache.kv_heads;
      sh->parts = over < 0 ? 1 : parts;
      sh->part = over < 0 ? 0 : over % parts;
      sh->slot = over < 0 ? 0 : over / parts;
    }
  }
  __syncthreads();
  if (!sh->found) return;
  if (warp == 0) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const KvSeq seq = kv_load_seq(p.batch, sh->b, p.cache.page_shift);
  const int rows = seq.q_len * p.group, row0 = sh->tile * C::kRows;
  const int last = min(rows, row0 + C::kRows) - 1;
  const KvRange range = kv_range(seq, row0 / p.group, last / p.group, p.window);
  const int key_lo = range.lo & ~(C::TK - 1), all_tiles = (range.hi - key_lo + C::TK - 1) / C::TK;
  const int head = sh->head, part = sh->part, parts = sh->parts;
  const int tile0 = int((long long)all_tiles * part / parts);
  const int n_tiles = int((long long)all_tiles * (part + 1) / parts) - tile0, key0 = key_lo + tile0 * C::TK;
  constexpr int kMmaWarp = C::kSoftWarps + kKpConvWarps;

  if (warp < C::kSoftWarps) {
    // ------------------------------------------------ softmax: a thread per row
    const int t = warp >> 2, q = warp & 3;
    const int r = 32 * q + lane;                      // row of the tile, TMEM lane
    const int row = min(row0 + 128 * t + r, rows - 1);  // rows past the last repeat it and are not stored
    const bool live = row0 + 128 * t + r < rows;
    const int j = row / p.group, h = head * p.group + row - j * p.group;
    const uint32_t trow = uint32_t(32 * q) << 16;
    float f;
    {
      // q to fp16 with the row's power of two, [64-value block][row][128 bytes], swizzled
      const uint16_t* src = p.q.data + (long long)(seq.start + j) * p.q.token + h * p.q.head;
      float top = 0.f;
#pragma unroll 4
      for (int i = 0; i < D; i += 8) {
        float v[8];
        bf16x8_to_float(__ldcg(reinterpret_cast<const uint4*>(src + i)), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
      }
      const int e2 = ka_row_power(top);
      float up = __uint_as_float(uint32_t(127 + e2) << 23);
      f = __uint_as_float(uint32_t(127 - e2) << 23) * p.scale_log2;
      if (f < 0.f) {  // a negative scale goes into q, so that larger products stay larger scores
        f = -f;
        up = -up;
      }
#pragma unroll 4
      for (int i = 0; i < D; i += 8) {
        float v[8];
        bf16x8_to_float(__ldcg(reinterpret_cast<const uint4*>(src + i)), v);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 x = __floats2half2_rn(v[2 * e] * up, v[2 * e + 1] * up);
          w[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
        sts128(q0 + uint32_t(t) * C::kQ + uint32_t(i >> 6) * (128 * 128) + uint32_t(r) * 128u +
                   ((uint32_t((i >> 3) & 7) ^ uint32_t(r & 7)) << 4),
               w[0], w[1], w[2], w[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_full);
    }
    const int lim = seq.kv_len - seq.q_len + j;                      // last key of the row
    const int low = p.window > 0 ? lim - p.window + 1 : 0;           // first
    int lim0 = seq.kv_len - seq.q_len + (row0 + 128 * t) / p.group;         // last key of the tile's first row
    const int low1 = p.window > 0 ? range.hi - p.window : 0;         // first key of the CTA's last row
    float z = -INFINITY, l = 0.f;
    bool ok = true;
    for (int i = 0; i < n_tiles && ok; ++i) {
      const int slot = 2 * t + (i & 1);
      const uint32_t par = uint32_t((i >> 1) & 1);
      ok = kp_wait_warp(&sh->s_full[slot], par, sh, p.err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sbuf = tmem + trow + uint32_t(slot) * C::kSCols;
      const int key = key0 + i * C::TK;
      const float* ks = sh->ks[i & 7];
      const float* lv = sh->lv[i & 7];
      const float* iv = sh->iv[i & 7];
      const bool edge = key + C::TK - 1 > lim0 || key < low1;
      // ---- the row's largest score + log2(vs)
      float x = -INFINITY;
      uint32_t v[C::TK / 32][32];  // 64 scores
      if (!edge) {
#pragma unroll
        for (int c = 0; c < C::TK / 32; ++c) tmem_ld_32x32b_x32(sbuf + uint32_t(32 * c), v[c]);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < C::TK / 32; ++c) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            auto s = [&](int e) { return __uint_as_float(v[c][16 * g + e]); };
            const float m0 = max3(s(0), s(1), s(2)), m1 = max3(s(3), s(4), s(5)), m2 = max3(s(6), s(7), s(8));
            const float m3 = max3(s(9), s(10), s(11)), m4 = max3(s(12), s(13), s(14));
            const float top = fmaxf(max3(m0, m1, m2), max3(m3, m4, s(15)));
            x = fmaxf(x, fmaf(top, f * ks[2 * c + g], lv[2 * c + g]));
          }
        }
      } else {
#pragma unroll 1
        for (int g = 0; g < C::KG; ++g) {
          uint32_t y[16];
          tmem_ld_32x32b_x16(sbuf + uint32_t(16 * g), y);
          tc_wait_ld();
          const int k0g = key + 16 * g;
          float m = -INFINITY;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            m = fmaxf(m, k0g + e <= lim && k0g + e >= low ? __uint_as_float(y[e]) : -INFINITY);
          // (a group without a visible key stays at -inf, whatever its factor)
          if (m > -INFINITY) x = fmaxf(x, fmaf(m, f * ks[g], lv[g]));
        }
      }
      if (__any_sync(0xffffffffu, x - z > 15.f)) {  // (z = -inf: the first visible key)
        const float nz = fmaxf(z, __fadd_ru(x, -7.f));
        const float grow = z == -INFINITY ? 0.f : ex2(z - nz);
        if (i > 0) {
          // O's last product must be done
          ok = kp_wait_warp(&sh->pv_done[2 * t + ((i - 1) & 1)], uint32_t(((i - 1) >> 1) & 1), sh, p.err);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t y[16];
            const uint32_t at = tmem + trow + C::kOCol + uint32_t(t * D + c);
            tmem_ld_32x32b_x16(at, y);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * grow);
            tmem_st_32x32b_x16(at, y);
          }
          tc_wait_st();
        }
        l *= grow;
        z = nz;
        // Scores beyond 2^20 (of any row of the warp): this tile, once more, and the rest take the path of edge tiles, which
        // rounds t as it is rounded in z.  The other path has t and -z in one multiply-add, which differs from that by what
        // t's rounding lost: 2^-4 at 2^20, more than fp16's range from 2^24 on.
        if (__any_sync(0xffffffffu, fabsf(z) > 0x1p20f && z > -INFINITY)) {
          lim0 = -1;
          if (!edge) {
            --i;
            continue;
          }
        }
      }
      const float ref = z == -INFINITY ? 0.f : z;
      // ---- P' and the sum of p
      if (!edge) {
#pragma unroll
        for (int c = 0; c < C::TK / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float kf = f * ks[2 * c + g], off = lv[2 * c + g] - ref;
            const uint64_t kf2 = pack2(kf, kf), off2 = pack2(off, off);
            uint64_t sum = pack2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 x2 = unpack2(fma2(pack2(__uint_as_float(v[c][16 * g + e]), __uint_as_float(v[c][16 * g + e + 1])), kf2, off2));
              const float a = ex2(x2.x), b = ex2(x2.y);
              sum = q8_add2(sum, pack2(a, b));
              const __half2 hh = __floats2half2_rn(a, b);
              w[8 * g + e / 2] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            const float2 s2 = unpack2(sum);
            l = fmaf(s2.x + s2.y, iv[2 * c + g], l);
          }
          // (into the columns of scores that are read already)
          tmem_st_32x32b_x16(sbuf + uint32_t(16 * c), w);
        }
      } else {
#pragma unroll 1
        for (int g = 0; g < C::KG; ++g) {
          uint32_t y[16], w[8];
          tmem_ld_32x32b_x16(sbuf + uint32_t(16 * g), y);
          tc_wait_ld();
          const float kf = f * ks[g];
          const int k0g = key + 16 * g;
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float a = ex2(fmaf(__uint_as_float(y[e]), kf, lv[g]) - ref), b = ex2(fmaf(__uint_as_float(y[e + 1]), kf, lv[g]) - ref);
            a = k0g + e <= lim && k0g + e >= low ? a : 0.f;
            b = k0g + e + 1 <= lim && k0g + e + 1 >= low ? b : 0.f;
            sum += a + b;
            const __half2 hh = __floats2half2_rn(a, b);
            w[e / 2] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          l = fmaf(sum, iv[g], l);
          tmem_st_32x32b_x8(sbuf + uint32_t(8 * g), w);
        }
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full[slot]);
    }
    // ---- O / l
    if (ok) ok = kp_wait_warp(&sh->drain, 0, sh, p.err);
    tc_fence_after();
    uint16_t* dst = p.out.data + (long long)(seq.start + j) * p.out.token + h * p.out.head;
    const uint32_t ocol = tmem + trow + C::kOCol + uint32_t(t * D);
    if (parts == 1) {
      const float norm = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
#pragma unroll 1
      for (int c = 0; c < D && ok; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(ocol + uint32_t(c), v);
        tc_wait_ld();
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __uint_as_float(v[e + k]) * norm;
            *reinterpret_cast<uint4*>(dst + c + e) = float_to_bf16x8(o);
          }
        }
      }
    } else {
      // [part][O: D / 4][row][4], z [row], l [row]
      constexpr size_t kPart = size_t(C::kRows) * (D + 2);
      const int pr = 128 * t + r;
      float* slot = p.part + size_t(sh->slot) * parts * kPart;
      float* mine = slot + size_t(part) * kPart;
      if (n_tiles > 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(ocol + uint32_t(c), v);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4*>(mine + (size_t((c + e) / 4) * C::kRows + pr) * 4) =
                make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
      mine[C::kRows * D + pr] = ok ? z : -INFINITY;
      mine[C::kRows * D + C::kRows + pr] = l;
      __threadfence();
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kSoftWarps) : "memory");
      if (threadIdx.x == 0) sh->last = atomicAdd(p.counters + kKaMaxCtas + sh->slot, 1u) == unsigned(parts - 1);
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kSoftWarps) : "memory");
      if (sh->last) {
        __threadfence();
        float w[kKpMaxParts], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int s = 0; s < kKpMaxParts; ++s) {
          w[s] = s < parts ? __ldcg(slot + s * kPart + C::kRows * D + pr) : -INFINITY;
          top = fmaxf(top, w[s]);
        }
#pragma unroll
        for (int s = 0; s < kKpMaxParts; ++s) {  // (a part of which the row sees nothing has z = -inf, and O unset)
          w[s] = w[s] == -INFINITY ? 0.f : ex2(w[s] - top);
          if (w[s] > 0.f) sum = fmaf(w[s], __ldcg(slot + s * kPart + C::kRows * D + C::kRows + pr), sum);
        }
        const float norm = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
        if (live) {
#pragma unroll 2
          for (int c = 0; c < D; c += 8) {
            float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < kKpMaxParts; ++s)
              if (w[s] > 0.f) {
                const float* at = slot + s * kPart + (size_t(c / 4) * C::kRows + pr) * 4;
                const float4 a = __ldcg(reinterpret_cast<const float4*>(at));
                const float4 b = __ldcg(reinterpret_cast<const float4*>(at + 4 * C::kRows));
                o[0] = fmaf(w[s], a.x, o[0]), o[1] = fmaf(w[s], a.y, o[1]), o[2] = fmaf(w[s], a.z, o[2]);
                o[3] = fmaf(w[s], a.w, o[3]), o[4] = fmaf(w[s], b.x, o[4]), o[5] = fmaf(w[s], b.y, o[5]);
                o[6] = fmaf(w[s], b.z, o[6]), o[7] = fmaf(w[s], b.w, o[7]);
              }
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] *= norm;
            *reinterpret_cast<uint4*>(dst + c) = float_to_bf16x8(o);
          }
        }
        if (threadIdx.x == 0) p.counters[kKaMaxCtas + sh->slot] = 0u;  // ready for the next launch on this workspace
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------ converters
    constexpr int LPR = D / 16;              // lanes of a key (16 codes each)
    constexpr int RPP = 128 / LPR;           // keys of a pass
    constexpr int NP = C::TK / RPP;          // passes of a tile
    const int tid = threadIdx.x - 32 * C::kSoftWarps;
    const int sub = tid % LPR, r0 = tid / LPR;
    const int* table = p.batch.table + (long long)sh->b * p.batch.table_stride;
    const int ps = p.cache.page_shift;
    // Page ids of a tile's groups: lane g holds group g's (-1: nothing there).  What is fetched is looked at an
    // iteration later, so that no load is waited for.
    auto fetch_ids = [&](int i) {
      const int key = key0 + i * C::TK + 16 * lane;
      return i < n_tiles && lane < C::KG && key < range.hi ? __ldg(table + (key >> ps)) : -1;
    };
    auto checked = [&](int id, int i) {
      if (id >= p.cache.pages || (id < 0 && i < n_tiles && lane < C::KG && key0 + i * C::TK + 16 * lane < range.hi)) {
        record_error(p.err, kErrInput);
        id = -1;
      }
      return id;
    };
    // A group without a page reads page 0 instead (its values are zeroed when they are stored), so that the
    // loads are plain and stay in flight together.
    auto load = [&](int kind, int i, int ids, uint4 (&w)[NP]) {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const int r = n * RPP + r0;
        const int id = max(__shfl_sync(0xffffffffu, ids, r >> 4), 0);
        const long long at = ((((long long)id * p.cache.kv_heads + head) << ps) + ((key0 + i * C::TK + r) & ((1 << ps) - 1))) * D;
        w[n] = __ldg(reinterpret_cast<const uint4*>(p.cache.codes[kind] + at) + sub);
      }
    };
    auto fetch_scales = [&](int ids) {  // ks, vs of the lane's group
      const long long at = (long long)max(ids, 0) * p.cache.kv_heads + head;
      return make_float2(__ldg(p.cache.scales[0] + at), __ldg(p.cache.scales[1] + at));
    };
    // live: a bit per key group; a dead group's values are zeros.  16 codes are two 16-byte chunks of a row; lanes
    // 4 apart start with different halves (no bank conflict).  RPP is a multiple of 8, so a thread's chunks keep
    // their swizzle from pass to pass.
    static_assert(RPP % 8 == 0, "passes keep the swizzle");
    const uint32_t at_row = uint32_t(sub >> 2) * uint32_t(C::TK * 128) + uint32_t(r0) * 128u;
    const uint32_t ch = uint32_t(sub & 3) * 2u, sw = uint32_t(r0 & 7);
    const uint32_t at_a = at_row + (((ch + ((sub & 4) ? 1u : 0u)) ^ sw) << 4);
    const uint32_t at_b = at_row + (((ch + ((sub & 4) ? 0u : 1u)) ^ sw) << 4);
    auto store = [&](uint32_t base, const uint4 (&w)[NP], unsigned live) {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        // code + 128, or 128 (a zero) in a dead group
        uint32_t x[4] = {w[n].x ^ 0x80808080u, w[n].y ^ 0x80808080u, w[n].z ^ 0x80808080u, w[n].w ^ 0x80808080u};
        if (live != (1u << C::KG) - 1u && !((live >> ((n * RPP + r0) >> 4)) & 1u)) x[0] = x[1] = x[2] = x[3] = 0x80808080u;
        if (sub & 4) {
          const uint32_t y0 = x[0], y1 = x[1];
          x[0] = x[2], x[1] = x[3], x[2] = y0, x[3] = y1;
        }
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] = ka_codes(x[e], 0x4140u);
          o[2 * e + 1] = ka_codes(x[e], 0x4342u);
        }
        sts128(base + at_a + uint32_t(n * RPP * 128), o[0], o[1], o[2], o[3]);
        sts128(base + at_b + uint32_t(n * RPP * 128), o[4], o[5], o[6], o[7]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    uint4 wk[NP], wv[NP];
    // (the first tile may start in pages that the window has passed)
    int ids = key0 + 16 * lane < kv_first_key(range, ps) ? -1 : checked(fetch_ids(0), 0), raw = fetch_ids(1);
    load(0, 0, ids, wk);
    load(1, 0, ids, wv);
    float2 sc = fetch_scales(ids);
    bool ok = true, k_free = true, v_free = true;
    int st = 0;
    uint32_t phase = 1;
    for (int i = 0; i < n_tiles && ok; ++i) {
      const bool here = lane < C::KG && ids >= 0;
      const float s_k = here ? sc.x : 0.f, s_v = here ? sc.y : 0.f;
      const unsigned has = __ballot_sync(0xffffffffu, here), live_v = __ballot_sync(0xffffffffu, s_v >= kKvLeastScale);
      if (!k_free) ok = kp_wait_warp(&sh->k_empty[st], phase, sh, p.err);
      if (!ok) break;
      if (tid < C::KG) {
        // a page without a V scale counts in the sum of p like any other: its values are zeros at a stand-in scale
        const float v = fmaxf(s_v, kKvLeastScale);
        sh->ks[i & 7][tid] = s_k;
        sh->lv[i & 7][tid] = __log2f(v);
        sh->iv[i & 7][tid] = __fdiv_rn(1.f, v);
      }
      store(k0 + uint32_t(st) * C::kKV, wk, has);
      if (lane == 0) mbar_arrive(&sh->k_full[st]);
      ids = checked(raw, i + 1);
      load(0, i + 1, ids, wk);
      sc = fetch_scales(ids);
      raw = fetch_ids(i + 2);
      if (!v_free) ok = kp_wait_warp(&sh->v_empty[st], phase, sh, p.err);
      if (!ok) break;
      store(v0 + uint32_t(st) * C::kKV, wv, live_v);
      if (lane == 0) mbar_arrive(&sh->v_full[st]);
      load(1, i + 1, ids, wv);
      if (++st == C::kStages) { st = 0; phase ^= 1u; }
      // (a look at a barrier costs a warp about 150 clocks if it waits for the answer)
      k_free = mbar_test_wait(&sh->k_empty[st], phase);
      v_free = mbar_test_wait(&sh->v_empty[st], phase);
      k_free = __all_sync(0xffffffffu, k_free);
      v_free = __all_sync(0xffffffffu, v_free);
    }
  } else if (lane == 0) {
    // ------------------------------------------------ MMA issuers
    // The issuing thread's own instructions must stay few: descriptors are bases with constants added to their low
    // word (the address field; shared memory ends below 256 KiB, so nothing carries out of it), and as a wait costs
    // about 150 clocks even on a barrier that is complete (measured), each barrier is probed ahead of the MMAs that
    // come before it and waited for only where the probe found it incomplete.
    auto plus = [](uint64_t d, uint32_t bytes) {
      return (d & 0xFFFFFFFF00000000ull) | uint64_t(uint32_t(d) + (bytes >> 4));
    };
    bool ok = true;
    int st = 0;          // stage of tile i
    uint32_t phase = 0;  // and its phase
    if (warp == kMmaWarp) {
      // ---- scores: tile i into buffer i & 1, whose P' the product of tile i - 2 must have read
      const uint64_t qd0 = sw128_desc(q0), kd0 = sw128_desc(k0);
      ok = kp_wait(&sh->q_full, 0, sh, p.err);
      bool k_in = false, f_in = false;
      for (int i = 0; i < n_tiles && ok; ++i) {
        if (!k_in) ok = kp_wait(&sh->k_full[st], phase, sh, p.err);
        if (!ok) break;
        const uint64_t kd = plus(kd0, uint32_t(st) * C::kKV);
        for (int t = 0; t < C::kTiles; ++t) {
          if (i >= 2 && !f_in) ok = kp_wait(&sh->pv_done[2 * t + (i & 1)], uint32_t(((i - 2) >> 1) & 1), sh, p.err);
          if (!ok) break;
          tc_fence_after();
          f_in = t + 1 < C::kTiles ? i >= 2 && mbar_test_wait(&sh->pv_done[2 + (i & 1)], uint32_t(((i - 2) >> 1) & 1)) : false;
          const uint64_t qd = plus(qd0, uint32_t(t) * C::kQ);
          const int slot = 2 * t + (i & 1);
          const uint32_t at = tmem + uint32_t(slot) * C::kSCols;
#pragma unroll
          for (int d = 0; d < D; d += 16)
            tc_mma_ss_f16(at, plus(qd, uint32_t(d >> 6) * (128u * 128u) + uint32_t(d & 63) * 2u),
                          plus(kd, uint32_t(d >> 6) * uint32_t(C::TK * 128) + uint32_t(d & 63) * 2u), C::kIdescQK,
                          d ? 1u : 0u);
          tc_commit(&sh->s_full[slot]);
        }
        if (!ok) break;
        tc_commit(&sh->k_empty[st]);
        if (++st == C::kStages) { st = 0; phase ^= 1u; }
        k_in = i + 1 < n_tiles && mbar_test_wait(&sh->k_full[st], phase);
        f_in = i >= 1 && mbar_test_wait(&sh->pv_done[(i + 1) & 1], uint32_t(((i - 1) >> 1) & 1));
      }
    } else {
      // ---- O += P' V
      const uint64_t vd0 = sw128_mn_desc(v0, C::TK * 128);
      bool v_in = false, p_in = false;
      for (int i = 0; i < n_tiles && ok; ++i) {
        const uint32_t pp = uint32_t((i >> 1) & 1);
        if (!v_in) ok = kp_wait(&sh->v_full[st], phase, sh, p.err);
        const uint64_t vd = plus(vd0, uint32_t(st) * C::kKV);
        for (int t = 0; t < C::kTiles && ok; ++t) {
          if (!p_in) ok = kp_wait(&sh->p_full[2 * t + (i & 1)], pp, sh, p.err);
          if (!ok) break;
          tc_fence_after();
          p_in = t + 1 < C::kTiles ? mbar_test_wait(&sh->p_full[2 + (i & 1)], pp) : false;
          const uint32_t at = tmem + C::kOCol + uint32_t(t * D), ap = tmem + uint32_t(2 * t + (i & 1)) * C::kSCols;
#pragma unroll
          for (int k = 0; k < C::TK; k += 16)
            tc_mma_ts_f16(at, ap + uint32_t(k / 2), plus(vd, uint32_t(k) * 128u), C::kIdescPV, (i | k) ? 1u : 0u);
          tc_commit(&sh->pv_done[2 * t + (i & 1)]);
        }
        if (!ok) break;
        tc_commit(&sh->v_empty[st]);
        if (++st == C::kStages) { st = 0; phase ^= 1u; }
        v_in = i + 1 < n_tiles && mbar_test_wait(&sh->v_full[st], phase);
        p_in = i + 1 < n_tiles && mbar_test_wait(&sh->p_full[(i + 1) & 1], uint32_t(((i + 1) >> 1) & 1));
      }
    }
    pdl_launch_dependents();  // (late: the next kernel's bounded waits must not last as long as this one)
    tc_commit(&sh->drain);  // everything that this thread issued
    mbar_wait_bounded(&sh->drain, 0, p.err, 1u << 20);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace w4a8
