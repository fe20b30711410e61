// int8 x int8 product on the tensor cores (tcgen05.mma kind::i8, int32
// accumulation in TMEM):
//
//   y[m, n] = bf16( s_x[m] * s_w[n] * sum_k x_q[m, k] w_q[n, k] )
//
// The sum is exact: |code| <= 128 and K <= 32768 keep it below 2^29.  It is
// rounded once to fp32, scaled in fp32 and rounded to bf16.
//
// The product is computed transposed like the other GEMMs here: a tile is
// 128 weight rows (the MMA's M, TMEM lanes) x NT tokens (its N), k in blocks
// of 128 bytes loaded by TMA into 128-byte-swizzled stages.  TMA fills rows
// past M or N and k past K with zeros, so every ragged edge is plain.
//
// The work is a list of items (tile, k block), tiles in [row tile][token
// tile] order.  Each CTA (one per SM) takes a contiguous range of items, so
// the weight stream of a few wide rows spreads over every SM; a tile that is
// cut between CTAs is joined from int32 partial tiles by its last CTA to
// arrive (integer sums, so the order does not matter).  Three roles: a TMA
// thread, an MMA thread and four epilogue warps; two accumulators let the
// epilogue of a tile run under the next tile's MMAs.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "gemm_sk.cuh"
#include "gemm_tc.cuh"

namespace w4a8 {

constexpr int kQ8Rows = 128;
constexpr int kQ8BK = 128;       // k per stage (bytes)
constexpr int kQ8Threads = 192;  // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr int kQ8MaxCtas = 160;  // CTAs of a launch (one per SM)

template <int NT>
struct Q8Cfg {
  static constexpr uint32_t kA = kQ8Rows * kQ8BK;
  static constexpr uint32_t kB = NT * kQ8BK;
  static constexpr uint32_t kStage = kA + kB;
  static constexpr uint32_t kTrans = 4 * 2048;  // the epilogue warps' 32 x 32 bf16 blocks
  static constexpr int kStages = int((232448 - 3072 - kTrans) / kStage) > 12 ? 12 : int((232448 - 3072 - kTrans) / kStage);
  static constexpr size_t kSmem = 3072 + kTrans + size_t(kStages) * kStage;
  static constexpr uint32_t kTmemCols = 2 * NT < 32 ? 32 : 2 * NT;
  // kind::i8: S32 accumulator (2 at bit 4), S8 A and B (1 at bits 7 and 10),
  // both K-major, N >> 3 at bit 17, M >> 4 at bit 24
  static constexpr uint32_t kIdesc =
      (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(NT >> 3) << 17) | (uint32_t(kQ8Rows >> 4) << 24);
  static_assert(kStage % 1024 == 0 && kStages >= 3, "1024-byte aligned stages, a pipeline");
  static_assert(NT % 16 == 0 && NT >= 16 && NT <= 256, "token tile");
};

struct Q8Params {
  const float* s_x;
  const float* s_w;
  uint16_t* y;
  int* part;           // [CTA][2][NT][128] int32: the CTA's first and last partial tile
  unsigned* counters;  // [CTA][4]: arrivals at the tile that starts in the CTA, per lane quarter
  unsigned* err;
  int M, N, K, KB, TM;  // KB: k blocks, TM: token tiles
  int G;                // CTAs
  int whole;            // ranges are cut between tiles only
  long long items;      // tiles * KB
};

struct Q8Shared {
  uint64_t full[12];
  uint64_t empty[12];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort;
};

// First item of CTA c: an even share, or the nearest tile border.
__host__ __device__ inline long long q8_cta_item(long long c, const Q8Params& p) {
  if (p.whole) return (p.items / p.KB) * c / p.G * p.KB;
  return p.items * c / p.G;
}
// The CTA whose range holds item i.
__host__ __device__ inline int q8_item_cta(long long i, const Q8Params& p) {
  long long c = i * p.G / p.items;
  while (c + 1 < p.G && q8_cta_item(c + 1, p) <= i) ++c;
  while (c > 0 && q8_cta_item(c, p) > i) --c;
  return int(c);
}

__device__ __forceinline__ bool q8_wait(uint64_t* bar, uint32_t parity, Q8Shared* sh, unsigned* err) {
  for (uint32_t i = 0; i < (1u << 20); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 1023u && sh->abort) return false;
  }
  sh->abort = 1;
  record_error(err, kErrTimeout);
  return false;
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::i8.
__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int NT>
__global__ void __launch_bounds__(kQ8Threads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                     const Q8Params p) {
  using C = Q8Cfg<NT>;
  extern __shared__ __align__(1024) uint8_t q8_smem[];
  pdl_launch_dependents();
  Q8Shared* sh = reinterpret_cast<Q8Shared*>(q8_smem);
  const uint32_t stage0 = (smem_u32(q8_smem) + uint32_t(sizeof(Q8Shared)) + 1023u) & ~1023u;
  const uint32_t trans0 = stage0 + uint32_t(C::kStages) * C::kStage;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long i0 = q8_cta_item(blockIdx.x, p), i1 = q8_cta_item(blockIdx.x + 1, p);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], 4);  // one arrival per epilogue warp
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------ producer
    if (lane == 0 && i0 < i1) {
      tma_prefetch_desc(&tmap_w);
      tma_prefetch_desc(&tmap_x);
      // The first stages' weights do not depend on the previous kernel: they
      // are loaded before the wait for it, their tokens after.
      int kb = int(i0 % p.KB);
      long long tile = i0 / p.KB;
      const int n_pre = int(i1 - i0 < C::kStages ? i1 - i0 : C::kStages);
      {
        int k = kb;
        long long t = tile;
        for (int j = 0; j < n_pre; ++j) {
          mbar_arrive_expect_tx(&sh->full[j], C::kStage);
          tma_load_2d(stage0 + uint32_t(j) * C::kStage, &tmap_w, &sh->full[j], k * kQ8BK, int(t / p.TM) * kQ8Rows);
          if (++k == p.KB) { k = 0; ++t; }
        }
      }
      pdl_wait();
      int s = 0;
      uint32_t phase = 0;
      for (long long i = i0; i < i1; ++i) {
        const uint32_t a = stage0 + uint32_t(s) * C::kStage;
        const int rt = int(tile / p.TM), mt = int(tile - (long long)rt * p.TM);
        if (i - i0 >= n_pre) {
          if (!q8_wait(&sh->empty[s], phase ^ 1u, sh, p.err)) break;
          mbar_arrive_expect_tx(&sh->full[s], C::kStage);
          tma_load_2d(a, &tmap_w, &sh->full[s], kb * kQ8BK, rt * kQ8Rows);
        }
        tma_load_2d(a + C::kA, &tmap_x, &sh->full[s], kb * kQ8BK, mt * NT);
        if (++kb == p.KB) { kb = 0; ++tile; }
        if (++s == C::kStages) { s = 0; phase ^= 1u; }
      }
      if (sh->abort) {
        // let the copies in flight land before the CTA exits (bounded: 50 us)
        unsigned long long t0, t1;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        do {
          asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
        } while (t1 - t0 < 50000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0 && i0 < i1) {
      bool ok = true;
      int kb = int(i0 % p.KB), seg = 0, s = 0;
      uint32_t phase = 0;
      for (long long i = i0; i < i1; ++i) {
        const int buf = seg & 1;
        const bool first = i == i0 || kb == 0;
        if (first && seg >= 2) {
          ok = q8_wait(&sh->acc_empty[buf], ((seg >> 1) - 1) & 1, sh, p.err);
          if (!ok) break;
        }
        ok = q8_wait(&sh->full[s], phase, sh, p.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = stage0 + uint32_t(s) * C::kStage;
        const uint64_t ad = sw128_desc(a), bd = sw128_desc(a + C::kA);
#pragma unroll
        for (int j = 0; j < kQ8BK / 32; ++j)
          tc_mma_i8(tmem + uint32_t(buf) * NT, ad + uint64_t(2 * j), bd + uint64_t(2 * j), C::kIdesc,
                    (first && j == 0) ? 0u : 1u);
        tc_commit(&sh->empty[s]);
        if (++kb == p.KB || i + 1 == i1) {
          tc_commit(&sh->acc_full[buf]);
          kb = kb == p.KB ? 0 : kb;
          ++seg;
        }
        if (++s == C::kStages) { s = 0; phase ^= 1u; }
      }
      if (!ok) {  // wait for the tensor-core work already issued before the TMEM is freed
        tc_commit(&sh->drain);
        mbar_wait_bounded(&sh->drain, 0, p.err, 1u << 20);
      }
    }
  } else {
    // ------------------------------------------------ epilogue: a warp per TMEM lane quarter
    const int q = warp & 3;
    const uint32_t tbuf = trans0 + uint32_t(q) * 2048u;
    bool ok = true;
    int seg = 0;
    if (i0 < i1) pdl_wait();  // s_x, and the buffers that the previous kernels used
    for (long long i = i0; i < i1 && ok; ++seg) {
      const long long tile = i / p.KB, t0 = tile * p.KB;
      const long long end = t0 + p.KB < i1 ? t0 + p.KB : i1;
      const bool whole = i == t0 && end == t0 + p.KB;
      const int rt = int(tile / p.TM), mt = int(tile - (long long)rt * p.TM);
      const int n0 = rt * kQ8Rows + 32 * q, m0 = mt * NT;
      const int buf = seg & 1;
      const int w_ok = lane == 0 ? int(q8_wait(&sh->acc_full[buf], (seg >> 1) & 1, sh, p.err)) : 0;
      ok = __shfl_sync(0xffffffffu, w_ok, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t(32 * q) << 16) + uint32_t(buf) * NT;
      const int n = n0 + lane;
      const float sw = n < p.N ? p.s_w[n] : 0.f;
      const int slot = int(blockIdx.x) * 2 + (i0 >= t0 ? 0 : 1);
      constexpr int CW = NT < 32 ? NT : 32;  // columns at a time
#pragma unroll 1
      for (int c = 0; c < NT && m0 + c < p.M; c += CW) {
        uint32_t v[32];
        if constexpr (CW == 32) {
          tmem_ld_32x32b_x32(acc + uint32_t(c), v);
        } else {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < CW / 8; ++e) {
            tmem_ld_32x32b_x8(acc + uint32_t(c + 8 * e), h);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * e + j] = h[j];
          }
#pragma unroll
          for (int j = CW; j < 32; ++j) v[j] = 0u;
        }
        tc_wait_ld();
        if (whole) {
          store_block_transposed(p.y, min(p.M, m0 + NT), p.N, m0 + c, n0, tbuf, lane, [&](int j) {
            const float sx = m0 + c + j < p.M ? p.s_x[m0 + c + j] : 0.f;
            return __bfloat16_as_ushort(__float2bfloat16_rn(__int2float_rn(int(v[j])) * sw * sx));
          });
        } else {
#pragma unroll
          for (int j = 0; j < CW; ++j)
            if (m0 + c + j < p.M) p.part[(size_t(slot) * NT + c + j) * kQ8Rows + 32 * q + lane] = int(v[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->acc_empty[buf]);
      if (!whole) {
        // count in at the tile's first CTA; the last to arrive adds the partial tiles
        const int c_first = q8_item_cta(t0, p), c_last = q8_item_cta(t0 + p.KB - 1, p);
        unsigned* cnt = p.counters + c_first * 4 + q;
        __threadfence();
        __syncwarp();
        unsigned old = 0;
        if (lane == 0) old = atomicAdd(cnt, 1u);
        old = __shfl_sync(0xffffffffu, old, 0);
        if (old == unsigned(c_last - c_first)) {
          __threadfence();
#pragma unroll 1
          for (int c = 0; c < NT && m0 + c < p.M; c += CW) {
            int v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0;
            const int live = min(CW, p.M - m0 - c);
            for (int cc = c_first; cc <= c_last; ++cc) {
              const int sl = cc * 2 + (q8_cta_item(cc, p) >= t0 ? 0 : 1);
              const int* src = p.part + (size_t(sl) * NT + c) * kQ8Rows + 32 * q + lane;
#pragma unroll
              for (int j = 0; j < CW; ++j)
                if (j < live) v[j] += __ldcg(src + j * kQ8Rows);
            }
            store_block_transposed(p.y, min(p.M, m0 + NT), p.N, m0 + c, n0, tbuf, lane, [&](int j) {
              const float sx = m0 + c + j < p.M ? p.s_x[m0 + c + j] : 0.f;
              return __bfloat16_as_ushort(__float2bfloat16_rn(__int2float_rn(v[j]) * sw * sx));
            });
          }
          __syncwarp();
          if (lane == 0) *cnt = 0u;  // ready for the next launch on this workspace
        }
      }
      i = end;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace w4a8
