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
// Tile kernel (this file): one tile per cluster.  Where tiles are few, the
// 1 to 8 CTAs of a cluster share a tile's k blocks and join their int32
// accumulators through distributed shared memory, each CTA finishing its
// share of the token columns.  Integer sums, so the split does not change
// the result, and no global scratch is needed.
// Three roles: a TMA thread, an MMA thread and four epilogue warps.  The
// weights do not depend on the previous kernel, so the first stages' weight
// tiles are loaded before the wait for it.
// With the quantiser, 1 token of K = 5120, N = 17408 takes 15.7 us (5.7 TB/s of
// weights) and 45 tokens of K = 4304, N = 10010 16.8 (79 row tiles on 148 SMs).
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "common.cuh"
#include "gemm_sk.cuh"
#include "gemm_tc.cuh"

namespace w4a8 {

constexpr int kQ8Rows = 128;
constexpr int kQ8BK = 128;       // k per stage (bytes)
constexpr int kQ8Threads = 192;  // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr int kQ8MaxSplit = 8;   // CTAs of a cluster

template <int NT, int CPS>  // CPS: CTAs that share an SM
struct Q8Cfg {
  static constexpr uint32_t kA = kQ8Rows * kQ8BK;
  static constexpr uint32_t kB = NT * kQ8BK;
  static constexpr uint32_t kStage = kA + kB;
  static constexpr size_t kBudget = (CPS == 1 ? 232448 : size_t(233472 / CPS) - 1024) - 2048;
  static constexpr int kStages = int(kBudget / kStage) > 12 ? 12 : int(kBudget / kStage);
  static constexpr size_t kSmem = 2048 + size_t(kStages) * kStage;
  static constexpr uint32_t kTmemCols = NT < 32 ? 32 : NT;
  // kind::i8: S32 accumulator (2 at bit 4), S8 A and B (1 at bits 7 and 10),
  // both K-major, N >> 3 at bit 17, M >> 4 at bit 24
  static constexpr uint32_t kIdesc =
      (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(NT >> 3) << 17) | (uint32_t(kQ8Rows >> 4) << 24);
  static_assert(kStage % 1024 == 0 && kStages >= 3, "1024-byte aligned stages, a pipeline");
  static_assert(size_t(kStages) * kStage >= size_t(NT) * kQ8Rows * 4, "the stages hold an int32 tile");
  static_assert(NT % 16 == 0 && NT >= 16 && NT <= 256, "token tile");
};

struct Q8Params {
  const float* s_x;
  const float* s_w;
  uint16_t* y;
  unsigned* err;
  int M, N, KB;  // KB: k blocks
};

struct Q8Shared {
  uint64_t full[12];
  uint64_t empty[12];
  uint64_t acc_full;
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort;
};

template <typename Shared>
__device__ __forceinline__ bool q8_wait(uint64_t* bar, uint32_t parity, Shared* sh, unsigned* err) {
  for (uint32_t i = 0; i < (1u << 20); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 1023u && sh->abort) return false;
  }
  sh->abort = 1;
  record_error(err, kErrTimeout);
  return false;
}

// Bounded pause that lets copies in flight land before a CTA that gave up exits.
__device__ __forceinline__ void q8_settle() {
  unsigned long long t0, t1;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
  } while (t1 - t0 < 50000ull);  // 50 us
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

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

template <int NT>
__device__ __forceinline__ void q8_load_acc(uint32_t acc, int c, uint32_t (&v)[32]) {
  if constexpr (NT >= 32) {
    tmem_ld_32x32b_x32(acc + uint32_t(c), v);
    tc_wait_ld();
  } else {
#pragma unroll
    for (int e = 0; e < NT / 8; ++e) {
      uint32_t h[8];
      tmem_ld_32x32b_x8(acc + uint32_t(c + 8 * e), h);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * e + j] = h[j];
    }
#pragma unroll
    for (int j = NT; j < 32; ++j) v[j] = 0u;
  }
}

template <int NT, int CPS>
__global__ void __launch_bounds__(kQ8Threads, CPS)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                     const Q8Params p) {
  using C = Q8Cfg<NT, CPS>;
  extern __shared__ __align__(1024) uint8_t q8_smem[];
  pdl_launch_dependents();
  Q8Shared* sh = reinterpret_cast<Q8Shared*>(q8_smem);
  const uint32_t stage0 = (smem_u32(q8_smem) + uint32_t(sizeof(Q8Shared)) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = int(cluster_nctarank()), rank = int(cluster_ctarank());
  const int n0 = (int(blockIdx.x) / split) * kQ8Rows, m0 = int(blockIdx.y) * NT;
  const int k0 = int((long long)p.KB * rank / split), k1 = int((long long)p.KB * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->acc_full, 1);
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
    if (lane == 0) {
      const int pre = min(k1 - k0, C::kStages);
      for (int j = 0; j < pre; ++j) {
        mbar_arrive_expect_tx(&sh->full[j], C::kStage);
        tma_load_2d(stage0 + uint32_t(j) * C::kStage, &tmap_w, &sh->full[j], (k0 + j) * kQ8BK, n0);
      }
      pdl_wait();
      int s = 0;
      uint32_t phase = 0;
      for (int kb = k0; kb < k1; ++kb) {
        const uint32_t a = stage0 + uint32_t(s) * C::kStage;
        if (kb - k0 >= pre) {
          if (!q8_wait(&sh->empty[s], phase ^ 1u, sh, p.err)) break;
          mbar_arrive_expect_tx(&sh->full[s], C::kStage);
          tma_load_2d(a, &tmap_w, &sh->full[s], kb * kQ8BK, n0);
        }
        tma_load_2d(a + C::kA, &tmap_x, &sh->full[s], kb * kQ8BK, m0);
        if (++s == C::kStages) { s = 0; phase ^= 1u; }
      }
      if (sh->abort) q8_settle();
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      pdl_wait();  // (the bounded waits below are for this launch's own loads, not for the kernels before it)
      bool ok = true;
      int s = 0;
      uint32_t phase = 0;
      for (int kb = k0; kb < k1; ++kb) {
        ok = q8_wait(&sh->full[s], phase, sh, p.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = stage0 + uint32_t(s) * C::kStage;
        const uint64_t ad = sw128_desc(a), bd = sw128_desc(a + C::kA);
#pragma unroll
        for (int j = 0; j < kQ8BK / 32; ++j)
          tc_mma_i8(tmem, ad + uint64_t(2 * j), bd + uint64_t(2 * j), C::kIdesc, (kb > k0 || j > 0) ? 1u : 0u);
        tc_commit(&sh->empty[s]);
        if (++s == C::kStages) { s = 0; phase ^= 1u; }
      }
      if (ok) {
        tc_commit(&sh->acc_full);
      } else {  // wait for the tensor-core work already issued before the TMEM is freed
        tc_commit(&sh->drain);
        mbar_wait_bounded(&sh->drain, 0, p.err, 1u << 20);
      }
    }
  } else {
    // ------------------------------------------------ epilogue: a warp per TMEM lane quarter
    const int q = warp & 3;
    const uint32_t acc = tmem + (uint32_t(32 * q) << 16);
    pdl_wait();  // s_x, and y's earlier readers
    const int w_ok = lane == 0 ? int(q8_wait(&sh->acc_full, 0, sh, p.err)) : 0;
    if (__shfl_sync(0xffffffffu, w_ok, 0) != 0) {
      tc_fence_after();
      if (split == 1) {
        const int n = n0 + 32 * q + lane;
        const float sw = n < p.N ? p.s_w[n] : 0.f;
        const uint32_t tbuf = stage0 + uint32_t(q) * 2048u;  // every stage is free by now
#pragma unroll 1
        for (int c = 0; c < NT && m0 + c < p.M; c += 32) {
          uint32_t v[32];
          q8_load_acc<NT>(acc, c, v);
          const int end = min(p.M, m0 + NT);
          auto value = [&](int j) {
            const float sx = m0 + c + j < end ? p.s_x[m0 + c + j] : 0.f;
            return __bfloat16_as_ushort(__float2bfloat16_rn(__int2float_rn(int(v[j])) * sw * sx));
          };
          if (p.N & 7) {
            // rows of y that are not 16-byte aligned: a warp's 32 outputs of a token as they lie (2 bytes a lane)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (m0 + c + j < end && n < p.N) p.y[size_t(m0 + c + j) * p.N + n] = value(j);
          } else {
            store_block_transposed(p.y, end, p.N, m0 + c, n0 + 32 * q, tbuf, lane, value);
          }
        }
      } else {
        // the CTA's int32 tile into its shared memory: [token][row]
#pragma unroll 1
        for (int c = 0; c < NT && m0 + c < p.M; c += 32) {
          uint32_t v[32];
          q8_load_acc<NT>(acc, c, v);
#pragma unroll
          for (int j = 0; j < (NT < 32 ? NT : 32); ++j)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage0 + uint32_t((c + j) * kQ8Rows + 32 * q + lane) * 4u), "r"(v[j]));
        }
      }
    }
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync_all();  // every CTA's tile is written and visible
    pdl_wait();
    // Token columns are dealt to the cluster's CTAs, and (column, 32 rows) to a CTA's warps.
    const int cols = min(NT, p.M - m0);
    const int c0 = cols * rank / split, c1 = cols * (rank + 1) / split;
    for (int i = warp; i < 4 * (c1 - c0); i += kQ8Threads / 32) {
      const int c = c0 + (i >> 2), r = 32 * (i & 3) + lane, n = n0 + r;
      const uint32_t at = stage0 + uint32_t(c * kQ8Rows + r) * 4u;
      int v[kQ8MaxSplit];
#pragma unroll
      for (int s = 0; s < kQ8MaxSplit; ++s) v[s] = s < split ? ld_cluster_s32(at, uint32_t(s)) : 0;
      int sum = 0;
#pragma unroll
      for (int s = 0; s < kQ8MaxSplit; ++s) sum += v[s];
      if (n < p.N)
        p.y[size_t(m0 + c) * p.N + n] =
            __bfloat16_as_ushort(__float2bfloat16_rn(__int2float_rn(sum) * p.s_w[n] * p.s_x[m0 + c]));
    }
    cluster_sync_all();  // no CTA leaves while another reads its tile
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace w4a8
