// int8 x int8 product for many tokens: pairs of CTAs (tcgen05 cta_group::2).
//
// Same product as int8_gemm.cuh.  A tile is 256 tokens x 256 weight rows:
// each CTA of a cluster of two holds 128 of the tokens (its TMEM lanes) and
// loads 128 of the weight rows, and one thread of the first CTA issues the
// MMAs that read both CTAs' shared memory.  Every byte loaded then serves 256
// rows or tokens instead of 128 or 256: an SM takes 64 bytes a clock at the
// int8 MMAs' full rate (a single CTA's 128 x 256 tile: 96, more than L2
// delivers to it).  Persistent: a pair walks tiles [row tile][token tile] with
// two accumulators, so the epilogue runs under the next tile's MMAs.
//
// Tokens are the MMA's M here (the weights are, in the tile kernel): an
// epilogue thread then holds consecutive outputs of one token, 64 at a time,
// which leave as whole 128-byte rows: by a TMA store where the rows of y are
// 16-byte aligned, else a token at a time with 4-byte words.  (Weights as M
// and a transpose of 2-byte values took 11000 clocks a tile, 16-byte stores
// of each thread to its own row 15000, against 512 per 128 of K of MMAs.)
// Eight epilogue warps, two to a lane quarter, each half of the columns.
// With the quantiser (20 us), 4096 tokens of K = 5120, N = 17408 take 252 us.
//
// Barriers: `full` lives in the first CTA and counts both CTAs' bytes;
// `empty` and `acc_full` are in both, arrived at by commits that name both;
// `acc_empty` lives in the first CTA and counts both CTAs' epilogue warps.
#pragma once

#include "int8_gemm.cuh"

namespace w4a8 {

constexpr int kQ2Tile = 256;     // rows and tokens of a tile
constexpr int kQ2Threads = 320;  // warp 0 TMA, warp 1 MMA (first CTA), warps 2..9 epilogue
constexpr uint32_t kQ2Half = 128 * kQ8BK;      // a CTA's share of an operand's stage
constexpr uint32_t kQ2Stage = 2 * kQ2Half;
constexpr int kQ2Stages = 6;
constexpr uint32_t kQ2Block = 32 * 128;        // an epilogue warp's 32 tokens x 64 outputs
constexpr size_t kQ2Smem = 2048 + size_t(kQ2Stages) * kQ2Stage + 8 * kQ2Block;
constexpr uint32_t kQ2Idesc =
    (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kQ2Tile >> 3) << 17) | (uint32_t(kQ2Tile >> 4) << 24);

struct Q2Shared {
  uint64_t full[kQ2Stages];
  uint64_t empty[kQ2Stages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort;
};

__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 2-D tiled load into this CTA's shared memory, its bytes counted by a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t smem_dst, const void* desc, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(smem_dst),
      "l"(desc), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive at the barrier of this offset in both CTAs once this thread's MMAs so far have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// s_w[n .. n + 3] (n a multiple of 4); past N the values do not matter, but the reads stay inside.
__device__ __forceinline__ float4 q2_scales(const float* __restrict__ s_w, int n, int N) {
  if (n + 4 <= N) return __ldg(reinterpret_cast<const float4*>(s_w + n));
  return make_float4(__ldg(s_w + min(n, N - 1)), __ldg(s_w + min(n + 1, N - 1)), __ldg(s_w + min(n + 2, N - 1)),
                     __ldg(s_w + min(n + 3, N - 1)));
}

// Outputs [n, n + 64) of 32 tokens from the warp's block (swizzled rows of
// 128 bytes) to rows of y that are not 16-byte aligned: a token at a time,
// every lane a 4-byte word of it.  Where a row starts on an odd element the
// words are taken one element on, and its two end elements go alone.
__device__ __forceinline__ uint32_t q2_word(const uint8_t* block, int r, int i) {
  return *reinterpret_cast<const uint32_t*>(block + r * 128 + ((((i >> 2) ^ (r & 7)) << 4) | ((i & 3) << 2)));
}
__device__ __forceinline__ void q2_store_rows(const Q8Params& p, const uint8_t* block, int mb, int n, int lane) {
  const int rows = min(32, p.M - mb), cols = min(64, p.N - n);
  const size_t at = size_t(mb) * p.N + n;
  uint16_t* dst = p.y + at;
  if (cols == 64) {
    const int odd = int(at & 1), step = p.N & 1;  // row r starts on an odd element if odd ^ (r & step)
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      if (r < rows) {
        const uint32_t a = q2_word(block, r, lane), b = q2_word(block, r, min(lane + 1, 31));
        if (!(odd ^ (r & step))) {
          *reinterpret_cast<uint32_t*>(dst + 2 * lane) = a;
        } else if (lane < 31) {
          *reinterpret_cast<uint32_t*>(dst + 2 * lane + 1) = (a >> 16) | (b << 16);
        } else {
          dst[0] = uint16_t(q2_word(block, r, 0));
          dst[63] = uint16_t(a >> 16);
        }
        dst += p.N;
      }
    }
  } else {
    for (int r = 0; r < rows; ++r, dst += p.N) {
      const uint32_t a = q2_word(block, r, lane);
      if (2 * lane < cols) dst[2 * lane] = uint16_t(a);
      if (2 * lane + 1 < cols) dst[2 * lane + 1] = uint16_t(a >> 16);
    }
  }
}

__global__ void __launch_bounds__(kQ2Threads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                     const __grid_constant__ CUtensorMap tmap_y, const Q8Params p) {
  extern __shared__ __align__(1024) uint8_t q2_smem[];
  Q2Shared* sh = reinterpret_cast<Q2Shared*>(q2_smem);
  const uint32_t stage0 = (smem_u32(q2_smem) + uint32_t(sizeof(Q2Shared)) + 1023u) & ~1023u;
  const uint32_t trans0 = stage0 + uint32_t(kQ2Stages) * kQ2Stage;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = int(blockIdx.x) >> 1, pairs = int(gridDim.x) >> 1;
  const int TM = (p.M + kQ2Tile - 1) / kQ2Tile;
  const long long tiles = (long long)((p.N + kQ2Tile - 1) / kQ2Tile) * TM;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kQ2Stages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], 16);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh->tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either's loads or commits name them
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------ producer: this CTA's rows and tokens
    if (lane == 0) {
      tma_prefetch_desc(&tmap_w);
      tma_prefetch_desc(&tmap_x);
      pdl_wait();
      const uint32_t full0 = map_to_rank(smem_u32(&sh->full[0]), 0);
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (long long t = pair; t < tiles && ok; t += pairs) {
        const int rt = int(t / TM), mt = int(t - (long long)rt * TM);
        const int n0 = rt * kQ2Tile + int(rank) * 128, m0 = mt * kQ2Tile + int(rank) * 128;
        for (int kb = 0; kb < p.KB; ++kb) {
          ok = q8_wait(&sh->empty[s], phase ^ 1u, sh, p.err);
          if (!ok) break;
          const uint32_t a = stage0 + uint32_t(s) * kQ2Stage, bar = full0 + uint32_t(s) * 8u;
          if (rank == 0) mbar_arrive_expect_tx(&sh->full[s], 2 * kQ2Stage);
          tma_load_2d_pair(a, &tmap_x, bar, kb * kQ8BK, m0);
          tma_load_2d_pair(a + kQ2Half, &tmap_w, bar, kb * kQ8BK, n0);
          if (++s == kQ2Stages) { s = 0; phase ^= 1u; }
        }
      }
      pdl_launch_dependents();  // (late: the next kernel's bounded waits must not last as long as this one)
      if (sh->abort) q8_settle();
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (first CTA)
    if (lane == 0 && rank == 0) {
      pdl_wait();  // (the bounded waits below are for this launch's own loads, not for the kernels before it)
      int s = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true, in = false;
      const uint64_t ad0 = sw128_desc(stage0), bd0 = sw128_desc(stage0 + kQ2Half);
      for (long long t = pair; t < tiles && ok; t += pairs, ++n) {
        const int buf = n & 1;
        if (n >= 2) ok = q8_wait(&sh->acc_empty[buf], uint32_t((n >> 1) - 1) & 1u, sh, p.err);
        if (!ok) break;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!in) ok = q8_wait(&sh->full[s], phase, sh, p.err);
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = uint64_t(uint32_t(s) * (kQ2Stage >> 4));
          if (++s == kQ2Stages) { s = 0; phase ^= 1u; }
          in = mbar_test_wait(&sh->full[s], phase);  // looked at ahead of this stage's MMAs
#pragma unroll
          for (int j = 0; j < kQ8BK / 32; ++j)
            tc_mma_i8_pair(tmem + uint32_t(buf) * kQ2Tile, ad0 + off + uint64_t(2 * j), bd0 + off + uint64_t(2 * j), kQ2Idesc,
                           (kb | j) ? 1u : 0u);
          tc_commit_pair(&sh->empty[s == 0 ? kQ2Stages - 1 : s - 1]);
        }
        if (ok) tc_commit_pair(&sh->acc_full[buf]);
      }
      if (!ok) {  // wait for the tensor-core work already issued before the TMEM is freed
        tc_commit_pair(&sh->drain);
        mbar_wait_bounded(&sh->drain, 0, p.err, 1u << 20);
      }
    }
  } else {
    // ------------------------------------------------ epilogue: a warp per TMEM lane quarter
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;  // which columns
    const uint32_t block_at = trans0 + uint32_t(warp - 2) * kQ2Block;
    const uint8_t* block = q2_smem + (block_at - smem_u32(q2_smem));
    const bool tma_store = (p.N & 7) == 0;
    const uint32_t empty0 = map_to_rank(smem_u32(&sh->acc_empty[0]), 0);
    pdl_wait();  // s_x, and y's earlier readers
    int n = 0;
    for (long long t = pair; t < tiles; t += pairs, ++n) {
      const int buf = n & 1;
      const int rt = int(t / TM), mt = int(t - (long long)rt * TM);
      const int n0 = rt * kQ2Tile, mb = mt * kQ2Tile + int(rank) * 128 + 32 * q, m = mb + lane;
      const float sx = m < p.M ? p.s_x[m] : 0.f;
      const int w_ok = lane == 0 ? int(q8_wait(&sh->acc_full[buf], uint32_t(n >> 1) & 1u, sh, p.err)) : 0;
      if (__shfl_sync(0xffffffffu, w_ok, 0) == 0) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t(32 * q) << 16) + uint32_t(buf) * kQ2Tile;
      if (mb < p.M) {
        // 64 outputs of a token at a time, as 32 words of two
        for (int c = 128 * half; c < 128 * half + 128 && n0 + c < p.N; c += 64) {
          uint32_t w[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(acc + uint32_t(c + 32 * h), v);
            const int nb = n0 + c + 32 * h;
            float4 sw[8];  // (rows past N, in the last tile only, are read as the last four that exist)
#pragma unroll
            for (int i = 0; i < 8; ++i) sw[i] = q2_scales(p.s_w, nb + 4 * i, p.N);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = __int2float_rn(int(v[4 * i])) * sw[i].x * sx, b = __int2float_rn(int(v[4 * i + 1])) * sw[i].y * sx;
              const float d = __int2float_rn(int(v[4 * i + 2])) * sw[i].z * sx, e = __int2float_rn(int(v[4 * i + 3])) * sw[i].w * sx;
              const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(d, e);
              w[16 * h + 2 * i] = *reinterpret_cast<const uint32_t*>(&x);
              w[16 * h + 2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
          // the warp's block: its last store must have been read
          if (tma_store && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(block_at + uint32_t(lane) * 128u +
                                                                       (uint32_t(i ^ (lane & 7)) << 4)),
                         "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                         : "memory");
          if (tma_store) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {  // (rows past M and outputs past N are not written)
              asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(&tmap_y),
                           "r"(block_at), "r"(n0 + c), "r"(mb)
                           : "memory");
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          } else {
            __syncwarp();
            q2_store_rows(p, block, mb, n0 + c, lane);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(empty0 + uint32_t(buf) * 8u);
    }
  }
  if (warp >= 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // y is written
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves, or frees its TMEM, while the other's loads, commits or MMAs name it
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

}  // namespace w4a8
