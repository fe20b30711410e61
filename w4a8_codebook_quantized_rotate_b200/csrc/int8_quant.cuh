// Row quantiser of the int8 layer: int8 codes and one fp32 scale per row.
//
//   v[r, k] = x[r, k], or the row rotated by H_256 / 16 per 256-block (act.cuh)
//   s[r]    = max_k |v[r, k]| / 127,  q = clamp(rint(v / s), -127, 127)
//
// Same arithmetic as the activation kernel (rotate_words_lane, quant_scale,
// quant_code), so a rotated bf16 row gets the codes and scale of
// w4a8_rotate_quant_act.  One CTA per row, read once: its values wait in
// registers or, in fp32, in shared memory until the row's maximum is known.
// Few rows take as many threads as a row has groups of 8 (latency counts);
// many rows the second kernel below.
#pragma once

#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "qk_rope.cuh"

namespace w4a8 {

template <bool F32>
__device__ __forceinline__ void q8_load8(const void* x, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 raw = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// Codes of four values in a word: clamp(rint(v / s)) as in quant_code, rounded by adding 1.5 * 2^23, whose last byte
// is then the code (exact, and half to even, for what the clamp lets through; the rounding and conversion
// instructions run at a quarter of the rate).
template <bool FAST>
__device__ __forceinline__ uint32_t q8_code4(const float (&v)[4], const QuantScale& q) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x;
    if constexpr (FAST) {
      const float q0 = v[i] * q.r;
      x = fmaf(fmaf(-q0, q.s, v[i]), q.r, q0);
    } else {
      x = q.s > 0.f ? __fdiv_rn(v[i], q.s) : 0.f;
    }
    w[i] = __float_as_uint(fminf(fmaxf(x, -127.f), 127.f) + 12582912.f);
  }
  return prmt(prmt(w[0], w[1], 0x0040u), prmt(w[2], w[3], 0x0040u), 0x5410u);
}

__device__ __forceinline__ float q8_row_max(float amax, float* warp_max) {
  const int lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (lane == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = warp_max[0];
  for (int i = 1; i < nwarps; ++i) amax = fmaxf(amax, warp_max[i]);
  return amax;
}

constexpr int64_t kQ8FewRows = 296;  // two CTAs an SM
__host__ __device__ inline int q8_threads(int64_t K) {
  const int64_t t = (K / 8 + 31) / 32 * 32;
  return int(t < 64 ? 64 : t > 1024 ? 1024 : t);
}

// `early`: the next kernel may launch now, if it waits for this one before it
// reads the codes.  The layer's product does so for activations; weights it
// fetches before that wait, so a call of the quantiser alone is not early.
template <bool F32>
__global__ void __launch_bounds__(1024) int8_quant_kernel(const void* __restrict__ x, int K, int rotate, bool early,
                                                          int8_t* __restrict__ codes, float* __restrict__ scale) {
  extern __shared__ __align__(16) float q8_row[];  // [K]
  __shared__ float warp_max[32];
  if (early) pdl_launch_dependents();
  pdl_wait();
  const int64_t base = int64_t(blockIdx.x) * K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  float amax = 0.f;
  // A warp takes 256 consecutive values at a time (a rotation block when
  // rotating; K is then a multiple of 256 and every lane is live).
  for (int k0 = warp * 256; k0 < K; k0 += nwarps * 256) {
    const int k = k0 + lane * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (k < K) q8_load8<F32>(x, base + k, v);
    if (rotate) rotate_vals_lane(v, lane);
    if (k < K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
      float4* dst = reinterpret_cast<float4*>(q8_row + k);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  const float s = quant_scale(q8_row_max(amax, warp_max));
  const QuantScale qs = quant_prepare(s);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
  auto quantise = [&](auto fast) {
    for (int k0 = warp * 256; k0 < K; k0 += nwarps * 256) {  // the values this thread staged
      const int k = k0 + lane * 8;
      if (k >= K) break;
      const float4 a = *reinterpret_cast<const float4*>(q8_row + k);
      const float4 b = *reinterpret_cast<const float4*>(q8_row + k + 4);
      const float v[4] = {a.x, a.y, a.z, a.w}, w[4] = {b.x, b.y, b.z, b.w};
      *reinterpret_cast<uint2*>(codes + base + k) =
          make_uint2(q8_code4<decltype(fast)::value>(v, qs), q8_code4<decltype(fast)::value>(w, qs));
    }
  };
  if (qs.fast)
    quantise(std::true_type{});
  else
    quantise(std::false_type{});
}

// Many rows: a lane holds 32 values of a 256-block, four groups of 8 that
// are 64 apart (so that 8 lanes' loads are 128 consecutive bytes), which
// leaves three of the rotation's eight stages to exchanges between lanes
// instead of five, and its sums go two to an instruction.  A warp takes 1024
// values at a time; the last round's stay in registers.  4096 rotated rows of
// 5120 take 20.4 us (25 with the kernel above and 256 threads a row), 14.4
// without the rotation, against 9.6 for the bytes: what is left is the
// instructions, about nine a value, and the barrier before the second half.
struct Q8Wide {
  int warps, rounds;
};
__host__ __device__ inline Q8Wide q8_wide(int64_t K) {
  const int units = int((K + 1023) / 1024), rounds = (units + 7) / 8;
  return Q8Wide{(units + rounds - 1) / rounds, rounds};
}

__device__ __forceinline__ uint64_t q8_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The stages of bits 0 .. 7 in that order, as in rotate_vals_lane: v[4 c + i] holds values 64 c + 8 (lane % 8) + 2 i
// and the next.
__device__ __forceinline__ void q8_rotate_wide(uint64_t (&v)[16], int lane) {
  const uint64_t neg = pack2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = unpack2(v[i]);
    v[i] = pack2(x.x + x.y, x.x - x.y);
  }
  auto stage = [&](int step) {  // pairs `step` apart
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & step)) {
        const uint64_t a = v[i], b = v[i + step];
        v[i] = q8_add2(a, b);
        v[i + step] = fma2(b, neg, a);
      }
  };
  stage(1);
  stage(2);
#pragma unroll
  for (int bit = 1; bit < 8; bit <<= 1) {
    const float sign = (lane & bit) ? -1.f : 1.f;
    const uint64_t sign2 = pack2(sign, sign);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = unpack2(v[i]);
      v[i] = fma2(v[i], sign2, pack2(__shfl_xor_sync(0xffffffffu, x.x, bit), __shfl_xor_sync(0xffffffffu, x.y, bit)));
    }
  }
  stage(4);
  stage(8);
  const uint64_t sixteenth = pack2(0.0625f, 0.0625f);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], sixteenth);
}

template <bool F32>
__global__ void __launch_bounds__(256, 3)
    int8_quant_wide_kernel(const void* __restrict__ x, int K, int rotate, bool early, int8_t* __restrict__ codes,
                           float* __restrict__ scale, int rounds) {
  extern __shared__ __align__(16) float4 q8_staged[];  // [round][warp][8][lane], all rounds but the last
  __shared__ float warp_max[8];
  if (early) pdl_launch_dependents();
  pdl_wait();
  const int64_t base = int64_t(blockIdx.x) * K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  auto first = [&](int r) { return (r * nwarps + warp) * 1024 + (lane >> 3) * 256 + (lane & 7) * 8; };
  auto staged = [&](int r) { return q8_staged + (r * nwarps + warp) * 256 + lane; };
  float amax = 0.f;
  uint64_t v[16];
  for (int r = 0; r < rounds; ++r) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = first(r) + 64 * c;
      float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (k < K) q8_load8<F32>(x, base + k, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * c + i] = pack2(u[2 * i], u[2 * i + 1]);
    }
    if (rotate) q8_rotate_wide(v, lane);  // (blocks past K are zeros)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 u = unpack2(v[i]);
      amax = fmaxf(amax, fmaxf(fabsf(u.x), fabsf(u.y)));
    }
    if (r + 1 < rounds) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 a = unpack2(v[2 * i]), b = unpack2(v[2 * i + 1]);
        staged(r)[32 * i] = make_float4(a.x, a.y, b.x, b.y);
      }
    }
  }
  const float s = quant_scale(q8_row_max(amax, warp_max));
  const QuantScale qs = quant_prepare(s);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
  auto quantise = [&](auto fast) {
    for (int r = rounds - 1; r >= 0; --r) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 a = unpack2(v[4 * c + 2 * h]), b = unpack2(v[4 * c + 2 * h + 1]);
          const float u[4] = {a.x, a.y, b.x, b.y};
          w[h] = q8_code4<decltype(fast)::value>(u, qs);
        }
        const int k = first(r) + 64 * c;
        if (k < K) *reinterpret_cast<uint2*>(codes + base + k) = make_uint2(w[0], w[1]);
      }
      if (r > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 u = staged(r - 1)[32 * i];
          v[2 * i] = pack2(u.x, u.y);
          v[2 * i + 1] = pack2(u.z, u.w);
        }
      }
    }
  };
  if (qs.fast)
    quantise(std::true_type{});
  else
    quantise(std::false_type{});
}

}  // namespace w4a8
