// Row quantiser of the int8 layer: int8 codes and one fp32 scale per row.
//
//   v[r, k] = x[r, k], or the row rotated by H_256 / 16 per 256-block (act.cuh)
//   s[r]    = max_k |v[r, k]| / 127,  q = clamp(rint(v / s), -127, 127)
//
// Same arithmetic as the activation kernel (rotate_words_lane, quant_scale,
// quant_code), so a rotated bf16 row gets the codes and scale of
// w4a8_rotate_quant_act.  One CTA per row; the row is staged in shared
// memory in fp32 until its maximum is known, so it is read once.
#pragma once

#include <type_traits>

#include "act.cuh"
#include "common.cuh"

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

// Threads per row: few rows take as many threads as the row has groups of 8
// (latency counts), many rows 256 (more rows share an SM).
__host__ __device__ inline int q8_threads(int64_t rows, int64_t K) {
  if (rows > 296) return 256;
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
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (lane == 0) warp_max[warp] = amax;
  __syncthreads();
  amax = warp_max[0];
  for (int i = 1; i < nwarps; ++i) amax = fmaxf(amax, warp_max[i]);
  const float s = quant_scale(amax);
  const QuantScale qs = quant_prepare(s);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
  auto quantise = [&](auto fast) {
    for (int k0 = warp * 256; k0 < K; k0 += nwarps * 256) {  // the values this thread staged
      const int k = k0 + lane * 8;
      if (k >= K) break;
      const float4 a = *reinterpret_cast<const float4*>(q8_row + k);
      const float4 b = *reinterpret_cast<const float4*>(q8_row + k + 4);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo |= (uint32_t(int(quant_code<decltype(fast)::value>(v[i], qs))) & 0xFFu) << (8 * i);
        hi |= (uint32_t(int(quant_code<decltype(fast)::value>(v[i + 4], qs))) & 0xFFu) << (8 * i);
      }
      *reinterpret_cast<uint2*>(codes + base + k) = make_uint2(lo, hi);
    }
  };
  if (qs.fast)
    quantise(std::true_type{});
  else
    quantise(std::false_type{});
}

}  // namespace w4a8
