// RMS norm of query and key heads with the position rotation in one pass.
//
//   n[i] = x[i] * rsqrt(mean(x^2) + eps) * weight[i]        (a head of D values)
//   pair (a, b) of the first rot_dim values turns by t = position * inv_freq:
//     a' = (a cos t - b sin t) f,  b' = (b cos t + a sin t) f
//   pairs are (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1); f is the
//   attention factor of a frequency scaling; the rest of the head stays n.
//
// Sums and products are fp32 and the result is rounded once.  The angle is
// formed in fp64 as a number of turns, position * (inv_freq / 2 pi), and its
// whole turns are dropped there: in fp32 the angle of a position of 10^6
// would be off by 0.03 rad.  What is left (|t| <= 1/2 turn) goes to fp32.
//
// A head is held by D / 8 neighbouring lanes, 8 values (16 bytes) each, so
// a row's loads are whole 16-byte words, the norm is a few shuffles, and as
// rot_dim is a multiple of 16 a half-layout partner is a whole lane away.
#pragma once

#include "common.cuh"
#include "kv_index.h"

namespace w4a8 {

struct RopeParams {
  const double* inv_freq;  // [rot_dim / 2], or NULL: no rotation
  int rot_dim;
  int interleaved;
  float factor;
};

struct HeadRows {  // bf16 [token][head][D] with element strides
  uint16_t* data;
  long long token, head;
  int heads;
};

constexpr double kInvTwoPi = 0.15915494309189533577;

// cos and sin (times the factor) of pair i at a position.
__device__ __forceinline__ float2 rope_cs(const RopeParams& r, int pos, int i) {
  const double turns = double(pos) * (__ldg(r.inv_freq + i) * kInvTwoPi);
  const float t = float(turns - rint(turns));
  float s, c;
  sincospif(2.0f * t, &s, &c);
  return make_float2(c * r.factor, s * r.factor);
}

__device__ __forceinline__ void bf16x8_to_float(const uint4 raw, float (&v)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 float_to_bf16x8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The lane's 8 weights (ones without a weight).
template <int LPH>
__device__ __forceinline__ void head_weight(const float* weight, int sub, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (weight) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(weight) + 2 * sub);
    const float4 b = __ldg(reinterpret_cast<const float4*>(weight) + 2 * sub + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// Norm of a head held by LPH neighbouring lanes (8 values each); the whole
// warp takes part.
template <int LPH>
__device__ __forceinline__ void head_norm(float (&v)[8], const float (&w)[8], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
  for (int off = LPH / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float r = rsqrtf(ss * (1.0f / float(8 * LPH)) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
}

// The lane's cos/sin values: interleaved, pair 4 sub + i / 2 for value i;
// half layout, pair (8 sub + i) % (rot_dim / 2).  `cs(pair)` gives them.
template <int LPH, typename Cs>
__device__ __forceinline__ void head_rope(float (&v)[8], const RopeParams& r, int sub, Cs cs) {
  const int span = r.rot_dim >> 3;  // lanes that hold rotated values
  if (r.interleaved) {
    if (sub < span) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = cs(4 * sub + i);
        const float a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = a * t.x - b * t.y;
        v[2 * i + 1] = b * t.x + a * t.y;
      }
    }
  } else {
    const int half = span >> 1;
    const bool low = sub < half;
    const int lane = threadIdx.x & 31;
    const int src = sub < span ? (low ? lane + half : lane - half) : lane;
    const int p0 = low ? 8 * sub : 8 * (sub - half);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, v[i], src);
      if (sub < span) {
        const float2 t = cs(p0 + i);
        v[i] = low ? v[i] * t.x - o * t.y : v[i] * t.x + o * t.y;
      }
    }
  }
}

struct QkParams {
  HeadRows q, k;          // inputs (data NULL: none)
  HeadRows q_out, k_out;
  const float* q_weight;  // [D] or NULL (no norm)
  const float* k_weight;
  float eps;
  RopeParams rope;
  const int* positions;   // [tokens]
  int tokens;
};

constexpr int kQkThreads = 256;
constexpr int kQkMaxPairs = 128;  // rot_dim / 2 at most (heads of 256)

// One head row of the warp's current group: load, norm, rotate, store.
template <int D>
__device__ __forceinline__ void qk_head(const HeadRows& in, const HeadRows& out, const float* weight, float eps,
                                        const RopeParams& rope, const float2* cs, int token, int head, bool live) {
  constexpr int LPH = D / 8;
  const int sub = threadIdx.x & (LPH - 1);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live)
    bf16x8_to_float(__ldcg(reinterpret_cast<const uint4*>(in.data + token * in.token + head * in.head) + sub), v);
  if (weight) {
    float w[8];
    head_weight<LPH>(weight, sub, w);
    head_norm<LPH>(v, w, eps);
  }
  if (rope.inv_freq) head_rope<LPH>(v, rope, sub, [&](int i) { return cs[i]; });
  if (live)
    reinterpret_cast<uint4*>(out.data + token * out.token + head * out.head)[sub] = float_to_bf16x8(v);
}

// A CTA per token: its angles once, then every head of q and k.
template <int D>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkParams p) {
  __shared__ float2 cs[kQkMaxPairs];
  constexpr int LPH = D / 8, HPC = kQkThreads / LPH;  // heads per pass
  pdl_wait();
  pdl_launch_dependents();
  const int token = blockIdx.x;
  if (p.rope.inv_freq) {
    const int pos = p.positions[token];
    for (int i = threadIdx.x; i < p.rope.rot_dim / 2; i += kQkThreads) cs[i] = rope_cs(p.rope, pos, i);
    __syncthreads();
  }
  const int hq = p.q.data ? p.q.heads : 0, hk = p.k.data ? p.k.heads : 0;
  const int g = threadIdx.x / LPH;
  for (int h0 = 0; h0 < hq; h0 += HPC)
    qk_head<D>(p.q, p.q_out, p.q_weight, p.eps, p.rope, cs, token, h0 + g, h0 + g < hq);
  for (int h0 = 0; h0 < hk; h0 += HPC)
    qk_head<D>(p.k, p.k_out, p.k_weight, p.eps, p.rope, cs, token, h0 + g, h0 + g < hk);
}

}  // namespace w4a8
