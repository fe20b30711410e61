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
// would be off by 0.03 rad.  What is left (|t| <= 1/2 turn) goes to fp32 and
// to the hardware's sine and cosine (2^-21 off at most, against the 2^-9 of
// the bf16 result or the 2^-8 of an int8 code).
//
// A head is held by D / 8 neighbouring lanes, 8 values (16 bytes) each, so
// a row's loads are whole 16-byte words, the norm is a few shuffles, and as
// rot_dim is a multiple of 16 a half-layout partner is a whole lane away.  A
// lane's angles and weights are the same for every head of a token and stay
// in registers; a warp walks a token's heads with nothing shared and no
// barrier.  The kernel's instructions (about 75 a lane and head) and its
// bytes then take about the same time.
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
  const float t = float(turns - rint(turns)) * 6.28318530717958647692f;
  return make_float2(__cosf(t) * r.factor, __sinf(t) * r.factor);
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

// The lane's cosines and sines at a position: interleaved, pair 4 sub + i / 2
// for value i (the first four); half layout, pair (8 sub + i) % (rot_dim / 2).
__device__ __forceinline__ void lane_angles(const RopeParams& r, int sub, int pos, float2 (&cs)[8]) {
  const int span = r.rot_dim >> 3, half = span >> 1;
  if (sub < span) {
    if (r.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) cs[i] = rope_cs(r, pos, 4 * sub + i);
    } else {
      const int p0 = 8 * (sub < half ? sub : sub - half);
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = rope_cs(r, pos, p0 + i);
    }
  }
}

// Rotation of a head's values; the whole warp takes part.
__device__ __forceinline__ void head_rope(float (&v)[8], const RopeParams& r, int sub, const float2 (&cs)[8]) {
  const int span = r.rot_dim >> 3;  // lanes that hold rotated values
  if (r.interleaved) {
    if (sub < span) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = a * cs[i].x - b * cs[i].y;
        v[2 * i + 1] = b * cs[i].x + a * cs[i].y;
      }
    }
  } else {
    const int half = span >> 1, lane = threadIdx.x & 31;
    const bool low = sub < half;
    const int src = sub < span ? (low ? lane + half : lane - half) : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, v[i], src);
      if (sub < span) v[i] = v[i] * cs[i].x + (low ? -o : o) * cs[i].y;
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

// Heads [h0, h1) of one token's rows, by a warp.
template <int D>
__device__ __forceinline__ void qk_rows(const HeadRows& in, const HeadRows& out, const float* weight, float eps,
                                        const RopeParams& rope, const float2 (&cs)[8], int token, int h0, int h1) {
  constexpr int LPH = D / 8, HPW = 32 / LPH;  // heads of a warp at a time
  const int lane = threadIdx.x & 31, sub = lane & (LPH - 1), g = lane / LPH;
  float w[8];
  head_weight<LPH>(weight, sub, w);
  const uint16_t* src = in.data + token * in.token + 8 * sub;
  uint16_t* dst = out.data + token * out.token + 8 * sub;
  auto load = [&](int h) {
    return h + g < h1 ? __ldcg(reinterpret_cast<const uint4*>(src + (h + g) * in.head)) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 raw = load(h0), next = load(h0 + HPW);
  for (int h = h0; h < h1; h += HPW) {
    float v[8];
    bf16x8_to_float(raw, v);
    raw = next;
    next = load(h + 2 * HPW);
    if (weight) head_norm<LPH>(v, w, eps);
    if (rope.inv_freq) head_rope(v, rope, sub, cs);
    if (h + g < h1) *reinterpret_cast<uint4*>(dst + (h + g) * out.head) = float_to_bf16x8(v);
  }
}

// How many warps share a token's heads: enough to fill the SMs where tokens
// are few, one where there are many (its angles are then formed once).
__host__ __device__ inline int qk_parts(int64_t tokens, int heads, int D) {
  const int64_t most = (heads + 256 / D - 1) / (256 / D), fill = (148 * 16 + tokens - 1) / tokens;
  return int(fill < most ? fill : most);
}

// Part `part` of `parts` of a token's heads, q's then k's, in steps of a warp's heads.
template <int D>
__device__ __forceinline__ void qk_token(const QkParams& p, int token, int pos, int part, int parts) {
  constexpr int HPW = 256 / D;
  float2 cs[8];
  if (p.rope.inv_freq) lane_angles(p.rope, threadIdx.x & (D / 8 - 1), pos, cs);
  const int sq = p.q.data ? (p.q.heads + HPW - 1) / HPW : 0, sk = p.k.data ? (p.k.heads + HPW - 1) / HPW : 0;
  const int s0 = (sq + sk) * part / parts, s1 = (sq + sk) * (part + 1) / parts;
  if (s0 < sq)
    qk_rows<D>(p.q, p.q_out, p.q_weight, p.eps, p.rope, cs, token, s0 * HPW, min(p.q.heads, min(s1, sq) * HPW));
  if (s1 > sq)
    qk_rows<D>(p.k, p.k_out, p.k_weight, p.eps, p.rope, cs, token, max(s0 - sq, 0) * HPW, min(p.k.heads, (s1 - sq) * HPW));
}

template <int D>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkParams p, int parts) {
  pdl_wait();
  pdl_launch_dependents();
  const long long unit = ((long long)blockIdx.x * kQkThreads + threadIdx.x) >> 5;
  const int token = int(unit / parts), part = int(unit - (long long)token * parts);
  if (token >= p.tokens) return;
  qk_token<D>(p, token, p.rope.inv_freq ? __ldg(p.positions + token) : 0, part, parts);
}

}  // namespace w4a8
