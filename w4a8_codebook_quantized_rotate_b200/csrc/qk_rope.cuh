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
// bytes then take about the same time: 8197 tokens of 32/8 heads of 128, 168
// MB, in 32.3 us (5.2 TB/s); 16 tokens of 24/4 heads of 256 in 2.6.  Four CTAs
// an SM cap the registers at 64; 36 to 56 bytes a thread spill.
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

// Two fp32 values as one operand of the packed fp32 instructions (each half
// rounded like the scalar one; half the issue slots, which bound these kernels).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t d) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(d));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

struct Head8 {  // a lane's 8 values of a head, neighbouring values paired
  uint64_t p[4];
};
__device__ __forceinline__ Head8 head_unpack(const uint4 raw) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  Head8 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h.p[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return h;
}
__device__ __forceinline__ uint4 head_pack(const Head8& h) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(h.p[i]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void head_values(const Head8& h, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2(h.p[i]);
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
}

// The lane's 8 weights (ones without a weight).
__device__ __forceinline__ Head8 head_weight(const float* weight, int sub) {
  Head8 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w.p[i] = pack2(1.f, 1.f);
  if (weight) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(weight) + 2 * sub);
    const float4 b = __ldg(reinterpret_cast<const float4*>(weight) + 2 * sub + 1);
    w.p[0] = pack2(a.x, a.y), w.p[1] = pack2(a.z, a.w), w.p[2] = pack2(b.x, b.y), w.p[3] = pack2(b.z, b.w);
  }
  return w;
}

// Norm of a head held by LPH neighbouring lanes (8 values each); the whole
// warp takes part.
template <int LPH>
__device__ __forceinline__ void head_norm(Head8& h, const Head8& w, float eps) {
  uint64_t sq = mul2(h.p[0], h.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) sq = fma2(h.p[i], h.p[i], sq);
  const float2 s2 = unpack2(sq);
  float ss = s2.x + s2.y;
#pragma unroll
  for (int off = LPH / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float r = rsqrtf(ss * (1.0f / float(8 * LPH)) + eps);
  const uint64_t r2 = pack2(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) h.p[i] = mul2(mul2(h.p[i], r2), w.p[i]);
}

// The lane's cosines and (signed) sines at a position, so that a value turns
// to v * c + (its partner) * s: half layout, pair (8 sub + i) % (rot_dim / 2)
// for value i, the sine negative in the first half; interleaved, pair 4 sub +
// i / 2, negative for the even value.  Lanes past the rotated part hold 1, 0.
// The lanes of a head form M angles each and hand them round (where a quarter
// of a head turns, its few lanes would form eight each while the others wait).
struct Turn8 {
  uint64_t c[4], s[4];
  int src;  // half layout: the lane that holds the partners
};
template <int LPH, int M>
__device__ __forceinline__ Turn8 head_turn_by(const RopeParams& r, int sub, int pos) {
  const int span = r.rot_dim >> 3, half = span >> 1, lane = threadIdx.x & 31, group = lane & ~(LPH - 1);
  const bool low = sub < half, in = sub < span;
  float2 mine[M];
#pragma unroll
  for (int i = 0; i < M; ++i)
    mine[i] = 2 * (sub * M + i) < r.rot_dim ? rope_cs(r, pos, sub * M + i) : make_float2(1.f, 0.f);
  const int p0 = !in ? 0 : r.interleaved ? 4 * sub : 8 * (low ? sub : sub - half);  // the lane's first pair
  auto pair = [&](int i) {  // p0 is a multiple of 4, so pair p0 + i is number i % M of its lane
    const int from = group + (p0 + i) / M;
    return make_float2(__shfl_sync(0xffffffffu, mine[i % M].x, from), __shfl_sync(0xffffffffu, mine[i % M].y, from));
  };
  Turn8 t;
  t.src = in && !r.interleaved ? (low ? lane + half : lane - half) : lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 a, b;
    if (r.interleaved) {
      a = b = pair(i);
      a.y = -a.y;
    } else {
      a = pair(2 * i);
      b = pair(2 * i + 1);
      if (low) a.y = -a.y, b.y = -b.y;
    }
    t.c[i] = in ? pack2(a.x, b.x) : pack2(1.f, 1.f);
    t.s[i] = in ? pack2(a.y, b.y) : pack2(0.f, 0.f);
  }
  return t;
}
template <int LPH>
__device__ __forceinline__ Turn8 head_turn(const RopeParams& r, int sub, int pos) {
  if (r.rot_dim <= 2 * LPH) return head_turn_by<LPH, 1>(r, sub, pos);
  if (r.rot_dim <= 4 * LPH) return head_turn_by<LPH, 2>(r, sub, pos);
  return head_turn_by<LPH, 4>(r, sub, pos);
}

// Rotation of a head's values; the whole warp takes part.
__device__ __forceinline__ void head_rope(Head8& h, int interleaved, const Turn8& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(h.p[i]);
    const uint64_t o = interleaved ? pack2(v.y, v.x)
                                   : pack2(__shfl_sync(0xffffffffu, v.x, t.src), __shfl_sync(0xffffffffu, v.y, t.src));
    h.p[i] = fma2(o, t.s[i], mul2(h.p[i], t.c[i]));
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
constexpr int kQkAhead = 4;  // head rows of a lane group in flight

// Heads [h0, h1) of one token's rows, by a warp.
template <int D>
__device__ __forceinline__ void qk_rows(const HeadRows& in, const HeadRows& out, const float* weight, float eps,
                                        const RopeParams& rope, const Turn8& turn, int token, int h0, int h1) {
  constexpr int LPH = D / 8, HPW = 32 / LPH;  // heads of a warp at a time
  const int lane = threadIdx.x & 31, sub = lane & (LPH - 1), g = lane / LPH;
  const Head8 w = head_weight(weight, sub);
  const uint16_t* src = in.data + token * in.token + (h0 + g) * in.head + 8 * sub;
  uint16_t* dst = out.data + token * out.token + (h0 + g) * out.head + 8 * sub;
  const long long step_in = HPW * in.head, step_out = HPW * out.head;
  int left = h1 - h0 - g;  // heads of this lane group, HPW apart
  for (; left + g > 0; left -= kQkAhead * HPW) {  // (left + g is the same for all lanes: the shuffles below)
    uint4 raw[kQkAhead];
#pragma unroll
    for (int a = 0; a < kQkAhead; ++a)
      raw[a] = left > a * HPW ? __ldcg(reinterpret_cast<const uint4*>(src + a * step_in)) : make_uint4(0u, 0u, 0u, 0u);
    src += kQkAhead * step_in;
#pragma unroll
    for (int a = 0; a < kQkAhead; ++a) {
      if (left + g <= a * HPW) break;
      Head8 v = head_unpack(raw[a]);
      if (weight) head_norm<LPH>(v, w, eps);
      if (rope.inv_freq) head_rope(v, rope.interleaved, turn);
      if (left > a * HPW) *reinterpret_cast<uint4*>(dst) = head_pack(v);
      dst += step_out;
    }
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
  Turn8 turn{};
  if (p.rope.inv_freq) turn = head_turn<D / 8>(p.rope, threadIdx.x & (D / 8 - 1), pos);
  const int sq = p.q.data ? (p.q.heads + HPW - 1) / HPW : 0, sk = p.k.data ? (p.k.heads + HPW - 1) / HPW : 0;
  const int s0 = (sq + sk) * part / parts, s1 = (sq + sk) * (part + 1) / parts;
  if (s0 < sq)
    qk_rows<D>(p.q, p.q_out, p.q_weight, p.eps, p.rope, turn, token, s0 * HPW, min(p.q.heads, min(s1, sq) * HPW));
  if (s1 > sq)
    qk_rows<D>(p.k, p.k_out, p.k_weight, p.eps, p.rope, turn, token, max(s0 - sq, 0) * HPW, min(p.k.heads, (s1 - sq) * HPW));
}

template <int D>
__global__ void __launch_bounds__(kQkThreads, 4) qk_norm_rope_kernel(const QkParams p, int parts) {
  pdl_launch_dependents();  // (the next kernel waits for this one, and this one for the last)
  pdl_wait();
  const long long unit = ((long long)blockIdx.x * kQkThreads + threadIdx.x) >> 5;
  const int token = int(unit / parts), part = int(unit - (long long)token * parts);
  if (token >= p.tokens) return;
  qk_token<D>(p, token, p.rope.inv_freq ? __ldg(p.positions + token) : 0, part, parts);
}

}  // namespace w4a8
