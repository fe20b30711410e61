// C ABI of the 8-bit integer path (include/w4a8_int8.h): argument checks and
// launches.  Part of the library's single translation unit (w4a8_api.cu),
// whose per-device state and launch helpers it uses.
#pragma once

#include <cmath>

namespace w4a8 {
namespace {

w4a8_status status_of(cudaError_t e) { return e == cudaSuccess ? W4A8_OK : W4A8_ERR_CUDA; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// ------------------------------------------------------------------ int8 layer

bool q8_rows_ok(int64_t R) { return R > 0 && R <= (int64_t(1) << 24); }
bool q8_k_ok(int64_t K, int rotate) { return K > 0 && K % 16 == 0 && K <= kMaxK && (!rotate || K % kRotBlock == 0); }
bool q8_shape_ok(int64_t M, int64_t N, int64_t K, int rotate) {
  return M > 0 && M <= kMaxTokens && q8_rows_ok(N) && q8_k_ok(K, rotate);
}

// Kernel, token tile, k split and CTAs per SM of a product: the choice with
// the least estimated time (in clocks).  A CTA takes its k blocks at the
// slowest of its loads, the latency of a pipeline that its stages do not
// cover, and its MMAs; then an epilogue, or the joining of a split tile; the
// rounds of CTAs that fit at once add up, and memory bounds it all.  The
// constants are fitted to measured times: up to 128 tokens to the times and
// choices of 48 shapes (K 64 to 17408, N 16 to 17408; the choice is 2.2 %
// slower than the best measured one on average), beyond to 1250 times of 120 shapes of up
// to 8192 tokens (3 to 4 %).  For example 1 token, K = 17408, N = 5120: split
// 1 / 4 / 6 took 38.6 / 17.3 / 16.3 us; 727 tokens, K = 512, N = 91: tiles of 16 /
// 256 tokens 4.1 / 19.7 us; 4096 tokens, K = 5120, N = 17408: pairs 236 us, tiles
// of 128 / 256 tokens 386 / 367.
struct Q8Plan {
  int nt, cps, split;
  bool pair;  // int8_pair_kernel (the rest is then unused)
};
struct Q8Model {
  double rate, latency, epi, epi_nt, odd, join, join_nt, join_share, mma, start, memory, write;
};
constexpr Q8Model kQ8Few = {43.9, 3000, 2299, 18, 1, 2543, 8.7, 140, 1.41, 2001, 3105, 1e9};
constexpr Q8Model kQ8Many = {47.7, 2594, 413, 33.3, 2.46, 2918, 11.3, 160, 1.18, 3030, 2239, 691};

// Clusters of 1 .. 8 CTAs that fit at one CTA per SM (the GPU's answer,
// cudaOccupancyMaxActiveClusters; a cluster stays inside one of its
// processing clusters).
constexpr int kQ8Clusters[kQ8MaxSplit + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15};

Q8Plan q8_plan(int64_t M, int64_t K, int64_t N) {
  const int64_t kb = (K + kQ8BK - 1) / kQ8BK, rows = (N + kQ8Rows - 1) / kQ8Rows;
  const bool few = M <= 128;
  const Q8Model& c = few ? kQ8Few : kQ8Many;
  const double weights = double(N) * K + double(M) * K;
  Q8Plan best{};
  double least = 1e300;
  for (const int nt : {16, 32, 64, 128, 256}) {
    const int64_t tokens = (M + nt - 1) / nt;
    if ((nt > 16 && nt >= 2 * M) || tokens > 65535) continue;
    for (int split = 1; split <= kQ8MaxSplit && split <= kb; ++split) {
      const double ctas = double(rows * tokens) * split, fit = kQ8Clusters[split] * split;
      const int cps = nt <= 128 && ctas > fit ? 2 : 1;
      const double slots = fit * cps, rounds = ctas > slots ? std::ceil(ctas / slots) : 1.0;
      const double share = std::max(1.0, std::min(ctas, slots) / fit);
      const double stage = double(kQ8Rows + nt) * kQ8BK;
      const double stages = std::min(12.0, std::floor(((cps == 1 ? 232448 : 115712) - 2048) / stage));
      const double step = std::max({stage / c.rate * share, c.latency / stages, c.mma * nt * share});
      const double epilogue = split == 1 ? (c.epi + c.epi_nt * nt) * (N % 8 ? c.odd : 1.0)
                                         : c.join + c.join_nt * nt + c.join_share * nt / split;
      const double busy = rounds * (double((kb + split - 1) / split) * step + epilogue * share);
      // (a tenth of the CTAs' time, so that choices that memory bounds alike are told apart)
      const double t = std::max(busy, weights / c.memory + double(M) * N * 2 / c.write) + 0.1 * busy * few + c.start;
      if (t < least) {
        least = t;
        best = Q8Plan{nt, cps, split, false};
      }
    }
  }
  if (!few) {
    // pairs: rounds of 74 tiles at the slower of the MMAs (with their loads) and the epilogue
    const double tiles = double((N + kQ2Tile - 1) / kQ2Tile) * double((M + kQ2Tile - 1) / kQ2Tile);
    const double epilogue = N % 8 == 0 ? 6113 : N % 2 == 0 ? 11616 : 15989;
    const double t = std::max(std::ceil(tiles / 74) * std::max(kb * 740.0, epilogue) + epilogue / 2 + 5760, weights / 2080) + 1550;
    best.pair = t < least;
  }
  return best;
}

// Workspace of the layer: the quantised activations.
struct Q8Ws {
  size_t off_s, total;
};
Q8Ws q8_ws(int64_t M, int64_t K) {
  Q8Ws w;
  w.off_s = round_up(size_t(M) * K, 256);
  w.total = w.off_s + round_up(size_t(M) * 4, 256);
  return w;
}

cudaError_t q8_quantize(const void* x, int f32, int64_t R, int64_t K, int rotate, bool early, int8_t* codes, float* s,
                        cudaStream_t st) {
  const dim3 grid{unsigned(R)};
  if (R > kQ8FewRows) {
    const Q8Wide w = q8_wide(K);
    const dim3 block{unsigned(32 * w.warps)};
    const size_t smem = size_t(w.rounds - 1) * w.warps * 4096;
    return f32 ? launch_pdl(int8_quant_wide_kernel<true>, grid, block, smem, st, x, int(K), int(rotate), early, codes, s, w.rounds)
               : launch_pdl(int8_quant_wide_kernel<false>, grid, block, smem, st, x, int(K), int(rotate), early, codes, s, w.rounds);
  }
  const dim3 block{unsigned(q8_threads(K))};
  return f32 ? launch_pdl(int8_quant_kernel<true>, grid, block, size_t(K) * 4, st, x, int(K), int(rotate), early, codes, s)
             : launch_pdl(int8_quant_kernel<false>, grid, block, size_t(K) * 4, st, x, int(K), int(rotate), early, codes, s);
}

// 2-D map of rows of bytes, box [box_cols x box_rows].
bool byte_map(CUtensorMap* m, const void* data, int64_t cols, int64_t rows, uint32_t box_cols, uint32_t box_rows,
              CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dim[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  const cuuint64_t stride[1] = {cuuint64_t(cols)};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t step[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(data), dim, stride, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, int CPS>
cudaError_t q8_launch(const CUtensorMap& tw, const CUtensorMap& tx, const Q8Params& p, int split, cudaStream_t st) {
  const dim3 grid(unsigned((p.N + kQ8Rows - 1) / kQ8Rows * split), unsigned((p.M + NT - 1) / NT));
  return launch_pdl_cluster(int8_gemm_kernel<NT, CPS>, grid, dim3(kQ8Threads), unsigned(split), Q8Cfg<NT, CPS>::kSmem, st,
                            tw, tx, p);
}

w4a8_status q8_gemm(const int8_t* x_q, const float* s_x, int64_t M, const int8_t* w_q, const float* s_w, int64_t N,
                    int64_t K, uint16_t* y, const DeviceState* d, cudaStream_t st) {
  const Q8Plan P = q8_plan(M, K, N);
  const int nt = P.pair ? 128 : P.nt;  // token rows of a load
  CUtensorMap tw, tx;
  if (!byte_map(&tw, w_q, K, N, kQ8BK, kQ8Rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !byte_map(&tx, x_q, K, M, kQ8BK, uint32_t(nt), CU_TENSOR_MAP_SWIZZLE_128B))
    return W4A8_ERR_CUDA;
  Q8Params p;
  p.s_x = s_x;
  p.s_w = s_w;
  p.y = y;
  p.err = d->err;
  p.M = int(M);
  p.N = int(N);
  p.KB = int((K + kQ8BK - 1) / kQ8BK);
  if (P.pair) {
    const int64_t tiles = ((N + kQ2Tile - 1) / kQ2Tile) * ((M + kQ2Tile - 1) / kQ2Tile);
    const unsigned ctas = unsigned(2 * std::min<int64_t>(tiles, d->sms / 2));
    CUtensorMap ty = tx;  // (used where the rows of y are 16-byte aligned)
    if (N % 8 == 0) {
      EncodeTiledFn enc = encode_fn();
      const cuuint64_t dim[2] = {cuuint64_t(N), cuuint64_t(M)}, stride[1] = {cuuint64_t(N) * 2};
      const cuuint32_t box[2] = {64, 32}, step[2] = {1, 1};
      if (enc(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, y, dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
          CUDA_SUCCESS)
        return W4A8_ERR_CUDA;
    }
    return status_of(launch_pdl_cluster(int8_pair_kernel, dim3(ctas), dim3(kQ2Threads), 2u, kQ2Smem, st, tw, tx, ty, p));
  }
  cudaError_t e;
  switch (P.nt * 2 + P.cps - 1) {
    case 32: e = q8_launch<16, 1>(tw, tx, p, P.split, st); break;
    case 33: e = q8_launch<16, 2>(tw, tx, p, P.split, st); break;
    case 64: e = q8_launch<32, 1>(tw, tx, p, P.split, st); break;
    case 65: e = q8_launch<32, 2>(tw, tx, p, P.split, st); break;
    case 128: e = q8_launch<64, 1>(tw, tx, p, P.split, st); break;
    case 129: e = q8_launch<64, 2>(tw, tx, p, P.split, st); break;
    case 256: e = q8_launch<128, 1>(tw, tx, p, P.split, st); break;
    case 257: e = q8_launch<128, 2>(tw, tx, p, P.split, st); break;
    default: e = q8_launch<256, 1>(tw, tx, p, P.split, st); break;
  }
  return e == cudaSuccess ? W4A8_OK : W4A8_ERR_CUDA;
}

// ------------------------------------------------------------------ heads and cache

bool head_dim_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

w4a8_status heads_ok(const w4a8_heads& h, int64_t D) {
  if (h.heads < 1 || h.heads > 65536) return W4A8_ERR_SHAPE;
  if (h.token_stride < 0 || h.head_stride < 0 || h.token_stride % 8 || h.head_stride % 8 || h.token_stride > (int64_t(1) << 40) ||
      h.head_stride > (int64_t(1) << 40) || (h.heads > 1 && h.head_stride < D))
    return W4A8_ERR_SHAPE;
  return aligned16(h.data) ? W4A8_OK : W4A8_ERR_ALIGN;
}
// Rows of tokens that are written must not share memory.
w4a8_status heads_out_ok(const w4a8_heads& h, int64_t tokens, int64_t D) {
  if (w4a8_status st = heads_ok(h, D); st != W4A8_OK) return st;
  const int64_t token = (h.heads - 1) * (h.heads > 1 ? h.head_stride : 0) + D;  // values from a token's first to its last
  const int64_t head = (tokens - 1) * h.token_stride + D;                       // and of a head over the tokens
  const bool apart = tokens == 1 || h.token_stride >= token || (h.token_stride >= D && (h.heads == 1 || h.head_stride >= head));
  return apart ? W4A8_OK : W4A8_ERR_SHAPE;
}
// An output that starts where its input does must be that input, row for row: under other strides rows would be written
// that other threads have yet to read.
bool heads_in_place_ok(const w4a8_heads& in, const w4a8_heads& out, int64_t tokens) {
  return in.data != out.data || ((tokens == 1 || in.token_stride == out.token_stride) &&
                                 (in.heads == 1 || in.head_stride == out.head_stride));
}
HeadRows head_rows(const w4a8_heads* h) {
  if (!h || !h->data) return HeadRows{nullptr, 0, 0, 0};
  return HeadRows{h->data, h->token_stride, h->head_stride, h->heads};
}

w4a8_status rope_ok(const w4a8_rope* r, int64_t D) {
  if (!r || !r->inv_freq) return W4A8_OK;
  if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > D) return W4A8_ERR_SHAPE;
  return (reinterpret_cast<uintptr_t>(r->inv_freq) & 7u) ? W4A8_ERR_ALIGN : W4A8_OK;
}
RopeParams rope_params(const w4a8_rope* r) {
  if (!r || !r->inv_freq) return RopeParams{nullptr, 0, 0, 1.f};
  return RopeParams{r->inv_freq, r->rot_dim, r->interleaved != 0, r->factor};
}

int page_shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

w4a8_status cache_ok(const w4a8_kv_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return W4A8_ERR_NULL;
  if (!head_dim_ok(c->head_dim) || page_shift_of(c->page) < 0 || c->kv_heads < 1 || c->kv_heads > 65536 || c->pages < 1 ||
      c->pages > (int64_t(1) << 31) || c->pages * c->kv_heads * c->page >= (int64_t(1) << 31))
    return W4A8_ERR_SHAPE;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) || !aligned16(c->v_scales))
    return W4A8_ERR_ALIGN;
  return W4A8_OK;
}
KvCacheParams cache_params(const w4a8_kv_cache* c) {
  KvCacheParams p;
  p.codes[0] = c->k_codes;
  p.codes[1] = c->v_codes;
  p.scales[0] = c->k_scales;
  p.scales[1] = c->v_scales;
  p.pages = c->pages;
  p.kv_heads = c->kv_heads;
  p.page_shift = page_shift_of(c->page);
  p.D = c->head_dim;
  return p;
}

w4a8_status batch_ok(const w4a8_kv_batch* b, int page) {
  if (!b || !b->table || !b->q_start || !b->kv_len) return W4A8_ERR_NULL;
  if (b->batch < 1 || b->batch > 65536 || b->tokens < 1 || b->tokens > (int64_t(1) << 24) || b->table_stride < 1 ||
      b->table_stride > kKvMaxTokens / page)
    return W4A8_ERR_SHAPE;
  if (!aligned4(b->table) || !aligned4(b->q_start) || !aligned4(b->kv_len)) return W4A8_ERR_ALIGN;
  return W4A8_OK;
}
KvBatchParams batch_params(const w4a8_kv_batch* b) {
  return KvBatchParams{b->table, b->table_stride, b->q_start, b->kv_len, int(b->batch), int(b->tokens)};
}

bool ka_shape_ok(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t D) {
  return tokens >= 1 && tokens <= (int64_t(1) << 24) && head_dim_ok(D) && kv_heads >= 1 && q_heads >= 1 &&
         q_heads <= 65536 && q_heads % kv_heads == 0 && q_heads / kv_heads <= 128 &&
         tokens * (q_heads / kv_heads) < (int64_t(1) << 31);
}

constexpr size_t kKaZeroBytes = 1024;
static_assert((kKaMaxCtas + kKaMaxCtas / 2) * 4 <= kKaZeroBytes, "counters fit");

// Row tiles of 8 where a sequence has that many rows on average (a decode
// step of up to 8 query heads to a key head), else of 16.
bool ka_few_rows(int64_t tokens, int64_t batch, int group) { return tokens * group <= 8 * batch; }

template <int D, int NR>
cudaError_t ka_launch(const KaParams& p, const w4a8_kv_cache* c, int ctas, cudaStream_t st) {
  using C = KaCfg<D, NR>;
  const int box = std::min(C::TK, int(c->page));
  const auto swizzle = D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const int64_t slots = c->pages * c->kv_heads * c->page;
  CUtensorMap tk, tv;
  if (!byte_map(&tk, c->k_codes, D, slots, C::kRowBytes, uint32_t(box), swizzle) ||
      !byte_map(&tv, c->v_codes, D, slots, C::kRowBytes, uint32_t(box), swizzle))
    return cudaErrorUnknown;
  KaParams q = p;
  q.box_shift = page_shift_of(box);
  // The tensor-memory kernel goes first where the batch may have rows for it (each kernel decides from the
  // sequences' lengths which of them are its own).
  q.both = kv_tiles_may_pay(p.batch.tokens, p.batch.batch, p.group, c->kv_heads, p.batch.table_stride * c->page, p.window,
                            D, p.sms);
  if (q.both) {
    const int64_t units = kp_tiles_bound(int64_t(p.batch.tokens) * p.group, p.batch.batch, kp_rows(D)) * c->kv_heads;
    const int64_t grid = units + p.sms;  // (the units' parts are at most one wave)
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    if (cudaError_t e = launch_pdl(kv_prefill_kernel<D>, dim3(unsigned(grid)), dim3(KpCfg<D>::kThreads),
                                   KpCfg<D>::kSmem, st, q);
        e != cudaSuccess)
      return e;
  }
  return launch_pdl(kv_attention_kernel<D, NR>, dim3(ctas), dim3(C::kThreads), C::kSmem, st, tk, tv, q);
}

// Shared-memory opt-ins of this file's kernels, once per device.
bool int8_allow_smem() {
  return allow_smem(int8_quant_kernel<false>, size_t(kMaxK) * 4) == cudaSuccess &&
         allow_smem(int8_quant_kernel<true>, size_t(kMaxK) * 4) == cudaSuccess &&
         allow_smem(int8_quant_wide_kernel<false>, size_t(kMaxK) * 4) == cudaSuccess &&
         allow_smem(int8_quant_wide_kernel<true>, size_t(kMaxK) * 4) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<16, 2>, Q8Cfg<16, 2>::kSmem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<16, 1>, Q8Cfg<16, 1>::kSmem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<32, 2>, Q8Cfg<32, 2>::kSmem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<32, 1>, Q8Cfg<32, 1>::kSmem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<64, 2>, Q8Cfg<64, 2>::kSmem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<64, 1>, Q8Cfg<64, 1>::kSmem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<128, 2>, Q8Cfg<128, 2>::kSmem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<128, 1>, Q8Cfg<128, 1>::kSmem) == cudaSuccess &&
         allow_smem(int8_pair_kernel, kQ2Smem) == cudaSuccess &&
         allow_smem(int8_gemm_kernel<256, 1>, Q8Cfg<256, 1>::kSmem) == cudaSuccess &&
         allow_smem(kv_attention_kernel<64, 1>, KaCfg<64, 1>::kSmem) == cudaSuccess &&
         allow_smem(kv_attention_kernel<64, 2>, KaCfg<64, 2>::kSmem) == cudaSuccess &&
         allow_smem(kv_attention_kernel<128, 1>, KaCfg<128, 1>::kSmem) == cudaSuccess &&
         allow_smem(kv_attention_kernel<128, 2>, KaCfg<128, 2>::kSmem) == cudaSuccess &&
         allow_smem(kv_attention_kernel<256, 1>, KaCfg<256, 1>::kSmem) == cudaSuccess &&
         allow_smem(kv_attention_kernel<256, 2>, KaCfg<256, 2>::kSmem) == cudaSuccess &&
         allow_smem(kv_prefill_kernel<64>, KpCfg<64>::kSmem) == cudaSuccess &&
         allow_smem(kv_prefill_kernel<128>, KpCfg<128>::kSmem) == cudaSuccess &&
         allow_smem(kv_prefill_kernel<256>, KpCfg<256>::kSmem) == cudaSuccess;
}

// device_state, and the opt-ins above the first time on a device.
w4a8_status int8_state(DeviceState** out) {
  if (w4a8_status st = device_state(out); st != W4A8_OK) return st;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!(*out)->int8_ready) {
    if (!int8_allow_smem()) return W4A8_ERR_CUDA;
    (*out)->int8_ready = true;
  }
  return W4A8_OK;
}

}  // namespace
}  // namespace w4a8

extern "C" {

w4a8_status w4a8_int8_quantize(const void* x, int32_t x_is_f32, int64_t R, int64_t K, int32_t rotate, int8_t* codes,
                               float* s, void* stream) {
  if (!x || !codes || !s) return W4A8_ERR_NULL;
  if (!q8_rows_ok(R) || !q8_k_ok(K, rotate)) return W4A8_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(s)) return W4A8_ERR_ALIGN;
  DeviceState* d = nullptr;
  if (w4a8_status st = int8_state(&d); st != W4A8_OK) return st;
  return status_of(q8_quantize(x, x_is_f32, R, K, rotate, false, codes, s, static_cast<cudaStream_t>(stream)));
}

w4a8_status w4a8_int8_gemm(const int8_t* x_q, const float* s_x, int64_t M, const int8_t* w_q, const float* s_w,
                           int64_t N, int64_t K, uint16_t* y, void* stream) {
  if (!x_q || !s_x || !w_q || !s_w || !y) return W4A8_ERR_NULL;
  if (!q8_shape_ok(M, N, K, 0)) return W4A8_ERR_SHAPE;
  if (!aligned16(x_q) || !aligned16(s_x) || !aligned16(w_q) || !aligned16(s_w) || !aligned16(y)) return W4A8_ERR_ALIGN;
  DeviceState* d = nullptr;
  if (w4a8_status st = int8_state(&d); st != W4A8_OK) return st;
  return q8_gemm(x_q, s_x, M, w_q, s_w, N, K, y, d, static_cast<cudaStream_t>(stream));
}

size_t w4a8_int8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  return q8_shape_ok(M, N, K, 0) ? q8_ws(M, K).total : 0;
}

w4a8_status w4a8_int8_linear(const uint16_t* x, int64_t M, int64_t K, int32_t rotate, const int8_t* w_q,
                             const float* s_w, int64_t N, uint16_t* y, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!x || !w_q || !s_w || !y || !workspace) return W4A8_ERR_NULL;
  if (!q8_shape_ok(M, N, K, rotate)) return W4A8_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(w_q) || !aligned16(s_w) || !aligned16(y) || !aligned16(workspace)) return W4A8_ERR_ALIGN;
  const Q8Ws w = q8_ws(M, K);
  if (workspace_bytes < w.total) return W4A8_ERR_WORKSPACE;
  DeviceState* d = nullptr;
  if (w4a8_status st = int8_state(&d); st != W4A8_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int8_t* codes = static_cast<int8_t*>(workspace);
  float* s_x = reinterpret_cast<float*>(codes + w.off_s);
  if (q8_quantize(x, 0, M, K, rotate, true, codes, s_x, s) != cudaSuccess) return W4A8_ERR_CUDA;
  return q8_gemm(codes, s_x, M, w_q, s_w, N, K, y, d, s);
}

w4a8_status w4a8_qk_norm_rope(const w4a8_heads* q, const w4a8_heads* k, int64_t T, int32_t D, const float* q_weight,
                              const float* k_weight, float eps, const int32_t* positions, const w4a8_rope* rope,
                              const w4a8_heads* q_out, const w4a8_heads* k_out, void* stream) {
  const bool has_q = q && q->data, has_k = k && k->data;
  if ((!has_q && !has_k) || (has_q && (!q_out || !q_out->data)) || (has_k && (!k_out || !k_out->data))) return W4A8_ERR_NULL;
  if (rope && rope->inv_freq && !positions) return W4A8_ERR_NULL;
  if (T < 1 || T > (int64_t(1) << 24) || !head_dim_ok(D)) return W4A8_ERR_SHAPE;
  for (const w4a8_heads* h : {has_q ? q : nullptr, has_k ? k : nullptr})
    if (h)
      if (w4a8_status st = heads_ok(*h, D); st != W4A8_OK) return st;
  for (const w4a8_heads* h : {has_q ? q_out : nullptr, has_k ? k_out : nullptr})
    if (h)
      if (w4a8_status st = heads_out_ok(*h, T, D); st != W4A8_OK) return st;
  if ((has_q && q->heads != q_out->heads) || (has_k && k->heads != k_out->heads)) return W4A8_ERR_SHAPE;
  if ((has_q && !heads_in_place_ok(*q, *q_out, T)) || (has_k && !heads_in_place_ok(*k, *k_out, T))) return W4A8_ERR_SHAPE;
  if (w4a8_status st = rope_ok(rope, D); st != W4A8_OK) return st;
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)) || !aligned4(positions)) return W4A8_ERR_ALIGN;
  DeviceState* d = nullptr;
  if (w4a8_status st = int8_state(&d); st != W4A8_OK) return st;
  QkParams p{head_rows(q), head_rows(k), head_rows(q_out), head_rows(k_out), q_weight, k_weight, eps,
             rope_params(rope), positions, int(T)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int parts = qk_parts(T, (has_q ? q->heads : 0) + (has_k ? k->heads : 0), D);
  const dim3 grid{unsigned((T * parts * 32 + kQkThreads - 1) / kQkThreads)}, block{kQkThreads};
  return status_of(D == 64    ? launch_pdl(qk_norm_rope_kernel<64>, grid, block, 0, s, p, parts)
                   : D == 128 ? launch_pdl(qk_norm_rope_kernel<128>, grid, block, 0, s, p, parts)
                              : launch_pdl(qk_norm_rope_kernel<256>, grid, block, 0, s, p, parts));
}

w4a8_status w4a8_kv_update(const w4a8_kv_cache* cache, const w4a8_kv_batch* batch, const w4a8_heads* k,
                           const w4a8_heads* v, const w4a8_heads* q, const float* q_weight, const float* k_weight,
                           float eps, const int32_t* positions, const w4a8_rope* rope, const w4a8_heads* q_out,
                           void* stream) {
  const bool has_q = q && q->data;
  if (!k || !k->data || !v || !v->data || (has_q && (!q_out || !q_out->data))) return W4A8_ERR_NULL;
  if (w4a8_status st = cache_ok(cache); st != W4A8_OK) return st;
  if (w4a8_status st = batch_ok(batch, cache->page); st != W4A8_OK) return st;
  const int D = cache->head_dim;
  for (const w4a8_heads* h : {k, v, has_q ? q : nullptr})
    if (h)
      if (w4a8_status st = heads_ok(*h, D); st != W4A8_OK) return st;
  if (has_q)
    if (w4a8_status st = heads_out_ok(*q_out, batch->tokens, D); st != W4A8_OK) return st;
  if (k->heads != cache->kv_heads || v->heads != cache->kv_heads || (has_q && q->heads != q_out->heads)) return W4A8_ERR_SHAPE;
  if (has_q && !heads_in_place_ok(*q, *q_out, batch->tokens)) return W4A8_ERR_SHAPE;
  if (w4a8_status st = rope_ok(rope, D); st != W4A8_OK) return st;
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)) || !aligned4(positions)) return W4A8_ERR_ALIGN;
  const int64_t units = kv_touched_bound(batch->tokens, batch->batch, cache->page);
  const int64_t page_ctas = units * cache->kv_heads * 2;
  if (page_ctas + batch->tokens >= (int64_t(1) << 31)) return W4A8_ERR_SHAPE;
  DeviceState* d = nullptr;
  if (w4a8_status st = int8_state(&d); st != W4A8_OK) return st;
  KvUpdateParams p;
  p.qk = QkParams{head_rows(q), head_rows(k), head_rows(q_out), HeadRows{nullptr, 0, 0, 0}, q_weight, k_weight, eps,
                  rope_params(rope), positions, int(batch->tokens)};
  p.v = head_rows(v);
  p.cache = cache_params(cache);
  p.batch = batch_params(batch);
  p.page_ctas = int(page_ctas);
  p.err = d->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.q_parts = has_q ? qk_parts(batch->tokens, q->heads, D) : 1;
  // Few new tokens a sequence: small CTAs.
  const bool small = batch->tokens <= 4 * batch->batch;
  const int threads = small ? 64 : 256;
  const int64_t q_ctas = has_q ? (batch->tokens * p.q_parts * 32 + threads - 1) / threads : 0;
  p.stride = int((page_ctas + q_ctas) / page_ctas);
  p.rest_cta = batch->batch > 32 ? int(page_ctas + q_ctas) : -1;
  const dim3 grid{unsigned(page_ctas + q_ctas + (p.rest_cta >= 0))}, block{unsigned(threads)};
  switch (D + small) {
    case 64: return status_of(launch_pdl(kv_update_kernel<64, 256>, grid, block, 0, s, p));
    case 65: return status_of(launch_pdl(kv_update_kernel<64, 64>, grid, block, 0, s, p));
    case 128: return status_of(launch_pdl(kv_update_kernel<128, 256>, grid, block, 0, s, p));
    case 129: return status_of(launch_pdl(kv_update_kernel<128, 64>, grid, block, 0, s, p));
    case 256: return status_of(launch_pdl(kv_update_kernel<256, 256>, grid, block, 0, s, p));
    default: return status_of(launch_pdl(kv_update_kernel<256, 64>, grid, block, 0, s, p));
  }
}

w4a8_status w4a8_kv_dequant(const w4a8_kv_cache* cache, const int32_t* ids, int64_t n, uint16_t* k_out, uint16_t* v_out,
                            void* stream) {
  if (!ids || !k_out || !v_out) return W4A8_ERR_NULL;
  if (w4a8_status st = cache_ok(cache); st != W4A8_OK) return st;
  if (n < 1 || n >= (int64_t(1) << 31)) return W4A8_ERR_SHAPE;
  const int slab = cache->page * cache->head_dim, parts = (slab + 16 * kDqThreads - 1) / (16 * kDqThreads);
  const int64_t ctas = 2 * n * cache->kv_heads * parts;
  if (ctas >= (int64_t(1) << 31)) return W4A8_ERR_SHAPE;
  if (!aligned4(ids) || !aligned16(k_out) || !aligned16(v_out)) return W4A8_ERR_ALIGN;
  DeviceState* d = nullptr;
  if (w4a8_status st = int8_state(&d); st != W4A8_OK) return st;
  return status_of(launch_pdl(kv_dequant_kernel, dim3(unsigned(ctas)), dim3(kDqThreads), 0,
                              static_cast<cudaStream_t>(stream), cache_params(cache), ids, int(n), k_out, v_out, d->err));
}

size_t w4a8_kv_attention_workspace_bytes(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (!ka_shape_ok(tokens, q_heads, kv_heads, head_dim)) return 0;
  const int64_t rows = tokens * (q_heads / kv_heads);
  const size_t stream = size_t(kKaMaxCtas) * 2 * (size_t(kKaMaxRows) * head_dim + 2 * kKaMaxRows) * 4;
  const size_t parts = size_t(kKaMaxCtas) * (head_dim <= 128 ? 256 : 128) * (head_dim + 2) * 4;
  return kKaZeroBytes + (kp_tiles_bound(rows, tokens, 256) * kv_heads >= kKpMinCtas ? std::max(stream, parts) : stream);
}

w4a8_status w4a8_kv_attention(const w4a8_heads* q, const w4a8_kv_cache* cache, const w4a8_kv_batch* batch, float scale,
                              int32_t window, const w4a8_heads* out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (!q || !q->data || !out || !out->data || !workspace) return W4A8_ERR_NULL;
  if (w4a8_status st = cache_ok(cache); st != W4A8_OK) return st;
  if (w4a8_status st = batch_ok(batch, cache->page); st != W4A8_OK) return st;
  const int D = cache->head_dim;
  if (w4a8_status st = heads_ok(*q, D); st != W4A8_OK) return st;
  if (w4a8_status st = heads_out_ok(*out, batch->tokens, D); st != W4A8_OK) return st;
  if (q->heads != out->heads || window < 0 || !ka_shape_ok(batch->tokens, q->heads, cache->kv_heads, D)) return W4A8_ERR_SHAPE;
  if (!heads_in_place_ok(*q, *out, batch->tokens)) return W4A8_ERR_SHAPE;
  if (!aligned16(workspace)) return W4A8_ERR_ALIGN;
  if (workspace_bytes < w4a8_kv_attention_workspace_bytes(batch->tokens, q->heads, cache->kv_heads, D))
    return W4A8_ERR_WORKSPACE;
  DeviceState* d = nullptr;
  if (w4a8_status st = int8_state(&d); st != W4A8_OK) return st;
  KaParams p;
  p.q = head_rows(q);
  p.out = head_rows(out);
  p.cache = cache_params(cache);
  p.batch = batch_params(batch);
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.window = window;
  p.group = q->heads / cache->kv_heads;
  p.box_shift = 0;
  p.both = 0;
  p.sms = std::min(d->sms, kKaMaxCtas);
  p.counters = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kKaZeroBytes);
  p.err = d->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int ctas = p.sms;
  const bool few = ka_few_rows(batch->tokens, batch->batch, p.group);
  switch (D + few) {
    case 64: return status_of(ka_launch<64, 2>(p, cache, ctas, s));
    case 65: return status_of(ka_launch<64, 1>(p, cache, ctas, s));
    case 128: return status_of(ka_launch<128, 2>(p, cache, ctas, s));
    case 129: return status_of(ka_launch<128, 1>(p, cache, ctas, s));
    case 256: return status_of(ka_launch<256, 2>(p, cache, ctas, s));
    default: return status_of(ka_launch<256, 1>(p, cache, ctas, s));
  }
}

}  // extern "C"
