// pa_stream.cu -- the host side of the streams' attention (pa_stream.cuh): argument checks, workspace, tensor maps and the
// launches of a call.
#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_decode.h"
#include "pa_host.h"
#include "pa_launch.h"
#include "pa_stream_launch.cuh"

namespace pa {

namespace {

constexpr int kMaxSplits = 4096, kAutoParts = 256;
constexpr int kMaxQuery = 1 << 30;
// Longest context: the ends of the stages behind it, two of 128 tokens, are still tokens below 2^31.
constexpr int kMaxContext = INT_MAX - 512;
// Fixed cost of a piece of work in the partition, as the tokens that a CTA passes meanwhile (256, 512, 1024: a prompt of
// 8192 tokens 476, 471, 495 us; FP8 single tokens 92.9, 88.8, 95.4).
constexpr int kPieceCost = 512;
// Least share of a CTA, in tokens, where the number of shares is left to the call: below two stages, one for each
// softmax group, a share takes as long and only adds to what is merged (128, 256: one token 14.1, 15.3 us).
constexpr int kMinShare = 128;
// Pairs of at most so many tokens are not cut, where the number of shares is left to the call (400, 768: single tokens and chunks
// in a window of 512 30.1, 28.1 us; 1100 gains nothing there, and one token over 1028 takes 18.1 us for 14.1).  The rule does not
// look at how much work there is beside them: a lone token over 768 tokens and 8 key heads takes 14.3 us whole and 13.0 in six
// shares a head, over FP8 19.8 and 16.6; over 512 it is 12.5 and 12.1, over 256 whole is as fast.
constexpr int kWhole = 768;

// How a call's query rows are tiled, and where its workspace's parts lie.
struct StreamPlan {
  int G, qt, QT, nparts_max;
  size_t off_status, off_lse, off_o, off_half, total;
};

int stream_plan(int batch, int max_query, int Hq, int Hkv, int D, int max_ctx, int P, int num_splits, StreamPlan *pl) {
  if (batch < 0 || max_query <= 0 || Hq <= 0 || Hkv <= 0 || max_ctx < 0 || num_splits < 0 || Hq % Hkv != 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (max_query > kMaxQuery || num_splits > kMaxSplits || (D != 64 && D != 128 && D != 256) || !is_pow2(P) || P < 8 ||
      P > 256 || max_ctx > kMaxContext || Hq / Hkv > kTreeRows)
    return PA_ERR_UNSUPPORTED;
  pl->G = Hq / Hkv;
  pl->qt = kTreeRows / pl->G;
  pl->QT = D <= 128 && max_query > pl->qt ? 2 : 1;
  pl->nparts_max = num_splits > 0 ? num_splits : kAutoParts;
  const size_t np = (size_t)pl->nparts_max, rows = np * 2 * pl->QT * kTreeRows;
  size_t off = sizeof(WsHeader);
  pl->off_status = off;
  off = round_up(off + np * sizeof(uint32_t), 256);
  pl->off_lse = off;
  off = round_up(off + rows * sizeof(float), 256);
  pl->off_o = off;
  off = round_up(off + rows * D * sizeof(float), 256);
  pl->off_half = off;
  off = round_up(off + np * 2 * kTreeRows * sizeof(StreamHalf), 256);
  pl->total = off;
  return PA_OK;
}

int stream_call(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table, const int32_t *context_lens,
                const int32_t *query_start, const int32_t *granted, void *out, float *lse, int batch, int tokens, int max_query,
                int Hq, int Hkv, int D, int P, int num_pages, int max_pages, int max_ctx, float scale, int fmt, float k_scale,
                float v_scale, int window, int first, int num_splits, void *workspace, size_t workspace_bytes,
                cudaStream_t stream) {
  note_launches(0);
  StreamPlan pl;
  const int rc = stream_plan(batch, max_query, Hq, Hkv, D, max_ctx, P, num_splits, &pl);
  if (rc != PA_OK) return rc;
  if (tokens < 0 || num_pages <= 0 || max_pages <= 0 || first < 0 || !std::isfinite(scale)) return PA_ERR_INVALID_ARGUMENT;
  if (fmt != TREE_BF16 && !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARGUMENT;
  const float qscale = scale * LOG2E * (fmt == TREE_BF16 ? 1.f : k_scale);
  if (!std::isfinite(qscale)) return PA_ERR_INVALID_ARGUMENT;
  if ((long long)max_pages * P < (long long)max_ctx) return PA_ERR_INVALID_ARGUMENT;
  if (batch == 0 || tokens == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !block_table || !context_lens || !query_start || !out || !workspace)
    return PA_ERR_INVALID_ARGUMENT;
  const void *vecs[] = {q, k_pool, v_pool, out, workspace};
  for (const void *p : vecs)
    if (!aligned_to(p, 16)) return PA_ERR_MISALIGNED;
  const void *words[] = {block_table, context_lens, query_start, granted, lse};
  for (const void *p : words)
    if (!aligned_to(p, 4)) return PA_ERR_MISALIGNED;
  if (workspace_bytes < pl.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  const int BN = stream_stage(D, fmt, pl.QT), BH = P < BN ? P : BN;  // tokens of a stage, and of a TMA box: a unit
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaSuccess);
  CUtensorMap tm_k, tm_v, tm_q;
  const bool codes = fmt != TREE_BF16;
  const int rowb = tree_row_bytes(fmt, D);
  // bf16 pools: groups of 8 tokens, whose rows of 64 values (planes) of one head lie 128 bytes apart; codes: whole rows
  const cuuint64_t pool[4] = {(cuuint64_t)rowb, (cuuint64_t)Hkv, (cuuint64_t)P, (cuuint64_t)num_pages};
  const cuuint32_t pbox[4] = {(cuuint32_t)rowb, 1u, (cuuint32_t)BH, 1u};
  const cuuint64_t token = (cuuint64_t)Hkv * D * 2;  // bytes
  const cuuint64_t group[4] = {64u, 8u, (cuuint64_t)Hkv * (D / 64), (cuuint64_t)num_pages * (P / 8)};
  const cuuint64_t apart[3] = {token, 128u, 8 * token};
  const cuuint32_t gbox[4] = {64u, 8u, (cuuint32_t)(D / 64), (cuuint32_t)(BH / 8)};
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)tokens};
  const cuuint32_t qbox[3] = {64u, (cuuint32_t)pl.G, (cuuint32_t)(pl.qt < max_query ? pl.qt : max_query)};
  auto pool_map = [&](CUtensorMap *m, const void *base) {
    return codes ? encode_map(m, base, pool, pbox, true) : encode_map(m, base, group, gbox, false, apart);
  };
  if ((long long)num_pages * (P / 8) > INT_MAX || !pool_map(&tm_k, k_pool) || !pool_map(&tm_v, v_pool) ||
      !encode_map(&tm_q, q, qd, qbox, false))
    return PA_ERR_UNSUPPORTED;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  StreamArgs a;
  a.v_pool = static_cast<const uint8_t *>(v_pool);
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.granted = granted;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.cta_status = reinterpret_cast<uint32_t *>(ws + pl.off_status);
  a.part_lse = reinterpret_cast<float *>(ws + pl.off_lse);
  a.part_o = reinterpret_cast<float *>(ws + pl.off_o);
  a.halves = reinterpret_cast<StreamHalf *>(ws + pl.off_half);
  a.batch = batch;
  a.tokens = tokens;
  a.max_query = max_query;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = pl.G;
  a.qt = pl.qt;
  a.q2 = pl.QT * pl.qt;
  a.single = max_query <= a.q2;
  a.log2_page = ilog2(P);
  a.log2_bh = ilog2(BH);
  a.num_pages = num_pages;
  a.max_pages_per_seq = max_pages;
  a.max_context_len = max_ctx;
  a.window = window > 0 ? window : 0;
  a.first = window <= 0 ? 0 : first < max_ctx ? first : max_ctx;
  a.piece_cost = kPieceCost;
  a.whole = num_splits > 0 ? 0 : kWhole;  // (a caller's number of shares is what it gets)
  a.log2_share = num_splits > 0 ? 0 : ilog2(kMinShare);
  a.nparts = num_splits > 0 ? num_splits : sms < kAutoParts ? sms : kAutoParts;
  // groups of a CTA for each key head, unless more than a tenth of the CTAs would be left over (8 heads on 152: single tokens
  // over FP8 89.1 us for 92.0 with one line of all heads, NVFP4 189.5 for 191.3; bf16 59.9 for 59.3)
  a.hg = 10 * (a.nparts / Hkv * Hkv) >= 9 * a.nparts ? Hkv : 1;
  a.hl = Hkv / a.hg;
  a.qscale = qscale;
  a.vscale = codes ? v_scale : 1.f;
  uint32_t *status = &reinterpret_cast<WsHeader *>(ws)->status;
  const StreamLaunch l = {tm_k, tm_v, tm_q, a, status, D, pl.QT};
  const cudaError_t e = fmt == TREE_BF16  ? launch_stream_bf16(l, stream)
                        : fmt == TREE_FP8 ? launch_stream_fp8(l, stream)
                                          : launch_stream_nvfp4(l, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launches(2);
  return PA_OK;
}

}  // namespace

}  // namespace pa

extern "C" size_t pa_stream_workspace_size(int batch, int max_query, int num_q_heads, int num_kv_heads, int head_dim,
                                           int max_context_len, int page_size, int num_splits) {
  pa::StreamPlan pl;
  return pa::stream_plan(batch, max_query, num_q_heads, num_kv_heads, head_dim, max_context_len, page_size, num_splits, &pl) ==
                 PA_OK
             ? pl.total
             : 0;
}

extern "C" int pa_stream_gqa(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                             const int32_t *context_lens, const int32_t *query_start, const int32_t *granted, void *out,
                             float *lse, int batch, int num_tokens, int max_query, int num_q_heads, int num_kv_heads,
                             int head_dim, int page_size, int num_pages, int max_pages_per_seq, int max_context_len,
                             float scale, int window, int first, int num_splits, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  return pa::stream_call(q, k_pool, v_pool, block_table, context_lens, query_start, granted, out, lse, batch, num_tokens,
                         max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                         max_context_len, scale, pa::TREE_BF16, 1.f, 1.f, window, first, num_splits, workspace,
                         workspace_bytes, stream);
}

extern "C" int pa_stream_gqa_fp8(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                                 const int32_t *context_lens, const int32_t *query_start, const int32_t *granted, void *out,
                                 float *lse, int batch, int num_tokens, int max_query, int num_q_heads, int num_kv_heads,
                                 int head_dim, int page_size, int num_pages, int max_pages_per_seq, int max_context_len,
                                 float scale, float k_scale, float v_scale, int window, int first, int num_splits,
                                 void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return pa::stream_call(q, k_pool, v_pool, block_table, context_lens, query_start, granted, out, lse, batch, num_tokens,
                         max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                         max_context_len, scale, pa::TREE_FP8, k_scale, v_scale, window, first, num_splits, workspace,
                         workspace_bytes, stream);
}

extern "C" int pa_stream_gqa_nvfp4(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                                   const int32_t *context_lens, const int32_t *query_start, const int32_t *granted, void *out,
                                   float *lse, int batch, int num_tokens, int max_query, int num_q_heads, int num_kv_heads,
                                   int head_dim, int page_size, int num_pages, int max_pages_per_seq, int max_context_len,
                                   float scale, float k_scale, float v_scale, int window, int first, int num_splits,
                                   void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return pa::stream_call(q, k_pool, v_pool, block_table, context_lens, query_start, granted, out, lse, batch, num_tokens,
                         max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                         max_context_len, scale, pa::TREE_NVFP4, k_scale, v_scale, window, first, num_splits, workspace,
                         workspace_bytes, stream);
}
