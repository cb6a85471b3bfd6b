// pa_tree.cu -- the host side of the tree attention (pa_tree.cuh): argument checks, workspace, tensor maps
// and the launches of a call.
#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_decode.h"
#include "pa_host.h"
#include "pa_launch.h"
#include "pa_tree_launch.cuh"

namespace pa {

namespace {

constexpr int kMaxSplits = 4096, kAutoParts = 256;
// Fixed cost of a piece of work in the partition, as the tokens that a CTA passes meanwhile (256, 512, 768, 1024: the
// serving mix over FP8 109, 111, 117, 123 us, 8 rows of 33 nodes 46.3, 43.9, 43.6, 43.1).
constexpr int kPieceCost = 512;
// Least share of a group, in tokens, where the number of shares is left to the call: below two stages, one for each
// softmax group, a share takes as long and only adds to what is merged (none, 64, 128, 256: 4 rows of 8 nodes over 200
// to 3000 tokens 17.8, 17.9, 15.3, 15.6 us; 40 nodes over 1000 tokens 16.0, 16.1, 14.4, 15.3).
constexpr int kMinShare = 128;

// Longest context: the ends of the stages behind it, two of 64 tokens, are still tokens below 2^31.
constexpr int kMaxContext = INT_MAX - 128;

// How a call's query rows are tiled, and where its workspace's parts lie.
struct TreePlan {
  int G, gt, qt, nsub, QT, nseqh, nparts_max;
  size_t off_status, off_lse, off_o, off_half, total;
};

int tree_plan(int batch, int max_query, int Hq, int Hkv, int D, int max_ctx, int P, int num_splits, TreePlan *pl) {
  if (batch < 0 || max_query <= 0 || Hq <= 0 || Hkv <= 0 || max_ctx < 0 || num_splits < 0 || Hq % Hkv != 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (max_query > kTreeNodes || num_splits > kMaxSplits || (D != 64 && D != 128 && D != 256) || !is_pow2(P) || P < 8 ||
      P > 256 || max_ctx > kMaxContext)
    return PA_ERR_UNSUPPORTED;
  pl->G = Hq / Hkv;
  pl->gt = pl->G < kTreeRows ? pl->G : kTreeRows;
  pl->nsub = (pl->G + kTreeRows - 1) / kTreeRows;
  pl->qt = pl->nsub > 1 ? 1 : kTreeRows / pl->G;
  const int ntile = pl->nsub > 1 ? max_query * pl->nsub : (max_query + pl->qt - 1) / pl->qt;
  pl->QT = D <= 128 && ntile > 1 ? 2 : 1;
  pl->nseqh = (ntile + pl->QT - 1) / pl->QT;
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
  off = round_up(off + np * 2 * kTreeRows * sizeof(TreeHalf), 256);
  pl->total = off;
  return PA_OK;
}

int tree_call(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
              const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask, const int32_t *granted,
              void *out, float *lse, int batch, int tokens, int max_query, int Hq, int Hkv, int D, int P, int num_pages, int max_pages,
              int max_ctx, float scale, int fmt, float k_scale, float v_scale, int window, int num_splits, void *workspace,
              size_t workspace_bytes, cudaStream_t stream) {
  note_launches(0);
  TreePlan pl;
  const int rc = tree_plan(batch, max_query, Hq, Hkv, D, max_ctx, P, num_splits, &pl);
  if (rc != PA_OK) return rc;
  if (tokens < 0 || num_pages <= 0 || max_pages <= 0 || !std::isfinite(scale)) return PA_ERR_INVALID_ARGUMENT;
  if (fmt != TREE_BF16 && !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARGUMENT;
  if ((long long)max_pages * P < (long long)max_ctx) return PA_ERR_INVALID_ARGUMENT;
  if ((long long)batch * Hkv * pl.nseqh > INT_MAX) return PA_ERR_UNSUPPORTED;
  if (batch == 0 || tokens == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !block_table || !context_lens || !query_start || !tree_mask || !out || !workspace)
    return PA_ERR_INVALID_ARGUMENT;
  const void *vecs[] = {q, k_pool, v_pool, out, workspace};
  for (const void *p : vecs)
    if (!aligned_to(p, 16)) return PA_ERR_MISALIGNED;
  const void *words[] = {block_table, context_lens, query_start, granted, lse};
  for (const void *p : words)
    if (!aligned_to(p, 4)) return PA_ERR_MISALIGNED;
  if (!aligned_to(tree_mask, 8)) return PA_ERR_MISALIGNED;
  if (workspace_bytes < pl.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  const int BN = 64;                   // tokens per stage (TreeCfg::BN)
  const int BH = P < BN ? P : BN;      // tokens per TMA box: a unit
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaSuccess);
  CUtensorMap tm_k, tm_v, tm_q;
  const bool codes = fmt != TREE_BF16;
  const int rowb = tree_row_bytes(fmt, D);
  const cuuint64_t pool[4] = {(cuuint64_t)(codes ? rowb : D), (cuuint64_t)Hkv, (cuuint64_t)P, (cuuint64_t)num_pages};
  const cuuint32_t pbox[4] = {codes ? (cuuint32_t)rowb : 64u, 1u, (cuuint32_t)BH, 1u};
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)tokens};
  const cuuint32_t qbox[3] = {64u, (cuuint32_t)pl.gt, (cuuint32_t)(pl.qt < max_query ? pl.qt : max_query)};
  if (!encode_map(&tm_k, k_pool, pool, pbox, codes) || !encode_map(&tm_v, v_pool, pool, pbox, codes) ||
      !encode_map(&tm_q, q, qd, qbox, false))
    return PA_ERR_UNSUPPORTED;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  TreeArgs a;
  a.v_pool = static_cast<const uint8_t *>(v_pool);
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.tree_mask = tree_mask;
  a.granted = granted;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.cta_status = reinterpret_cast<uint32_t *>(ws + pl.off_status);
  a.part_lse = reinterpret_cast<float *>(ws + pl.off_lse);
  a.part_o = reinterpret_cast<float *>(ws + pl.off_o);
  a.halves = reinterpret_cast<TreeHalf *>(ws + pl.off_half);
  a.batch = batch;
  a.tokens = tokens;
  a.max_query = max_query;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = pl.G;
  a.gt = pl.gt;
  a.qt = pl.qt;
  a.nsub = pl.nsub;
  a.nseqh = pl.nseqh;
  a.log2_page = ilog2(P);
  a.log2_bh = ilog2(BH);
  a.num_pages = num_pages;
  a.max_pages_per_seq = max_pages;
  a.max_context_len = max_ctx;
  a.window = window > 0 ? window : 0;
  a.piece_cost = kPieceCost / BH;
  a.log2_share = num_splits > 0 ? 0 : ilog2(kMinShare / BH);
  a.nparts = num_splits > 0 ? num_splits : sms < kAutoParts ? sms : kAutoParts;
  const int hs = Hkv * pl.nseqh;
  a.hg = hs < a.nparts ? hs : a.nparts;
  a.qscale = scale * LOG2E * (codes ? k_scale : 1.f);
  a.vscale = codes ? v_scale : 1.f;
  uint32_t *status = &reinterpret_cast<WsHeader *>(ws)->status;
  const TreeLaunch l = {tm_k, tm_v, tm_q, a, status, D, pl.QT};
  const cudaError_t e = fmt == TREE_BF16  ? launch_tree_bf16(l, stream)
                        : fmt == TREE_FP8 ? launch_tree_fp8(l, stream)
                                          : launch_tree_nvfp4(l, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launches(2);
  return PA_OK;
}

}  // namespace

}  // namespace pa

extern "C" size_t pa_tree_workspace_size(int batch, int max_query, int num_q_heads, int num_kv_heads, int head_dim,
                                         int max_context_len, int page_size, int num_splits) {
  pa::TreePlan pl;
  return pa::tree_plan(batch, max_query, num_q_heads, num_kv_heads, head_dim, max_context_len, page_size, num_splits,
                       &pl) == PA_OK
             ? pl.total
             : 0;
}

extern "C" int pa_tree_gqa(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                           const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask,
                           void *out, float *lse, int batch, int num_tokens, int max_query, int num_q_heads,
                           int num_kv_heads, int head_dim, int page_size, int num_pages, int max_pages_per_seq,
                           int max_context_len, float scale, int window, int num_splits, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, nullptr, out, lse, batch,
                       num_tokens, max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                       max_pages_per_seq, max_context_len, scale, pa::TREE_BF16, 1.f, 1.f, window, num_splits,
                       workspace, workspace_bytes, stream);
}

extern "C" int pa_tree_gqa_granted(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                                   const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask,
                                   const int32_t *granted, void *out, float *lse, int batch, int num_tokens,
                                   int max_query, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                                   int num_pages, int max_pages_per_seq, int max_context_len, float scale, int window,
                                   int num_splits, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, granted, out, lse, batch,
                       num_tokens, max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                       max_pages_per_seq, max_context_len, scale, pa::TREE_BF16, 1.f, 1.f, window, num_splits,
                       workspace, workspace_bytes, stream);
}

extern "C" int pa_tree_gqa_fp8(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                               const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask,
                               void *out, float *lse, int batch, int num_tokens, int max_query, int num_q_heads,
                               int num_kv_heads, int head_dim, int page_size, int num_pages, int max_pages_per_seq,
                               int max_context_len, float scale, float k_scale, float v_scale, int window,
                               int num_splits, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, nullptr, out, lse, batch,
                       num_tokens, max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                       max_pages_per_seq, max_context_len, scale, pa::TREE_FP8, k_scale, v_scale, window, num_splits,
                       workspace, workspace_bytes, stream);
}

extern "C" int pa_tree_gqa_fp8_granted(const void *q, const void *k_pool, const void *v_pool,
                                       const int32_t *block_table, const int32_t *context_lens,
                                       const int32_t *query_start, const uint64_t *tree_mask, const int32_t *granted,
                                       void *out, float *lse, int batch, int num_tokens, int max_query, int num_q_heads,
                                       int num_kv_heads, int head_dim, int page_size, int num_pages,
                                       int max_pages_per_seq, int max_context_len, float scale, float k_scale,
                                       float v_scale, int window, int num_splits, void *workspace,
                                       size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, granted, out, lse, batch,
                       num_tokens, max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                       max_pages_per_seq, max_context_len, scale, pa::TREE_FP8, k_scale, v_scale, window, num_splits,
                       workspace, workspace_bytes, stream);
}

extern "C" int pa_tree_gqa_nvfp4(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                                 const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask,
                                 void *out, float *lse, int batch, int num_tokens, int max_query, int num_q_heads,
                                 int num_kv_heads, int head_dim, int page_size, int num_pages, int max_pages_per_seq,
                                 int max_context_len, float scale, float k_scale, float v_scale, int window,
                                 int num_splits, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, nullptr, out, lse, batch,
                       num_tokens, max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                       max_pages_per_seq, max_context_len, scale, pa::TREE_NVFP4, k_scale, v_scale, window, num_splits,
                       workspace, workspace_bytes, stream);
}

extern "C" int pa_tree_gqa_nvfp4_granted(const void *q, const void *k_pool, const void *v_pool,
                                         const int32_t *block_table, const int32_t *context_lens,
                                         const int32_t *query_start, const uint64_t *tree_mask, const int32_t *granted,
                                         void *out, float *lse, int batch, int num_tokens, int max_query,
                                         int num_q_heads, int num_kv_heads, int head_dim, int page_size, int num_pages,
                                         int max_pages_per_seq, int max_context_len, float scale, float k_scale,
                                         float v_scale, int window, int num_splits, void *workspace,
                                         size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, granted, out, lse, batch,
                       num_tokens, max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                       max_pages_per_seq, max_context_len, scale, pa::TREE_NVFP4, k_scale, v_scale, window, num_splits,
                       workspace, workspace_bytes, stream);
}
