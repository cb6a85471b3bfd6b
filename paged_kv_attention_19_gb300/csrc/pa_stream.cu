// pa_stream.cu -- the host side of the streams' attention (pa_stream.cuh): argument checks, workspace, tensor maps and the
// launches of a call.
#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_decode.h"
#include "pa_host.h"
#include "pa_launch.h"
#include "pa_stream.cuh"
#include "pa_tree_launch.cuh"

namespace pa {

namespace {

constexpr int kMaxSplits = 4096;
constexpr int kMaxQuery = 1 << 30;
constexpr int kMaxContext = INT_MAX - 512;

struct StreamPlan {
  size_t total;
};

int stream_plan(int batch, int max_query, int Hq, int Hkv, int D, int max_ctx, int P, int num_splits, StreamPlan *pl) {
  if (batch < 0 || max_query <= 0 || Hq <= 0 || Hkv <= 0 || max_ctx < 0 || num_splits < 0 || Hq % Hkv != 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (max_query > kMaxQuery || num_splits > kMaxSplits || (D != 64 && D != 128 && D != 256) || !is_pow2(P) || P < 8 ||
      P > 256 || max_ctx > kMaxContext || Hq / Hkv > kTreeRows)
    return PA_ERR_UNSUPPORTED;
  pl->total = sizeof(WsHeader);
  return PA_OK;
}

template <int D>
cudaError_t launch_rows(int fmt, const StreamArgs &a, cudaStream_t stream) {
  const dim3 grid((unsigned)a.tokens, (unsigned)a.Hq);
  auto kernel = fmt == TREE_BF16 ? stream_rows_kernel<D, TREE_BF16> : fmt == TREE_FP8 ? stream_rows_kernel<D, TREE_FP8> : stream_rows_kernel<D, TREE_NVFP4>;
  return launch_pdl(kernel, grid, 128, 0, stream, a);
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
  StreamArgs a;
  a.q = static_cast<const uint8_t *>(q);
  a.k_pool = static_cast<const uint8_t *>(k_pool);
  a.v_pool = static_cast<const uint8_t *>(v_pool);
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.granted = granted;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.status = &static_cast<WsHeader *>(workspace)->status;
  a.batch = batch;
  a.tokens = tokens;
  a.max_query = max_query;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.log2_page = ilog2(P);
  a.num_pages = num_pages;
  a.max_pages_per_seq = max_pages;
  a.max_context_len = max_ctx;
  a.window = window > 0 ? window : 0;
  a.first = window > 0 ? first : 0;
  a.scale = scale;
  a.kscale = fmt == TREE_BF16 ? 1.f : k_scale;
  a.vscale = fmt == TREE_BF16 ? 1.f : v_scale;
  cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(uint32_t), stream);
  if (e != cudaSuccess) return cuda_fail(e);
  e = D == 64 ? launch_rows<64>(fmt, a, stream) : D == 128 ? launch_rows<128>(fmt, a, stream) : launch_rows<256>(fmt, a, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launches(1);
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
