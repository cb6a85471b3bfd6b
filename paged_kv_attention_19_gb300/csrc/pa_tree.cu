// pa_tree.cu -- attention of drafted trees over the paged cache.
//
// Mathematics: node i of row b (n nodes, L tokens with them, prefix = L - n) attends to the set A of
// prefix tokens and of the nodes its mask names (under a window those fewer than `window` positions
// back, a node's position being prefix + its number of other mask bits):
//   out = sum_{t in A} exp(s_t - m) v_t / l,  lse = m + ln l,  s_t = scale q . k_t,
//   m = max s_t,  l = sum exp(s_t - m), in fp32 and rounded once.
#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_launch.h"
#include "pa_quant.cuh"

namespace pa {

namespace {

enum TreeFmt { TREE_BF16 = 0, TREE_FP8 = 1, TREE_NVFP4 = 2 };
constexpr int kTreeNodes = 64;

struct TreeArgs {
  const uint16_t *q;
  const uint8_t *k_pool, *v_pool;
  const int32_t *block_table, *context_lens, *query_start;
  const uint64_t *tree_mask;
  uint16_t *out;
  float *lse;  // or null
  uint32_t *status;
  int batch, tokens, max_query, Hq, Hkv, G, page_size, num_pages, max_pages_per_seq, max_context_len, window;
  float qscale, kscale, vscale;  // scale * log2(e); the pools' scales
};

template <int FMT, int D>
__device__ __forceinline__ float cache_value(const uint8_t *row, int d) {
  if constexpr (FMT == TREE_BF16) {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[d] << 16);
  } else if constexpr (FMT == TREE_FP8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(row[d], __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half *>(&h));
  } else {
    const uint32_t c = (row[d >> 1] >> (4 * (d & 1))) & 15u;
    const float mag = (c & 7u) < 2 ? 0.5f * (float)(c & 7u) : __uint_as_float((((c & 7u) >> 1) + 126u) << 23 | (c & 1u) << 22);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(row[D / 2 + (d >> 4)], __NV_E4M3);
    return (c & 8u ? -mag : mag) * __half2float(*reinterpret_cast<const __half *>(&h));
  }
}

// One block per (token, query head), a warp per fourth key.
template <int FMT, int D>
__global__ void __launch_bounds__(128) tree_plain_kernel(const TreeArgs a) {
  constexpr int PER = D / 32, W = 4;
  constexpr int ROW = FMT == TREE_BF16 ? 2 * D : FMT == TREE_FP8 ? D : (D / 2 + D / 16 + 15) / 16 * 16;
  __shared__ float so[W][D], sm[W], sl[W];
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b = 0;
  while (b < a.batch && !(a.query_start[b] <= t && t < a.query_start[b + 1])) ++b;
  if (b == a.batch) return;
  const int start = a.query_start[b], n = a.query_start[b + 1] - start, i = t - start, L = a.context_lens[b];
  if (n > a.max_query || L < n || L > a.max_context_len) {
    if (threadIdx.x == 0) atomicOr(a.status, PA_DEV_BAD_LEN);
    return;
  }
  const int prefix = L - n;
  const uint64_t mask = a.tree_mask[t] & (n < 64 ? (1ull << n) - 1 : ~0ull);
  const int depth = __popcll(mask & ~(1ull << i));
  float q[PER], acc[PER] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < PER; ++e) q[e] = __uint_as_float((uint32_t)a.q[((size_t)t * a.Hq + h) * D + e * 32 + lane] << 16);
  for (int j = warp; j < L; j += W) {
    int back = prefix + depth - j;
    if (j >= prefix) {
      if (!((mask >> (j - prefix)) & 1)) continue;
      const uint64_t mj = a.tree_mask[start + j - prefix] & (n < 64 ? (1ull << n) - 1 : ~0ull);
      back = depth - __popcll(mj & ~(1ull << (j - prefix)));
    }
    if (a.window > 0 && back >= a.window) continue;
    const int page = a.block_table[(size_t)b * a.max_pages_per_seq + j / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, PA_DEV_BAD_PAGE);
      continue;
    }
    const size_t row = (((size_t)page * a.page_size + j % a.page_size) * a.Hkv + h / a.G) * ROW;
    float s = 0.f;
    for (int e = 0; e < PER; ++e) s += q[e] * cache_value<FMT, D>(a.k_pool + row, e * 32 + lane);
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    s *= a.qscale * a.kscale;
    const float mn = fmaxf(m, s), al = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * al + p;
    for (int e = 0; e < PER; ++e) acc[e] = acc[e] * al + p * cache_value<FMT, D>(a.v_pool + row, e * 32 + lane);
  }
  for (int e = 0; e < PER; ++e) so[warp][e * 32 + lane] = acc[e];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  __syncthreads();
  float M = -INFINITY, Z = 0.f;
  for (int w = 0; w < W; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < W; ++w) Z += sl[w] == 0.f ? 0.f : sl[w] * exp2f(sm[w] - M);  // a NaN stays one
  for (int d = threadIdx.x; d < D; d += 128) {
    float o = 0.f;
    for (int w = 0; w < W; ++w)
      if (sl[w] != 0.f) o += so[w][d] * exp2f(sm[w] - M);
    a.out[((size_t)t * a.Hq + h) * D + d] = (uint16_t)(pack_bf16x2(Z != 0.f ? o * a.vscale / Z : 0.f, 0.f) & 0xffffu);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(size_t)t * a.Hq + h] = Z != 0.f ? (M + log2f(Z)) * LN2 : -INFINITY;
}

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

int tree_shape(int batch, int max_query, int Hq, int Hkv, int D, int max_ctx, int P, int num_splits, size_t *total) {
  if (batch < 0 || max_query <= 0 || Hq <= 0 || Hkv <= 0 || max_ctx < 0 || num_splits < 0 || Hq % Hkv != 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (max_query > kTreeNodes || num_splits > 4096 || (D != 64 && D != 128 && D != 256) || !is_pow2(P) || P < 8 ||
      P > 256)
    return PA_ERR_UNSUPPORTED;
  *total = sizeof(WsHeader);
  return PA_OK;
}

int tree_call(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
              const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask, void *out, float *lse,
              int batch, int tokens, int max_query, int Hq, int Hkv, int D, int P, int num_pages, int max_pages,
              int max_ctx, float scale, int fmt, float k_scale, float v_scale, int window, int num_splits, void *workspace,
              size_t workspace_bytes, cudaStream_t stream) {
  note_launches(0);
  size_t need = 0;
  const int rc = tree_shape(batch, max_query, Hq, Hkv, D, max_ctx, P, num_splits, &need);
  if (rc != PA_OK) return rc;
  if (tokens < 0 || num_pages <= 0 || max_pages <= 0 || !std::isfinite(scale)) return PA_ERR_INVALID_ARGUMENT;
  if (fmt != TREE_BF16 && !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARGUMENT;
  if ((long long)max_pages * P < (long long)max_ctx) return PA_ERR_INVALID_ARGUMENT;
  if (batch == 0 || tokens == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !block_table || !context_lens || !query_start || !tree_mask || !out || !workspace)
    return PA_ERR_INVALID_ARGUMENT;
  const void *vecs[] = {q, k_pool, v_pool, out, workspace};
  for (const void *p : vecs)
    if (!aligned_to(p, 16)) return PA_ERR_MISALIGNED;
  const void *words[] = {block_table, context_lens, query_start, lse};
  for (const void *p : words)
    if (!aligned_to(p, 4)) return PA_ERR_MISALIGNED;
  if (!aligned_to(tree_mask, 8)) return PA_ERR_MISALIGNED;
  if (workspace_bytes < need) return PA_ERR_WORKSPACE_TOO_SMALL;
  TreeArgs a = {static_cast<const uint16_t *>(q), static_cast<const uint8_t *>(k_pool), static_cast<const uint8_t *>(v_pool),
                block_table, context_lens, query_start, tree_mask, static_cast<uint16_t *>(out), lse,
                &static_cast<WsHeader *>(workspace)->status, batch, tokens, max_query, Hq, Hkv, Hq / Hkv, P, num_pages,
                max_pages, max_ctx, window > 0 ? window : 0, scale * LOG2E, fmt == TREE_BF16 ? 1.f : k_scale,
                fmt == TREE_BF16 ? 1.f : v_scale};
  if (const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(WsHeader), stream); e != cudaSuccess) return cuda_fail(e);
  const dim3 grid((unsigned)tokens, (unsigned)Hq);
  auto run = [&](auto kernel) { kernel<<<grid, 128, 0, stream>>>(a); };
  if (fmt == TREE_BF16)
    D == 64 ? run(tree_plain_kernel<TREE_BF16, 64>) : D == 128 ? run(tree_plain_kernel<TREE_BF16, 128>) : run(tree_plain_kernel<TREE_BF16, 256>);
  else if (fmt == TREE_FP8)
    D == 64 ? run(tree_plain_kernel<TREE_FP8, 64>) : D == 128 ? run(tree_plain_kernel<TREE_FP8, 128>) : run(tree_plain_kernel<TREE_FP8, 256>);
  else
    D == 64 ? run(tree_plain_kernel<TREE_NVFP4, 64>) : D == 128 ? run(tree_plain_kernel<TREE_NVFP4, 128>) : run(tree_plain_kernel<TREE_NVFP4, 256>);
  if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return cuda_fail(e);
  note_launches(1);
  return PA_OK;
}

}  // namespace

}  // namespace pa

extern "C" size_t pa_tree_workspace_size(int batch, int max_query, int num_q_heads, int num_kv_heads, int head_dim,
                                         int max_context_len, int page_size, int num_splits) {
  size_t n = 0;
  return pa::tree_shape(batch, max_query, num_q_heads, num_kv_heads, head_dim, max_context_len, page_size, num_splits,
                        &n) == PA_OK
             ? n
             : 0;
}

extern "C" int pa_tree_gqa(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                           const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask,
                           void *out, float *lse, int batch, int num_tokens, int max_query, int num_q_heads,
                           int num_kv_heads, int head_dim, int page_size, int num_pages, int max_pages_per_seq,
                           int max_context_len, float scale, int window, int num_splits, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse, batch, num_tokens,
                       max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                       max_context_len, scale, pa::TREE_BF16, 1.f, 1.f, window, num_splits, workspace, workspace_bytes,
                       stream);
}

extern "C" int pa_tree_gqa_fp8(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                               const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask,
                               void *out, float *lse, int batch, int num_tokens, int max_query, int num_q_heads,
                               int num_kv_heads, int head_dim, int page_size, int num_pages, int max_pages_per_seq,
                               int max_context_len, float scale, float k_scale, float v_scale, int window,
                               int num_splits, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse, batch, num_tokens,
                       max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                       max_context_len, scale, pa::TREE_FP8, k_scale, v_scale, window, num_splits, workspace,
                       workspace_bytes, stream);
}

extern "C" int pa_tree_gqa_nvfp4(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                                 const int32_t *context_lens, const int32_t *query_start, const uint64_t *tree_mask,
                                 void *out, float *lse, int batch, int num_tokens, int max_query, int num_q_heads,
                                 int num_kv_heads, int head_dim, int page_size, int num_pages, int max_pages_per_seq,
                                 int max_context_len, float scale, float k_scale, float v_scale, int window,
                                 int num_splits, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return pa::tree_call(q, k_pool, v_pool, block_table, context_lens, query_start, tree_mask, out, lse, batch, num_tokens,
                       max_query, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                       max_context_len, scale, pa::TREE_NVFP4, k_scale, v_scale, window, num_splits, workspace,
                       workspace_bytes, stream);
}
