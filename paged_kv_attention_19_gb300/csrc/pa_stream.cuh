// pa_stream.cuh -- attention of each row's newest tokens over its paged cache, in a window beside which the row's first
// tokens stay visible.
//
// Mathematics.  The query at position p attends to A = {t <= p : t > p - window or t < first}:
//   out = sum_{t in A} exp(s_t - m) v_t / l,  lse = m + ln l,  s_t = scale q . k_t,  m = max s_t,  l = sum exp(s_t - m).
#pragma once

#include "pa_tree.cuh"

namespace pa {

struct StreamArgs {
  const uint8_t *q, *k_pool, *v_pool;
  const int32_t *block_table, *context_lens, *query_start;
  const int32_t *granted;  // or null: all rows
  uint16_t *out;
  float *lse;  // or null
  uint32_t *status;
  int batch, tokens, max_query, Hq, Hkv, G;
  int log2_page, num_pages, max_pages_per_seq, max_context_len;
  int window, first;  // window 0: none
  float scale, kscale, vscale;
};

// A block for one token and query head: four warps, each with 32 tokens at a time (a lane's product each), a running
// maximum and sum, and the output's values spread over the lanes; merged at the end.
template <int D, int FMT>
__global__ void __launch_bounds__(128) stream_rows_kernel(const StreamArgs a) {
  __shared__ float q[D], m_w[4], l_w[4], o_w[4][D];
  const int t = blockIdx.x, head = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  // the token's row: the last one that starts at or before it
  int b = -1, n = 0, L = 0;
  for (int i = 0; i < a.batch; ++i) {
    const int s = a.query_start[i], e = a.query_start[i + 1];
    if (a.granted && a.granted[i] == 0) continue;
    const int len = a.context_lens[i];
    if (s < 0 || e < s || e > a.tokens || e - s > a.max_query || len < e - s || len > a.max_context_len) {
      if (threadIdx.x == 0) atomicOr(a.status, PA_DEV_BAD_LEN);
      continue;
    }
    if (t >= s && t < e) {
      b = i;
      n = e - t;  // tokens from this one on
      L = len;
    }
  }
  if (b < 0) return;
  const int p = L - n, lo = a.window > 0 ? max(p - a.window + 1, 0) : 0, first = min(a.first, lo);
  constexpr int ROWB = tree_row_bytes(FMT, D);
  const int g = head / a.G;
  const uint16_t *qr = reinterpret_cast<const uint16_t *>(a.q) + ((size_t)t * a.Hq + head) * D;
  for (int d = threadIdx.x; d < D; d += 128) q[d] = __uint_as_float((uint32_t)qr[d] << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  const int count = first + (p + 1 - lo);
  auto row = [&](int i) -> long long {  // the i-th visible token's place in the pools, or -1
    const int tok = i < first ? i : lo + (i - first);
    const int page = a.block_table[(size_t)b * a.max_pages_per_seq + (tok >> a.log2_page)];
    if (page < 0 || page >= a.num_pages) return -1;
    return ((((long long)page << a.log2_page) + (tok & ((1 << a.log2_page) - 1))) * a.Hkv + g) * ROWB;
  };
  for (int i0 = warp * 32; i0 < count; i0 += 128) {
    const long long at = i0 + lane < count ? row(i0 + lane) : -1;
    if (i0 + lane < count && at < 0) atomicOr(a.status, PA_DEV_BAD_PAGE);
    float s = -INFINITY;
    if (at >= 0) {
      s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(q[d], cache_value<FMT, D>(a.k_pool + at, d), s);
      s *= a.scale * a.kscale * LOG2E;
    }
    float mx = s;
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, x));
    if (__any_sync(FULL, s != s)) mx = NAN;
    const float mn = mx != mx ? mx : fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float al = m == -INFINITY ? 0.f : fast_exp2(m - mn), w = at >= 0 ? fast_exp2(s - mn) : 0.f;
    m = mn;
    l = l * al + w;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] *= al;
    for (int j = 0; j < 32; ++j) {
      const long long aj = __shfl_sync(FULL, at, j);
      const float wj = __shfl_sync(FULL, w, j);
      if (aj < 0) continue;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] = fmaf(wj, cache_value<FMT, D>(a.v_pool + aj, 32 * e + lane), o[e]);
    }
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(FULL, l, x);
  if (lane == 0) {
    m_w[warp] = m;
    l_w[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o_w[warp][32 * e + lane] = o[e];
  __syncthreads();
  float M = -INFINITY, Z = 0.f;
  for (int w = 0; w < 4; ++w) M = m_w[w] != m_w[w] ? m_w[w] : fmaxf(M, m_w[w]);
  float f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = m_w[w] == -INFINITY ? 0.f : fast_exp2(m_w[w] - M);
    Z += f[w] * l_w[w];
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w)
      if (f[w] != 0.f) x += f[w] * o_w[w][d];
    x = Z == 0.f ? 0.f : x * a.vscale / Z;
    a.out[((size_t)t * a.Hq + head) * D + d] = (uint16_t)pack_bf16x2(x, 0.f);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(size_t)t * a.Hq + head] = Z == 0.f ? -INFINITY : (M + __log2f(Z)) * LN2;
}

}  // namespace pa
