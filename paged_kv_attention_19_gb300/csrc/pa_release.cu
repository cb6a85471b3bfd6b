// pa_release.cu -- pages that a window has left behind go back to the free list.
#include <climits>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_host.h"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kReleaseThreads = 512;
constexpr int kReleaseMaxBatch = 8192;
constexpr int kReleaseMaxCluster = 8;  // the portable cluster size
constexpr int kReleaseMostCtas = 152;

struct ReleaseArgs {
  const int32_t *context_lens, *held_pages, *window_start;
  const int32_t *ended;  // or null
  int32_t *free_list;
  const int32_t *free_count;
  const int32_t *block_table;
  int32_t *context_lens_out, *held_pages_out, *window_start_out, *free_count_out, *block_table_out;
  uint32_t *status;  // or null
  int batch, page_size, num_pages, max_pages_per_seq, window;
  int kept;  // pages of the first tokens
};

// What a row gives back: its pages [0, part) and then those from `from` on; `before`: how many the rows before it give.
struct ReleaseRow {
  int32_t before, part, from;
};

struct ReleaseState {  // of a row after the step
  int32_t ctx, held, start;
};

// Row b: its pages to give back in *r (`before` aside), how many they are, and its state after the step.
__device__ __forceinline__ int release_row(const ReleaseArgs &a, int b, ReleaseRow *r, ReleaseState *s, uint32_t &bad) {
  *s = {a.context_lens[b], a.held_pages[b], a.window_start[b]};
  const bool ended = a.ended && a.ended[b] != 0;
  *r = {0, 0, 0};
  if (s->ctx < 0 || s->held < 0 || s->held > a.max_pages_per_seq || s->start < 0 || s->start > s->held) {
    bad |= PA_DEV_BAD_LEN;
    return 0;
  }
  if (ended) {
    const int gone = max(s->start - a.kept, 0), held = s->held;  // (then kept < start <= held)
    r->part = gone > 0 ? a.kept : held;
    r->from = s->start;
    *s = {0, 0, 0};
    return held - gone;
  }
  const int behind = min(max(s->ctx - (a.window - 1), 0) / a.page_size, s->held);
  r->from = max(a.kept, s->start);
  if (behind <= r->from) return 0;
  s->start = behind;
  return behind - r->from;
}

__device__ __forceinline__ int release_scan(int v, int *total, int *part) {  // exclusive, over the CTA's threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += u;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int s = lane < kReleaseThreads / 32 ? part[lane] : 0, p = s;
#pragma unroll
  for (int o = 1; o < kReleaseThreads / 32; o <<= 1) {
    const int u = __shfl_up_sync(FULL, p, o);
    if (lane >= o) p += u;
  }
  *total = __shfl_sync(FULL, p, kReleaseThreads / 32 - 1);
  const int before = __shfl_sync(FULL, p - s, warp);
  __syncthreads();
  return before + x - v;
}

// Integers in and out, bound by the launch and three dependent trips to memory (lengths, entries, list).  Each CTA has all
// rows' counts from one scan of its own and moves its share of the pages, flat over the grid; no CTA waits for
// another's sums.  Only state that is updated in place makes them meet, at a barrier of the one cluster that they
// then form, when all have read it.  Measured: 512 rows of a decode step 3.1 us, 64 rows that give back 7367 pages 3.2 us.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kReleaseThreads) release_kernel(const ReleaseArgs a) {
  extern __shared__ ReleaseRow rows[];  // [batch]
  __shared__ int part[kReleaseThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, first = (int)blockIdx.x * kReleaseThreads + tid, stride = (int)gridDim.x * kReleaseThreads;
  uint32_t bad = 0;
  const int free0 = *a.free_count;
  int total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kReleaseThreads) {
    const int b = b0 + tid;
    ReleaseRow r = {0, 0, 0};
    ReleaseState s;
    const int n = b < a.batch ? release_row(a, b, &r, &s, bad) : 0;
    int sum;
    r.before = total + release_scan(n, &sum, part);
    total += sum;
    if (b < a.batch) rows[b] = r;
  }
  const int count = min(max(free0, 0), a.num_pages), room = a.num_pages - count;
  if (count != free0 || total > room) bad |= PA_DEV_BAD_LEN;
  __syncthreads();
  for (int j = first; j < total; j += stride) {
    int lo = 0, hi = a.batch - 1;  // the last row with `before` at most j
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (rows[mid].before <= j) lo = mid;
      else hi = mid - 1;
    }
    const ReleaseRow r = rows[lo];
    const int i = j - r.before, k = i < r.part ? i : r.from + (i - r.part);
    const size_t at = (size_t)lo * a.max_pages_per_seq + k;
    const int page = a.block_table[at];
    if (page < 0 || page >= a.num_pages) bad |= PA_DEV_BAD_PAGE;
    if (j < room) a.free_list[count + j] = page;
    a.block_table_out[at] = -1;
  }
  // the states: all rows' are read, by everybody, before any is written
  // (a state depends on its own row alone, so its thread reads it again behind the barrier, just before it writes it)
  if constexpr (IN_PLACE) asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int b = first; b < a.batch; b += stride) {
    ReleaseRow r;
    ReleaseState s;
    uint32_t again = 0;
    release_row(a, b, &r, &s, again);
    a.context_lens_out[b] = s.ctx;
    a.held_pages_out[b] = s.held;
    a.window_start_out[b] = s.start;
  }
  if (first == 0) *a.free_count_out = count + min(total, room);
  if (bad && a.status) atomicOr(a.status, bad);
}

}  // namespace

}  // namespace pa

extern "C" int pa_release_pages(const int32_t *context_lens, const int32_t *held_pages, const int32_t *window_start,
                                const int32_t *ended, int32_t *free_list, const int32_t *free_count,
                                const int32_t *block_table, int32_t *context_lens_out, int32_t *held_pages_out,
                                int32_t *window_start_out, int32_t *free_count_out, int32_t *block_table_out,
                                int batch, int page_size, int num_pages, int max_pages_per_seq, int window, int first,
                                uint32_t *status, cudaStream_t stream) {
  using namespace pa;
  note_launches(0);
  if (batch < 0 || page_size <= 0 || num_pages <= 0 || max_pages_per_seq <= 0 || window <= 0 || first < 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (batch > kReleaseMaxBatch || (long long)max_pages_per_seq * page_size > INT_MAX ||
      (long long)max_pages_per_seq * batch > INT_MAX)
    return PA_ERR_UNSUPPORTED;
  if (!free_list || !free_count || !free_count_out) return PA_ERR_INVALID_ARGUMENT;
  if (batch > 0 && (!context_lens || !held_pages || !window_start || !block_table || !context_lens_out || !held_pages_out ||
                    !window_start_out || !block_table_out))
    return PA_ERR_INVALID_ARGUMENT;
  const void *words[] = {context_lens, held_pages, window_start, ended, free_list, free_count, block_table, context_lens_out,
                         held_pages_out, window_start_out, free_count_out, block_table_out, status};
  for (const void *p : words)
    if (!aligned_to(p, 4)) return PA_ERR_MISALIGNED;
  // every output against every input and every other output; in place means the same array
  const size_t nb = (size_t)batch * 4, nt = (size_t)max_pages_per_seq * nb;
  struct Range {
    const void *p;
    size_t n;
  };
  const Range in[] = {{context_lens, nb}, {held_pages, nb}, {window_start, nb}, {free_count, 4}, {block_table, nt}, {ended, ended ? nb : 0}};
  const Range out[] = {{context_lens_out, nb}, {held_pages_out, nb}, {window_start_out, nb}, {free_count_out, 4},
                       {block_table_out, nt}, {free_list, (size_t)num_pages * 4}, {status, status ? 4u : 0u}};
  constexpr int n_in = sizeof(in) / sizeof(in[0]), n_out = sizeof(out) / sizeof(out[0]);
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j) {
      const bool same = i == j && i < 5 && out[i].p == in[j].p;
      if (!same && overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return PA_ERR_INVALID_ARGUMENT;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return PA_ERR_INVALID_ARGUMENT;
  }
  const int kept = (int)(((long long)first + page_size - 1) / page_size);
  const ReleaseArgs a = {context_lens, held_pages, window_start, ended, free_list, free_count, block_table, context_lens_out,
                         held_pages_out, window_start_out, free_count_out, block_table_out, status, batch, page_size, num_pages,
                         max_pages_per_seq, window, kept};
  const bool in_place = context_lens_out == context_lens || held_pages_out == held_pages || window_start_out == window_start ||
                        free_count_out == free_count;
  // a CTA for each 64 rows and for each 4096 pages that the table can name
  const long long pages = ((long long)batch * max_pages_per_seq + 4095) / 4096, most = in_place ? kReleaseMaxCluster : kReleaseMostCtas;
  int ctas = (int)(pages > (batch + 63) / 64 ? (pages < most ? pages : most) : (batch + 63) / 64);
  ctas = ctas < 1 ? 1 : ctas < (int)most ? ctas : (int)most;
  int cluster = 0;
  if (in_place) {
    for (cluster = 1; cluster < ctas;) cluster *= 2;
    ctas = cluster;
  }
  auto kernel = in_place ? release_kernel<true> : release_kernel<false>;
  const size_t smem = (size_t)batch * sizeof(ReleaseRow);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kReleaseMaxBatch * (int)sizeof(ReleaseRow));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  const cudaError_t e = launch(kernel, dim3((unsigned)ctas), kReleaseThreads, smem, cluster, a, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launches(1);
  return PA_OK;
}
