// pa_plan.cu -- the plan of a step (pages, block tables, slots, positions and tree masks of its new
// tokens) and the compaction of an accepted path in the paged cache.
#include <climits>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_host.h"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxBatch = 8192;
constexpr int kPlanMaxCluster = 8;  // the portable cluster size
constexpr int kTreeNodes = 64;      // nodes of a tree: bits of a mask

struct PlanArgs {
  const int32_t *context_lens, *new_lens, *held_pages;
  int32_t *free_list;
  const int32_t *free_count;
  const int32_t *parents;  // or null: chains
  int32_t *block_table, *context_lens_out, *held_pages_out, *free_count_out, *query_start;
  int64_t *slot_mapping;
  int32_t *positions;
  uint64_t *tree_mask;
  int32_t *granted;  // or null
  uint32_t *status;  // or null
  int batch, page_size, num_pages, max_pages_per_seq, max_tokens;
};

// What a CTA keeps of a row, in shared memory.  need: pages to take; PLAN_REFUSED: a row with bad lengths;
// PLAN_ENDED: its pages are given back.
struct PlanRow {
  int32_t ctx, held, start, need;
  int32_t first;  // pages needed by the rows before it
  int32_t given;  // pages given back by the rows before it
};
constexpr int32_t PLAN_REFUSED = -1, PLAN_ENDED = -2;

// All threads of the cluster's CTAs; global writes before it are visible to all of them behind it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive scan over the CTA's threads of a 64-bit and two 32-bit values; the totals in *sum.
struct PlanSums {
  long long tokens;
  int given, need;
};
template <typename T>
__device__ __forceinline__ T lanes_scan(T x) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(FULL, x, o);
    if ((int)(threadIdx.x & 31) >= o) x += u;
  }
  return x;
}
__device__ __forceinline__ PlanSums block_scan(PlanSums v, PlanSums *sum, PlanSums *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PlanSums x = {lanes_scan(v.tokens), lanes_scan(v.given), lanes_scan(v.need)};
  if (lane == 31) part[warp] = x;
  __syncthreads();
  // the warps' sums: lane w has warp w's
  const PlanSums s = lane < kPlanThreads / 32 ? part[lane] : PlanSums{0, 0, 0};
  const PlanSums p = {lanes_scan(s.tokens), lanes_scan(s.given), lanes_scan(s.need)};
  *sum = {__shfl_sync(FULL, p.tokens, 31), __shfl_sync(FULL, p.given, 31), __shfl_sync(FULL, p.need, 31)};
  const PlanSums before = {__shfl_sync(FULL, p.tokens - s.tokens, warp), __shfl_sync(FULL, p.given - s.given, warp),
                           __shfl_sync(FULL, p.need - s.need, warp)};
  __syncthreads();
  return {before.tokens + x.tokens - v.tokens, before.given + x.given - v.given, before.need + x.need - v.need};
}

struct PlanTotals {
  int count, top, total;  // free pages before; with the given ones; tokens
  int need;               // pages needed by all rows
};

// All rows into shared memory, with the sums before each (every CTA of the plan does this for itself: the
// lengths are few, and to hand the sums over would take a launch).
__device__ __forceinline__ PlanTotals plan_rows(const PlanArgs &a, PlanRow *rows, PlanSums *part, uint32_t &bad) {
  const int tid = threadIdx.x, P = a.page_size;
  const int free0 = *a.free_count;
  PlanSums sums;
  // a row's need is 0 where its tokens pass max_tokens, which only the sum of the tokens tells: the first pass
  // takes that as not so, and a second follows in the rare call where it is
  for (int pass = 0; pass < 2; ++pass) {
    sums = {0, 0, 0};
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
      const int b = b0 + tid;
      int ctx = 0, n = 0, held = 0;
      if (b < a.batch) {
        ctx = a.context_lens[b];
        n = a.new_lens[b];
        held = a.held_pages[b];
      }
      const bool ended = n < 0, held_ok = held >= 0 && held <= a.max_pages_per_seq;
      const long long add = max(n, 0);
      bool ok = ctx >= 0 && held_ok && ctx + add <= INT_MAX - P;
      const int pages = ok ? (int)(((unsigned)ctx + (unsigned)add + (unsigned)P - 1u) / (unsigned)P) : 0;  // behind this step
      ok = ok && pages <= a.max_pages_per_seq;
      if (pass > 0) ok = ok && b < a.batch && rows[b].start + add <= a.max_tokens;
      if (ended ? !held_ok : !ok) bad |= PA_DEV_BAD_LEN;
      const int need = ok && !ended ? max(pages - held, 0) : 0;
      PlanSums all;
      const PlanSums v = block_scan({add, ended && held_ok ? held : 0, need}, &all, part);
      if (b < a.batch) {
        PlanRow r;
        r.ctx = ctx;
        r.held = held_ok ? held : 0;
        r.start = (int)min(sums.tokens + v.tokens, (long long)INT_MAX);
        r.need = ended ? PLAN_ENDED : ok ? need : PLAN_REFUSED;
        r.first = sums.need + v.need;
        r.given = sums.given + v.given;
        rows[b] = r;
      }
      sums = {sums.tokens + all.tokens, sums.given + all.given, sums.need + all.need};
    }
    if (sums.tokens <= a.max_tokens) break;
  }
  PlanTotals t;
  t.count = min(max(free0, 0), a.num_pages);
  if (free0 != t.count) bad |= PA_DEV_BAD_LEN;
  if ((long long)t.count + sums.given > a.num_pages) bad |= PA_DEV_BAD_LEN;  // more pages than there are: the ones past the list are lost
  t.top = (int)min((long long)t.count + sums.given, (long long)a.num_pages);
  t.total = (int)min(sums.tokens, (long long)INT_MAX);
  t.need = sums.need;
  if (tid == 0) rows[a.batch].start = t.total;
  __syncthreads();
  return t;
}

__device__ __forceinline__ bool plan_granted(const PlanRow &r, int top) {
  return r.need == 0 || (r.need > 0 && (long long)r.first + r.need <= top);
}

// The last row with key at most x.
template <int32_t PlanRow::*key>
__device__ __forceinline__ int plan_find(const PlanRow *rows, int batch, int x) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (rows[mid].*key <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Page r of those given back, from its ended row's own table entries.
__device__ __forceinline__ int plan_given(const PlanArgs &a, const PlanRow *rows, int r) {
  const int b = plan_find<&PlanRow::given>(rows, a.batch, r);
  return a.block_table[(size_t)b * a.max_pages_per_seq + (r - rows[b].given)];
}

// Page j of the step: entry top - 1 - j of the list with the given pages on it, without waiting for anyone to have
// put them there.
__device__ __forceinline__ int plan_page(const PlanArgs &a, const PlanRow *rows, const PlanTotals &t, int j) {
  const int s = t.top - 1 - j;
  return s < t.count ? a.free_list[s] : plan_given(a, rows, s - t.count);
}

// Row b's state after the step, and with it (one row's) the count of the free pages: what may be updated in place.
// The needs are granted, in row order, up to the first that passes the list; of the refused rows only that one has
// no more than the list before it.
__device__ __forceinline__ void plan_state(const PlanArgs &a, const PlanRow *rows, const PlanTotals &t, int b) {
  const PlanRow r = rows[b];
  const bool ok = plan_granted(r, t.top), ended = r.need == PLAN_ENDED;
  a.context_lens_out[b] = ended ? 0 : ok ? r.ctx + (rows[b + 1].start - r.start) : r.ctx;
  // (a refused row keeps what it said, a bad count included)
  if (ended) a.held_pages_out[b] = 0;
  else if (ok) a.held_pages_out[b] = r.held + r.need;
  else if (a.held_pages_out != a.held_pages) a.held_pages_out[b] = a.held_pages[b];
  if (r.need > 0 && !ok && r.first <= t.top) *a.free_count_out = t.top - r.first;
}
__device__ __forceinline__ void plan_state_all_granted(const PlanArgs &a, const PlanTotals &t) {
  if (t.need <= t.top) *a.free_count_out = t.top - (int)t.need;
}

// A few thousand integers in and out, bound by the launch and by the few dependent trips to memory.  The CTAs are
// independent: each has all rows' sums, writes its share of the rows' table entries and of the tokens, and reads of
// the table and the list what no CTA writes.  Only state that is updated in place makes them meet: with few CTAs
// (PLAN_CLUSTER) at a barrier of the one cluster that they form, when all have read all of their inputs, with many
// (PLAN_AFTER) in a launch of its own behind this one.  48 rows of trees: 4.9 us; 512 rows of 1 to 1024 tokens: 6.0 us
// (one cluster of eight CTAs for those, waiting for one another's sums: 38 us); in place the first 0.4 us more, the second,
// with its second launch, 2.2.
enum PlanMode { PLAN_APART = 0, PLAN_CLUSTER = 1, PLAN_AFTER = 2 };
template <int MODE>
__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const PlanArgs a) {
  extern __shared__ PlanRow rows[];  // [batch + 1]: the last one holds the total of the tokens
  __shared__ PlanSums part[kPlanThreads / 32];
  __shared__ int8_t up[kTreeNodes - 1 + kPlanThreads];  // parents of the chunk's tokens and 63 before it
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int rank = (int)blockIdx.x, nranks = (int)gridDim.x;
  const int P = a.page_size;
  uint32_t bad = 0;
  // the chunk's parents, whose loads go along with the lengths' (entries behind the last row are not looked at)
  auto load_parents = [&](int t0) {
    for (int e = tid; e < kTreeNodes - 1 + kPlanThreads; e += kPlanThreads) {
      const int s = t0 - (kTreeNodes - 1) + e;
      const int p = s >= 0 && s < a.max_tokens ? a.parents[s] : -1;
      up[e] = (int8_t)(p < -1 || p >= kTreeNodes ? -2 : p);
    }
  };
  if (a.parents) load_parents(rank * kPlanThreads);
  const PlanTotals tot = plan_rows(a, rows, part, bad);
  const int total = tot.total;
  if constexpr (MODE == PLAN_CLUSTER) cluster_barrier();

  // rows, then the pages given back onto the list and the step's pages into the table, each a thread's
  const int first = rank * kPlanThreads + tid, stride = nranks * kPlanThreads;
  for (int b = first; b < a.batch; b += stride) {
    a.query_start[b] = rows[b].start;
    if (a.granted) a.granted[b] = plan_granted(rows[b], tot.top);
    if (rows[b].need > 0 && !plan_granted(rows[b], tot.top)) bad |= PA_DEV_NO_PAGES;
    if constexpr (MODE != PLAN_AFTER) plan_state(a, rows, tot, b);
  }
  if (first == 0) {
    a.query_start[a.batch] = total;
    if constexpr (MODE != PLAN_AFTER) plan_state_all_granted(a, tot);
  }
  for (int r = first; r < tot.top - tot.count; r += stride) {
    const int page = plan_given(a, rows, r);
    if (page < 0 || page >= a.num_pages) bad |= PA_DEV_BAD_PAGE;
    a.free_list[tot.count + r] = page;
  }
  for (int j = first; j < min(tot.need, tot.top); j += stride) {
    const int b = plan_find<&PlanRow::first>(rows, a.batch, j);
    const PlanRow r = rows[b];
    if (r.need <= 0 || !plan_granted(r, tot.top)) continue;  // behind the last page that was granted
    const int page = plan_page(a, rows, tot, j);
    if (page < 0 || page >= a.num_pages) bad |= PA_DEV_BAD_PAGE;
    a.block_table[(size_t)b * a.max_pages_per_seq + r.held + (j - r.first)] = page;
  }

  // tokens, a chunk of kPlanThreads at a time
  for (int t0 = rank * kPlanThreads; t0 < a.max_tokens; t0 += nranks * kPlanThreads) {
    const int t = t0 + tid;
    if (a.parents && t0 != rank * kPlanThreads) {
      __syncthreads();
      load_parents(t0);
      __syncthreads();
    }
    if (t >= a.max_tokens) continue;
    int64_t slot = -1;
    int pos = 0;
    uint64_t mask = 0;
    if (t < total) {
      const int lo = plan_find<&PlanRow::start>(rows, a.batch, t);
      const PlanRow r = rows[lo];
      const int i = t - r.start, n = rows[lo + 1].start - r.start;
      const long long at = (long long)r.ctx + i;
      int page = 0;
      unsigned k = 0;
      const bool ok = plan_granted(r, tot.top);
      if (ok) {  // then at < max_pages_per_seq * P, which the host keeps below 2^31
        k = (unsigned)at / (unsigned)P;
        page = (int)k < r.held ? a.block_table[(size_t)lo * a.max_pages_per_seq + k]
                               : plan_page(a, rows, tot, r.first + ((int)k - r.held));
      }
      int depth = i;
      if (a.parents && n <= kTreeNodes) {
        for (int j = i;;) {  // up the ancestors: each step goes to a smaller index
          mask |= 1ull << j;
          const int p = up[kTreeNodes - 1 + tid - i + j];
          if (p < 0 || p >= j) {
            if (p != -1) bad |= PA_DEV_BAD_TREE;
            break;
          }
          j = p;
        }
        depth = __popcll(mask) - 1;
      }
      pos = (int)min((long long)r.ctx + depth, (long long)INT_MAX);
      if (ok) {
        if (page < 0 || page >= a.num_pages) bad |= PA_DEV_BAD_PAGE;
        else slot = (int64_t)page * P + ((unsigned)at - k * (unsigned)P);
      }
    }
    a.slot_mapping[t] = slot;
    a.positions[t] = pos;
    if (a.tree_mask) a.tree_mask[t] = mask;
  }
  if (bad && a.status) atomicOr(a.status, bad);
}

__global__ void __launch_bounds__(kPlanThreads) plan_state_kernel(const PlanArgs a) {
  extern __shared__ PlanRow rows[];
  __shared__ PlanSums part[kPlanThreads / 32];
  pdl_wait();  // for the step kernel, which reads what is written here
  pdl_launch_dependents();
  uint32_t bad = 0;  // (said by the step kernel)
  const PlanTotals tot = plan_rows(a, rows, part, bad);
  for (int b = threadIdx.x; b < a.batch; b += kPlanThreads) plan_state(a, rows, tot, b);
  if (threadIdx.x == 0) plan_state_all_granted(a, tot);
}

// Accepted paths.  Block (x, y) moves 256 16-byte columns of row y: a column is one 16-byte piece of
// a token in one pool of one layer, and each thread moves its column's accepted nodes in ascending
// order, eight loads in flight (sixteen: 14.0 us for 12.2, fewer threads fit an SM).  A node's target lies
// at or before its source and behind every earlier source, so no source is overwritten before it is read.
// Bound by memory and, before it, by two dependent trips (lengths and path, pages): 48 FP8 layers of 64 rows,
// 9 nodes of 63 each, 11.8 us (4.2 TB/s read and written); one layer 2.4 us in a graph.
constexpr int kCompactThreads = 256;

struct CompactArgs {
  uint4 *k_pool, *v_pool;
  const int32_t *block_table, *context_lens, *query_start, *accepted, *num_accepted;
  const int32_t *granted;  // or null: all rows
  int32_t *context_lens_out;
  uint32_t *status;
  long long columns;      // 2 * layers * vectors per token
  long long layer_vecs;   // vectors of a layer's pool
  int vecs;               // 16-byte vectors per token
  int max_accepted, page_size, num_pages, max_pages_per_seq;
};

__global__ void __launch_bounds__(kCompactThreads) kv_compact_kernel(const CompactArgs a) {
  __shared__ long long src[kTreeNodes], dst[kTreeNodes];  // slots; -1: not moved
  __shared__ int moves;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    // the path's first 64 entries, the lengths and the count: loads that wait for nothing
    const int32_t *path = a.accepted + (size_t)b * a.max_accepted;
    const int p0 = lane < a.max_accepted ? path[lane] : 0, p1 = lane + 32 < a.max_accepted ? path[lane + 32] : 0;
    uint32_t bad = 0;
    const int L = a.context_lens[b], n = a.query_start[b + 1] - a.query_start[b];
    const bool granted = !a.granted || a.granted[b] != 0;
    int m = a.num_accepted[b];
    const long long room = (long long)a.max_pages_per_seq * a.page_size;
    // a row whose tokens are not in the cache, or that is no tree (a plan's chain of more than 64), stays as it is
    const bool whole = !granted || (n > kTreeNodes && L >= n && L <= room);
    if (whole) m = 0;
    const bool ok = whole || (n >= 0 && L >= n && L <= room && m >= 0 && m <= a.max_accepted);
    if (!ok) {
      bad |= PA_DEV_BAD_LEN;
      m = 0;
    }
    const int prefix = L - n;
    int good = 0;  // entries before the first bad one
    bool stop = false;
    int tail = -1;  // the entry before this round's first
    for (int i0 = 0; i0 < m && !stop; i0 += 32) {
      const int i = i0 + lane, p = i0 == 0 ? p0 : p1;
      const int up = __shfl_up_sync(FULL, p, 1), before = lane == 0 ? tail : up;
      tail = __shfl_sync(FULL, p, 31);
      const uint32_t wrong = __ballot_sync(FULL, i < m && (p <= before || p < 0 || p >= n));
      stop = wrong != 0;
      good = stop ? i0 + __ffs((int)wrong) - 1 : min(m, i0 + 32);
      if (i < good) {
        const int32_t *bt = a.block_table + (size_t)b * a.max_pages_per_seq;
        const int s = prefix + p, d = prefix + i;
        const int ps = bt[s / a.page_size], pd = bt[d / a.page_size];
        const bool in = ps >= 0 && ps < a.num_pages && pd >= 0 && pd < a.num_pages;
        if (!in) bad |= PA_DEV_BAD_PAGE;
        src[i] = in && s != d ? (long long)ps * a.page_size + s % a.page_size : -1;
        dst[i] = (long long)pd * a.page_size + d % a.page_size;
      }
    }
    if (stop) bad |= PA_DEV_BAD_TREE;
    if (lane == 0) {
      moves = good;
      if (blockIdx.x == 0) a.context_lens_out[b] = whole ? L : ok ? prefix + good : max(L, 0);
    }
    if (bad && a.status && blockIdx.x == 0) atomicOr(a.status, bad);
  }
  __syncthreads();
  const long long col = (long long)blockIdx.x * kCompactThreads + tid;
  if (col >= a.columns) return;
  const int e = (int)(col % a.vecs);
  const long long lp = col / a.vecs;  // layer * 2 + pool
  uint4 *pool = ((lp & 1) ? a.v_pool : a.k_pool) + (lp >> 1) * a.layer_vecs + e;
  const int m = moves;
  constexpr int U = 8;
  for (int i0 = 0; i0 < m; i0 += U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < m && src[i0 + u] >= 0) x[u] = pool[src[i0 + u] * a.vecs];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < m && src[i0 + u] >= 0) pool[dst[i0 + u] * a.vecs] = x[u];
  }
}

}  // namespace

}  // namespace pa

extern "C" int pa_plan_step(const int32_t *context_lens, const int32_t *new_lens, const int32_t *held_pages,
                            int32_t *free_list, const int32_t *free_count, const int32_t *parents,
                            int32_t *block_table, int32_t *context_lens_out, int32_t *held_pages_out,
                            int32_t *free_count_out, int32_t *query_start, int64_t *slot_mapping,
                            int32_t *positions, uint64_t *tree_mask, int batch, int page_size, int num_pages,
                            int max_pages_per_seq, int max_tokens, uint32_t *status, cudaStream_t stream) {
  return pa_plan_step_granted(context_lens, new_lens, held_pages, free_list, free_count, parents, block_table,
                              context_lens_out, held_pages_out, free_count_out, query_start, slot_mapping, positions,
                              tree_mask, nullptr, batch, page_size, num_pages, max_pages_per_seq, max_tokens, status, stream);
}

extern "C" int pa_plan_step_granted(const int32_t *context_lens, const int32_t *new_lens, const int32_t *held_pages,
                                    int32_t *free_list, const int32_t *free_count, const int32_t *parents,
                                    int32_t *block_table, int32_t *context_lens_out, int32_t *held_pages_out,
                                    int32_t *free_count_out, int32_t *query_start, int64_t *slot_mapping,
                                    int32_t *positions, uint64_t *tree_mask, int32_t *granted, int batch, int page_size,
                                    int num_pages, int max_pages_per_seq, int max_tokens, uint32_t *status,
                                    cudaStream_t stream) {
  using namespace pa;
  note_launches(0);
  if (batch < 0 || page_size <= 0 || num_pages <= 0 || max_pages_per_seq <= 0 || max_tokens < 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (batch > kPlanMaxBatch || (long long)max_pages_per_seq * page_size > INT_MAX ||
      (long long)max_pages_per_seq * batch > INT_MAX)
    return PA_ERR_UNSUPPORTED;
  if (!free_list || !free_count || !free_count_out || !query_start) return PA_ERR_INVALID_ARGUMENT;
  if (batch > 0 && (!context_lens || !new_lens || !held_pages || !block_table || !context_lens_out || !held_pages_out))
    return PA_ERR_INVALID_ARGUMENT;
  if (max_tokens > 0 && (!slot_mapping || !positions)) return PA_ERR_INVALID_ARGUMENT;
  if ((parents != nullptr) != (tree_mask != nullptr)) return PA_ERR_INVALID_ARGUMENT;
  const void *words[] = {context_lens, new_lens, held_pages, free_list, free_count, parents, block_table,
                         context_lens_out, held_pages_out, free_count_out, query_start, positions, granted, status};
  for (const void *p : words)
    if (!aligned_to(p, 4)) return PA_ERR_MISALIGNED;
  if (!aligned_to(slot_mapping, 8) || !aligned_to(tree_mask, 8)) return PA_ERR_MISALIGNED;
  // every output against every input and every other output; in place means the same array
  const size_t nb = (size_t)batch * 4, nt = (size_t)max_tokens;
  struct Range {
    const void *p;
    size_t n;
  };
  const Range in[] = {{context_lens, nb}, {held_pages, nb}, {free_count, 4}, {new_lens, nb}, {parents, parents ? nt * 4 : 0}};
  const Range out[] = {{context_lens_out, nb}, {held_pages_out, nb}, {free_count_out, 4}, {query_start, nb + 4},
                       {slot_mapping, nt * 8}, {positions, nt * 4}, {tree_mask, tree_mask ? nt * 8 : 0},
                       {block_table, (size_t)max_pages_per_seq * nb}, {free_list, (size_t)num_pages * 4},
                       {granted, granted ? nb : 0}, {status, status ? 4u : 0u}};
  constexpr int n_in = sizeof(in) / sizeof(in[0]), n_out = sizeof(out) / sizeof(out[0]);
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j) {
      const bool same = i == j && i < 3 && out[i].p == in[j].p;
      if (!same && overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return PA_ERR_INVALID_ARGUMENT;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return PA_ERR_INVALID_ARGUMENT;
  }
  PlanArgs a = {context_lens, new_lens, held_pages, free_list, free_count, parents, block_table, context_lens_out,
                held_pages_out, free_count_out, query_start, slot_mapping, positions, tree_mask, granted, status, batch,
                page_size, num_pages, max_pages_per_seq, max_tokens};
  const size_t smem = (size_t)(batch + 1) * sizeof(PlanRow);
  const int chunks = (max_tokens + kPlanThreads - 1) / kPlanThreads;
  // A CTA for each chunk of tokens and for 64 rows.  State in place: up to eight of them in one cluster, more with
  // a second launch for the state.
  const bool in_place = context_lens_out == context_lens || held_pages_out == held_pages || free_count_out == free_count;
  constexpr int kPlanMostCtas = 304;  // two on each SM
  int ctas = chunks > (batch + 63) / 64 ? chunks : (batch + 63) / 64;
  ctas = ctas < 1 ? 1 : ctas < kPlanMostCtas ? ctas : kPlanMostCtas;
  int cluster = 0;
  if (in_place && chunks <= kPlanMaxCluster) {
    for (cluster = 1; cluster < kPlanMaxCluster && cluster < ctas;) cluster *= 2;
    ctas = cluster;
  }
  auto kernel = !in_place ? plan_step_kernel<PLAN_APART> : cluster ? plan_step_kernel<PLAN_CLUSTER> : plan_step_kernel<PLAN_AFTER>;
  const bool after = in_place && !cluster;
  if (smem > 40 * 1024) {
    constexpr int most = (kPlanMaxBatch + 1) * (int)sizeof(PlanRow);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess && after) e = cudaFuncSetAttribute(plan_state_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  cudaError_t e = launch(kernel, dim3((unsigned)ctas), kPlanThreads, smem, cluster, a, stream);
  if (e == cudaSuccess && after) e = launch(plan_state_kernel, dim3(1), kPlanThreads, smem, 0, a, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launches(after ? 2 : 1);
  return PA_OK;
}

extern "C" int pa_kv_compact(void *k_pool, void *v_pool, const int32_t *block_table, const int32_t *context_lens,
                             const int32_t *query_start, const int32_t *accepted, const int32_t *num_accepted,
                             int32_t *context_lens_out, int num_layers, int batch, int max_accepted, int token_bytes,
                             int page_size, int num_pages, int max_pages_per_seq, uint32_t *status,
                             cudaStream_t stream) {
  return pa_kv_compact_granted(k_pool, v_pool, block_table, context_lens, query_start, accepted, num_accepted, nullptr,
                               context_lens_out, num_layers, batch, max_accepted, token_bytes, page_size, num_pages,
                               max_pages_per_seq, status, stream);
}

extern "C" int pa_kv_compact_granted(void *k_pool, void *v_pool, const int32_t *block_table, const int32_t *context_lens,
                                     const int32_t *query_start, const int32_t *accepted, const int32_t *num_accepted,
                                     const int32_t *granted, int32_t *context_lens_out, int num_layers, int batch,
                                     int max_accepted, int token_bytes, int page_size, int num_pages,
                                     int max_pages_per_seq, uint32_t *status, cudaStream_t stream) {
  using namespace pa;
  note_launches(0);
  if (num_layers <= 0 || batch < 0 || token_bytes <= 0 || page_size <= 0 || num_pages <= 0 || max_pages_per_seq <= 0 ||
      max_accepted <= 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (token_bytes % 16 != 0 || max_accepted > kTreeNodes || batch > 65535 ||
      (long long)max_pages_per_seq * page_size > INT_MAX)
    return PA_ERR_UNSUPPORTED;
  if (batch == 0) return PA_OK;
  if (!k_pool || !v_pool || !block_table || !context_lens || !query_start || !accepted || !num_accepted ||
      !context_lens_out)
    return PA_ERR_INVALID_ARGUMENT;
  if (!aligned_to(k_pool, 16) || !aligned_to(v_pool, 16)) return PA_ERR_MISALIGNED;
  const void *words[] = {block_table, context_lens, query_start, accepted, num_accepted, granted, context_lens_out, status};
  for (const void *p : words)
    if (!aligned_to(p, 4)) return PA_ERR_MISALIGNED;
  const size_t nb = (size_t)batch * 4;
  const size_t pool = (size_t)num_layers * num_pages * page_size * token_bytes;
  if (overlap(context_lens_out, nb, context_lens, nb) || overlap(context_lens_out, nb, query_start, nb + 4) ||
      overlap(context_lens_out, nb, num_accepted, nb) || overlap(context_lens_out, nb, accepted, nb * max_accepted) ||
      overlap(context_lens_out, nb, block_table, nb * max_pages_per_seq) ||
      overlap(context_lens_out, nb, granted, granted ? nb : 0) || overlap(k_pool, pool, v_pool, pool))
    return PA_ERR_INVALID_ARGUMENT;
  CompactArgs a;
  a.k_pool = static_cast<uint4 *>(k_pool);
  a.v_pool = static_cast<uint4 *>(v_pool);
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.accepted = accepted;
  a.num_accepted = num_accepted;
  a.granted = granted;
  a.context_lens_out = context_lens_out;
  a.status = status;
  a.vecs = token_bytes / 16;
  a.columns = 2ll * num_layers * a.vecs;
  a.layer_vecs = (long long)num_pages * page_size * a.vecs;
  a.max_accepted = max_accepted;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages_per_seq = max_pages_per_seq;
  const long long gx = (a.columns + kCompactThreads - 1) / kCompactThreads;
  if (gx > INT_MAX) return PA_ERR_UNSUPPORTED;
  if (const cudaError_t e = launch(kv_compact_kernel, dim3((unsigned)gx, (unsigned)batch), kCompactThreads, 0, 0, a, stream);
      e != cudaSuccess)
    return cuda_fail(e);
  note_launches(1);
  return PA_OK;
}
