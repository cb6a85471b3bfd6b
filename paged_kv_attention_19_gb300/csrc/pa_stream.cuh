// pa_stream.cuh -- attention of each row's newest tokens -- one, a chunk or a whole prompt -- over its paged cache, in a
// window beside which the row's first tokens stay visible, on the 5th-generation tensor cores (sm_103a).
//
// Mathematics.  The query at position p attends to A = {t <= p : t > p - window or t < first}:
//   out = sum_{t in A} exp(s_t - m) v_t / l,  lse = m + ln l,  s_t = scale q . k_t,  m = max s_t,  l = sum exp(s_t - m).
// One pass over the keys with a running maximum and sum in fp32; the maximum is only raised when it grows by more than
// 2^8, so the weights stay below 2^8 and are rounded once, as the operand of the second product (bf16, half a step
// 2^-8 of each weight, or f16, 2^-11; the sum l is of the unrounded ones).
//
// What bounds it.  A key head's 128 (or, in pairs of tiles, 256) query rows -- tokens x the G heads that share it -- read a key
// and a value once: 4 D flops a row for 4 D bytes (bf16).  Single tokens are bound by memory, chunks and prompts by the tensor
// cores, and by the weights on the way between the two products.
//
// Work.  An item is (row, key head, pair of tiles); a pair's keys are those that some query of it sees: a run of the row's
// first tokens and a run that ends at its last query.  The items of all rows are laid end to end, each with its number of
// tokens and a fixed cost, and the line is cut into equal shares, one for each group of hg CTAs: long rows are split, short ones
// share a CTA, whatever the mix.  CTA r of a group serves key head r of its share, so that the key heads' parts of a page are
// read at the same time; where the number of key heads would leave CTAs idle a group is one CTA and the line holds all heads.
// Where an item lies on the line is known in closed form, so a CTA finds its own without walking the others.
// Only a CTA's first and last pieces can be part of an item that another CTA also touches: at most two partial results each.
//
// Roles of a CTA (one per SM):
//   * warp 3: the K and V tiles of a stage (64 or 128 tokens) into two rings of slots (TMA, 128-byte swizzle); its quarter of the SM
//     has no softmax warp that works where a tile has up to 96 rows, as single tokens' do;
//   * warps 1 and 2, one thread each: the products of softmax group x = 0, 1.  With two tiles thread x takes tile x of every
//     stage; with one tile the threads take alternate stages of the same rows, by their parity, and the two outputs are
//     merged at the end of the piece, which then has an even number of stages: the last may be without tokens;
//   * warp 0: the query tiles of each piece; and looks over V tiles that hold tokens which not every query sees before they
//     are used: a token that nobody sees becomes zero, and infinities and NaN of the others are taken out of the product
//     and handed to the queries that do see them (0 x inf must not reach the ones that do not);
//   * FP8 and NVFP4 pools: the tiles of codes land in a ring of their own, and eight more warps convert them to f16 operands
//     (exact; four warps K tiles, four V tiles), and the query rows, scaled by a power of two each, in place; those of
//     the V tiles then look them over;
//   * two groups of four warps: one thread per score row.
// Tensor memory: scores at 0 (the weights over a half of their buffer), outputs at 256.  At head_dim 256 one output fills
// the rest: one tile, one softmax group and one issuing thread.
//
// Measured (head_dim 128; per call, calls back to back, inputs in turn).  bf16: a prompt of 8192 tokens x 32 heads 470 us (1.17 PFLOP/s,
// 62 % of the measured 1886 TFLOP/s; a stage of two tiles takes 3640 cycles for 2048 of products, tensor pipe 45 % at 4096 tokens);
// 32 single tokens x 64 heads, 128 to 16384 tokens in a window of 4096 + 128, 60 us (266 MB, 4.4 TB/s; 30500 of 103000 cycles
// before the first weights).  The same shape over FP8, without a window, 89 us, issue slots 38 %.  NVFP4: 64 x 32 heads to 32768 tokens 189 us,
// issue slots 44 %.  Over codes at head_dim 64 (where 96 registers a thread spill 132 to 164 bytes) 32 x 64 heads to 16384 tokens 72 us, FP8
// and NVFP4 alike; at head_dim 256 32 x 32 heads 90 and 88.
#pragma once

#include "pa_tree.cuh"

namespace pa {

struct StreamArgs {
  const uint8_t *v_pool;
  const int32_t *block_table, *context_lens, *query_start;
  const int32_t *granted;  // or null: all rows
  uint16_t *out;
  float *lse;              // or null
  uint32_t *cta_status;    // [nparts]: PA_DEV_* bits
  float *part_o;           // [nparts, 2, D / 4, QT * 128, 4]: rows beside each other, so that a warp's stores are whole lines
  float *part_lse;         // [nparts, 2, QT * 128], log2 units
  struct StreamHalf *halves;  // [nparts, 2, 128]: the groups' halves of a one-tile piece
  int batch, tokens, max_query, Hq, Hkv, G;
  int qt, q2;              // queries of a tile (each with its G heads), and of a pair
  int log2_page, log2_bh, num_pages, max_pages_per_seq, max_context_len;
  int window, first;       // window 0: none
  int piece_cost, whole, log2_share, nparts;  // (in tokens)
  int single;              // no row has more than one pair
  int hg, hl;              // CTAs of a group, one for each of hg key heads; key heads of a group's line (hg hl = Hkv)
  float qscale;            // scale * log2(e) (* the keys' scale)
  float vscale;
};

struct StreamHalf {  // one row's state in one softmax group, for the merge of a one-tile piece
  float m, l;
};

// Tokens of a stage: what two groups' scores, or four buffers of one group's, have room for in the tensor memory beside the
// outputs; with pairs of tiles over codes half of that, or the shared memory would hold one tile of codes of each kind only
// (head_dim 128: FP8 chunks 673 us for 635, NVFP4 286 for 255).
constexpr int stream_stage(int D, int fmt, int QT) { return D == 256 || (D == 128 && fmt != TREE_BF16 && QT == 2) ? 64 : 128; }

template <int D_, int FMT_, int QT_>
struct StreamCfg {
  static constexpr int D = D_, FMT = FMT_, QT = QT_;
  static constexpr bool QUANT = FMT != TREE_BF16;  // codes in the cache, f16 operands
  static constexpr int ROWB = tree_row_bytes(FMT, D);
  static constexpr int GROUPS = D <= 128 ? 2 : 1;  // softmax groups, and output regions
  static constexpr int BN = stream_stage(D, FMT, QT);
  static constexpr int NB = 256 / BN;              // score buffers
  static constexpr int BACK = NB / GROUPS;         // of each issuing thread
  static constexpr int NPL = D / 64;               // 128-byte swizzle planes of a row
  // a tile: groups of 8 tokens, of each the planes' 8 rows one plane after the other, so that one copy brings all planes of a unit
  static constexpr int PLANE = 1024, GROUP = NPL * PLANE, SLOT = BN / 8 * GROUP, QPLANE = kTreeRows * 128;
  static constexpr int Q_BYTES = QT * NPL * QPLANE;
  static constexpr int ROOM = 229376 - Q_BYTES;
  // codes: up to eight slots of a tile each, copied in order K, V, K, V...; operands converted from them
  static constexpr int RAW_SLOT = QUANT ? (BN * ROWB + 1023) / 1024 * 1024 : 0;
  static constexpr int NS_QUANT = D == 64 ? 8 : D == 128 ? (QT == 1 ? 4 : 6) : 3;
  static constexpr int NR_FIT = QUANT ? (ROOM - NS_QUANT * SLOT) / (RAW_SLOT > 0 ? RAW_SLOT : 1) : 0;
  static constexpr int NR = (NR_FIT < 8 ? NR_FIT : 8) & ~1;  // (even: a slot holds tiles of one kind)
  static constexpr int NS_FIT = QUANT ? NS_QUANT : ROOM / SLOT < 12 ? ROOM / SLOT : 12;
  // Two rings of slots: a K tile is free after the scores of its stage, a V tile later.  Copies complete out of order,
  // and a wait for a phase of a slot must not come before the phase before it is known to be complete, so whoever
  // waits for the tiles of one kind, or of one parity of the stages, needs slots that hold those only.
  static constexpr int NK = GROUPS == 1 ? NS_FIT / 2 : NS_FIT / 4 * 2;
  static constexpr int NV = GROUPS == 1 ? NS_FIT - NK : (NS_FIT - NK) / 2 * 2, NS = NK + NV;
  static constexpr int SOFTMAX_WARPS = 4 * GROUPS;
  static constexpr int CONVERT_WARPS = QUANT ? 8 : 0;
  static constexpr int TILE_WARPS = CONVERT_WARPS / 2;           // half of them for K tiles, half for V tiles
  static constexpr int CLEAN_WARPS = QUANT ? TILE_WARPS : 1;     // warps that look over the V tiles
  static constexpr int THREADS = (4 + SOFTMAX_WARPS + CONVERT_WARPS) * 32;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
  // (formats 0: f16 operands)
  static constexpr uint32_t IDESC_F16 = QUANT ? (1u << 7) | (1u << 10) : 0u;
  static constexpr uint32_t IDESC_S = tc_idesc_bf16(kTreeRows, BN, false) & ~IDESC_F16;
  static constexpr uint32_t IDESC_PV = tc_idesc_bf16(kTreeRows, D, true) & ~IDESC_F16;
  // the maximum is raised when it grows by more than 2^TAU; f16 weights are 2^LIFT times as large: below 2^15, and one of
  // 2^-21 of the largest still has all its bits (its step is 2^-24, so none is off by more than 2^-32 of the largest)
  static constexpr float TAU = 8.f, LIFT = QUANT ? 7.f : 0.f, WEIGHTS = QUANT ? 32768.f : 256.f;  // 2^(LIFT + TAU)
  // score buffer of item i of group (issuing thread) x, and the parity of its use
  __host__ __device__ static constexpr uint32_t buffer(int x, uint32_t i) {
    return GROUPS == 2 ? (uint32_t)x + 2 * (i % BACK) : i % BACK;
  }
  __host__ __device__ static constexpr uint32_t buffer_phase(uint32_t i) { return (i / BACK) & 1; }
  // the weights in a score buffer: of 128 scores over the second half, which is in registers when they are written
  static constexpr uint32_t P_AT = BN == 128 ? 64 : 0;
  // with one buffer a half of an item's weights is handed over by itself, so that its product runs beside the rest
  static constexpr bool HALVES = BACK == 1;
  // and the groups take turns at the exponentials: in step they would share the units for them and then both wait for the products
  // (prompt 470 us for 476 without, chunks 782 for 790)
  static constexpr bool TURNS = BACK == 1 && QT == 2;
  // registers a thread: what the softmax warps hold of a row and its output does not fit the launch's share
  // (384 x 168 or 640 x 96), so the other warps hand some over
  static constexpr bool REG_SPLIT = GROUPS == 2;
  static constexpr int REGS = QUANT ? 96 : 168;
  static constexpr int REGS_CONTROL = QUANT ? 72 : 104, REGS_SOFTMAX = QUANT ? 128 : 200, REGS_CONVERT = 72;
  static_assert(!REG_SPLIT || 128 * REGS_CONTROL + 256 * REGS_SOFTMAX + 32 * CONVERT_WARPS * REGS_CONVERT <= THREADS * REGS,
                "the register split stays within the launch's registers");
  static constexpr int META = 16;  // stage records kept: a record is rewritten sixteen stages later, once the K tile of a
                                   // stage at least six later is free, and with that its own softmax long done
  static_assert(NK >= 1 && NK + NR / 2 <= 10 && (GROUPS == 1 || NK % 2 + NV % 2 == 0), "rings within the records");
  static_assert(QT <= GROUPS, "two tiles need two groups");
  static_assert(NB * BN <= 256 && GROUPS * D <= 256, "tensor-memory budget");
};

struct alignas(16) StreamPieceRec {  // written by the query warp before the piece's query is announced
  int32_t end, stages, two, slot;    // stages with tokens; slot: -1 whole item, else partial slot
  int32_t b, pos0, nq, tok0;         // position and packed index of the pair's first query; its queries
  int32_t g, lo_min, lo_max, pad;    // key head; first token in the window of the pair's first and of its last query
};
static_assert(sizeof(StreamPieceRec) == 48, "records of 16-byte words");

constexpr int kStreamBits = 8;  // words of the set of a pair's partly seen tokens: fewer than 256 queries
struct StreamMisc {
  uint32_t status, tmem;
  int32_t npieces, pad;
  TreePart part;
};

template <class C>
struct StreamSmem {
  static constexpr int OFF_RING = C::Q_BYTES;
  static constexpr int OFF_RAW = OFF_RING + C::NS * C::SLOT;
  static constexpr int OFF_META = OFF_RAW + C::NR * C::RAW_SLOT;
  static constexpr int OFF_PIECE = OFF_META + C::META * (int)sizeof(TreeStage);       // [2]
  // sets of tokens with infinities or NaN, of the last four pieces: behind the first query, and at the window's edge
  static constexpr int OFF_SET = OFF_PIECE + 2 * (int)sizeof(StreamPieceRec);         // [4][2][kStreamBits]
  // full[NS], empty[NS], clean[META], q_full, q_empty, s_full[NB], p_ready[NB], pv_done[NB], o_free, half[2], drain[2],
  // q_conv, p_half[2], pv_half[2], turn[2][4], raw_full[NR], raw_empty[NR]
  static constexpr int OFF_BAR = OFF_SET + 4 * 2 * kStreamBits * 4;
  static constexpr int NBAR = 2 * C::NS + C::META + 20 + 3 * C::NB + 2 * C::NR;
  static constexpr int OFF_SHIFT = OFF_BAR + NBAR * 8;  // int8 [2][QT * 128]: exponents of the query rows' scales
  static constexpr int OFF_MISC = (OFF_SHIFT + (C::QUANT ? 2 * C::QT * kTreeRows : 0) + 7) & ~7;
  static constexpr int BYTES = OFF_MISC + (int)sizeof(StreamMisc) + 1024;
  static_assert(BYTES <= 232448, "fits the 227 KB opt-in shared memory of one CTA");
};

// ---------------------------------------------------------------------------------------- rows, items

struct StreamRow {
  int start, n, L;  // n = 0: nothing to do
};

// Row b, its lengths checked: a bad row has no queries and sets PA_DEV_BAD_LEN; one that was not granted has none.  (From L2: the
// combine kernel reads them before the grids that come before it are known to it as complete.)
__device__ __forceinline__ StreamRow stream_row(const StreamArgs &a, int b, uint32_t *bad) {
  StreamRow r;
  r.start = __ldcg(a.query_start + b);
  r.L = __ldcg(a.context_lens + b);
  const int end = __ldcg(a.query_start + b + 1);
  r.n = end - r.start;
  if (a.granted && __ldcg(a.granted + b) == 0) {  // (whatever its lengths say)
    r.n = 0;
  } else if (r.start < 0 || end < r.start || end > a.tokens || r.n > a.max_query || r.L < r.n || r.L > a.max_context_len) {
    *bad |= PA_DEV_BAD_LEN;
    r.n = 0;
  }
  return r;
}

__device__ __forceinline__ int stream_pairs(const StreamArgs &a, const StreamRow &r) {
  return a.single ? r.n > 0 : (int)(((unsigned)r.n + (unsigned)a.q2 - 1u) / (unsigned)a.q2);
}

// Cost of the first p pairs of a row.  Pair i has the tokens up to its last query, less those behind its window and the first
// ones: hi - max(0, A + i q2) with hi = prefix + min((i + 1) q2, n), A = prefix + 1 - window - first.
__device__ __forceinline__ long long stream_cost(const StreamArgs &a, const StreamRow &r, int p) {
  if (p <= 0) return 0;
  if (a.single)
    return (long long)a.piece_cost + r.L - (a.window > 0 ? max(0ll, (long long)(r.L - r.n + 1 - a.window) - a.first) : 0ll);
  const long long prefix = r.L - r.n, q2 = a.q2, P = p;
  long long c = P * (a.piece_cost + prefix) + q2 * (P * (P + 1) / 2);
  c -= max(0ll, P * q2 - r.n);  // (the last pair's queries)
  if (a.window > 0) {
    const long long A = prefix + 1 - a.window - a.first;
    const long long i0 = A > 0 ? 0 : (long long)((unsigned)(-A) / (unsigned)a.q2) + 1;  // the first pair that leaves tokens out
    if (P > i0) c -= (P - i0) * A + q2 * (P * (P - 1) / 2 - i0 * (i0 - 1) / 2);
  }
  return c;
}

// The keys of a pair, in units of one TMA box: `su` units of the row's first tokens, then those from wlo on.
struct StreamSpan {
  int i0, nq, pos0, lo_min, lo_max, su, wlo, units, cost;  // cost: of the tokens, without the fixed one
};
__device__ __forceinline__ StreamSpan stream_span(const StreamArgs &a, const StreamRow &r, int p) {
  StreamSpan s;
  s.i0 = p * a.q2;
  s.nq = min(a.q2, r.n - s.i0);
  s.pos0 = r.L - r.n + s.i0;
  const int last = s.pos0 + s.nq - 1;
  s.lo_min = a.window > 0 ? max(s.pos0 - (a.window - 1), 0) : 0;
  s.lo_max = a.window > 0 ? max(last - (a.window - 1), 0) : 0;
  const int fu = (a.first + (1 << a.log2_bh) - 1) >> a.log2_bh;
  s.wlo = s.lo_min >> a.log2_bh;
  s.su = fu;
  if (fu >= s.wlo && fu > 0) s.su = s.wlo = 0;  // the two runs meet
  s.units = s.su + (last >> a.log2_bh) + 1 - s.wlo;
  s.cost = last + 1 - max(0, s.lo_min - (s.lo_min > 0 ? a.first : 0));
  return s;
}

// Units that lie before cost c of a pair.  (A pair has at least as many units as its tokens would fill; what the edges of its runs
// add comes with the last ones.)
__device__ __forceinline__ int stream_unit(const StreamArgs &a, const StreamSpan &s, long long c) {
  // a short pair is not cut: its middle says whose it is
  if (s.cost <= a.whole) return 2 * c >= (long long)a.piece_cost + s.cost ? s.units : 0;
  const long long x = c - a.piece_cost;
  return x <= 0 ? 0 : x >= s.cost ? s.units : (int)x >> a.log2_bh;
}

// ---------------------------------------------------------------------------------------- partition

// The total cost W of a line, all rows and its key heads; and the row for which is(W, x, v) holds (at most one; x: the costs before it, v:
// its own) as found_b (-1: none) and found_x = x.
template <int THREADS, class Is>
__device__ __forceinline__ long long stream_find(const StreamArgs &a, TreePart *ps, uint32_t *bad, const Is &is) {
  const int tid = threadIdx.x;
  if (tid == 0) ps->found_b = -1;
  auto cost = [&](int b, uint32_t *bits) {
    const StreamRow r = stream_row(a, b, bits);
    return r.n > 0 ? a.hl * stream_cost(a, r, stream_pairs(a, r)) : 0ll;
  };
  // up to THREADS rows: one scan gives the total and the place; more: a pass for the total, one for the place
  const bool once = a.batch <= THREADS;
  long long v = 0, ex = 0;
  for (int b = tid; b < a.batch; b += THREADS) v += cost(b, bad);
  const long long W = tree_scan<THREADS>(v, &ex, ps->warp_part);
  long long base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    if (!once) {
      uint32_t again = 0;
      v = b0 + tid < a.batch ? cost(b0 + tid, &again) : 0;
      const long long total = tree_scan<THREADS>(v, &ex, ps->warp_part);
      ex += base;
      base += total;
    }
    if (v > 0 && is(W, ex, v)) {
      ps->found_b = b0 + tid;
      ps->found_x = ex;
    }
    __syncthreads();
    if (ps->found_b >= 0) break;
  }
  return W;
}

// The groups that work on a total cost W, none on less than 2^log2_share, and their shares: group g has [cut(g), cut(g + 1)).
struct StreamShares {
  int groups, more;  // the first `more` groups have one unit of cost more than `each`
  long long each;
  __device__ __forceinline__ StreamShares(const StreamArgs &a, long long W) {
    groups = (int)max(1ll, min((long long)(a.nparts / a.hg), W >> a.log2_share));
    each = W >> 32 ? W / groups : (long long)((uint32_t)W / (uint32_t)groups);
    more = (int)(W - each * groups);
  }
  __device__ __forceinline__ long long cut(int g) const { return g * each + min(g, more); }
};

// Where cost x of a row lies on its line: key head, pair, and the cost within it.
struct StreamPlace {
  int h, p;
  long long off;
};
__device__ __forceinline__ StreamPlace stream_place(const StreamArgs &a, const StreamRow &r, long long x) {
  const int pairs = stream_pairs(a, r);
  StreamPlace s = {0, 0, x};
  if (pairs == 0) return s;
  if (a.hl > 1) {
    const long long head = stream_cost(a, r, pairs);
    s.h = (x | head) >> 32 ? (int)(x / head) : (int)((uint32_t)x / (uint32_t)head);
    s.off = x -= s.h * head;
  }
  if (a.single) return s;
  int lo = 0, hi = pairs - 1;  // the last pair that begins at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (stream_cost(a, r, mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  s.p = lo;
  s.off = x - stream_cost(a, r, lo);
  return s;
}

// This CTA's range [x_begin, x_end) of the costs, and the row that it begins in.
template <int THREADS>
__device__ __forceinline__ void stream_partition(const StreamArgs &a, TreePart *ps, uint32_t *status) {
  const int grp = (int)blockIdx.x / a.hg;
  uint32_t bad = 0;
  stream_find<THREADS>(a, ps, &bad, [&](long long W, long long x, long long v) {
    const StreamShares s(a, W);
    const long long xb = grp < s.groups ? s.cut(grp) : 0, xe = grp < s.groups ? s.cut(grp + 1) : 0;
    const bool mine = xb < xe && xb >= x && xb < x + v;
    if (mine) {
      ps->x_begin = xb;
      ps->x_end = xe;
    }
    return mine;
  });
  if (bad) atomicOr(status, bad);
}

// One piece: units [ub, ue) of a pair's.
struct StreamPiece {
  int b, g, tok0, ub, ue;  // tok0: packed index of the pair's first query
  bool starts, ends;
  StreamSpan span;
};

// Where a piece's results go: -1 the outputs (it is a whole item); else the CTA's partial slot 1 (it begins an
// item that another CTA ends) or 0.
__device__ __forceinline__ int stream_slot(const StreamPiece &p) { return p.starts ? (p.ends ? -1 : 1) : 0; }

// A warp's walk over its CTA's pieces (all lanes call together); each walker sees the same pieces.
struct StreamWalker {
  const StreamArgs &a;
  int lane;
  long long R;      // cost that is left of the range
  int b, h, p;      // the item (h: key head of the line)
  long long off;    // cost of it that is behind the walker
  int rb, w_start, w_n, w_L;  // lane l holds row rb + l

  __device__ StreamWalker(const StreamArgs &args, const TreePart *ps, int lane_) : a(args), lane(lane_) {
    b = max(ps->found_b, 0);
    R = ps->found_b >= 0 ? ps->x_end - ps->x_begin : 0;
    fill(b);
    const StreamPlace at = stream_place(a, row_of(b), ps->found_b >= 0 ? ps->x_begin - ps->found_x : 0);
    h = at.h;
    p = at.p;
    off = at.off;
  }
  __device__ void fill(int row) {
    rb = row;
    uint32_t ignored = 0;
    StreamRow r = {0, 0, 0};
    if (rb + lane < a.batch) r = stream_row(a, rb + lane, &ignored);
    w_start = r.start;
    w_n = r.n;
    w_L = r.L;
  }
  __device__ StreamRow row_of(int row) {
    if (row < rb || row >= rb + 32) fill(row);
    StreamRow r;
    r.start = __shfl_sync(FULL, w_start, row - rb);
    r.n = __shfl_sync(FULL, w_n, row - rb);
    r.L = __shfl_sync(FULL, w_L, row - rb);
    return r;
  }

  __device__ bool take(StreamPiece &pc) {
    while (R > 0 && b < a.batch) {
      const StreamRow r = row_of(b);
      if (r.n == 0) {
        ++b;
        continue;
      }
      pc.span = stream_span(a, r, p);
      const long long cost = (long long)pc.span.cost + a.piece_cost, part = min(cost - off, R);
      pc.b = b;
      pc.g = h * a.hg + (int)blockIdx.x % a.hg;
      pc.tok0 = r.start + pc.span.i0;
      pc.ub = stream_unit(a, pc.span, off);
      pc.ue = stream_unit(a, pc.span, off + part);
      pc.starts = pc.ub == 0;
      pc.ends = pc.ue == pc.span.units;
      R -= part;
      off += part;
      if (off >= cost) {
        off = 0;
        if (++p >= stream_pairs(a, r)) {
          p = 0;
          if (++h >= a.hl) {
            h = 0;
            ++b;
          }
        }
      }
      if (pc.ue > pc.ub) return true;
    }
    return false;
  }
};

// Stages of units [ub, ue), whose first `su` are a run of their own.
__device__ __forceinline__ int stream_stages(int ub, int ue, int su, int nbox) {
  const int n0 = max(min(ue, su) - ub, 0), n1 = ue - max(ub, su);
  return (n0 + nbox - 1) / nbox + (n1 > 0 ? (n1 + nbox - 1) / nbox : 0);
}

// A run of consecutive units of a piece, for the copies.
struct StreamRun {
  int b, g, ub, ue;           // units of the row
  int hi, pos0, lo_max;       // tokens that some query of the pair sees end at hi
  bool first, last, odd;      // of the piece's runs; a stage without tokens makes its stages even in number
};

// A tile's queries, and whether any of them sees a token of [tok, tok + count).
struct StreamTile {
  int pos0, pos1, lo;  // positions of the first and the last; first token in the first one's window
  __device__ __forceinline__ StreamTile(const StreamArgs &a, int pair_pos0, int nq, int x) {
    pos0 = pair_pos0 + x * a.qt;
    pos1 = pair_pos0 + min(nq, (x + 1) * a.qt) - 1;
    lo = a.window > 0 ? max(pos0 - (a.window - 1), 0) : 0;
  }
  __device__ __forceinline__ bool sees(const StreamArgs &a, int tok, int count) const {
    return tok <= pos1 && (tok + count > lo || tok < a.first);
  }
};

// ---------------------------------------------------------------------------------------- tensor memory

// Warp-wide: lane l reads 64 consecutive columns of tensor-memory lane (taddr.lane + l).  The wait is part of the statement: no
// use of the values can be moved before it.
__device__ __forceinline__ void stream_ld(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// The same for 16 columns: where code is run once in a while a short loop costs less than the fetch of a long one.
__device__ __forceinline__ void stream_ld(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void stream_st(uint32_t taddr, const float (&v)[16]) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
  tc_st16(taddr, w);
}

// ---------------------------------------------------------------------------------------- the kernel

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    stream_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_q, const StreamArgs a) {
  using S = StreamSmem<C>;
  constexpr int D = C::D, BN = C::BN, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::OFF_BAR), *empty = full + NS, *clean = empty + NS;
  uint64_t *q_full = clean + C::META, *q_empty = q_full + 1, *s_full = q_full + 2, *p_ready = s_full + C::NB,
           *pv_done = p_ready + C::NB, *o_free = pv_done + C::NB, *half_in = o_free + 1, *drain = half_in + 2, *q_conv = drain + 2,
           *p_half = q_conv + 1, *pv_half = p_half + 2, *turn = pv_half + 2, *raw_full = turn + 8, *raw_empty = raw_full + C::NR;
  TreeStage *meta = reinterpret_cast<TreeStage *>(smem + S::OFF_META);
  StreamPieceRec *prec = reinterpret_cast<StreamPieceRec *>(smem + S::OFF_PIECE);
  uint32_t *sets = reinterpret_cast<uint32_t *>(smem + S::OFF_SET);
  StreamMisc *misc = reinterpret_cast<StreamMisc *>(smem + S::OFF_MISC);
  uint32_t *status = &misc->status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nbox = BN >> a.log2_bh;

  if (lane == 0 && warp < 4) {  // (four threads' worth of barriers)
    if (warp == 0) {
      for (int s = 0; s < NS; ++s) mbar_init(&full[s], C::QUANT ? C::TILE_WARPS : 1);
      for (int s = 0; s < NS; ++s) mbar_init(&empty[s], C::GROUPS);  // an arrival of each issuing thread (both of one where the stage is its own)
      misc->status = 0;
      misc->npieces = 0;
    } else if (warp == 1) {
      for (int s = 0; s < C::META; ++s) mbar_init(&clean[s], C::CLEAN_WARPS);
    } else if (warp == 2) {
      for (int s = 0; s < C::NR; ++s) {
        mbar_init(&raw_full[s], 1);
        mbar_init(&raw_empty[s], C::TILE_WARPS);
      }
      mbar_init(q_conv, C::QUANT ? C::TILE_WARPS : 1);
      mbar_init(q_full, 1);
      mbar_init(q_empty, C::GROUPS);
      mbar_init(o_free, C::SOFTMAX_WARPS);
    } else {
      for (int b = 0; b < C::NB; ++b) {
        mbar_init(&s_full[b], 2);  // the scores' commit and the issuing thread's arrive
        mbar_init(&p_ready[b], 4);
        mbar_init(&pv_done[b], 1);
      }
      for (int w = 0; w < 8; ++w) mbar_init(&turn[w], 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(&pv_half[x], 1);
        mbar_init(&p_half[x], 4);
        mbar_init(&half_in[x], 4);
        mbar_init(&drain[x], 1);
      }
    }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    prefetch_tensormap(&tm_q);
  }
  if (warp == 1) tc_alloc(&misc->tmem, C::TM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;
  pdl_wait();               // what the stream's previous kernel wrote is visible from here on
  pdl_launch_dependents();  // the combine kernel may be scheduled; it waits for this grid to finish
  stream_partition<C::THREADS>(a, &misc->part, status);

  if (warp < 4) {
  if constexpr (C::REG_SPLIT) setmaxnreg_dec<C::REGS_CONTROL>();
  if (warp == 3) {
    // ------------------------------------------------------------ K and V tiles
    const int P = 1 << a.log2_page;
    uint32_t t = 0;
    int in_flight = 0;  // tiles of stage t whose copies were issued
    // where the next K and V tile go: slots, the rings' sizes, and the parity of the phase that frees a slot (a slot's first use
    // waits for the phase before the first, which counts as complete)
    constexpr int K0 = 0, V0 = C::QUANT ? 1 : C::NK, STEP = C::QUANT ? 2 : 1, KEND = C::QUANT ? C::NR : C::NK, VEND = C::QUANT ? C::NR + 1 : C::NS;
    int slot[2] = {K0, V0};
    uint32_t freed[2] = {1u, 1u};
    uint64_t *const r_full = C::QUANT ? raw_full : full, *const r_empty = C::QUANT ? raw_empty : empty;
    bool ok = true;
    StreamWalker walker(a, &misc->part, lane);
    StreamPiece pc;
    int npieces = 0, next_part = 2;  // the run of `pc` that comes next: 0 the first tokens', 1 the window's, 2 none
    auto next_run = [&](StreamRun &r) -> bool {
      bool begins = false;
      if (next_part == 2) {
        if (!walker.take(pc)) return false;
        next_part = pc.ub < pc.span.su ? 0 : 1;
        begins = true;
      }
      const StreamSpan &s = pc.span;
      r.b = pc.b;
      r.g = pc.g;
      r.hi = s.pos0 + s.nq;
      r.pos0 = s.pos0;
      r.lo_max = s.lo_max;
      r.first = begins;
      r.last = next_part == 1 || pc.ue <= s.su;
      r.odd = C::GROUPS == 2 && s.nq <= a.qt && (stream_stages(pc.ub, pc.ue, s.su, nbox) & 1);
      r.ub = next_part == 0 ? pc.ub : max(pc.ub, s.su) - s.su + s.wlo;
      r.ue = next_part == 0 ? min(pc.ue, s.su) : pc.ue - s.su + s.wlo;
      next_part = r.last ? 2 : 1;
      return true;
    };
    auto window_of = [&](const StreamRun &r, int w) {  // block-table entries [32 w, 32 w + 32) of a run
      const int pb = (r.ub << a.log2_bh) >> a.log2_page;
      const int np = ((((r.ue << a.log2_bh) - 1) >> a.log2_page) + 1) - pb;
      return 32 * w + lane < np ? a.block_table[(size_t)r.b * a.max_pages_per_seq + pb + 32 * w + lane] : 0;
    };
    // The tile kv of a stage goes to the next slot of its ring.
    auto next_slot = [&](int kv) {
      slot[kv] += STEP;
      if (slot[kv] >= (kv ? VEND : KEND)) {
        slot[kv] = kv ? V0 : K0;
        freed[kv] ^= 1u;
      }
    };
    // Stage t of units [unit0, ue) of run r, whose pages are in `page` of the first lanes; absent: without tokens.
    auto stage = [&](const StreamRun &r, int unit0, int page, bool absent, bool begins) {
      const bool mine = !absent && lane < nbox && unit0 + lane < r.ue, load = mine && page >= 0 && page < a.num_pages;
      if (mine && !load) atomicOr(status, PA_DEV_BAD_PAGE);
      const uint32_t bad = __ballot_sync(FULL, mine && !load);
      const int boxes = absent ? 0 : min(nbox, r.ue - unit0) - __popc(bad);
      const int btok = (unit0 + lane) << a.log2_bh;
#pragma unroll
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int s = slot[kv];
        ok = warp_wait(&r_empty[s], freed[kv], status);
        if (!ok) break;
        in_flight = kv + 1;
        if (lane == 0) {
          if (kv == 0) {
            const int tok0 = unit0 << a.log2_bh, tok_hi = min(r.hi, r.ue << a.log2_bh);
            const bool whole = tok0 + BN <= min(r.pos0 + 1, tok_hi) && (tok0 >= r.lo_max || tok0 + BN <= a.first) && bad == 0;
            *reinterpret_cast<int4 *>(&meta[t % C::META]) =
                make_int4((absent ? STAGE_ABSENT : whole ? 0 : STAGE_MASKED) | (begins ? STAGE_FIRST : 0), tok0, tok_hi, (int)bad);
          }
          mbar_arrive_expect_tx(&r_full[s], (uint32_t)boxes * (uint32_t)(C::ROWB << a.log2_bh));
        }
        __syncwarp();
        if (load) {
          if constexpr (C::QUANT) {  // whole rows of codes, one after the other
            tma_load_4d(smem + S::OFF_RAW + s * C::RAW_SLOT + (lane << a.log2_bh) * C::ROWB, kv ? &tm_v : &tm_k, 0, r.g,
                        btok & (P - 1), page, &r_full[s]);
          } else {
            tma_load_4d(smem + S::OFF_RING + s * C::SLOT + (lane << a.log2_bh) * C::ROWB, kv ? &tm_v : &tm_k, 0, 0, r.g * C::NPL,
                        (page << (a.log2_page - 3)) + ((btok & (P - 1)) >> 3), &full[s]);
          }
        }
        next_slot(kv);
      }
      if (ok) {
        ++t;
        in_flight = 0;
      }
    };
    StreamRun cur = {}, nxt = {};
    int cwin = 0, nwin = 0;
    for (bool has = false;;) {  // cur, if there is one, with the run behind it known
      const bool has_next = next_run(nxt);
      if (has_next) nwin = window_of(nxt, 0);
      if (has) {
        const int pb = (cur.ub << a.log2_bh) >> a.log2_page;
        int wi = 0, fwin = window_of(cur, 1);
        for (int unit0 = cur.ub; unit0 < cur.ue && ok; unit0 += nbox) {
          // the pages of one stage never straddle a window of 32 (nbox divides 32)
          const int pwin = (((unit0 << a.log2_bh) >> a.log2_page) - pb) >> 5;
          while (wi < pwin) {
            cwin = fwin;
            ++wi;
            fwin = window_of(cur, wi + 1);
          }
          const int page = __shfl_sync(FULL, cwin, ((((unit0 + lane) << a.log2_bh) >> a.log2_page) - pb) & 31);
          stage(cur, unit0, page, false, cur.first && unit0 == cur.ub);
        }
        if (ok && cur.last && cur.odd) stage(cur, cur.ue, 0, true, false);
        if (!ok) break;
        if (cur.last) ++npieces;
      }
      if (!has_next) break;
      has = true;
      cur = nxt;
      cwin = nwin;
    }
    // the end, for the converting warps: the next stage's tiles, which are none
    for (int kv = 0; C::QUANT && kv < 2 && ok; ++kv) {
      ok = warp_wait(&r_empty[slot[kv]], freed[kv], status);
      if (ok && lane == 0) {
        if (kv == 0) meta[t % C::META].flags = STAGE_END;
        mbar_arrive(&r_full[slot[kv]]);
      }
    }
    if (!ok) {  // copies in flight land before the CTA exits
      if constexpr (C::QUANT) {
        const uint32_t nf_ = 2 * t + (uint32_t)in_flight;
        for (uint32_t i = nf_ > C::NR ? nf_ - C::NR : 0u; i < nf_; ++i)
          warp_wait(&raw_full[i % C::NR], (i / C::NR) & 1, status);
      } else {
        const uint32_t nk = t + (in_flight > 0), nv = t + (in_flight > 1);
        for (uint32_t i = nk > C::NK ? nk - C::NK : 0u; i < nk; ++i) warp_wait(&full[i % C::NK], (i / C::NK) & 1, status);
        for (uint32_t i = nv > C::NV ? nv - C::NV : 0u; i < nv; ++i)
          warp_wait(&full[C::NK + i % C::NV], (i / C::NV) & 1, status);
      }
    }
    if (lane == 0) misc->npieces = npieces;
  } else if (warp == 1 || (warp == 2 && C::GROUPS == 2)) {
    // ------------------------------------------------------------ products (one thread of the warp, elected: with the
    // first one, which the compiler cannot know to be alone, each instruction's operands take a detour)
    if (elect_one()) {
      const int x = warp - 1;
      const uint32_t ring = smem_u32(smem + S::OFF_RING), qb = smem_u32(smem);
      uint32_t t0 = 0, c = 0, d = 0;  // the piece's first stage; items begun and finished
      bool ok = true;
      auto buf = [&](uint32_t i) { return C::buffer(x, i); };
      auto par = [&](uint32_t i) { return C::buffer_phase(i); };
      // the slot of a tile is free for whoever shares it: with this thread's operations, or at once
      auto release = [&](uint64_t *bar, bool read, bool alone) {
        if (read) tc_commit(bar);
        else mbar_arrive(bar);
        if (C::GROUPS == 2 && alone) mbar_arrive(bar);
      };
      // the scores of the next item: query tile qx, stage t; are there any?
      auto begin = [&](uint32_t t, int qx, const StreamTile &tile, bool alone, bool &present) -> bool {
        const uint32_t b = buf(c);
        if (!mbar_wait(&full[t % C::NK], (t / C::NK) & 1, status)) return false;
        if (c >= (uint32_t)C::BACK && !mbar_wait(&pv_done[b], par(c - C::BACK), status)) return false;
        const int4 m = *reinterpret_cast<const int4 *>(&meta[t % C::META]);  // flags, tok0, tok_hi, badmask
        present = !(m.x & STAGE_ABSENT) && (!(m.x & STAGE_MASKED) || tile.sees(a, m.y, BN));
        mbar_arrive(&s_full[b]);
        if (present) {
          tc_fence_after();
          const uint64_t qd = tc_sdesc_sw128(qb + qx * (C::NPL * C::QPLANE), 16, 1024);
          const uint64_t kd = tc_sdesc_sw128(ring + (t % C::NK) * C::SLOT, 16, C::GROUP);
#pragma unroll
          for (int p = 0; p < C::NPL; ++p)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_ss(tmem + C::TM_S + b * BN, qd + (uint64_t)((p * C::QPLANE + 32 * kk) >> 4),
                        kd + (uint64_t)((p * C::PLANE + 32 * kk) >> 4), C::IDESC_S, (p | kk) != 0 ? 1u : 0u);
          tc_commit(&s_full[b]);
        } else {
          mbar_arrive(&s_full[b]);  // no scores: the record alone
        }
        release(&empty[t % C::NK], present, alone);
        ++c;
        return true;
      };
      // the second product of the oldest item; fresh: the piece's output has had none yet.  (What usually is there already is
      // waited for first; next: the stage whose scores follow at once, or none)
      auto finish = [&](uint32_t t, uint32_t piece, bool first, bool &fresh, bool present, bool alone, int next) -> bool {
        const uint32_t b = buf(d), vs = C::NK + t % C::NV;
        // the previous piece's outputs have been read, and all its V tiles with that (before any wait for this one's: the other
        // thread's tiles of that piece may have been in its slot)
        if (first && piece > 0 && !mbar_wait(o_free, (piece - 1) & 1, status)) return false;
        // (bf16: whoever looked it over has waited for it)
        if (C::QUANT ? !mbar_wait(&full[vs], (t / C::NV) & 1, status)
                     : !mbar_wait(&clean[t % C::META], (t / C::META) & 1, status))
          return false;
        if (C::BACK == 1 && next >= 0 && !mbar_wait(&full[next % C::NK], (next / C::NK) & 1, status)) return false;
        if (!(C::HALVES ? mbar_wait(&p_half[x], d & 1, status) : mbar_wait(&p_ready[b], par(d), status))) return false;
        if (present) {
          tc_fence_after();
          const int o = C::GROUPS == 2 ? x : 0;
          const uint64_t vd = tc_sdesc_sw128(ring + vs * C::SLOT, C::PLANE, C::GROUP);
#pragma unroll
          for (int i = 0; i < BN / 16; ++i) {
            if (C::HALVES && i == BN / 32) {
              tc_commit(&pv_half[x]);
              if (!mbar_wait(&p_ready[b], par(d), status)) return false;
              tc_fence_after();
            }
            const int kk = C::HALVES ? i ^ (BN / 32) : i;  // (the second half of the weights is there first)
            tc_mma_ts(tmem + C::TM_O + o * D, tmem + C::TM_S + b * BN + C::P_AT + 8 * kk, vd + (uint64_t)((kk * 2 * C::GROUP) >> 4),
                      C::IDESC_PV, fresh && i == 0 ? 0u : 1u);
          }
          fresh = false;
        } else if (C::HALVES) {
          mbar_arrive(&pv_half[x]);
          if (!mbar_wait(&p_ready[b], par(d), status)) return false;
        }
        tc_commit(&pv_done[b]);
        release(&empty[vs], present, alone);
        ++d;
        return true;
      };
      for (uint32_t piece = 0; ok; ++piece) {
        ok = mbar_wait(C::QUANT ? q_conv : q_full, piece & 1, status);
        if (!ok) break;
        const int4 r = *reinterpret_cast<const int4 *>(&prec[piece & 1]);  // end, stages, two, slot
        const int4 r1 = *(reinterpret_cast<const int4 *>(&prec[piece & 1]) + 1);  // b, pos0, nq, tok0
        if (r.x) {
          for (int k = 0; k < 2; ++k) mbar_arrive(&s_full[buf(c)]);  // the softmax groups stop here
          break;
        }
        const bool two = r.z != 0, alone = !two;
        const uint32_t stages = (uint32_t)r.y, count = C::GROUPS == 2 && alone ? (stages + 1) & ~1u : stages;
        const StreamTile tile(a, r1.y, r1.z, two ? x : 0);
        // this thread's stages: all of them, or those of its parity
        const uint32_t j0 = C::GROUPS == 2 && alone ? (x + t0) & 1 : 0, dj = C::GROUPS == 2 && alone ? 2 : 1;
        bool fresh = true, now = false, before = false, told = false;
        for (uint32_t j = j0; j < count + dj && ok; j += dj) {
          // with more than one buffer the next scores come before the second product of the item before them
          if (C::BACK == 1 && j > j0) ok = finish(t0 + j - dj, piece, j == j0 + dj, fresh, before, alone, j < count ? (int)(t0 + j) : -1);
          if (ok && j < count) ok = begin(t0 + j, two ? x : 0, tile, alone, now);
          if (!told && j + dj >= stages) {  // the query tiles have been read
            tc_commit(q_empty);
            told = true;
          }
          if (C::BACK > 1 && ok && j > j0) ok = finish(t0 + j - dj, piece, j == j0 + dj, fresh, before, alone, -1);
          before = now;
        }
        t0 += count;
      }
      // every operation of this thread has completed before the tensor memory is released
      tc_commit(&drain[x]);
      mbar_wait(&drain[x], 0, status);
    }
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------ query tiles; V tiles looked over (bf16)
    StreamWalker walker(a, &misc->part, lane);
    StreamPiece pc;
    uint32_t k = 0, t = 0;
    int stages = 0;
    bool ok = true;
    // the last piece's scores are done: of all the kernel's waits the one that lasts as long as a piece.  65536 stages
    // take some 60 ms; a second more for each
    auto scored = [&]() -> bool {
      const bool r = mbar_wait_warp(q_empty, (k - 1) & 1, WAIT_LIMIT_NS * (1 + ((uint64_t)stages >> 16)));
      if (!r && lane == 0) atomicOr(status, PA_DEV_TIMEOUT);
      return r;
    };
    while (ok && walker.take(pc)) {
      if (k > 0) ok = scored();
      if (!ok) break;
      const StreamSpan &sp = pc.span;
      stages = stream_stages(pc.ub, pc.ue, sp.su, nbox);
      const bool two = sp.nq > a.qt;
      // (the sets of four pieces before: whoever reads those of the piece before the last may still be at it)
      uint32_t *set = sets + (k & 3) * (2 * kStreamBits);
      if (lane < 2 * kStreamBits) set[lane] = 0;
      __syncwarp();
      if (lane == 0) {
        prec[k & 1] = StreamPieceRec{0, stages, two, stream_slot(pc), pc.b, sp.pos0, sp.nq, pc.tok0, pc.g, sp.lo_min, sp.lo_max, 0};
        const int boxes = min(a.qt, a.max_query) * a.G * 128;  // bytes of one plane's box
        mbar_arrive_expect_tx(q_full, (uint32_t)(C::NPL * boxes * (two ? 2 : 1)));
        for (int x = 0; x < (two ? 2 : 1); ++x) {
#pragma unroll
          for (int p = 0; p < C::NPL; ++p)
            tma_load_3d(smem + (x * C::NPL + p) * C::QPLANE, &tm_q, p * 64, pc.g * a.G, pc.tok0 + x * a.qt, q_full);
        }
      }
      __syncwarp();
      ++k;
      if constexpr (!C::QUANT) {
        for (int st = 0; st < (C::GROUPS == 2 && !two ? (stages + 1) & ~1 : stages) && ok; ++st, ++t) {
          const int s = C::NK + t % C::NV;
          ok = warp_wait(&full[s], (t / C::NV) & 1, status);
          if (!ok) break;
          const int4 m = *reinterpret_cast<const int4 *>(&meta[t % C::META]);  // flags, tok0, tok_hi, badmask
          if (m.x & STAGE_MASKED) {
            uint8_t *v = smem + S::OFF_RING + s * C::SLOT;
#pragma unroll 1
            for (int r = lane; r < BN; r += 32) {
              const int tok = m.y + r;
              const bool any = tok < m.z && (tok >= sp.lo_min || tok < a.first) &&
                               ((loaded_bits((uint32_t)m.w, r >> 5, a.log2_bh) >> (r & 31)) & 1u);
              const bool some = tok > sp.pos0 || (tok < sp.lo_max && tok >= a.first);  // seen by some and not by others
              if (any && !some) continue;
              auto chunk = [&](int c) {
                return reinterpret_cast<uint4 *>(v + (r >> 3) * C::GROUP + (c >> 3) * C::PLANE + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
              };
              if (!any) {
#pragma unroll 8
                for (int c = 0; c < C::NPL * 8; ++c) *chunk(c) = make_uint4(0, 0, 0, 0);
                continue;
              }
              // exponents of all ones (infinities and NaN) carry into the sign's place
              auto odd = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
              uint32_t seen = 0;
#pragma unroll 8
              for (int c = 0; c < C::NPL * 8; ++c) {
                const uint4 x = *chunk(c);
                seen |= odd(x.x) | odd(x.y) | odd(x.z) | odd(x.w);
              }
              const bool found = seen & 0x80008000u;
              if (__builtin_expect(found, 0)) {
#pragma unroll 1
                for (int c = 0; c < C::NPL * 8; ++c) {
                  uint4 x = *chunk(c);
                  auto without = [&](uint32_t w) { return w & ~((odd(w) >> 15 & 0x00010001u) * 0xffffu); };
                  *chunk(c) = make_uint4(without(x.x), without(x.y), without(x.z), without(x.w));
                }
              }
              if (found) {
                const int bit = tok > sp.pos0 ? tok - sp.pos0 - 1 : kStreamBits * 32 + tok - sp.lo_min;
                atomicOr(&set[bit >> 5], 1u << (bit & 31));
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&clean[t % C::META]);
        }
      }
    }
    // no copy is in flight when the CTA exits, and the issuing threads learn of the end
    if (k > 0) {
      warp_wait(q_full, (k - 1) & 1, status);
      if (ok) ok = scored();
    }
    if (ok && lane == 0) {
      prec[k & 1].end = 1;
      mbar_arrive(q_full);
    }
  }
  } else if (warp >= 4 + C::SOFTMAX_WARPS) {
    if constexpr (C::REG_SPLIT) setmaxnreg_dec<C::REGS_CONVERT>();
    // ------------------------------------------------------------ codes to f16 operands
    // Each thread takes 16 codes at a time: two 16-byte chunks of a swizzled f16 row.  Eight lanes take a plane
    // (64 values) of one row and the plane beside it of the next row: in the swizzled rows one half's chunks are
    // then the even and the other's the odd ones, and the codes are in different banks too.
    if constexpr (C::QUANT) {
      const int ct = tid - (4 + C::SOFTMAX_WARPS) * 32, cw = ct >> 5;
      constexpr int TPR = D / 16, NTASK = BN * TPR, STEP = C::TILE_WARPS * 32, ROUND = NTASK / STEP < 4 ? NTASK / STEP : 4;
      static_assert(NTASK % (ROUND * STEP) == 0 && STEP % TPR == 0, "whole rounds of tasks");
      const int kv = cw / C::TILE_WARPS, tt = ct % STEP;  // this warp's kind of tile; the thread among its warps'
      uint32_t kp = 0;  // pieces begun
      int pos0 = 0, lo_min = 0, lo_max = 0;
      for (uint32_t t = 0;; ++t) {
        const uint32_t f = 2 * t + kv;
        const int rs = f % C::NR;
        bool ok = warp_wait(&raw_full[rs], (f / C::NR) & 1, status);
        if (!ok) break;
        const int4 m = *reinterpret_cast<const int4 *>(&meta[t % C::META]);  // flags, tok0, tok_hi, badmask
        // a new piece, or the end: the warps of the V tiles, which are needed later, take the query rows
        if (__builtin_expect(kv == 1 && (m.x & (STAGE_FIRST | STAGE_END)), 0)) {
          ok = warp_wait(q_full, kp & 1, status);
          if (!ok) break;
          const StreamPieceRec &r = prec[kp & 1];
          pos0 = r.pos0;
          lo_min = r.lo_min;
          lo_max = r.lo_max;
          if (!(m.x & STAGE_END)) {
            const int nq = r.nq;
            // times 2^s (largest magnitude in [2^14, 2^15)) to f16, in place
            int8_t *shift = reinterpret_cast<int8_t *>(smem + S::OFF_SHIFT) + (kp & 1) * (C::QT * kTreeRows);
            for (int i = tt; i < nq * a.G; i += STEP) {  // (the rows that hold a query)
              const int r = i < a.qt * a.G ? i : kTreeRows + i - a.qt * a.G;
              uint8_t *row = smem + (r >> 7) * (C::NPL * C::QPLANE) + (r & 127) * 128;
              auto chunk = [&](int c) {
                return reinterpret_cast<uint4 *>(row + (c >> 3) * C::QPLANE + (((c & 7) ^ (r & 7)) << 4));
              };
              constexpr int CH = 8;  // chunks of the row in registers at a time
              uint4 w[CH];
              float amax = 0.f;
#pragma unroll 1
              for (int c0 = 0; c0 < C::NPL * 8; c0 += CH) {
#pragma unroll
                for (int c = 0; c < CH; ++c) w[c] = *chunk(c0 + c);
#pragma unroll
                for (int c = 0; c < CH; ++c) amax = fmaxf(amax, absmax8(w[c]));
              }
              const int sh = min(14 - ((int)(__float_as_uint(amax) >> 23) - 127), 126);  // at least -114
              const float p2 = __uint_as_float((uint32_t)(sh + 127) << 23);
              shift[r] = (int8_t)sh;
#pragma unroll 1
              for (int c0 = C::NPL * 8 - CH; c0 >= 0; c0 -= CH) {  // (the last ones read are still there)
                if (c0 != C::NPL * 8 - CH) {
#pragma unroll
                  for (int c = 0; c < CH; ++c) w[c] = *chunk(c0 + c);
                }
#pragma unroll
                for (int c = 0; c < CH; ++c)
                  *chunk(c0 + c) = make_uint4(scaled_f16x2(w[c].x, p2), scaled_f16x2(w[c].y, p2), scaled_f16x2(w[c].z, p2),
                                              scaled_f16x2(w[c].w, p2));
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(q_conv);
          ++kp;
        }
        if (m.x & STAGE_END) break;
        {
          const int s = kv ? C::NK + t % C::NV : t % C::NK;
          const uint32_t u = kv ? t / C::NV : t / C::NK;
          if (u > 0) ok = warp_wait(&empty[s], (u - 1) & 1, status);
          if (!ok) break;
          const uint8_t *raw = smem + S::OFF_RAW + rs * C::RAW_SLOT;
          uint8_t *op = smem + S::OFF_RING + s * C::SLOT;
          const bool look = kv == 1 && (m.x & STAGE_MASKED);
          auto put = [&](int r, int pc, const uint32_t (&h)[8]) {
            uint8_t *row = op + (r >> 3) * C::GROUP + (pc >> 2) * C::PLANE + (r & 7) * 128;
            const int c0 = 2 * (pc & 3);
            *reinterpret_cast<uint4 *>(row + ((c0 ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(row + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          };
          // this thread's place: 16 codes pc of row r0, and of every (STEP / TPR)-th row from there; four loads in flight
          const int pl = (tt >> 3) % C::NPL, odd = (tt >> 2) & 1;
          const int pc = (C::NPL > 1 ? pl ^ odd : pl) * 4 + (tt & 3), r0 = (tt >> 3) / C::NPL * 2 + odd;
          if (__builtin_expect(m.x & STAGE_ABSENT, 0)) {
            // nothing is there
          } else if (__builtin_expect(!look, 1)) {
#pragma unroll 1
            for (int i0 = 0; i0 < NTASK / STEP; i0 += ROUND) {
              Codes16<C::FMT, D> x[ROUND];
#pragma unroll
              for (int e = 0; e < ROUND; ++e) x[e].load(raw + (r0 + (i0 + e) * (STEP / TPR)) * C::ROWB, pc);
#pragma unroll
              for (int e = 0; e < ROUND; ++e) {
                uint32_t h[8];
                x[e].convert(h);
                put(r0 + (i0 + e) * (STEP / TPR), pc, h);
              }
            }
          } else {
            uint32_t *set = sets + ((kp - 1) & 3) * (2 * kStreamBits);
#pragma unroll 1
            for (int i = 0; i < NTASK / STEP; ++i) {
              const int r = r0 + i * (STEP / TPR), tok = m.y + r;
              Codes16<C::FMT, D> x;
              uint32_t h[8];
              x.load(raw + r * C::ROWB, pc);
              x.convert(h);
              const bool any = tok < m.z && (tok >= lo_min || tok < a.first) &&
                               ((loaded_bits((uint32_t)m.w, r >> 5, a.log2_bh) >> (r & 31)) & 1u);
              if (!any) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = 0u;
              } else if (tok > pos0 || (tok < lo_max && tok >= a.first)) {
                uint32_t hit = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint32_t bits = ((h[e] & 0x7c00u) == 0x7c00u ? 0xffffu : 0u) |
                                        ((h[e] & 0x7c000000u) == 0x7c000000u ? 0xffff0000u : 0u);
                  hit |= bits;
                  h[e] &= ~bits;
                }
                if (hit) {
                  const int bit = tok > pos0 ? tok - pos0 - 1 : kStreamBits * 32 + tok - lo_min;
                  atomicOr(&set[bit >> 5], 1u << (bit & 31));
                }
              }
              put(r, pc, h);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) {
            mbar_arrive(&full[s]);
            mbar_arrive(&raw_empty[rs]);
            if (kv == 1) mbar_arrive(&clean[t % C::META]);
          }
        }
      }
    }
  } else {
    if constexpr (C::REG_SPLIT) setmaxnreg_inc<C::REGS_SOFTMAX>();
    // ------------------------------------------------------------ softmax and output
    const int grp = (warp - 4) >> 2;              // softmax group
    const int row = 32 * (warp & 3) + lane;       // row of the tile, lane of the tensor memory
    const uint32_t tl_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // scores s to exponents s' * qs - m with qs > 0: s' = s * flip
    const float flip = a.qscale > 0.f ? 1.f : a.qscale < 0.f ? -1.f : 0.f, scale = a.qscale != 0.f ? fabsf(a.qscale) : 1.f;
    const int qi = row / a.G, qh = row - qi * a.G;  // query of the tile, head of the group
    float m_run = -INFINITY, l_run = 0.f, qs = scale;
    uint32_t kp = 0;  // pieces begun
    int pos = 0, lo_row = 0, node_tok = 0, head = 0, b = 0, slot = -1, g = 0, prow = 0, pos0 = 0, lo_min = 0;
    bool real = false, warp_real = false, had = false;  // had: this group's output has had a product in the piece
    uint32_t c = 0, k_half = 0;  // items done; merges
    uint32_t t0 = 0;             // the piece's first stage
    bool ok = true;
    auto buf = [&](uint32_t i) { return C::buffer(grp, i); };
    auto par = [&](uint32_t i) { return C::buffer_phase(i); };

    // the group's next item, of a stage with the record m (flags, tok0, tok_hi, badmask)
    // With pairs of tiles the two warps that share a quarter of the SM take turns at the exponentials, group 0's item first.  (Barriers
    // of their own, each of whose phases is waited for once: a barrier that goes on without its waiter, as those of the
    // weights do where one tile's stages alternate, can be a whole turn of its parity ahead.)
    uint32_t turns = 0;
    auto my_turn = [&]() -> bool {
      return grp == 0 ? turns == 0 || warp_wait(&turn[warp & 3], (turns - 1) & 1, status)
                      : warp_wait(&turn[4 + (warp & 3)], turns & 1, status);
    };
    auto your_turn = [&]() {
      if (lane == 0) mbar_arrive(&turn[(grp ? 0 : 4) + (warp & 3)]);
      ++turns;
    };
    auto item = [&](const StreamTile &tile, int4 m, bool two) -> bool {
      const uint32_t tS = tl_base + C::TM_S + buf(c) * BN;
      const int o = C::GROUPS == 2 ? grp : 0;
      const uint32_t tO = tl_base + C::TM_O + o * D;
      const bool partly = m.x & STAGE_MASKED;
      if (warp_real && !(m.x & STAGE_ABSENT) && (!partly || tile.sees(a, m.y, BN))) {
        // 64 weights at a time, of 128 the last 64 first.  Their sum tells whether the maximum is still good: while it is at most
        // 2^(LIFT + TAU), no weight is larger.
        const float2 q2 = make_float2(qs, qs);
        int k = BN / 64 - 1;
        // the maximum is looked for: over all scores in the first item of a piece, in stages that are seen in part and with scales that
        // are not positive (the last two change the scores on the way), over 64 of them where their sum says so
        bool all = partly || !had || flip != 1.f, find = all, looked = false;
        bool wanted = true;
        bool turned = false;
        while (k >= 0) {
          if (__builtin_expect(find, 0)) {
            float mx = -INFINITY;
#pragma unroll 1
            for (int e = all ? 0 : 64 * k; e < (all ? BN : 64 * k + 64); e += 32) {
              float v[32];
              tc_ld32(tS + e, v);
              if (all && (partly || flip != 1.f)) {
                const int base = m.y + e;
                const uint32_t vis = partly ? (range_bits(base, lo_row, pos + 1) | range_bits(base, 0, min(a.first, pos + 1))) &
                                                  range_bits(base, 0, m.z) & loaded_bits((uint32_t)m.w, e >> 5, a.log2_bh)
                                            : ~0u;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = (vis >> i) & 1u ? v[i] * flip : -INFINITY;
                tc_st32(tS + e, v);
              }
              float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], v[i]);
              mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            }
            tc_wait_st();
            // The maximum is raised, and the output and the sum so far with it.  (Only of rows that want it, so that no row's rounding
            // depends on what its neighbours attend to.)
            const float m_new = mx * qs - C::LIFT;
            const bool up = real && wanted && m_new > m_run + (all && m_run != -INFINITY ? C::TAU : 0.f);
            if (__any_sync(FULL, up)) {
              const float al = up && m_run != -INFINITY ? fast_exp2(m_run - m_new) : 1.f;
              if (up) m_run = m_new;
              l_run *= al;
              if (had) {
                // the output's products so far are complete: the items' before, and that of this one's other half
                if (!warp_wait(&pv_done[buf(c - 1)], par(c - 1), status)) return false;
                if (C::HALVES && k == 0 && !warp_wait(&pv_half[grp], c & 1, status)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < D; e += 16) {
                  float v[16];
                  stream_ld(tO + e, v);
#pragma unroll
                  for (int i = 0; i < 16; ++i) v[i] *= al;
                  stream_st(tO + e, v);
                }
                tc_wait_st();
              }
            }
            looked = !all;
            find = all = false;
          }
          uint32_t w[32];
          float x[64];
          stream_ld(tS + 64 * k, x);
          if (C::TURNS && two && !turned) {
            if (!my_turn()) return false;
            turned = true;
          }
          const float sub = m_run == -INFINITY ? 0.f : m_run;
          const float2 sub2 = make_float2(-sub, -sub);
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            const float2 y = fma_pair(make_float2(x[i], x[i + 1]), q2, sub2);
            const float2 pr = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            l2[(i >> 1) & 1] = add_pair(l2[(i >> 1) & 1], pr);
            w[i >> 1] = C::QUANT ? pack_f16x2(pr.x, pr.y) : pack_bf16x2(pr.x, pr.y);
          }
          l2[0] = add_pair(l2[0], l2[1]);
          const float sum = l2[0].x + l2[0].y;
          wanted = !(sum <= C::WEIGHTS) || (m_run == -INFINITY && !partly);
          if (__builtin_expect(!looked && __any_sync(FULL, real && wanted), 0)) {
            find = true;
            continue;
          }
          looked = false;
          if (C::TURNS && two && k == 0) your_turn();
          l_run += sum;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = w[16 * h + i];
            tc_st16(tS + C::P_AT + 32 * k + 16 * h, u);
          }
          had = true;
          if (C::HALVES && k == 1) {
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[grp]);
          }
          --k;
        }
        tc_wait_st();
      } else if (C::HALVES) {
        if (C::TURNS && two) {
          if (!my_turn()) return false;
          your_turn();
        }
        if (lane == 0) mbar_arrive(&p_half[grp]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[buf(c)]);
      ++c;
      return true;
    };

    while (ok) {
      // a new piece: its record comes with its first item
      if (!warp_wait(&s_full[buf(c)], par(c), status)) break;
      tc_fence_after();
      const int4 *rp = reinterpret_cast<const int4 *>(&prec[kp & 1]);
      const int4 r0 = rp[0], r1 = rp[1], r2 = rp[2];
      if (r0.x) break;
      const bool two = r0.z != 0;
      const uint32_t count = C::GROUPS == 2 && !two ? ((uint32_t)r0.y + 1) & ~1u : (uint32_t)r0.y;
      const int tx = two ? grp : 0;
      slot = r0.w;
      b = r1.x;
      pos0 = r1.y;
      g = r2.x;
      lo_min = r2.y;
      const StreamTile tile(a, pos0, r1.z, tx);
      {
        const int i = tx * a.qt + qi;  // query of the pair
        real = qi < a.qt && i < r1.z;
        warp_real = __any_sync(FULL, real);
        prow = tx * kTreeRows + row;
        if constexpr (C::QUANT) {  // the scores are 2^s times too large
          const int sh = reinterpret_cast<const int8_t *>(smem + S::OFF_SHIFT)[(kp & 1) * (C::QT * kTreeRows) + prow];
          // (never 0, which masked scores of -inf would make NaN of: these scores are below 2^35, so 2^-126 of them is nothing)
          qs = fmaxf(scale * __uint_as_float((uint32_t)(127 - sh) << 23), 0x1p-126f);
        }
        pos = pos0 + i;
        lo_row = a.window > 0 ? max(pos - (a.window - 1), 0) : 0;
        node_tok = r1.w + i;
        head = g * a.G + qh;
      }
      const uint32_t *set = sets + (kp & 3) * (2 * kStreamBits);
      ++kp;
      m_run = -INFINITY;
      l_run = 0.f;
      had = false;
      const uint32_t j0 = C::GROUPS == 2 && !two ? (grp + t0) & 1 : 0, dj = C::GROUPS == 2 && !two ? 2 : 1;
      for (uint32_t j = j0; j < count && ok; j += dj) {
        if (j != j0) {
          ok = warp_wait(&s_full[buf(c)], par(c), status);
          if (!ok) break;
          tc_fence_after();
        }
        ok = item(tile, *reinterpret_cast<const int4 *>(&meta[(t0 + j) % C::META]), two);
      }
      if (!ok) break;
      t0 += count;

      // ---- end of a piece: the products of the last item, and with them all before, are complete; and all V tiles looked over
      ok = warp_wait(&pv_done[buf(c - 1)], par(c - 1), status) &&
           warp_wait(&clean[(t0 - 1) % C::META], ((t0 - 1) / C::META) & 1, status);
      if (!ok) break;
      StreamHalf other = {-INFINITY, 0.f};
      const bool merge = C::GROUPS == 2 && !two && r0.y > 1;  // (one stage: one group, that of its parity, has had it)
      if (merge) {  // both groups have had as many items
        a.halves[((size_t)blockIdx.x * 2 + grp) * kTreeRows + row] = StreamHalf{m_run, l_run};
        __syncwarp();
        if (lane == 0) mbar_arrive(&half_in[grp]);
        ok = warp_wait(&half_in[grp ^ 1], k_half & 1, status) && warp_wait(&pv_done[C::buffer(grp ^ 1, c - 1)], par(c - 1), status);
        if (!ok) break;
        ++k_half;
        other = a.halves[((size_t)blockIdx.x * 2 + (grp ^ 1)) * kTreeRows + row];
      }
      __syncwarp();
      tc_fence_after();
      // weights of this group's output and of the other's; a sum of zero: nothing was attended to
      const float M = fmaxf(m_run, other.m);
      const float w_own = l_run == 0.f ? 0.f : fast_exp2(m_run - M), w_oth = other.l == 0.f ? 0.f : fast_exp2(other.m - M);
      const float Z = (l_run == 0.f ? 0.f : l_run * w_own) + (other.l == 0.f ? 0.f : other.l * w_oth);
      const float inv = Z == 0.f ? 0.f : a.vscale / Z;
      const float s_own = w_own * inv, s_oth = w_oth * inv;
      const bool use_own = l_run != 0.f, use_oth = merge && other.l != 0.f;
      const float lse2 = Z == 0.f ? -INFINITY : M + __log2f(Z);
      const int o = C::GROUPS == 2 ? grp : 0;
      const int c0 = merge ? grp * (D / 2) : 0, c1 = merge ? c0 + D / 2 : D;
      const size_t pi = ((size_t)blockIdx.x * 2 + (slot > 0 ? 1 : 0)) * (C::QT * kTreeRows) + prow;
      uint16_t *orow = a.out + ((size_t)node_tok * a.Hq + head) * D;
      constexpr int RS = C::QT * kTreeRows;
      float *po = a.part_o + (pi - prow) * D + prow * 4;  // value d of the row: po[d / 4 * 4 RS + d % 4]
      if (warp_real && (two || merge || C::GROUPS == 1 || grp == (int)(t0 & 1))) {
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          float v[16], u[16];
          stream_ld(tl_base + C::TM_O + o * D + c, v);
          if (merge) stream_ld(tl_base + C::TM_O + (o ^ 1) * D + c, u);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = use_own ? v[i] * s_own : 0.f;
            if (merge) v[i] = use_oth ? fmaf(u[i], s_oth, v[i]) : v[i];
          }
          if (real) {
            if (slot < 0) {
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                *reinterpret_cast<uint4 *>(orow + c + i) =
                    make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]), pack_bf16x2(v[i + 4], v[i + 5]),
                               pack_bf16x2(v[i + 6], v[i + 7]));
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4 *>(po + (size_t)(c + i) * RS) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
        }
        // (rare) the infinities and NaN of the partly seen tokens that this row sees, added to what its thread has just written
        uint32_t any = 0;
#pragma unroll
        for (int w = 0; w < 2 * kStreamBits; w += 4) {
          const uint4 x = *reinterpret_cast<const uint4 *>(set + w);
          any |= x.x | x.y | x.z | x.w;
        }
        if (__builtin_expect(real && any, 0)) {
#pragma unroll 1
          for (int w = 0; w < 2 * kStreamBits; ++w) {
            for (uint32_t rest = set[w]; rest; rest &= rest - 1) {
              const int at = 32 * (w % kStreamBits) + __ffs((int)rest) - 1, tok = w < kStreamBits ? pos0 + 1 + at : lo_min + at;
              if (tok > pos || (tok < lo_row && tok >= a.first)) continue;
              const size_t page = (size_t)a.block_table[(size_t)b * a.max_pages_per_seq + (tok >> a.log2_page)];
              const uint8_t *vr =
                  a.v_pool + (((page << a.log2_page) + (tok & ((1 << a.log2_page) - 1))) * a.Hkv + g) * (size_t)C::ROWB;
#pragma unroll 1
              for (int d = c0; d < c1; ++d) {
                const float x = cache_value<C::FMT, D>(vr, d);
                if (isfinite(x)) continue;
                if (slot < 0) orow[d] = (uint16_t)pack_bf16x2(__uint_as_float((uint32_t)orow[d] << 16) + x, 0.f);
                else po[(size_t)(d & ~3) * RS + (d & 3)] += x;
              }
            }
          }
        }
        if (real && c0 == 0) {
          if (slot >= 0) a.part_lse[pi] = lse2;
          else if (a.lse) a.lse[(size_t)node_tok * a.Hq + head] = lse2 * LN2;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tc_dealloc(tmem, C::TM_COLS);
  if (tid == 0) a.cta_status[blockIdx.x] = misc->status;
  if (misc->npieces == 0) {
    // a range that held no key can still lie between two pieces of an item: its slot 0 weighs nothing
    for (int h = tid; h < C::QT * kTreeRows; h += C::THREADS)
      a.part_lse[(size_t)blockIdx.x * 2 * C::QT * kTreeRows + h] = -INFINITY;
  }
}

// ---------------------------------------------------------------------------------------- combine
// Grid (CTAs of the split kernel, rows / rows per block): a block for some rows of the item that CTA x begins
// and does not end (at most one).  Its pieces lie in CTAs x, x + hg, ..., in ascending order of the keys.  Which one
// that is and where it ends follow from the partition, which a block works out while the split kernel's last CTAs run;
// behind it only the partial results are loaded.  A warp takes 8 rows x 32 columns: the partials of 8 rows lie beside
// each other, 16 bytes of each.  Several pieces' log-sum-exps and values are loaded together and merged in order.

template <int D, int QT>
__global__ void __launch_bounds__(kCombineThreads, QT == 2 ? 3 : 2) stream_combine_kernel(const StreamArgs a, uint32_t *status) {
  __shared__ TreePart part;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = (int)blockIdx.x, grp = cta / a.hg;
  // the row in which this CTA's range ends, neither with it nor at its start
  uint32_t ignored = 0;
  const long long W = stream_find<kCombineThreads>(a, &part, &ignored, [&](long long W, long long x, long long v) {
    const StreamShares s(a, W);
    return grp < s.groups && s.cut(grp + 1) > x && s.cut(grp + 1) < x + v;
  });
  int k = 0, h = 0;  // pieces of the item; its key head
  StreamRow r = {0, 0, 0};
  StreamSpan span = {};
  if (part.found_b >= 0) {
    const StreamShares s(a, W);
    r = stream_row(a, part.found_b, &ignored);
    const long long end = s.cut(grp + 1);
    const StreamPlace at = stream_place(a, r, end - part.found_x);
    span = stream_span(a, r, at.p);
    const long long begin = end - at.off, last = begin + a.piece_cost + span.cost;
    h = at.h * a.hg + cta % a.hg;
    const int u = stream_unit(a, span, at.off);
    if (u > 0 && u < span.units && stream_unit(a, span, s.cut(grp) - begin) == 0)
      for (k = 2; s.cut(grp + k) < last;) ++k;
  }
  pdl_wait();
  pdl_launch_dependents();
  if (cta == 0 && blockIdx.y == 0 && warp == 0) {
    uint32_t st = 0;
    for (int i = lane; i < a.nparts; i += 32) st |= a.cta_status[i];
    st = __reduce_or_sync(FULL, st);
    if (lane == 0) *status = st;
  }
  if (k == 0) return;
  constexpr int RS = QT * kTreeRows, WPR = D / 32, CHUNK = QT == 2 ? 4 : 8;  // warps for one row; pieces at a time
#pragma unroll 1
  for (int pr = (int)blockIdx.y * combine_rows(D) + warp / WPR * 8 + (lane & 7); pr < RS; pr += (int)gridDim.y * combine_rows(D)) {
    const int row = pr % kTreeRows, qi = row / a.G, i = pr / kTreeRows * a.qt + qi;
    if (qi >= a.qt || i >= span.nq) continue;  // (nothing below is the whole warp's)
    const int c0 = warp % WPR * 32 + (lane >> 3) * 4;  // this lane's values: c0 .. c0 + 3 and c0 + 16 .. c0 + 19
    float M = -INFINITY, Z = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < k; i0 += CHUNK) {
      float lc[CHUNK];
      float4 x[CHUNK][2];
#pragma unroll
      for (int u = 0; u < CHUNK; ++u) {
        lc[u] = -INFINITY;
        x[u][0] = x[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + u < k) {
          const size_t slot = (size_t)(cta + (i0 + u) * a.hg) * 2 + (i0 + u == 0 ? 1 : 0);
          lc[u] = a.part_lse[slot * RS + pr];
          const float *src = a.part_o + slot * RS * D + (size_t)c0 * RS + pr * 4;
          x[u][0] = *reinterpret_cast<const float4 *>(src);
          x[u][1] = *reinterpret_cast<const float4 *>(src + 16 * RS);
        }
      }
      float mn = M;
#pragma unroll
      for (int u = 0; u < CHUNK; ++u) mn = fmaxf(mn, lc[u]);
      const float sc = M == -INFINITY ? 0.f : fast_exp2(M - mn);
      M = mn;
      Z *= sc;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= sc;
#pragma unroll
      for (int u = 0; u < CHUNK; ++u) {
        // an empty piece (lse -inf) weighs nothing, and what lies in its place is not looked at: it was not written
        const float w = lc[u] == -INFINITY ? 0.f : fast_exp2(lc[u] - mn);
        if (w != 0.f) {
          Z += w;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            acc[4 * v] = fmaf(w, x[u][v].x, acc[4 * v]);
            acc[4 * v + 1] = fmaf(w, x[u][v].y, acc[4 * v + 1]);
            acc[4 * v + 2] = fmaf(w, x[u][v].z, acc[4 * v + 2]);
            acc[4 * v + 3] = fmaf(w, x[u][v].w, acc[4 * v + 3]);
          }
        }
      }
    }
    const float inv = Z == 0.f ? 0.f : 1.f / Z;
    const size_t at = (size_t)(r.start + span.i0 + i) * a.Hq + h * a.G + (row - qi * a.G);
#pragma unroll
    for (int v = 0; v < 2; ++v)
      *reinterpret_cast<uint2 *>(a.out + at * D + c0 + 16 * v) =
          make_uint2(pack_bf16x2(acc[4 * v] * inv, acc[4 * v + 1] * inv), pack_bf16x2(acc[4 * v + 2] * inv, acc[4 * v + 3] * inv));
    if (c0 == 0 && a.lse) a.lse[at] = Z == 0.f ? -INFINITY : (M + __log2f(Z)) * LN2;
  }
}

}  // namespace pa
