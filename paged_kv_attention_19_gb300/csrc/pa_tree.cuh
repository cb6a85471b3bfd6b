// pa_tree.cuh -- attention of drafted trees over the paged cache on the 5th-generation tensor cores
// (sm_103a).
//
// Mathematics.  Node i of row b (n nodes; L tokens with them; prefix = L - n) attends to the set A of
// the prefix tokens and of the nodes that its mask names (under a window those fewer than `window`
// positions back, a node's position being prefix + its number of other mask bits):
//   out = sum_{t in A} exp(s_t - m) v_t / l,  lse = m + ln l,  s_t = scale q . k_t,
//   m = max s_t,  l = sum exp(s_t - m).
// One pass over the keys with a running maximum and sum in fp32; the maximum is only raised when it
// grows by more than 2^8, so the weights stay below 2^8 and are rounded once, as the operand of
// the second product (bf16, half a step 2^-8 of each weight; the sum l is of the unrounded ones).
//
// What bounds it.  The cache is read once for all of a key head's query rows, n nodes x G heads of
// them, 4 D flops for each 4 D bytes of keys and values (bf16): memory up to about 280 rows, the
// tensor cores and the exponentials beyond.  16 rows of an mma.sync would read the cache again for
// each 16; here 128 rows are the M of one tcgen05.mma, two such tiles share every staged key.
//
// Work.  A sequence is (row, key head, pair of 128-row tiles); its keys are cut into units of one TMA
// box.  CTAs form groups of HG = sequences per row; a group takes an equal share of all rows' cost
// and CTA r of it serves sequence r, so that the tiles of one key head stream the same pages at the
// same time.  A CTA's range is a list of pieces (runs of one sequence); only its first and its last
// can be part of a sequence that another CTA also touches: at most two partial results a CTA.
//
// Roles of a CTA (one per SM):
//   * warp 0: the K and V tiles of 64 tokens into two rings of slots (TMA, 128-byte swizzle);
//   * warps 1 and 2, one thread each: the products.  Softmax group and output columns x = 0, 1 and two score
//     buffers each belong to thread x: it issues the scores of an item before the second product of the
//     one before it, so that the group has its next scores while its weights are being used.  With two tiles
//     thread x takes tile x of every stage; with one tile the threads take alternate stages of the same
//     rows, and the two outputs are merged at the end of the piece.  (One thread for both spent more time
//     on its waits and commits than the products took.)  A piece has an even number of stages, so that a
//     stage's parity says whose it is; the last may be without tokens;
//   * warp 3: the query tiles of each piece; and looks over V tiles that hold tokens which not every row
//     attends to (the tree, the edge of a window, the ends of a piece) before they are used: a token that
//     nobody attends to becomes zero, and infinities and NaN of the others are taken out of the product and
//     handed to the rows that do attend to them (0 x inf must not reach the ones that do not);
//   * FP8 and NVFP4 pools: the tiles of codes land in a ring of their own, and four more warps convert
//     them to f16 operands (exact; two warps K tiles, two V tiles), and the query rows, scaled by a
//     power of two each, in place; those of the V tiles then look them over.  The weights are rounded to
//     f16 (2^-11);
//   * two groups of four warps: one thread per score row, 32 of its item's scores at a time, for the maximum and
//     then for the weights (read twice: less code than all 64 held, 104 -> 99 us in the case below).
// Code.  The roles' code together passes the instruction cache of an SM (with codes 13% of its requests missed, and
// an SM's misses wait for its neighbours'), so what a stage rarely needs is kept out of its path, and with codes the
// loops over the products' instructions are not unrolled (32 ragged trees of up to 16 nodes x 8 heads over 128 to
// 16384 tokens, 8 key heads of 128: with these steps FP8 137 -> 111 us, NVFP4 134 -> 104, bf16 107 -> 99).
// Measured (GB300; bytes: the cache once): a request of 8 nodes x 32 heads over 1000 tokens 13.6 us, start-up and the
// combine kernel's trips; 16 rows of 64 nodes x 64 heads over 1024 to 8192 tokens 126 to 129 us, 900 to 920 TFLOP/s, the score
// products of N = 64; 16 windowed rows at head_dim 256 57 us, 4.4 TB/s; the ragged trees above 109 us over FP8 (2.1 TB/s
// of codes) and 105 over NVFP4 (1.4 TB/s), the chain from conversion to weights.
// Tensor memory: score buffer b (the weights over its first half) at 64 b, outputs at 256.  At head_dim 256 one
// output fills the rest: one tile, one softmax group and one issuing thread.
#pragma once

#include "pa_common.cuh"
#include "pa_quant.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

enum TreeFmt { TREE_BF16 = 0, TREE_FP8 = 1, TREE_NVFP4 = 2 };
constexpr int kTreeNodes = 64;   // most nodes of a row: bits of a mask
constexpr int kTreeRows = 128;   // query rows of a tile

struct TreeArgs {
  const uint8_t *v_pool;
  const int32_t *block_table, *context_lens, *query_start;
  const uint64_t *tree_mask;
  const int32_t *granted;  // or null: all rows
  uint16_t *out;
  float *lse;           // or null
  uint32_t *cta_status; // [nparts]: PA_DEV_* bits
  float *part_o;        // [nparts, 2, D / 4, QT * 128, 4]: rows beside each other, so that a warp's stores are whole lines
  float *part_lse;      // [nparts, 2, QT * 128], log2 units
  struct TreeHalf *halves;        // [nparts, 2, 128]: the groups' halves of a one-tile piece
  int batch, tokens, max_query, Hq, Hkv, G;
  int gt, qt, nsub;     // a tile: qt nodes x gt heads; nsub tiles for a node's heads (G > 128)
  int nseqh;            // sequences per key head
  int log2_page, log2_bh, num_pages, max_pages_per_seq, max_context_len, window;
  int piece_cost, log2_share, nparts, hg;  // (costs in units)
  float qscale;         // scale * log2(e) (* the keys' scale)
  float vscale;
};

struct TreeHalf {  // one row's state in one softmax group, for the merge of a one-tile piece
  float m, l;
  uint64_t bad_nodes, bad_edge;
};

// Bytes of one head's row of a token in the cache.
__host__ __device__ constexpr int tree_row_bytes(int fmt, int D) {
  return fmt == TREE_BF16 ? 2 * D : fmt == TREE_FP8 ? D : (D / 2 + D / 16 + 15) / 16 * 16;
}

template <int D_, int FMT_, int QT_>
struct TreeCfg {
  static constexpr int D = D_, FMT = FMT_, QT = QT_;
  static constexpr bool QUANT = FMT != TREE_BF16;  // codes in the cache, f16 operands
  static constexpr int ROWB = tree_row_bytes(FMT, D);
  static constexpr int GROUPS = D <= 128 ? 2 : 1;  // softmax groups, and output regions
  static constexpr int BN = 64;                    // tokens per stage
  static constexpr int NB = 4;                     // score buffers
  static constexpr int NPL = D / 64;               // 128-byte swizzle planes of a row
  static constexpr int PLANE = BN * 128, SLOT = NPL * PLANE, QPLANE = kTreeRows * 128;
  static constexpr int Q_BYTES = QT * NPL * QPLANE;
  static constexpr int ROOM = (QUANT ? 228352 : 229376) - Q_BYTES;
  // codes: up to eight slots of a tile each, copied in order K, V, K, V...; operands converted from them
  static constexpr int RAW_SLOT = QUANT ? (BN * ROWB + 1023) / 1024 * 1024 : 0;
  static constexpr int NS_QUANT = D == 64 ? 10 : D == 128 ? (QT == 1 ? 8 : 6) : 3;
  static constexpr int NR_FIT = QUANT ? (ROOM - NS_QUANT * SLOT) / (RAW_SLOT > 0 ? RAW_SLOT : 1) : 0;
  static constexpr int NR = (NR_FIT < 8 ? NR_FIT : 8) & ~1;  // (even: a slot holds tiles of one kind)
  static constexpr int NS_FIT = QUANT ? NS_QUANT : ROOM / SLOT < 12 ? ROOM / SLOT : 12;
  // Two rings of slots: a K tile is free after the scores of its stage, a V tile later.  Copies complete out of order,
  // and a wait for a phase of a slot must not come before the phase before it is known to be complete, so whoever
  // waits for the tiles of one kind, or of one parity of the stages, needs slots that hold those only.
  static constexpr int NK = GROUPS == 1 ? NS_FIT / 2 : NS_FIT / 4 * 2;
  static constexpr int NV = GROUPS == 1 ? NS_FIT - NK : (NS_FIT - NK) / 2 * 2, NS = NK + NV;
  static constexpr int SOFTMAX_WARPS = 4 * GROUPS;
  static constexpr int CONVERT_WARPS = QUANT ? 4 : 0;
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
  static constexpr float TAU = 8.f, LIFT = QUANT ? 7.f : 0.f;
  // score buffer of item i of group (issuing thread) x, and the parity of its use
  __host__ __device__ static constexpr uint32_t buffer(int x, uint32_t i) {
    return GROUPS == 2 ? (uint32_t)x + 2 * (i & 1) : i & 3;
  }
  __host__ __device__ static constexpr uint32_t buffer_phase(uint32_t i) { return GROUPS == 2 ? (i >> 1) & 1 : (i >> 2) & 1; }
  // registers a thread: what the softmax warps hold of a row and its output does not fit the launch's share
  // (384 x 168 or 512 x 128), so the other warps hand some over
  static constexpr bool REG_SPLIT = GROUPS == 2;
  static constexpr int REGS = QUANT ? 128 : 168;
  static constexpr int REGS_CONTROL = QUANT ? 80 : 88, REGS_SOFTMAX = QUANT ? 160 : 208, REGS_CONVERT = 104;
  static_assert(!REG_SPLIT || 128 * REGS_CONTROL + 256 * REGS_SOFTMAX + (QUANT ? 128 * REGS_CONVERT : 0) <= THREADS * REGS,
                "the register split stays within the launch's registers");
  static constexpr int META = 16;  // stage records kept: a record is rewritten sixteen stages later, once the K tile of a
                                   // stage at least six later is free, and with that its own softmax long done
  static_assert(NK >= 1 && NK + NR / 2 <= 10 && (GROUPS == 1 || NK % 2 + NV % 2 == 0), "rings within the records");
  static_assert(QT <= GROUPS, "two tiles need two groups");
  static_assert(NB * BN <= 256 && GROUPS * D <= 256, "tensor-memory budget");
};

enum : int32_t { STAGE_MASKED = 1, STAGE_ABSENT = 2, STAGE_FIRST = 4, STAGE_END = 8 };
struct alignas(16) TreeStage {
  int32_t flags;     // MASKED: not every row attends to every token; ABSENT: no tokens; FIRST: of a piece; END: none follows
  int32_t tok0, tok_hi;
  uint32_t badmask;  // bit k: box k of the stage was not loaded
};
struct alignas(16) TreePieceRec {  // written by the query warp before the piece's query is announced
  int32_t end, stages, two, slot;  // stages with tokens; slot: -1 whole sequence, else partial slot
  int32_t b, L, n, start;
  int32_t t0, g, lo_min, pad;      // first tile, key head, first token that any node's window reaches
};
static_assert(sizeof(TreeStage) == 16 && sizeof(TreePieceRec) == 48, "records of 16-byte words");

struct TreePart {
  int32_t found_b, pad;
  long long found_x, x_begin, x_end, warp_part[16];
};

struct TreeMisc {
  uint32_t status, tmem;
  int32_t npieces, pad;
  TreePart part;
};

template <class C>
struct TreeSmem {
  static constexpr int OFF_RING = C::Q_BYTES;
  static constexpr int OFF_RAW = OFF_RING + C::NS * C::SLOT;
  static constexpr int OFF_META = OFF_RAW + C::NR * C::RAW_SLOT;
  static constexpr int OFF_PIECE = OFF_META + C::META * (int)sizeof(TreeStage);       // [2]
  static constexpr int OFF_NF = OFF_PIECE + 2 * (int)sizeof(TreePieceRec);            // [META][CLEAN_WARPS][2] token bits
  // full[NS], empty[NS], clean[META], q_full, q_empty, s_full[NB], p_ready[NB], pv_done[NB], o_free, half[2], drain[2],
  // q_conv, raw_full[NR], raw_empty[NR]
  static constexpr int OFF_BAR = OFF_NF + C::META * C::CLEAN_WARPS * 16;
  static constexpr int NBAR = 2 * C::NS + C::META + 8 + 3 * C::NB + 2 * C::NR;
  static constexpr int OFF_SHIFT = OFF_BAR + NBAR * 8;  // int8 [2][QT * 128]: exponents of the query rows' scales
  static constexpr int OFF_MISC = OFF_SHIFT + (C::QUANT ? 2 * C::QT * kTreeRows : 0);
  static constexpr int BYTES = OFF_MISC + (int)sizeof(TreeMisc) + 1024;
  static_assert(BYTES <= 232448, "fits the 227 KB opt-in shared memory of one CTA");
};

// ---------------------------------------------------------------------------------------- rows, tiles

struct TreeRow {
  int start, n, L;  // n = 0: nothing to do
};

// Row b, its lengths checked: a bad row has no nodes and sets PA_DEV_BAD_LEN; one that was not granted has none.  (From L2: the combine kernel
// reads them before the grids that come before it are known to it as complete.)
__device__ __forceinline__ TreeRow tree_row(const TreeArgs &a, int b, uint32_t *bad) {
  TreeRow r;
  r.start = __ldcg(a.query_start + b);
  r.L = __ldcg(a.context_lens + b);
  const int end = __ldcg(a.query_start + b + 1);
  r.n = end - r.start;
  if (a.granted && __ldcg(a.granted + b) == 0) {  // (whatever its lengths say)
    r.n = 0;
  } else if (r.start < 0 || end < r.start || end > a.tokens || r.n > a.max_query || r.L < r.n || r.L < 0 ||
      r.L > a.max_context_len) {
    *bad |= PA_DEV_BAD_LEN;
    r.n = 0;
  }
  return r;
}

// First token that some node of the row can see: a node of depth 0 is at position L - n.
__device__ __forceinline__ int tree_lo(const TreeArgs &a, const TreeRow &r) {
  return a.window > 0 ? max(r.L - r.n + 1 - a.window, 0) : 0;
}

// Units of the row's keys: [*u_lo, *u_lo + the returned number).
__device__ __forceinline__ int tree_units(const TreeArgs &a, const TreeRow &r, int *u_lo) {
  *u_lo = tree_lo(a, r) >> a.log2_bh;
  return r.n > 0 ? ((r.L + (1 << a.log2_bh) - 1) >> a.log2_bh) - *u_lo : 0;
}

__device__ __forceinline__ int tree_cost(const TreeArgs &a, const TreeRow &r) {
  int ul;
  const int n = tree_units(a, r, &ul);
  return n > 0 ? n + a.piece_cost : 0;
}

__device__ __forceinline__ int tree_tiles(const TreeArgs &a, int n) {
  return a.nsub > 1 ? n * a.nsub : (n + a.qt - 1) / a.qt;
}

// Tile t: nodes [i0, i0 + nq), heads [h0, h0 + nh) of the group; its row r is node i0 + r / gt, head h0 + r % gt.
struct TreeTile {
  int i0, nq, h0, nh;
};
__device__ __forceinline__ TreeTile tree_tile(const TreeArgs &a, int t, int n) {
  TreeTile x;
  if (a.nsub > 1) {
    x.i0 = t / a.nsub;
    x.nq = 1;
    x.h0 = (t % a.nsub) * kTreeRows;
    x.nh = min(kTreeRows, a.G - x.h0);
  } else {
    x.i0 = t * a.qt;
    x.nq = min(a.qt, n - x.i0);
    x.h0 = 0;
    x.nh = a.G;
  }
  return x;
}

// ---------------------------------------------------------------------------------------- partition
// The rows' costs laid end to end are cut into one equal range per group of HG CTAs (see the top).

template <int THREADS>
__device__ __forceinline__ long long tree_scan(long long v, long long *excl, long long *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  __syncthreads();
  *excl = before + x - v;
  return total;
}

// The rows' total cost W; and the row for which is(W, x, v) holds (at most one; x: the costs of the rows before it, v: its
// own) as found_b (-1: none) and found_x = x.
template <int THREADS, class Is>
__device__ __forceinline__ long long tree_find(const TreeArgs &a, TreePart *ps, uint32_t *bad, const Is &is) {
  const int tid = threadIdx.x;
  if (tid == 0) ps->found_b = -1;
  // up to THREADS rows: one scan gives the total and the place; more: a pass for the total, one for the place
  const bool once = a.batch <= THREADS;
  long long v = 0, ex = 0;
  for (int b = tid; b < a.batch; b += THREADS) v += tree_cost(a, tree_row(a, b, bad));
  const long long W = tree_scan<THREADS>(v, &ex, ps->warp_part);
  long long base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    if (!once) {
      uint32_t again = 0;
      v = b0 + tid < a.batch ? tree_cost(a, tree_row(a, b0 + tid, &again)) : 0;
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

// The groups that work on a total cost W, none on less than 2^log2_share, and their shares: group g has the costs
// [cut(g), cut(g + 1)).
struct TreeShares {
  int groups, more;  // the first `more` groups have one unit of cost more than `each`
  long long each;
  __device__ __forceinline__ TreeShares(const TreeArgs &a, long long W) {
    groups = (int)max(1ll, min((long long)(a.nparts / a.hg), W >> a.log2_share));
    each = W >> 32 ? W / groups : (long long)((uint32_t)W / (uint32_t)groups);
    more = (int)(W - each * groups);
  }
  __device__ __forceinline__ long long cut(int g) const { return g * each + min(g, more); }
  // the group of cost x, x >= cut(g), counted from g
  __device__ __forceinline__ int behind(int g, long long x) const {
    int n = 0;
    while (g + n + 1 < groups && cut(g + n + 1) <= x) ++n;
    return n;
  }
};

// This CTA's range [x_begin, x_end) of the rows' costs, and the row that it begins in.
template <int THREADS>
__device__ __forceinline__ void tree_partition(const TreeArgs &a, TreePart *ps, uint32_t *status) {
  const int grp = (int)blockIdx.x / a.hg;
  uint32_t bad = 0;
  long long xb = 0, xe = 0;
  tree_find<THREADS>(a, ps, &bad, [&](long long W, long long x, long long v) {
    const TreeShares s(a, W);
    xb = grp < s.groups ? s.cut(grp) : 0;
    xe = grp < s.groups ? s.cut(grp + 1) : 0;
    const bool mine = xb < xe && xb >= x && xb < x + v;
    if (mine) {
      ps->x_begin = xb;
      ps->x_end = xe;
    }
    return mine;
  });
  if (bad) atomicOr(status, bad);
}

// One piece: units [ub, ue) of sequence hs of row b.
struct TreePiece {
  int b, hs, ub, ue, start, n, L, t0, g, two;
  bool starts, ends;
};

// Where a piece's results go: -1 the outputs (it is a whole sequence); else the CTA's partial slot 1 (it begins a
// sequence that another CTA ends) or 0.
__device__ __forceinline__ int tree_slot(const TreePiece &p) { return p.starts ? (p.ends ? -1 : 1) : 0; }

// A warp's walk over its CTA's pieces (all lanes call together); each walker sees the same pieces.
struct TreeWalker {
  const TreeArgs &a;
  int lane, hs_row, b_first, in_first;
  long long span, R;
  int rb, w_start, w_n, w_L;  // lane l holds row rb + l
  int it_hs, it_b, it_in;

  __device__ TreeWalker(const TreeArgs &args, const TreePart *ps, int lane_) : a(args), lane(lane_) {
    hs_row = a.Hkv * a.nseqh;
    b_first = max(ps->found_b, 0);
    in_first = ps->found_b >= 0 ? (int)(ps->x_begin - ps->found_x) : 0;
    span = ps->found_b >= 0 ? ps->x_end - ps->x_begin : 0;
    R = span;
    fill(b_first);
    it_hs = (int)blockIdx.x % a.hg;
    it_b = b_first;
    it_in = in_first;
  }
  __device__ void fill(int row) {
    rb = row;
    uint32_t ignored = 0;
    TreeRow r = {0, 0, 0};
    if (rb + lane < a.batch) r = tree_row(a, rb + lane, &ignored);
    w_start = r.start;
    w_n = r.n;
    w_L = r.L;
  }
  __device__ TreeRow row_of(int row) {
    if (row < rb || row >= rb + 32) fill(row);
    TreeRow r;
    r.start = __shfl_sync(FULL, w_start, row - rb);
    r.n = __shfl_sync(FULL, w_n, row - rb);
    r.L = __shfl_sync(FULL, w_L, row - rb);
    return r;
  }

  template <int QT>
  __device__ bool take(TreePiece &pc) {
    while (true) {
      if (R == 0) {
        it_hs += a.hg;
        if (span == 0 || it_hs >= hs_row) return false;
        R = span;
        it_b = b_first;
        it_in = in_first;
      }
      if (it_b >= a.batch) {
        R = 0;  // (what is left of the range lies in rows that exist)
        continue;
      }
      const TreeRow r = row_of(it_b);
      const int w = tree_cost(a, r);
      if (it_in >= w) {
        it_in = 0;
        ++it_b;
        continue;
      }
      const int b = it_b;
      const int take = (int)min((long long)(w - it_in), R);
      const int u0 = max(0, it_in - a.piece_cost), u1 = max(0, it_in + take - a.piece_cost);
      R -= take;
      it_in += take;
      const int t0 = (it_hs % a.nseqh) * QT;
      if (u1 > u0 && t0 < tree_tiles(a, r.n)) {
        int ul;
        const int units = tree_units(a, r, &ul);
        pc.b = b;
        pc.hs = it_hs;
        pc.start = r.start;
        pc.n = r.n;
        pc.L = r.L;
        pc.ub = ul + u0;
        pc.ue = ul + u1;
        pc.starts = u0 == 0;
        pc.ends = u1 == units;
        pc.t0 = t0;
        pc.g = it_hs / a.nseqh;
        pc.two = QT == 2 && t0 + 1 < tree_tiles(a, r.n);
        return true;
      }
    }
  }
};

// ---------------------------------------------------------------------------------------- values, bits

// Value d of a cache row (without the pool's scale).
template <int FMT, int D>
__device__ __forceinline__ float cache_value(const uint8_t *row, int d) {
  if constexpr (FMT == TREE_BF16) {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[d] << 16);
  } else if constexpr (FMT == TREE_FP8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(row[d], __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half *>(&h));
  } else {
    const uint32_t c = (row[d >> 1] >> (4 * (d & 1))) & 15u;
    const float mag = (c & 7u) < 2 ? 0.5f * (float)(c & 7u)
                                   : __uint_as_float((((c & 7u) >> 1) + 126u) << 23 | (c & 1u) << 22);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(row[D / 2 + (d >> 4)], __NV_E4M3);
    return (c & 8u ? -mag : mag) * __half2float(*reinterpret_cast<const __half *>(&h));
  }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Of 8 bf16 values: the largest magnitude (NaN aside); a pair times a power of two as an f16 pair.
__device__ __forceinline__ float absmax8(uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
  return m;
}
__device__ __forceinline__ uint32_t scaled_f16x2(uint32_t pair, float p2) {
  return pack_f16x2(__uint_as_float(pair << 16) * p2, __uint_as_float(pair & 0xffff0000u) * p2);
}

// Values 16 pc .. 16 pc + 15 of a row of codes as f16 pairs, without the pool's scale: exact (an E2M1 value
// times an E4M3 block scale has at most six significant bits and lies in [2^-10, 2688]).
template <int FMT, int D>
struct Codes16 {
  uint4 x;
  __device__ __forceinline__ void load(const uint8_t *row, int pc) {
    if constexpr (FMT == TREE_FP8) {
      x = *reinterpret_cast<const uint4 *>(row + 16 * pc);
    } else {
      const uint2 c = *reinterpret_cast<const uint2 *>(row + 8 * pc);
      x = make_uint4(c.x, c.y, row[D / 2 + pc], 0u);
    }
  }
  __device__ __forceinline__ void convert(uint32_t (&h)[8]) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (FMT == TREE_FP8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
        h[e] = (uint32_t)r.x | ((uint32_t)r.y << 16);
      }
    } else {
      const __half_raw b = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)w[2], __NV_E4M3);
      const __half2 by = __half2half2(*reinterpret_cast<const __half *>(&b));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w[e >> 2] >> (8 * (e & 3))), __NV_E2M1);
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&r), by);
        h[e] = *reinterpret_cast<const uint32_t *>(&v);
      }
    }
  }
};

// The low k bits (k clamped to [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int k) { return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u; }

// Bits of the 32 tokens from `base` on that lie in [lo, hi).
__device__ __forceinline__ uint32_t range_bits(int base, int lo, int hi) {
  return low_bits(hi - base) & ~low_bits(lo - base);
}

// Bits of the 32 tokens from `base` on of a 64-bit mask whose bit 0 is token `at`.
__device__ __forceinline__ uint32_t mask_bits(uint64_t m, int at, int base) {
  const int s = base - at;
  return s >= 64 || s <= -32 ? 0u : s >= 0 ? (uint32_t)(m >> s) : (uint32_t)(m << -s);
}

// Bits of the tokens of chunk c (32 tokens of a stage) whose boxes were loaded.
__device__ __forceinline__ uint32_t loaded_bits(uint32_t badmask, int c, int log2_bh) {
  if (badmask == 0) return ~0u;
  if (log2_bh >= 5) return (badmask >> ((32 * c) >> log2_bh)) & 1u ? 0u : ~0u;
  uint32_t ok = 0;
  const int per = 32 >> log2_bh;
  for (int k = 0; k < per; ++k)
    if (!((badmask >> (c * per + k)) & 1u)) ok |= low_bits(1 << log2_bh) << (k << log2_bh);
  return ok;
}

// ---------------------------------------------------------------------------------------- tensor memory
// Warp-wide: lane l reads 32 consecutive columns of tensor-memory lane (taddr.lane + l) at each of two addresses.
// The wait is part of the statement: no use of the values can be moved before it.
__device__ __forceinline__ void tree_ld_pair(uint32_t ta, uint32_t tb, float (&v)[32], float (&u)[32]) {
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
      : "r"(ta), "r"(tb));
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = __uint_as_float(r[i]);
    u[i] = __uint_as_float(r[32 + i]);
  }
}
// Pairs of fp32 in one instruction: a * b + c, and a + b.
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// One thread of a converged warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}

// A bounded wait of a whole warp, with one answer: a lane that gave up by itself would leave the others waiting for it at the
// warp's next common instruction, without a limit.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *status) {
  const bool ok = mbar_wait_warp(bar, parity, WAIT_LIMIT_NS);
  if (!ok && (threadIdx.x & 31) == 0) atomicOr(status, PA_DEV_TIMEOUT);
  return ok;
}

// ---------------------------------------------------------------------------------------- the kernel

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    tree_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_q, const TreeArgs a) {
  using S = TreeSmem<C>;
  constexpr int D = C::D, BN = C::BN, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::OFF_BAR), *empty = full + NS, *clean = empty + NS;
  uint64_t *q_full = clean + C::META, *q_empty = q_full + 1, *s_full = q_full + 2, *p_ready = s_full + C::NB,
           *pv_done = p_ready + C::NB, *o_free = pv_done + C::NB, *half_in = o_free + 1, *drain = half_in + 2, *q_conv = drain + 2,
           *raw_full = q_conv + 1, *raw_empty = raw_full + C::NR;
  TreeStage *meta = reinterpret_cast<TreeStage *>(smem + S::OFF_META);
  TreePieceRec *prec = reinterpret_cast<TreePieceRec *>(smem + S::OFF_PIECE);
  uint64_t *nf = reinterpret_cast<uint64_t *>(smem + S::OFF_NF);
  TreeMisc *misc = reinterpret_cast<TreeMisc *>(smem + S::OFF_MISC);
  uint32_t *status = &misc->status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], C::QUANT ? C::TILE_WARPS : 1);
      mbar_init(&empty[s], C::GROUPS);  // an arrival of each issuing thread (both of one where the stage is its own)
    }
    for (int s = 0; s < C::META; ++s) mbar_init(&clean[s], C::CLEAN_WARPS);
    for (int s = 0; s < C::NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], C::TILE_WARPS);
    }
    mbar_init(q_conv, C::QUANT ? C::TILE_WARPS : 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, C::GROUPS);
    for (int b = 0; b < C::NB; ++b) {
      mbar_init(&s_full[b], 2);  // the scores' commit and the issuing thread's arrive
      mbar_init(&p_ready[b], 4);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(&half_in[0], 4);
    mbar_init(&half_in[1], 4);
    mbar_init(o_free, C::SOFTMAX_WARPS);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    fence_mbar_init();
    misc->status = 0;
    misc->npieces = 0;
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
  tree_partition<C::THREADS>(a, &misc->part, status);

  if (warp < 4) {
  if constexpr (C::REG_SPLIT) setmaxnreg_dec<C::REGS_CONTROL>();
  if (warp == 0) {
    // ------------------------------------------------------------ K and V tiles
    const int nbox = BN >> a.log2_bh, P = 1 << a.log2_page;
    uint32_t t = 0;
    int in_flight = 0;  // tiles of stage t whose copies were issued
    // where tile kv of stage t goes: slot, its phase, and the barriers of the ring
    auto place = [&](int kv, uint32_t &u) -> int {
      if constexpr (C::QUANT) {
        u = (2 * t + kv) / C::NR;
        return (2 * t + kv) % C::NR;
      } else {
        u = kv ? t / C::NV : t / C::NK;
        return kv ? C::NK + t % C::NV : t % C::NK;
      }
    };
    uint64_t *const r_full = C::QUANT ? raw_full : full, *const r_empty = C::QUANT ? raw_empty : empty;
    bool ok = true;
    TreeWalker walker(a, &misc->part, lane);
    int npieces = 0;
    auto window_of = [&](const TreePiece &p, int w) {  // block-table entries [32 w, 32 w + 32) of a piece
      const int pb = (p.ub << a.log2_bh) >> a.log2_page;
      const int np = ((((p.ue << a.log2_bh) - 1) >> a.log2_page) + 1) - pb;
      return 32 * w + lane < np ? a.block_table[(size_t)p.b * a.max_pages_per_seq + pb + 32 * w + lane] : 0;
    };
    TreePiece cur = {}, nxt = {};
    int cwin = 0, nwin = 0;
    for (bool has = false;;) {  // cur, if there is one, with the piece behind it known
      const bool has_next = walker.take<C::QT>(nxt);
      if (has_next) nwin = window_of(nxt, 0);
      if (has) {
        const int prefix = cur.L - cur.n;
        // every node sees the tokens [lo_max, prefix): depths are below n
        const int lo_max = a.window > 0 ? max(cur.L - a.window, 0) : 0;
        const int tok_hi = min(cur.L, cur.ue << a.log2_bh);
        const int n_stages = (cur.ue - cur.ub + nbox - 1) / nbox;
        const int pb = (cur.ub << a.log2_bh) >> a.log2_page;
        int wi = 0, fwin = window_of(cur, 1);
        for (int st = 0; st < ((n_stages + 1) & ~1) && ok; ++st) {  // (the last one may be without tokens)
          const int unit0 = cur.ub + st * nbox, tok0 = unit0 << a.log2_bh;
          // the pages of one stage never straddle a window of 32 (nbox divides 32)
          const int pwin = ((tok0 >> a.log2_page) - pb) >> 5;
          while (wi < pwin) {
            cwin = fwin;
            ++wi;
            fwin = window_of(cur, wi + 1);
          }
          const int unit = unit0 + lane, btok = unit << a.log2_bh;
          const int phys = __shfl_sync(FULL, cwin, ((btok >> a.log2_page) - pb) & 31);
          bool load = false, isbad = false;
          if (lane < nbox && unit < cur.ue) {
            load = phys >= 0 && phys < a.num_pages;
            isbad = !load;
            if (isbad) atomicOr(status, PA_DEV_BAD_PAGE);
          }
          const uint32_t bad = __ballot_sync(FULL, isbad);
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(FULL, load)) * (uint32_t)(C::ROWB << a.log2_bh);
#pragma unroll
          for (int kv = 0; kv < 2 && ok; ++kv) {
            uint32_t u;
            const int s = place(kv, u);
            if (u > 0) ok = warp_wait(&r_empty[s], (u - 1) & 1, status);
            if (!ok) break;
            in_flight = kv + 1;
            if (lane == 0) {
              if (kv == 0) {
                TreeStage m;
                m.flags = st >= n_stages ? STAGE_ABSENT
                                         : (tok0 + BN > min(prefix, tok_hi) || tok0 < lo_max || bad != 0 ? STAGE_MASKED : 0);
                if (st == 0) m.flags |= STAGE_FIRST;
                m.tok0 = tok0;
                m.tok_hi = tok_hi;
                m.badmask = bad;
                meta[t % C::META] = m;
              }
              mbar_arrive_expect_tx(&r_full[s], bytes);
            }
            __syncwarp();
            if (load) {
              if constexpr (C::QUANT) {  // whole rows of codes, one after the other
                tma_load_4d(smem + S::OFF_RAW + s * C::RAW_SLOT + (lane << a.log2_bh) * C::ROWB, kv ? &tm_v : &tm_k, 0, cur.g,
                            btok & (P - 1), phys, &r_full[s]);
              } else {
                uint8_t *dst = smem + S::OFF_RING + s * C::SLOT + (lane << a.log2_bh) * 128;
#pragma unroll
                for (int p = 0; p < C::NPL; ++p)
                  tma_load_4d(dst + p * C::PLANE, kv ? &tm_v : &tm_k, p * 64, cur.g, btok & (P - 1), phys, &full[s]);
              }
            }
          }
          if (ok) {
            ++t;
            in_flight = 0;
          }
        }
        if (!ok) break;
        ++npieces;
      }
      if (!has_next) break;
      has = true;
      cur = nxt;
      cwin = nwin;
    }
    // the end, for the converting warps: the next stage's tiles, which are none
    for (int kv = 0; C::QUANT && kv < 2 && ok; ++kv) {
      uint32_t u;
      const int s = place(kv, u);
      if (u > 0) ok = warp_wait(&r_empty[s], (u - 1) & 1, status);
      if (ok && lane == 0) {
        if (kv == 0) meta[t % C::META].flags = STAGE_END;
        mbar_arrive(&r_full[s]);
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
    // first one, which the compiler cannot know to be alone, each instruction's operands take a detour, 64-node trees
    // 147 -> 133 us)
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
      // the scores of the next item: query tile qx, stage t
      auto begin = [&](uint32_t t, int qx, bool present, bool alone) -> bool {
        const uint32_t b = buf(c);
        constexpr uint32_t BACK = C::NB / C::GROUPS;  // items since this buffer's last
        if (!mbar_wait(&full[t % C::NK], (t / C::NK) & 1, status)) return false;
        if (c >= BACK && !mbar_wait(&pv_done[b], par(c - BACK), status)) return false;
        if (present) {
          tc_fence_after();
          const uint64_t qd = tc_sdesc_sw128(qb + qx * (C::NPL * C::QPLANE), 16, 1024);
          const uint64_t kd = tc_sdesc_sw128(ring + (t % C::NK) * C::SLOT, 16, 1024);
#pragma unroll(C::QUANT ? 1 : C::NPL)
          for (int p = 0; p < C::NPL; ++p)
#pragma unroll(C::QUANT ? 1 : 4)
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_ss(tmem + C::TM_S + b * BN, qd + (uint64_t)((p * C::QPLANE + 32 * kk) >> 4),
                        kd + (uint64_t)((p * C::PLANE + 32 * kk) >> 4), C::IDESC_S, (p | kk) != 0 ? 1u : 0u);
          tc_commit(&s_full[b]);
        } else {
          mbar_arrive(&s_full[b]);  // no scores: the record alone
        }
        mbar_arrive(&s_full[b]);
        release(&empty[t % C::NK], present, alone);
        ++c;
        return true;
      };
      // the second product of the oldest item; first: of this thread in the piece
      auto finish = [&](uint32_t t, uint32_t piece, bool first, bool present, bool alone) -> bool {
        const uint32_t b = buf(d), vs = C::NK + t % C::NV;
        if (!mbar_wait(&p_ready[b], par(d), status)) return false;
        // the previous piece's outputs have been read, and all its V tiles with that
        if (first && piece > 0 && !mbar_wait(o_free, (piece - 1) & 1, status)) return false;
        // (bf16: whoever looked it over has waited for it)
        if (C::QUANT ? !mbar_wait(&full[vs], (t / C::NV) & 1, status)
                     : !mbar_wait(&clean[t % C::META], (t / C::META) & 1, status))
          return false;
        if (present) {
          tc_fence_after();
          const int o = C::GROUPS == 2 ? x : 0;
          const uint64_t vd = tc_sdesc_sw128(ring + vs * C::SLOT, C::PLANE, 1024);
#pragma unroll(C::QUANT ? 1 : BN / 16)
          for (int kk = 0; kk < BN / 16; ++kk)
            tc_mma_ts(tmem + C::TM_O + o * D, tmem + C::TM_S + b * BN + 8 * kk, vd + (uint64_t)((kk * 16 * 128) >> 4),
                      C::IDESC_PV, first && kk == 0 ? 0u : 1u);
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
        if (r.x) {
          for (int k = 0; k < 2; ++k) mbar_arrive(&s_full[buf(c)]);  // the softmax groups stop here
          break;
        }
        const uint32_t n = (uint32_t)r.y, even = (n + 1) & ~1u;
        const bool two = r.z != 0, alone = !two;
        // this thread's stages: all of them, or every other one
        const uint32_t j0 = C::GROUPS == 2 && !two ? (uint32_t)x : 0, dj = C::GROUPS == 2 && !two ? 2 : 1;
        // the second product of an item behind the scores of the next one
        for (uint32_t j = j0; j < even + dj && ok; j += dj) {
          if (j < even) ok = begin(t0 + j, two ? x : 0, j < n, alone);
          if (j < even && j + dj >= even) tc_commit(q_empty);
          if (ok && j > j0) ok = finish(t0 + j - dj, piece, j == j0 + dj, j - dj < n, alone);
        }
        t0 += even;
      }
      // every operation of this thread has completed before the tensor memory is released
      tc_commit(&drain[x]);
      mbar_wait(&drain[x], 0, status);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ query tiles; V tiles looked over (bf16)
    TreeWalker walker(a, &misc->part, lane);
    TreePiece pc;
    uint32_t k = 0, t = 0;
    const int nbox = BN >> a.log2_bh;
    int stages = 0;
    bool ok = true;
    // the last piece's scores are done: of all the kernel's waits the one that lasts as long as a piece.  65536 stages
    // take some 60 ms; a second more for each
    auto scored = [&]() -> bool {
      const bool r = mbar_wait_warp(q_empty, (k - 1) & 1, WAIT_LIMIT_NS * (1 + ((uint64_t)stages >> 16)));
      if (!r && lane == 0) atomicOr(status, PA_DEV_TIMEOUT);
      return r;
    };
    while (ok && walker.take<C::QT>(pc)) {
      if (k > 0) ok = scored();
      if (!ok) break;
      stages = (pc.ue - pc.ub + nbox - 1) / nbox;
      const TreeRow row = {pc.start, pc.n, pc.L};
      const int prefix = pc.L - pc.n, lo_min = tree_lo(a, row), lo_max = a.window > 0 ? max(pc.L - a.window, 0) : 0;
      if (lane == 0) {
        prec[k & 1] = TreePieceRec{0, stages, pc.two, tree_slot(pc), pc.b, pc.L, pc.n, pc.start, pc.t0, pc.g, lo_min, 0};
        const int boxes = min(a.qt, a.max_query) * a.gt * 128;  // bytes of one plane's box
        mbar_arrive_expect_tx(q_full, (uint32_t)(C::NPL * boxes * (pc.two ? 2 : 1)));
        for (int x = 0; x < (pc.two ? 2 : 1); ++x) {
          const TreeTile tl = tree_tile(a, pc.t0 + x, pc.n);
#pragma unroll
          for (int p = 0; p < C::NPL; ++p)
            tma_load_3d(smem + (x * C::NPL + p) * C::QPLANE, &tm_q, p * 64, pc.g * a.G + tl.h0, pc.start + tl.i0, q_full);
        }
      }
      __syncwarp();
      ++k;
      if constexpr (!C::QUANT) {
        for (int st = 0; st < ((stages + 1) & ~1) && ok; ++st, ++t) {
          const int s = C::NK + t % C::NV;
          ok = warp_wait(&full[s], (t / C::NV) & 1, status);
          if (!ok) break;
          const int4 m = *reinterpret_cast<const int4 *>(&meta[t % C::META]);  // flags, tok0, tok_hi, badmask
          if (m.x & STAGE_MASKED) {
            uint64_t bad_nodes = 0, bad_edge = 0;
            uint8_t *v = smem + S::OFF_RING + s * C::SLOT;
            for (int r = lane; r < BN; r += 32) {
              const int tok = m.y + r;
              const bool any = tok >= lo_min && tok < m.z && ((loaded_bits((uint32_t)m.w, r >> 5, a.log2_bh) >> (r & 31)) & 1u);
              const bool some = tok >= prefix || tok < lo_max;  // seen by some nodes and not by others
              if (any && !some) continue;
              bool found = false;
#pragma unroll 4
              for (int c = 0; c < C::NPL * 8; ++c) {
                uint4 *p = reinterpret_cast<uint4 *>(v + (c >> 3) * C::PLANE + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                if (!any) {
                  *p = make_uint4(0, 0, 0, 0);
                  continue;
                }
                uint4 x = *p;
                uint32_t w[4] = {x.x, x.y, x.z, x.w}, hit = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // exponents of all ones: infinities and NaN
                  const uint32_t bits = ((w[e] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w[e] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
                  hit |= bits;
                  w[e] &= ~bits;
                }
                if (hit) {
                  found = true;
                  *p = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
              if (found) {
                if (tok >= prefix) bad_nodes |= 1ull << (tok - prefix);
                else bad_edge |= 1ull << (tok - lo_min);
              }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
              bad_nodes |= __shfl_xor_sync(FULL, bad_nodes, o);
              bad_edge |= __shfl_xor_sync(FULL, bad_edge, o);
            }
            if (lane == 0) {
              nf[(t % C::META) * 2] = bad_nodes;
              nf[(t % C::META) * 2 + 1] = bad_edge;
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
      int prefix = 0, lo_min = 0, lo_max = 0;
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
          const TreePieceRec &r = prec[kp & 1];
          if (!(m.x & STAGE_END)) {
            prefix = r.L - r.n;
            lo_min = r.lo_min;
            lo_max = a.window > 0 ? max(r.L - a.window, 0) : 0;
            const bool two = r.two != 0;
            // times 2^s (largest magnitude in [2^14, 2^15)) to f16, in place
            int8_t *shift = reinterpret_cast<int8_t *>(smem + S::OFF_SHIFT) + (kp & 1) * (C::QT * kTreeRows);
            for (int r = tt; r < (two ? 2 : 1) * kTreeRows; r += STEP) {
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
          uint64_t bad_nodes = 0, bad_edge = 0;
          auto put = [&](int r, int pc, const uint32_t (&h)[8]) {
            uint8_t *row = op + (pc >> 2) * C::PLANE + r * 128;
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
#pragma unroll 1
            for (int i = 0; i < NTASK / STEP; ++i) {
              const int r = r0 + i * (STEP / TPR), tok = m.y + r;
              Codes16<C::FMT, D> x;
              uint32_t h[8];
              x.load(raw + r * C::ROWB, pc);
              x.convert(h);
              const bool any = tok >= lo_min && tok < m.z && ((loaded_bits((uint32_t)m.w, r >> 5, a.log2_bh) >> (r & 31)) & 1u);
              if (!any) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = 0u;
              } else if (tok >= prefix || tok < lo_max) {
                uint32_t hit = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint32_t bits = ((h[e] & 0x7c00u) == 0x7c00u ? 0xffffu : 0u) |
                                        ((h[e] & 0x7c000000u) == 0x7c000000u ? 0xffff0000u : 0u);
                  hit |= bits;
                  h[e] &= ~bits;
                }
                if (hit) {
                  if (tok >= prefix) bad_nodes |= 1ull << (tok - prefix);
                  else bad_edge |= 1ull << (tok - lo_min);
                }
              }
              put(r, pc, h);
            }
          }
          if (__builtin_expect(look, 0)) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
              bad_nodes |= __shfl_xor_sync(FULL, bad_nodes, o);
              bad_edge |= __shfl_xor_sync(FULL, bad_edge, o);
            }
            if (lane == 0) {
              const int w = cw % C::TILE_WARPS;
              nf[((t % C::META) * C::CLEAN_WARPS + w) * 2] = bad_nodes;
              nf[((t % C::META) * C::CLEAN_WARPS + w) * 2 + 1] = bad_edge;
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
    float m_run = -INFINITY, l_run = 0.f, qs = scale;
    uint32_t kp = 0;  // pieces begun
    uint64_t eff = 0, bad_nodes = 0, bad_edge = 0;
    int lo_row = 0, prefix = 0, node_tok = 0, head = 0, start = 0, n = 0, lo_min = 0, b = 0, slot = -1, g = 0, prow = 0;
    bool real = false, warp_real = false, had = false;  // had: this group's output has had a product in the piece
    uint32_t c = 0, k_half = 0;  // items done; merges
    uint32_t t0 = 0;             // the piece's first stage
    bool ok = true;
    auto buf = [&](uint32_t i) { return C::buffer(grp, i); };
    auto par = [&](uint32_t i) { return C::buffer_phase(i); };
    int seen = -1;  // the stage of the item before, if its V tile was looked over: what was found is not taken up yet
    auto take_up = [&]() -> bool {  // (its second product is complete)
      if (seen < 0) return true;
      if (!warp_wait(&clean[seen % C::META], (seen / C::META) & 1, status)) return false;
#pragma unroll
      for (int w = 0; w < C::CLEAN_WARPS; ++w) {
        bad_nodes |= nf[((seen % C::META) * C::CLEAN_WARPS + w) * 2];
        bad_edge |= nf[((seen % C::META) * C::CLEAN_WARPS + w) * 2 + 1];
      }
      seen = -1;
      return true;
    };

    // the group's next item: stage tt, whose record is m (flags, tok0, tok_hi, badmask)
    auto item = [&](uint32_t tt, int4 m) -> bool {
      const uint32_t tS = tl_base + C::TM_S + buf(c) * BN;
      const int o = C::GROUPS == 2 ? grp : 0;
      const uint32_t tO = tl_base + C::TM_O + o * D;
      if (warp_real && !(m.x & STAGE_ABSENT)) {
        if (__builtin_expect(seen >= 0, 0)) {  // of the item before, whose record is soon another's
          if (!warp_wait(&pv_done[buf(c - 1)], par(c - 1), status) || !take_up()) return false;
        }
        const bool masked = m.x & STAGE_MASKED;
        if (__builtin_expect(masked || flip != 1.f, 0)) {
          // (few stages, or a scale that is not positive: what the code below would carry along in every stage, and
          // the instruction cache with it)
          if (masked) seen = (int)tt;
#pragma unroll 1
          for (int k = 0; k < BN / 32; ++k) {
            const int base = m.y + 32 * k;
            const uint32_t vis = masked ? (range_bits(base, lo_row, prefix) | mask_bits(eff, prefix, base)) & range_bits(base, 0, m.z) &
                                              loaded_bits((uint32_t)m.w, k, a.log2_bh)
                                        : ~0u;
            float v[32];
            tc_ld32(tS + 32 * k, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = (vis >> i) & 1u ? v[i] * flip : -INFINITY;
            tc_st32(tS + 32 * k, v);
          }
          tc_wait_st();
        }
        float mx = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < BN / 32; ++k) {
          float v[32];
          tc_ld32(tS + 32 * k, v);
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], fmaxf(v[i + e], v[i + 4 + e]));
          mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
        }
        mx = mx * qs - C::LIFT;
        if (!had) {
          m_run = mx;
        } else if (__builtin_expect(__any_sync(FULL, real && m_run != -INFINITY && mx > m_run + C::TAU), 0)) {
          // raise the maximum: the output so far is scaled, once its products are complete
          if (!warp_wait(&pv_done[buf(c - 1)], par(c - 1), status)) return false;
          tc_fence_after();
          // (only of rows past the threshold, so that no row's rounding depends on what its neighbours attend to)
          const bool raise = m_run == -INFINITY || mx > m_run + C::TAU;
          const float al = raise && m_run != -INFINITY ? fast_exp2(m_run - mx) : 1.f;
          if (raise) m_run = mx;
          l_run *= al;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float v[32];
            tc_ld32(tO + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= al;
            tc_st32(tO + c, v);
          }
          tc_wait_st();
        } else if (m_run == -INFINITY) {
          m_run = mx;  // nothing attended to so far: the output is zero
        }
        const float sub = m_run == -INFINITY ? 0.f : m_run;
        const float2 q2 = make_float2(qs, qs), sub2 = make_float2(-sub, -sub);
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int k = 0; k < BN / 32; ++k) {
          uint32_t w[16];
          float x[32];
          tc_ld32(tS + 32 * k, x);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 y = fma_pair(make_float2(x[i], x[i + 1]), q2, sub2);
            const float2 pr = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            l2[(i >> 1) & 1] = add_pair(l2[(i >> 1) & 1], pr);
            w[i >> 1] = C::QUANT ? pack_f16x2(pr.x, pr.y) : pack_bf16x2(pr.x, pr.y);
          }
          tc_st16(tS + 16 * k, w);
        }
        l2[0] = add_pair(l2[0], l2[1]);
        l_run += l2[0].x + l2[0].y;
        tc_wait_st();
        had = true;
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
      const uint32_t stages = (uint32_t)r0.y, even = (stages + 1) & ~1u;
      const bool two = r0.z != 0;
      slot = r0.w;
      b = r1.x;
      n = r1.z;
      prefix = r1.y - n;
      start = r1.w;
      g = r2.y;
      lo_min = r2.z;
      {
        const int tx = two ? grp : 0;
        const TreeTile tile = tree_tile(a, r2.x + tx, n);
        const int pos = row / a.gt, h = row - pos * a.gt;
        real = pos < tile.nq && h < tile.nh;
        warp_real = __any_sync(FULL, real);
        prow = tx * kTreeRows + row;
        if constexpr (C::QUANT) {  // the scores are 2^s times too large
          const int sh = reinterpret_cast<const int8_t *>(smem + S::OFF_SHIFT)[(kp & 1) * (C::QT * kTreeRows) + prow];
          qs = scale * __uint_as_float((uint32_t)(127 - sh) << 23);
        }
        head = g * a.G + tile.h0 + h;
        node_tok = start + tile.i0 + pos;
        eff = 0;
        lo_row = 0;
        if (real) {
          const uint64_t keep = n < 64 ? (1ull << n) - 1 : ~0ull;
          const int node = tile.i0 + pos;
          eff = a.tree_mask[node_tok] & keep;
          if (a.window > 0) {
            const int depth = __popcll(eff & ~(1ull << node));
            lo_row = max(prefix + depth - a.window + 1, 0);
            for (uint64_t rest = eff; rest; rest &= rest - 1) {
              const int j = __ffsll((long long)rest) - 1;
              const uint64_t mj = a.tree_mask[start + j] & keep;
              if (depth - __popcll(mj & ~(1ull << j)) >= a.window) eff &= ~(1ull << j);
            }
          }
        }
      }
      ++kp;
      m_run = -INFINITY;
      l_run = 0.f;
      bad_nodes = bad_edge = 0;
      had = false;
      const uint32_t j0 = C::GROUPS == 2 && !two ? (uint32_t)grp : 0, dj = C::GROUPS == 2 && !two ? 2 : 1;
      for (uint32_t j = j0; j < even && ok; j += dj) {
        if (j != j0) {
          ok = warp_wait(&s_full[buf(c)], par(c), status);
          if (!ok) break;
          tc_fence_after();
        }
        ok = item(t0 + j, *reinterpret_cast<const int4 *>(&meta[(t0 + j) % C::META]));
      }
      if (!ok) break;
      t0 += even;

      // ---- end of a piece: the products of the last item, and with them all before, are complete
      ok = warp_wait(&pv_done[buf(c - 1)], par(c - 1), status) && take_up();
      if (!ok) break;
      TreeHalf other = {-INFINITY, 0.f, 0, 0};
      const bool merge = C::GROUPS == 2 && !two;
      if (merge) {  // both groups have had as many items
        TreeHalf *mine = a.halves + ((size_t)blockIdx.x * 2 + grp) * kTreeRows + row;
        *mine = TreeHalf{m_run, l_run, bad_nodes, bad_edge};
        __syncwarp();
        if (lane == 0) mbar_arrive(&half_in[grp]);
        ok = warp_wait(&half_in[grp ^ 1], k_half & 1, status) && warp_wait(&pv_done[C::buffer(grp ^ 1, c - 1)], par(c - 1), status);
        if (!ok) break;
        ++k_half;
        other = a.halves[((size_t)blockIdx.x * 2 + (grp ^ 1)) * kTreeRows + row];
        bad_nodes |= other.bad_nodes;
        bad_edge |= other.bad_edge;
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
      // tokens with infinities or NaN that this row attends to
      uint64_t hit_nodes = bad_nodes & eff, hit_edge = bad_edge;
      if (hit_edge) hit_edge = lo_row - lo_min >= 64 ? 0 : hit_edge >> (lo_row - lo_min) << (lo_row - lo_min);
      if (warp_real) {
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          float v[32], u[32];
          if (merge) {
            tree_ld_pair(tl_base + C::TM_O + o * D + c, tl_base + C::TM_O + (o ^ 1) * D + c, v, u);
          } else {
            tc_ld32(tl_base + C::TM_O + o * D + c, v);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = use_own ? v[i] * s_own : 0.f;
          if (merge) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = use_oth ? fmaf(u[i], s_oth, v[i]) : v[i];
          }
          if (real) {
            if (slot < 0) {
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4 *>(orow + c + i) =
                    make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]), pack_bf16x2(v[i + 4], v[i + 5]),
                               pack_bf16x2(v[i + 6], v[i + 7]));
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4 *>(po + (size_t)(c + i) * RS) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
        }
        if (real && (hit_nodes | hit_edge)) {
          // (rare) their infinities and NaN, added to what this thread has just written
          for (int half = 0; half < 2; ++half) {
            for (uint64_t rest = half ? hit_edge : hit_nodes; rest; rest &= rest - 1) {
              const int tok = (half ? lo_min : prefix) + __ffsll((long long)rest) - 1;
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
    // a range that held no key can still lie between two pieces of a sequence: its slot 0 weighs nothing
    for (int h = tid; h < C::QT * kTreeRows; h += C::THREADS)
      a.part_lse[(size_t)blockIdx.x * 2 * C::QT * kTreeRows + h] = -INFINITY;
  }
}

// ---------------------------------------------------------------------------------------- combine
// Grid (CTAs of the split kernel, rows / rows per block): a block for some rows of the sequence that CTA x begins
// and does not end (at most one).  Its pieces lie in CTAs x, x + HG, ..., in ascending order of the keys.  Which one
// that is and where it ends follow from the partition, which a block works out while the split kernel's last CTAs run;
// behind it only the partial results are loaded.  A warp takes 8 rows x 32 columns: the partials of 8 rows lie beside
// each other, 16 bytes of each.  Eight pieces' log-sum-exps and values are loaded together and merged in order; of
// sequences of two tiles, whose many rows want more warps and which are cut into fewer pieces, four (64-node trees
// 153 -> 149 us; a single request of one tile, cut into 19, would lose 15.8 -> 16.7).  At most four blocks share a
// sequence's rows (64-node trees: two 152, four 153, sixteen, one for each 16 rows, 158 us; windowed at head_dim 256:
// 59.5, 57.3, 59.7).

constexpr int kCombineThreads = 256, kCombineBlocks = 4;  // most blocks for one sequence
__host__ __device__ constexpr int combine_rows(int D) { return 8 * (kCombineThreads / 32) / (D / 32); }  // rows of a block

// The rows that a sequence can have: of a single tile those that it holds.
__host__ __device__ inline int tree_max_rows(const TreeArgs &a, int QT) {
  const int nodes = a.qt < a.max_query ? a.qt : a.max_query;
  return a.nseqh * QT > 1 ? QT * kTreeRows : a.gt * nodes;
}

template <int D, int QT>
__global__ void __launch_bounds__(kCombineThreads, QT == 2 ? 3 : 2) tree_combine_kernel(const TreeArgs a, uint32_t *status) {
  __shared__ TreePart part;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = (int)blockIdx.x;
  const int grp = cta / a.hg, hs = cta % a.hg;
  // the row whose first unit lies in this range, and whose last one does not; k: the ranges that it lies in
  uint32_t ignored = 0;
  const long long W = tree_find<kCombineThreads>(a, &part, &ignored, [&](long long W, long long x, long long v) {
    const TreeShares s(a, W);
    const long long first = x + a.piece_cost;
    return grp < s.groups && s.cut(grp) <= first && first < s.cut(grp + 1) && s.cut(grp + 1) < x + v;
  });
  const int b = part.found_b;
  const TreeRow r = b >= 0 ? tree_row(a, b, &ignored) : TreeRow{0, 0, 0};
  const long long end = b >= 0 ? part.found_x + tree_cost(a, r) : 0;
  const int k = b >= 0 ? TreeShares(a, W).behind(grp, end - 1) + 1 : 0;
  pdl_wait();
  pdl_launch_dependents();
  if (cta == 0 && blockIdx.y == 0 && warp == 0) {
    uint32_t st = 0;
    for (int i = lane; i < a.nparts; i += 32) st |= a.cta_status[i];
    st = __reduce_or_sync(FULL, st);
    if (lane == 0) *status = st;
  }
  if (b < 0) return;
  constexpr int RS = QT * kTreeRows, WPR = D / 32, CHUNK = QT == 2 ? 4 : 8;  // warps for one row; pieces at a time
  const int rows = tree_max_rows(a, QT);
#pragma unroll 1
  for (int pr = (int)blockIdx.y * combine_rows(D) + warp / WPR * 8 + (lane & 7); pr < rows; pr += (int)gridDim.y * combine_rows(D)) {
    const int t = (hs % a.nseqh) * QT + pr / kTreeRows, row = pr % kTreeRows;
    if (t >= tree_tiles(a, r.n)) return;
    const TreeTile tl = tree_tile(a, t, r.n);
    const int pos = row / a.gt, h = row - pos * a.gt;
    if (pos >= tl.nq || h >= tl.nh) continue;  // (nothing below is the whole warp's)
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
    const size_t at = (size_t)(r.start + tl.i0 + pos) * a.Hq + (hs / a.nseqh) * a.G + tl.h0 + h;
#pragma unroll
    for (int v = 0; v < 2; ++v)
      *reinterpret_cast<uint2 *>(a.out + at * D + c0 + 16 * v) =
          make_uint2(pack_bf16x2(acc[4 * v] * inv, acc[4 * v + 1] * inv), pack_bf16x2(acc[4 * v + 2] * inv, acc[4 * v + 3] * inv));
    if (c0 == 0 && a.lse) a.lse[at] = Z == 0.f ? -INFINITY : (M + __log2f(Z)) * LN2;
  }
}

}  // namespace pa
