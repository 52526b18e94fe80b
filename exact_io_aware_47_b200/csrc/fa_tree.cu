// Attention of drafted tokens over the paged cache (fa.h, fa_fwd_tree).
//
// The query rows of one K/V head (group heads x T tokens, consecutive in
// memory) share every key, so a work item is (sequence, K/V head, tile of R
// rows) and streams the sequence's keys once, 128 at a time.  With few rows the
// stream of K and V is what costs: 2 d bytes a key and head in e4m3.
//
// Transposed products.  The 128 keys of a tile are the M side of the tensor
// core's products and the rows are its N side (16 to 128), so nothing is spent
// on rows that do not exist:
//     S^T [keys x R] = K Q^T          A = K tile (K-major), B = Q (K-major)
//     O^T [d x R]   += V^T P^T        A = V tile (MN-major), B = P^T (MN-major)
// K and V go from the cache to shared memory by TMA and are read there by the
// tensor core as they are.  With an 8-bit cache the 16-bit operand is cut into
// 8-bit terms, whose kind::f8f6f4 products add up exactly in fp32:
//   * Q, scaled per row by a power of two to [128, 256): e4m3 terms (4
//     significant bits each), 2 for bf16 (8 bits), 3 for fp16 (11 bits); what
//     falls below the last term is at most 2^-17 of the row's largest value;
//   * P: fp16 first (11 bits), then e5m2 terms, whose byte is the high byte of
//     an fp16 value (3 bits each, down to steps of 2^-16 below a reference at
//     2^11, so that small probabilities are not lost beside a large one): 3
//     terms, rounded at the end (9 bits, finer than bf16), or all 4 (exact).
//   With 64 rows and more, where the softmax's instructions and the products
//   weigh more than the cache, P stays fp16 and four warps that have time
//   convert V to fp16 (exact; half the products and no terms to cut).
// The scale of a K row multiplies its row of S^T, the scale of a V row its
// row of P^T: both are one thread's.
// With a 16-bit cache P is rounded to the cache's type, as in the dense forward
// (both operands of a kind::f16 product have one type): half a step of it per
// probability.
//
// Measured (kernel and join, replayed from a graph; d 128, 32 query heads on 8 K/V
// heads): 64 sequences of 820..8192 keys, one token, e4m3: 108 us for 611 MB (5.7
// TB/s, 0.87 of a measured copy); 2 sequences of 105 to 131 thousand keys, 8
// tokens, bf16 cache: 160 us for 1008 MB (6.3 TB/s, 0.96); 16 sequences of
// 820..8192 keys, 32 tokens each (128 rows), e4m3: 113 us, of which a CTA's 34
// tiles take 69 (2.03 us, 3990 cycles at 1965 MHz, a tile: the softmax's steps in
// this arrangement; tensor core 23 % busy) and the rest launch, items' starts and
// ends and the join.
//
// Softmax.  A thread owns one key of a tile.  Rows keep a reference exponent r
// (shared memory); probabilities are 2^(z - r), their sums per thread and
// column stay in registers until the end of the item.  r follows a row's
// maximum only when a score passes it by a factor of 2^4 (2^8 for 16-bit P):
// the usual tile needs no maximum at all, only one vote of the 128 threads
// that no score did.  With an 8-bit cache what is stored is p times the V scale,
// and the reference follows that.  A row of zeros has the scale 1, some 2^9 times
// its neighbours', and adds nothing, so it may not move a reference (the others'
// probabilities would fall into the last steps of the terms): where a reference
// is about to move, rows of scale 1 are looked through, and those of zeros count
// as kTreeMinScale.  (Looked at for every row, it took 94.1 against 89.1 us for 64
// sequences of 820..8192 keys at d = 64, for the wait and the reads of V at every
// item's start; so 90.1 us.)  Two groups of 128 threads work at it.  Up to 32 rows they
// take turns, a tile each, with references, sums and an O of their own that
// meet at the item's end (two chains of dependent steps run at once: what a
// tile costs with few rows is latency); from 64 rows on they share each tile,
// half of the columns each (a thread holds its columns in registers).
//
// Roles (512 threads, one CTA per SM): warps 0-3 and 4-7 softmax, warp 8 loads K
// and the scales, warp 9 V (TMA), warp 10 issues the products of S, warp 11 those
// of O, warps 12-15 prepare Q (and convert V).
// An issuing thread pays about 60 cycles for an MMA and 210 for a commit
// (measured, whatever the size), so S and O have a thread each, and there is
// one commit per product: the barrier that gives a K or V slot back to the
// loader is also what the softmax waits on for S and for finished products of O
// (see below, at the rings).
//
// Work split.  All key tiles of all items form one line that is cut evenly
// into one piece per CTA, whatever the lengths (counting a few tiles for what
// an item costs beside its keys); an item that is cut leaves
// partial results (unnormalised O, r, sum) in the workspace, and
// fa_tree_join_kernel adds them up in order.
#include "fa_serve.h"

namespace fa {

constexpr int kTreeThreads = 512;
// Registers: 512 threads are launched with 128 each.  With 128 rows a softmax
// thread holds 64 columns (scores and sums) and needs more: its warpgroups take
// 176, the other two keep 80 (2 x 176 + 2 x 80 = 4 x 128; 16 sequences with 128
// rows: 113 us, with 184 and 72 116, with 192 and 64 116).
constexpr int kTreeLaunchRegs = 128, kTreeSoftmaxRegs = 176, kTreeOtherRegs = 80;
static_assert(2 * kTreeSoftmaxRegs + 2 * kTreeOtherRegs <= 4 * kTreeLaunchRegs, "register split");
// What an item's start and end cost, in tiles, where the line of work is cut.  One
// number serves all kinds of tile, the best or within 8 % of it for each.  Counted
// as 0, 2, 4, 7 (us; 32 query heads on 8, lengths from a tenth of the longest up):
//   8-bit, d 128, 16 rows: 64 sequences to 8192 keys 118, 109, 108, 108
//                          64 sequences to 2000 keys 67, 52, 46, 44
//     32 rows, fp16: 64 to 4000   120, 101, 90, 85     64 rows: 32 to 4000  96, 83, 76, 77
//     128 rows, fp16: 16 to 8192  134, 118, 113, 117
//   8-bit, d 64, 16 rows: 64 to 8192  110, 99, 90, 84  32 rows: 64 to 4000  110, 92, 81, 76
//   16-bit, d 128, 16 rows: 64 to 2000  65, 59, 60, 62  128 rows: 16 to 8192  112, 100, 95, 93
//   16-bit, d 64, 16 rows: 64 to 8192  113, 107, 106, 106
constexpr int kTreeItemCost = 4;
// V scales below this move a reference as if they were this: it keeps sums, which
// are without the scale, below 2^(90 + 15) a key.  (Their products keep their size,
// and lose their last bits: 2^-28 x 2^-90 of the largest p is a step of the terms.)
constexpr float kTreeMinScale = 0x1p-90f;
constexpr float kTreeMinScaleLog2 = -90.f;

template <int D_, bool BF16, bool E4M3, int R_>
struct TreeLayout {
  static constexpr int D = D_, R = R_;
  static constexpr bool kE4M3 = E4M3;
  static constexpr bool kTurns = R <= 32;                   // the groups take turns at the tiles
  static constexpr int kCols = kTurns ? R : R / 2;          // columns of a softmax thread
  static constexpr int kTermsQ = E4M3 ? (BF16 ? 2 : 3) : 1;
  // e4m3, many rows: V is converted to fp16 in shared memory (exact) and P is
  // fp16, see the top
  static constexpr bool kConvert = E4M3 && !kTurns;
  static constexpr bool kTerms8 = E4M3 && kTurns;           // P in e5m2 terms
  static constexpr int kTermsP = kTerms8 ? (BF16 ? 3 : 4) : 1;
  static constexpr int kPanels = (D * (E4M3 ? 1 : 2) + 127) / 128;  // 128-byte panels of a row
  static constexpr int kPanelElems = E4M3 ? 128 : 64;
  static constexpr int kSlotBytes = kPanels * 16384;
  static constexpr int kSteps = D * (E4M3 ? 1 : 2) / 32;    // MMAs of 32 bytes over d
  // with few rows the terms of Q and of P sit side by side (one product of N =
  // terms x R columns, summed afterwards); with many rows the terms of Q are
  // products into the same columns
  static constexpr bool kStackQ = kTurns && kTermsQ > 1;
  static constexpr int kSCols = kStackQ ? kTermsQ * R : R;
  static constexpr int kPRow = kTerms8 ? kTermsP * R : 2 * R;  // bytes of a key's row of P^T
  static constexpr int kPBytes = (kPRow + 127) / 128 * 16384;
  static constexpr int kPBufs = R == 128 ? 1 : 2;
  static constexpr int kQPanel = R * 128;
  static constexpr int kQBytes = kTermsQ * kPanels * kQPanel;
  static constexpr int kQBufs = R == 128 ? 1 : 2;
  static constexpr int kScales = E4M3 ? 8 : 0;              // ring of tile scales, 1 KB each (see below)
  static constexpr int kV16Bufs = kConvert ? 2 : 0;         // converted V tiles
  static constexpr int kV16Bytes = (D + 63) / 64 * 16384;
  // per row: Q scales; per group and column: reference, its last change and
  // factor, final weight; per softmax warp and column: one value
  static constexpr int kStatBytes = (kQBufs * R + 2 * kCols * 4 + 8 * kCols + R) * 4;
  static constexpr int kBarBytes = 640;
  static constexpr int kFixed = kV16Bufs * kV16Bytes + kPBufs * kPBytes + kQBufs * kQBytes + kScales * 1024 +
                                kStatBytes + kBarBytes + 1024;
  static constexpr int kSlotsFit = (232448 - kFixed) / kSlotBytes;
  static constexpr int kSlots = kSlotsFit < 12 ? kSlotsFit : 12;
  static constexpr int kSlotsK = kSlots / 2, kSlotsV = kSlots - kSlotsK;  // two rings
  static_assert(kSlotsK >= 2, "a slot is reused two tiles later at the earliest (see below)");
  static_assert(!E4M3 || kScales >= kSlotsK + 2, "scales are read before they are overwritten (see below)");
  static constexpr int kV = kSlotsK * kSlotBytes;
  static constexpr int kV16 = kSlots * kSlotBytes;
  static constexpr int kP = kV16 + kV16Bufs * kV16Bytes;
  static constexpr int kQ = kP + kPBufs * kPBytes;
  static constexpr int kScale = kQ + kQBufs * kQBytes;
  static constexpr int kStat = kScale + kScales * 1024;
  static constexpr int kBar = kStat + kStatBytes;
  static constexpr int kSmemBytes = kBar + kBarBytes + 1024;  // + slack to align to 1024
  // (3 terms are computed as 4: products with N = 48 or 96 columns take longer
  // than with 64 or 128, 129 against 124 us for 64 sequences of 4500 keys; the
  // last quarter is not read)
  static constexpr int kOCols = kTerms8 ? 4 * R : R;
  static constexpr int kTmemO = 2 * kSCols;                 // S twice, then O
  static constexpr int kTmemUsed = kTmemO + (kTurns ? 2 : 1) * kOCols;
  static_assert(kTmemUsed <= 512, "TMEM columns");
  static constexpr uint32_t kTmemCols = kTmemUsed <= 32 ? 32 : kTmemUsed <= 64 ? 64
                                        : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
};

// Lengths of sequence b, clamped into range.
struct TreeLens {
  int ctx, drafts;
  bool bad;
};
__device__ __forceinline__ TreeLens tree_lens(const TreeParams& p, int b) {
  // (positions stay within 32 bits, with a tile to spare)
  const long long room = min(p.c.room, (1ll << 31) - 256);
  const int n_in = p.draft_lens ? p.draft_lens[b] : p.T;
  const int ctx_in = p.ctx_lens[b];
  const int n_cap = static_cast<int>(min(static_cast<long long>(p.T), room));
  const int n = min(max(n_in, 0), n_cap);
  const int ctx = static_cast<int>(min(static_cast<long long>(max(ctx_in, 0)), room - n));
  return TreeLens{ctx, n, n != n_in || ctx != ctx_in};
}
__device__ __forceinline__ int tree_tiles(const TreeLens& l) {
  // (no drafted token: no row to compute)
  return l.drafts > 0 ? static_cast<int>((static_cast<long long>(l.ctx) + l.drafts + 127) / 128) : 0;
}

// This CTA's walk over its piece of the line, item by item.  An item takes
// `cost` units (its start and end) and then one per key tile.
struct TreeWalk {
  int b, hk, rt, nt;        // next item of sequence b (nt tiles each)
  int unit;                 // where in it this CTA begins
  int left;                 // units left in the piece
  int cost;
  int ctx, drafts;
};
struct TreeSeg {
  int b, hk, rt;          // the item
  int t0, t1, nt;         // its tiles [t0, t1) of nt
  int ctx, drafts;
};
__device__ __forceinline__ bool tree_next(TreeWalk& w, const TreeParams& p, TreeSeg& s) {
  if (w.left <= 0) return false;
  while (w.hk >= p.c.Hk || w.nt == 0) {
    const TreeLens l = tree_lens(p, ++w.b);
    w.nt = tree_tiles(l);
    w.ctx = l.ctx;
    w.drafts = l.drafts;
    w.hk = w.rt = 0;
  }
  s.b = w.b;
  s.hk = w.hk;
  s.rt = w.rt;
  s.t0 = max(0, w.unit - w.cost);
  s.t1 = min(w.nt, w.unit - w.cost + w.left);
  s.nt = w.nt;
  s.ctx = w.ctx;
  s.drafts = w.drafts;
  if (s.t1 <= s.t0) {  // (the piece ends within the item's cost)
    w.left = 0;
    return false;
  }
  w.left -= w.cost + w.nt - w.unit;
  w.unit = 0;
  if (++w.rt == p.row_tiles) {
    w.rt = 0;
    ++w.hk;
  }
  return true;
}

// Rings.  Tile i of a CTA uses slot i % n of the K and of the V ring (n slots) in round
// i / n.  A slot's "empty" barrier ends a round's phase when the product that
// reads the slot is complete: the loader waits for that, and so does the softmax:
// in tile i for S(i), for O of tile i - 1 or i - 2, and at an item's end for O of
// its last tile.  No phase can be missed there: with n >= 2 slots the next one
// of the same slot belongs to S(i + 2), O(i) or a later tile, whose product
// waits for that very softmax step or, S(i + 2), for all warps to have read
// S(i) (both issuing threads go in order).  The scales of tile i come with K(i)
// and are read once S(i) is complete, before S(i)'s columns are given back; tile
// i + 8's overwrite them after S(i + 8 - n), which waited for that (with barriers
// of their own the scales cost two more waits a tile: 112 against 106 us for 64
// sequences of 820..8192 keys, 121 against 115 for 16 with 128 rows).  Nor can
// a wait be early (a parity wait returns at once while the phase before is still
// open): whoever waits for a round of a slot has waited for the round before, or
// for what followed from it.

// The tiles of a CTA's piece in order, as the loading warps see them.  A tile
// takes 128 / box copies (one page may hold less than a tile); a warp looks up
// the places of 32 copies at once, i.e. of several tiles of an item, and the
// next batch's before it issues this one's, so that no copy waits for the page
// table.
struct TreeBatch {
  int tiles;        // tiles of the batch (0: none left)
  int left;         // keys of the sequence from the batch's first tile on
  int page, hk, y;  // this lane's copy: page, head, row in the page
};
struct TreeTiles {
  TreeWalk walk;
  TreeSeg seg;
  int tile;
  __device__ __forceinline__ TreeTiles(const TreeWalk& w) : walk(w), seg{}, tile(0) {}
  __device__ __forceinline__ TreeBatch next(const TreeParams& p, int lane) {
    TreeBatch b{0, 0, 0, 0, 0};
    if (tile == seg.t1) {
      if (!tree_next(walk, p, seg)) return b;
      tile = seg.t0;
    }
    const int per = 7 - p.box_log2;              // log2 of the copies of a tile
    b.tiles = min(32 >> per, seg.t1 - tile);
    b.left = seg.ctx + seg.drafts - tile * 128;
    b.hk = seg.hk;
    const int off = (lane >> per) * 128 + (lane & ((1 << per) - 1)) * p.box;
    if (off < min(b.left, b.tiles * 128)) {
      const unsigned key = tile * 128 + off;
      const unsigned at = __umulhi(key, p.c.page_mul) >> p.c.page_shift;   // key / page_size
      b.y = static_cast<int>(key - at * p.c.page_size);
      b.page = p.c.table ? p.c.table[static_cast<long long>(seg.b) * p.c.table_stride + at] : seg.b;
    }
    tile += b.tiles;
    return b;
  }
  // Copies of tile j of a batch; this lane does one if it is its turn.
  static __device__ __forceinline__ int copies(const TreeParams& p, const TreeBatch& b, int j) {
    return min(128, b.left - j * 128 + p.box - 1) >> p.box_log2;
  }
  static __device__ __forceinline__ int turn(const TreeParams& p, int j, int lane) {
    const int per = 7 - p.box_log2;
    return (lane >> per) == j ? lane & ((1 << per) - 1) : 128;
  }
};
// Slice (page and head) of a copy; -1 if its page is not in the pool.
__device__ __forceinline__ int tree_place(const TreeParams& p, const TreeBatch& b) {
  return b.page >= 0 && b.page < p.c.num_pages ? b.page * p.c.Hk + b.hk : -1;
}

// One MMA; operands by descriptor words (sdesc_lo, kSdescHi).
template <bool E4M3>
__device__ __forceinline__ void tree_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (E4M3) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kSdescHi)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kSdescHi)
        : "memory");
  }
}

// 16-byte aligned bulk copy global -> shared, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// Sums of TERMS sets of 8 columns, STEP columns apart, loaded with one wait.
template <int TERMS, int STEP>
__device__ __forceinline__ void tmem_sum8(uint32_t taddr, float (&s)[8]) {
  uint32_t r[TERMS][8];
#define FA_LD8(a, b) \
  "tcgen05.ld.sync.aligned.32x32b.x8.b32 {" a "}, [" b "];\n\t"
#define FA_OUT8(t) \
  "=r"(r[t][0]), "=r"(r[t][1]), "=r"(r[t][2]), "=r"(r[t][3]), "=r"(r[t][4]), "=r"(r[t][5]), "=r"(r[t][6]), "=r"(r[t][7])
  if constexpr (TERMS == 1) {
    tmem_ld8(taddr, r[0]);
  } else if constexpr (TERMS == 3) {
    asm volatile(FA_LD8("%0, %1, %2, %3, %4, %5, %6, %7", "%24")
                 FA_LD8("%8, %9, %10, %11, %12, %13, %14, %15", "%25")
                 FA_LD8("%16, %17, %18, %19, %20, %21, %22, %23", "%26")
                 "tcgen05.wait::ld.sync.aligned;"
                 : FA_OUT8(0), FA_OUT8(1), FA_OUT8(2)
                 : "r"(taddr), "r"(taddr + STEP), "r"(taddr + 2 * STEP)
                 : "memory");
  } else {
    static_assert(TERMS == 4, "1, 3 or 4 terms");
    asm volatile(FA_LD8("%0, %1, %2, %3, %4, %5, %6, %7", "%32")
                 FA_LD8("%8, %9, %10, %11, %12, %13, %14, %15", "%33")
                 FA_LD8("%16, %17, %18, %19, %20, %21, %22, %23", "%34")
                 FA_LD8("%24, %25, %26, %27, %28, %29, %30, %31", "%35")
                 "tcgen05.wait::ld.sync.aligned;"
                 : FA_OUT8(0), FA_OUT8(1), FA_OUT8(2), FA_OUT8(3)
                 : "r"(taddr), "r"(taddr + STEP), "r"(taddr + 2 * STEP), "r"(taddr + 3 * STEP)
                 : "memory");
  }
#undef FA_LD8
#undef FA_OUT8
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    s[e] = __uint_as_float(r[0][e]);
#pragma unroll
    for (int t = 1; t < TERMS; ++t) s[e] += __uint_as_float(r[t][e]);
  }
}
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_ld8(taddr, r);
  else if constexpr (N == 16) tmem_ld16(taddr, r);
  else if constexpr (N == 32) tmem_ld32(taddr, r);
  else tmem_ld64(taddr, r);
}

// True in all threads of the named barrier if any of them passes true.
__device__ __forceinline__ bool named_bar_or(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Maximum (which drops NaN) or sum over the warp's lanes of each of N columns,
// to out[0 .. N).  Every exchange halves the columns that a lane still holds:
// N - 1 shuffles (N <= 32) where one column at a time takes 5 N.
template <int N, bool MAX>
__device__ __forceinline__ void reduce_columns(float (&v)[N], int lane, float* out) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int step = 0; step < 5; ++step) {
    const int o = 16 >> step;
    const int held = N >> step;                  // columns before this exchange
    if (held > 1) {
      const bool hi = (lane & o) != 0;
#pragma unroll
      for (int j = 0; j < held / 2; ++j) {
        const float send = hi ? v[j] : v[j + held / 2];
        const float keep = hi ? v[j + held / 2] : v[j];
        v[j] = join(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    } else {
      v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  if constexpr (N >= 32) {
#pragma unroll
    for (int j = 0; j < N / 32; ++j) out[lane * (N / 32) + j] = v[j];
  } else {
    if (lane % (32 / N) == 0) out[lane / (32 / N)] = v[0];
  }
}

// e4m3 bytes back to fp32 (two per call).
__device__ __forceinline__ void unpack_e4m3x2(uint32_t pair, float& lo, float& hi) {
  uint32_t half2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(static_cast<unsigned short>(pair)));
  unpack2<false>(half2, lo, hi);
}

// Pairs between fp16 and e4m3.
__device__ __forceinline__ uint32_t pack_e4m3x2_f16(uint32_t half2) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(half2));
  return static_cast<uint32_t>(r);
}
__device__ __forceinline__ uint32_t unpack_e4m3x2_f16(uint32_t pair) {
  uint32_t half2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(static_cast<unsigned short>(pair)));
  return half2;
}

__device__ __forceinline__ uint32_t hsub2_bits(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Terms of P: four fp32 values as kTerms words of e5m2 bytes.
template <int TERMS>
__device__ __forceinline__ void e5m2_terms(float p0, float p1, float p2, float p3, uint32_t (&w)[TERMS]) {
  uint32_t a = pack_f16x2(p0, p1), b = pack_f16x2(p2, p3);
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    if (t + 1 == TERMS) {  // the last one takes what is left, rounded
      a += 0x00800080u;
      b += 0x00800080u;
    }
    w[t] = __byte_perm(a, b, 0x7531);
    if (t + 1 < TERMS) {
      a = hsub2_bits(a, a & 0xFF00FF00u);
      b = hsub2_bits(b, b & 0xFF00FF00u);
    }
  }
}

// Whether query row m (0 .. group * T - 1) sees drafted token u.
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int t, int u) {
  return p.mask ? p.mask[b * p.mask_stride + static_cast<long long>(t) * p.T + u] != 0 : u <= t;
}

// Partial results of a CTA in the workspace: slot 2 c holds the part of an item
// that an earlier CTA began, slot 2 c + 1 the part of one that a later CTA goes
// on with.  A slot is R rows of d fp32 columns, then R (reference, sum) pairs.
template <class Lay>
__host__ __device__ constexpr size_t tree_slot_floats() {
  return static_cast<size_t>(Lay::R) * (Lay::D + 2);
}

// Drafted V rows with values that are not finite were cleared for the products:
// adds those values of column d, of keys k0 .. k1 - 1, to the queries m0 ..
// m0 + n - 1 that see them (in the output, or in a partial result).
template <int D, bool BF16, bool E4M3>
__device__ __noinline__ void tree_add_not_finite(const TreeParams& p, int b, int hk, int ctx, int drafts,
                                                 int k0, int k1, int m0, int n, int d, float* partial) {
  uint16_t* o = reinterpret_cast<uint16_t*>(p.o) +
                ((static_cast<long long>(b) * p.Hq + static_cast<long long>(hk) * p.group) * p.T + m0) * D + d;
  for (int key = k0; key < k1; ++key) {
    const long long row = cache_row(p.c, b, hk, key);
    if (row < 0) continue;
    float v, skip;
    if constexpr (E4M3) unpack_e4m3x2(p.c.v[row * D + d], v, skip);
    else unpack2<BF16>(reinterpret_cast<const uint16_t*>(p.c.v)[row * D + d], v, skip);
    if (fabsf(v) < INFINITY) continue;
    for (int e = 0; e < n; ++e) {
      const int t = (m0 + e) % p.T;
      if (m0 + e >= p.group * p.T || t >= drafts || !tree_sees(p, b, t, key - ctx)) continue;
      if (partial != nullptr) {
        partial[e * D + d] += v;
      } else {
        float old;
        unpack2<BF16>(o[e * D], old, skip);
        o[e * D] = static_cast<uint16_t>(pack2<BF16>(old + v, 0.f));
      }
    }
  }
}

// Whether the V row of key tid of tile i (8-bit cache) holds zeros only.  (The lanes
// start at different 16-byte chunks: rows are 128 bytes apart.)
template <class Lay>
__device__ __forceinline__ bool tree_zero_row(const uint8_t* smem, int i, int tid) {
  constexpr int kRowPanels = Lay::kConvert ? (Lay::D + 63) / 64 : 1;
  const uint8_t* row = smem + tid * 128 +
                       (Lay::kConvert ? Lay::kV16 + (i & 1) * Lay::kV16Bytes
                                      : Lay::kV + i % Lay::kSlotsV * Lay::kSlotBytes);
  uint32_t any = 0u;
#pragma unroll
  for (int c = 0; c < 8 * kRowPanels; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + (c >> 3) * 16384 + (((c + tid) & 7) << 4));
    any |= v.x | v.y | v.z | v.w;
  }
  return (any & (Lay::kConvert ? 0x7FFF7FFFu : 0x7F7F7F7Fu)) == 0u;  // (signs apart)
}

// An item's Q, by WARPS warps of which this is number `worker` (four do 128 rows in
// the time of an item's end, 7000 cycles): loads a batch ahead, the first ones on construction; store() puts
// the rows in place, with an 8-bit cache as e4m3 terms and a scale per row.
template <class Lay, bool BF16, int WARPS>
struct TreeQ {
  static constexpr int kLanes = Lay::D / 8;      // lanes of a row, 8 values each
  static constexpr int kRowsWarp = 32 / kLanes;
  static constexpr int kPass = WARPS * kRowsWarp;  // rows of all warps at a time
  static constexpr int kBatch = Lay::R < 4 * kPass ? (Lay::R + kPass - 1) / kPass : 4;
  const uint8_t* q;
  int rows, first, l;                            // rows that exist, this lane's first, its part of a row
  uint4 next[kBatch];

  __device__ __forceinline__ uint4 load(int it) const {
    const int r = first + it * kPass;
    return r < Lay::R && r < rows ? *(reinterpret_cast<const uint4*>(q + static_cast<long long>(r) * Lay::D * 2) + l)
                               : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ TreeQ(const TreeParams& p, const TreeSeg& seg, int lane, int worker) {
    const long long row0 = (static_cast<long long>(seg.b) * p.Hq + static_cast<long long>(seg.hk) * p.group) * p.T +
                           static_cast<long long>(seg.rt) * Lay::R;
    q = p.q + row0 * Lay::D * 2;
    rows = p.group * p.T - seg.rt * Lay::R;
    first = worker * kRowsWarp + lane / kLanes;
    l = lane % kLanes;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) next[k] = load(k);
  }
  __device__ __forceinline__ void store(uint8_t* qdst, float* qs, float scale_log2) {
#pragma unroll 1
    for (int it0 = 0; it0 * kPass < Lay::R; it0 += kBatch) {
      uint4 xs[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        xs[k] = next[k];
        next[k] = load(it0 + kBatch + k);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = first + (it0 + k) * kPass;
        const uint4 x = xs[k];
        if constexpr (Lay::kE4M3) {
          float f[8];
          const float amax = row_amax<kLanes, BF16>(x);
          unpack8<BF16>(x, f);
          // up = 2^(7 - e), e the exponent of amax: amax up in [128, 256); the
          // scaled row is exact in fp16 (down to its steps of 2^-24)
          const int e = amax > 0.f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23), 8), 253) : 134;
          const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
          const float down = __uint_as_float(static_cast<uint32_t>(e - 7) << 23);
          if (l == 0 && r < Lay::R) qs[r] = amax < INFINITY ? down * scale_log2 : __int_as_float(0x7fffffff);
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = pack_f16x2(f[2 * i] * up, f[2 * i + 1] * up);
#pragma unroll
          for (int t = 0; t < Lay::kTermsQ; ++t) {
            uint32_t w[4];                       // pairs of codes
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = pack_e4m3x2_f16(h[i]);
              if (t + 1 < Lay::kTermsQ) h[i] = hsub2_bits(h[i], unpack_e4m3x2_f16(w[i]));
            }
            // 8 bytes at column 8 l of row r: chunk l / 2, swizzled by the row
            const uint32_t at = r * 128 + ((((l >> 1) ^ (r & 7)) << 4) | ((l & 1) << 3));
            if (r < Lay::R)
              *reinterpret_cast<uint2*>(qdst + t * Lay::kQPanel + at) =
                  make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
          }
        } else {
          const uint32_t at = (l >> 3) * Lay::kQPanel + r * 128 + (((l & 7) ^ (r & 7)) << 4);
          if (r < Lay::R) *reinterpret_cast<uint4*>(qdst + at) = x;
        }
      }
    }
  }
};

template <int D, bool BF16, bool E4M3, int R>
__global__ void __launch_bounds__(kTreeThreads, 1)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const __grid_constant__ TreeParams p) {
  using Lay = TreeLayout<D, BF16, E4M3, R>;
  constexpr int kCols = Lay::kCols;
  constexpr int kSlots = Lay::kSlots, kSlotsK = Lay::kSlotsK, kSlotsV = Lay::kSlotsV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float* s_qs = reinterpret_cast<float*>(smem + Lay::kStat);  // [kQBufs][R] Q unscale x scale_log2
  float* s_nr = s_qs + Lay::kQBufs * R;                       // [2][kCols] negated references
  float* s_move = s_nr + 2 * kCols;                           // [2][kCols] last change of s_nr
  float* s_alpha = s_move + 2 * kCols;                        // [2][kCols] 2^s_move
  float* s_weight = s_alpha + 2 * kCols;                      // [2][kCols] at the end: factor of O
  float* s_warp = s_weight + 2 * kCols;                       // [8][kCols] per-warp column values
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* kv_full = bars;                     // [kSlots]: the K ring, the V ring
  uint64_t* kv_empty = kv_full + kSlots;        // [kSlots]
  uint64_t* p_full = kv_empty + kSlots;         // [2]
  uint64_t* s_free = p_full + 2;                // [2]
  uint64_t* q_full = s_free + 2;                // [2]
  uint64_t* q_empty = q_full + 2;               // [2]
  uint64_t* v16_full = q_empty + 2;             // [2]
  uint64_t* v16_empty = v16_full + 2;           // [2]
  uint64_t* drain = v16_empty + 2;              // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_fix = abort_flag + 1;         // [4 items][4 warps or groups that look]
  TreeWalk* s_walk = reinterpret_cast<TreeWalk*>(const_cast<int*>(s_fix + 16));
  long long* s_scan = reinterpret_cast<long long*>(smem + Lay::kStat);  // setup only, one per warp
  static_assert(8 * (2 * kSlots + 14) + 4 * 18 + sizeof(TreeWalk) <= Lay::kBarBytes, "barrier area");
  static_assert(Lay::kStatBytes >= kTreeThreads / 32 * 16, "scan scratch");
  const WaitCtl wc{abort_flag, p.wait_ns};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], Lay::kConvert && s >= kSlotsK ? 4 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&p_full[s], Lay::kTurns ? 4 : 8);
      mbar_init(&s_free[s], Lay::kTurns ? 4 : 8);
      mbar_init(&q_full[s], 4);
      mbar_init(&q_empty[s], 8);
      mbar_init(&v16_full[s], 4);
      mbar_init(&v16_empty[s], 1);
      mbar_init(&drain[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 10) {
    tmem_alloc(tmem_slot, Lay::kTmemCols);
    tmem_relinquish();
  }
  // ------------------------------------------------- this CTA's piece of the line
  {
    const int per = (p.B + kTreeThreads - 1) / kTreeThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    const int items = p.c.Hk * p.row_tiles;
    long long tiles = 0, count = 0;              // of this thread's sequences
    for (int b = b0; b < b1; ++b) {
      const TreeLens l = tree_lens(p, b);
      if (l.bad && blockIdx.x == 0) record_error(kErrDeviceSeqlen, 60);
      const int nt = tree_tiles(l);
      tiles += static_cast<long long>(nt) * items;
      count += nt > 0 ? items : 0;
    }
    long long it = tiles, ic = count;            // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long ut = __shfl_up_sync(0xffffffffu, it, o), uc = __shfl_up_sync(0xffffffffu, ic, o);
      if (lane >= o) {
        it += ut;
        ic += uc;
      }
    }
    if (lane == 31) {
      s_scan[2 * warp] = it;
      s_scan[2 * warp + 1] = ic;
    }
    __syncthreads();
    long long bt = it - tiles, bc = ic - count, total_t = 0, total_c = 0;
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      const long long x = s_scan[2 * w], y = s_scan[2 * w + 1];
      if (w < warp) {
        bt += x;
        bc += y;
      }
      total_t += x;
      total_c += y;
    }
    // an item's start and end take about as long as kTreeItemCost tiles; where
    // there are fewer than two tiles for a CTA, they are spread evenly instead
    // (256 tiles: 15.8 us, with the cost 16.3; 512 tiles: 19.0, with it 16.8)
    const int cost = total_t >= 2ll * gridDim.x ? kTreeItemCost : 0;
    const long long total = total_t + cost * total_c, before = bt + cost * bc, sum = tiles + cost * count;
    const long long lo = total / gridDim.x, rest = total % gridDim.x;
    const long long c = blockIdx.x;
    const long long p0 = lo * c + min(c, rest), p1 = p0 + lo + (c < rest ? 1 : 0);
    if (threadIdx.x == 0 && p1 == p0) s_walk->left = 0;
    if (p1 > p0 && before <= p0 && p0 < before + sum) {  // exactly one thread
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        const TreeLens l = tree_lens(p, b);
        const int nt = tree_tiles(l);
        const long long here = nt > 0 ? static_cast<long long>(nt + cost) * items : 0;
        if (p0 < at + here) {
          const int item = static_cast<int>((p0 - at) / (nt + cost));
          s_walk->b = b;
          s_walk->hk = item / p.row_tiles;
          s_walk->rt = item % p.row_tiles;
          s_walk->nt = nt;
          s_walk->unit = static_cast<int>((p0 - at) % (nt + cost));
          s_walk->left = static_cast<int>(p1 - p0);
          s_walk->cost = cost;
          s_walk->ctx = l.ctx;
          s_walk->drafts = l.drafts;
          break;
        }
        at += here;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  TreeWalk walk = *s_walk;
  __syncthreads();  // s_scan's memory holds the statistics from here on
  // whether this CTA's first item was begun by an earlier CTA: the join reads it
  if (threadIdx.x == 0) {
    TreeWalk first = walk;
    TreeSeg seg;
    const bool cont = tree_next(first, p, seg) && seg.t0 > 0;
    *reinterpret_cast<int4*>(p.heads + blockIdx.x * 4) =
        cont ? make_int4(seg.b, seg.hk * p.row_tiles + seg.rt, seg.drafts, 0)
             : make_int4(-1, -1, 0, 0);
  }

  if (warp >= 8) {
  if constexpr (R == 128) regs_decrease<kTreeOtherRegs>();
  if (warp == 8 || warp == 9) {
    // ------------------------------------------------------------- K, V
    const bool is_v = warp == 9;
    const CUtensorMap* map = is_v ? &tmv : &tmk;
    const int ring = is_v ? kSlotsV : kSlotsK;
    uint64_t* full = kv_full + (is_v ? kSlotsK : 0);
    uint64_t* empty = kv_empty + (is_v ? kSlotsK : 0);
    uint8_t* slots = smem + (is_v ? Lay::kV : 0);
    int slot = 0, round = 0;
    if (lane == 0) tma_prefetch_desc(map);
    TreeTiles at(walk);
    TreeBatch next = at.next(p, lane);
    int loaded = 0;
    bool ok = true;
    while (ok && next.tiles > 0) {
      const TreeBatch cur = next;
      next = at.next(p, lane);
      int z = tree_place(p, cur);
      // (a bad page takes the scales of page 0)
      const long long row = static_cast<long long>(max(z, 0)) * p.c.page_size + cur.y;
      if (z < 0) {  // read as zeros, past the map's last slice
        z = p.c.num_pages * p.c.Hk;
        record_error(kErrDeviceSeqlen, 60);
      }
      for (int j = 0; j < cur.tiles; ++j) {
        ok = mbar_wait_warp(&empty[slot], (round & 1) ^ 1, wc, 61 + is_v);
        if (!ok) break;
        const int copies = TreeTiles::copies(p, cur, j), mine = TreeTiles::turn(p, j, lane);
        if (lane == 0)
          mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(copies * p.box * (128 * Lay::kPanels +
                                                                                     (E4M3 && !is_v ? 8 : 0))));
        __syncwarp();
        if (mine < copies) {
#pragma unroll
          for (int pn = 0; pn < Lay::kPanels; ++pn)
            tma_load_3d(slots + slot * Lay::kSlotBytes + pn * 16384 + mine * p.box * 128, map,
                        &full[slot], pn * Lay::kPanelElems, cur.y, z);
          if constexpr (E4M3) {
            if (!is_v) {                         // scales of both come with K
              float* dst = reinterpret_cast<float*>(smem + Lay::kScale + loaded % Lay::kScales * 1024) + mine * p.box;
              bulk_load(dst, p.c.k_scale + row, 4u * p.box, &full[slot]);
              bulk_load(dst + 128, p.c.v_scale + row, 4u * p.box, &full[slot]);
            }
          }
        }
        ++loaded;
        if (++slot == ring) {
          slot = 0;
          ++round;
        }
      }
    }
    // never leave with copies in flight: the last load into every slot
    for (int i = max(0, loaded - ring); i < loaded; ++i)
      mbar_wait_drain(&full[i % ring], (i / ring) & 1, 200000000ull);
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------- S^T = K Q^T
    if (lane == 0) {
      constexpr uint32_t kFormat = E4M3 ? 0u : (BF16 ? 1u : 0u);
      constexpr uint32_t kIdesc = (1u << 4) | (kFormat << 7) | (kFormat << 10) |
                                  (static_cast<uint32_t>(Lay::kSCols >> 3) << 17) | (8u << 24);
      constexpr int kPasses = Lay::kStackQ ? 1 : Lay::kTermsQ;
      const uint32_t base = smem_addr(smem);
      TreeSeg seg;
      int i = 0, slot = 0, round = 0;
      bool ok = true;
      for (int si = 0; ok && tree_next(walk, p, seg); ++si) {
        const int qb = si % Lay::kQBufs;
        ok = mbar_wait(&q_full[qb], (si / Lay::kQBufs) & 1, wc, 64);
        const uint32_t b0 = sdesc_lo(base + Lay::kQ + qb * Lay::kQBytes, false);
        for (int tile = seg.t0; ok && tile < seg.t1; ++tile, ++i) {
          // S(i - 2) has been read
          if (i >= 2) ok = mbar_wait(&s_free[i & 1], ((i >> 1) - 1) & 1, wc, 65);
          // With many rows the products take long, and O(i - 2) is what the softmax
          // waits for next: let it finish first, S(i) has time.
          if (!Lay::kTurns && ok && i >= 2)
            ok = Lay::kConvert ? mbar_wait(&v16_empty[i & 1], ((i >> 1) - 1) & 1, wc, 77)
                               : mbar_wait(&kv_empty[kSlotsK + (i - 2) % kSlotsV], ((i - 2) / kSlotsV) & 1, wc, 77);
          if (ok) ok = mbar_wait(&kv_full[slot], round & 1, wc, 66);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a0 = sdesc_lo(base + slot * Lay::kSlotBytes, false);
          const uint32_t d = tmem + (i & 1) * Lay::kSCols;
#pragma unroll
          for (int t = 0; t < kPasses; ++t) {
#pragma unroll
            for (int k = 0; k < Lay::kSteps; ++k)
              tree_mma<E4M3>(d, a0 + (k >> 2) * 1024 + (k & 3) * 2,
                             b0 + t * (Lay::kPanels * Lay::kQPanel >> 4) + (k >> 2) * (Lay::kQPanel >> 4) +
                                 (k & 3) * 2,
                             kIdesc, t + k > 0);
          }
          umma_commit(&kv_empty[slot]);
          if (++slot == kSlotsK) {
            slot = 0;
            ++round;
          }
          FA_TRACE_AT(i, 16);
        }
      }
      umma_commit(&drain[0]);
      mbar_wait_drain(&drain[0], 0, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------- O^T += V^T P^T
    if (lane == 0) {
      // both operands MN-major; e4m3 caches: A is e4m3 and B e5m2 (format 1), or
      // both are fp16
      constexpr bool k8 = Lay::kTerms8;
      constexpr uint32_t kFormatA = E4M3 ? 0u : (BF16 ? 1u : 0u), kFormatB = k8 ? 1u : kFormatA;
      constexpr uint32_t kIdesc = (1u << 4) | (kFormatA << 7) | (kFormatB << 10) | (1u << 15) | (1u << 16) |
                                  (static_cast<uint32_t>(Lay::kOCols >> 3) << 17) | (8u << 24);
      constexpr int kKeySteps = k8 ? 4 : 8;                    // 32 or 16 keys each
      constexpr uint32_t kKeyStep = k8 ? 256u : 128u;          // x 16 bytes
      const uint32_t base = smem_addr(smem);
      TreeSeg seg;
      int i = 0, slot = 0, round = 0;
      bool ok = true;
      while (ok && tree_next(walk, p, seg)) {
        for (int tile = seg.t0; tile < seg.t1; ++tile, ++i) {
          uint64_t* full = Lay::kConvert ? &v16_full[i & 1] : &kv_full[kSlotsK + slot];
          ok = mbar_wait(full, Lay::kConvert ? (i >> 1) & 1 : round & 1, wc, 67);
          if (ok) ok = mbar_wait(&p_full[i & 1], (i >> 1) & 1, wc, 68);
          if (!ok) break;
          FA_TRACE_AT(i, 17);
          tc_fence_after();
          const uint32_t a0 = sdesc_lo(base + (Lay::kConvert ? Lay::kV16 + (i & 1) * Lay::kV16Bytes
                                                             : Lay::kV + slot * Lay::kSlotBytes), true);
          const uint32_t b0 = sdesc_lo(base + Lay::kP + (i % Lay::kPBufs) * Lay::kPBytes, true);
          const uint32_t d = tmem + Lay::kTmemO + (Lay::kTurns ? (i & 1) * Lay::kOCols : 0);
          const bool first = tile - seg.t0 < (Lay::kTurns ? 2 : 1);
#pragma unroll
          for (int k = 0; k < kKeySteps; ++k)
            tree_mma<k8>(d, a0 + k * kKeyStep, b0 + k * kKeyStep, kIdesc, !first || k > 0);
          umma_commit(Lay::kConvert ? &v16_empty[i & 1] : &kv_empty[kSlotsK + slot]);
          if (++slot == kSlotsV) {
            slot = 0;
            ++round;
          }
          FA_TRACE_AT(i, 18);
        }
      }
      umma_commit(&drain[1]);
      mbar_wait_drain(&drain[1], 0, 200000000ull);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- Q
    bool ok = true;
    TreeWalk walk_q = walk;
    int si = 0;                                  // items whose Q is prepared
    auto prepare_q = [&]() {
      TreeSeg seg;
      if (!tree_next(walk_q, p, seg)) return false;
      const int qb = si % Lay::kQBufs;
      // (the first loads are issued before the buffer is free)
      TreeQ<Lay, BF16, 4> rows(p, seg, lane, warp - 12);
      ok = mbar_wait_warp(&q_empty[qb], ((si / Lay::kQBufs) & 1) ^ 1, wc, 69);
      if (!ok) return false;
      rows.store(smem + Lay::kQ + qb * Lay::kQBytes, s_qs + qb * R, p.scale_log2);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qb]);
      ++si;
      return true;
    };
    if constexpr (!Lay::kConvert) {
      while (prepare_q()) {
      }
    } else {
      // The same warps convert V: Q of the first items, then V of an item and Q of
      // the next one whose buffer that item's end gives back (never Q before the
      // V that its buffer waits for).
#pragma unroll 1
      for (int q = 0; q < Lay::kQBufs && prepare_q(); ++q) {
      }
      TreeSeg seg;
      int i = 0, slot = 0, round = 0;
      for (int item = 0; ok && tree_next(walk, p, seg); ++item) {
        const int L = seg.ctx + seg.drafts;
        volatile int* fix = s_fix + (item & 3) * 4 + warp - 12;
        if (lane == 0) *fix = 0;
        __syncwarp();
        for (int tile = seg.t0; tile < seg.t1; ++tile, ++i) {
          ok = mbar_wait_warp(&kv_full[kSlotsK + slot], round & 1, wc, 78);
          if (ok && i >= 2) ok = mbar_wait_warp(&v16_empty[i & 1], ((i >> 1) - 1) & 1, wc, 79);
          if (!ok) break;
          const uint8_t* from = smem + Lay::kV + slot * Lay::kSlotBytes;
          uint8_t* to = smem + Lay::kV16 + (i & 1) * Lay::kV16Bytes;
          const bool edge = tile * 128 + 128 > seg.ctx;
          bool found = false;
          // a unit: 16 columns of 32 rows, a row per lane
#pragma unroll 2
          for (int unit = warp - 12; unit < 4 * (D / 16); unit += 4) {
            const int row = (unit & 3) * 32 + lane, ch = unit >> 2, sw = row & 7;
            uint4 v = *reinterpret_cast<const uint4*>(from + row * 128 + ((ch ^ sw) << 4));
            if (edge) {
              const int key = tile * 128 + row;
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              if (key >= L) {                    // not in the cache
                w[0] = w[1] = w[2] = w[3] = 0u;
              } else if (key >= seg.ctx) {       // drafted: NaN codes apart (tree_add_not_finite)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t nan = ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                  found |= nan != 0;
                  w[e] &= ~((nan >> 7) * 0xFFu);
                }
              }
              v = make_uint4(w[0], w[1], w[2], w[3]);
            }
            uint32_t h[8];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = unpack_e4m3x2_f16(w[e >> 1] >> (16 * (e & 1)));
            uint8_t* out = to + (ch >> 2) * 16384 + row * 128;
            const int c16 = (ch & 3) * 2;
            *reinterpret_cast<uint4*>(out + ((c16 ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(out + (((c16 + 1) ^ sw) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          if (found) *fix = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v16_full[i & 1]);
            mbar_arrive(&kv_empty[kSlotsK + slot]);
          }
          if (++slot == kSlotsV) {
            slot = 0;
            ++round;
          }
        }
        if (ok) prepare_q();
      }
    }
    __syncwarp();
  }
  } else {
    if constexpr (R == 128) regs_increase<kTreeSoftmaxRegs>();
    // ------------------------------------------------------------- softmax
    const int grp = warp >> 2;
    const int tid = threadIdx.x & 127;           // key of the tile = TMEM lane; d at the end
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int col0 = Lay::kTurns ? 0 : grp * kCols;   // this thread's columns of S^T
    const int bar_id = 1 + grp;
    float* nr = s_nr + grp * kCols;
    float* move = s_move + grp * kCols;
    float* alpha = s_alpha + grp * kCols;
    const uint32_t tO = tmem + lane_off + Lay::kTmemO + (Lay::kTurns ? grp * Lay::kOCols : 0);
    constexpr int kEvery = Lay::kTurns ? 2 : 1;       // tiles from one of this group to its next
    // a row's reference stands for P = 2^kBias, and moves when P would pass
    // 2^kOver.  e5m2 terms reach from 2^15 down to steps of 2^-16: the reference
    // at 2^11 leaves 2^4 above it and 2^-27 below; fp16 has steps of 2^-24.
    constexpr float kBias = Lay::kTerms8 ? 11.f : (BF16 && !E4M3) ? 0.f : 7.f;
    constexpr float kOver = Lay::kTerms8 ? 15.f : kBias + 8.f;
    const int rows_all = p.group * p.T;
    bool ok = true;
    int i = 0;                                   // tile of this CTA
    // S(i), O(i) complete
    auto wait_s = [&](int i, unsigned site) {
      return mbar_wait_warp(&kv_empty[i % kSlotsK], (i / kSlotsK) & 1, wc, site);
    };
    auto wait_o = [&](int i, unsigned site) {
      if constexpr (Lay::kConvert) return mbar_wait_warp(&v16_empty[i & 1], (i >> 1) & 1, wc, site);
      else return mbar_wait_warp(&kv_empty[kSlotsK + i % kSlotsV], (i / kSlotsV) & 1, wc, site);
    };
    // V(i) is in shared memory, as the product reads it
    auto wait_v = [&](int i, unsigned site) {
      if constexpr (Lay::kConvert) return mbar_wait_warp(&v16_full[i & 1], (i >> 1) & 1, wc, site);
      else return mbar_wait_warp(&kv_full[kSlotsK + i % kSlotsV], (i / kSlotsV) & 1, wc, site);
    };
    TreeSeg seg;
    for (int si = 0; tree_next(walk, p, seg); ++si) {
      const int qb = si % Lay::kQBufs;
      const float* qs = s_qs + qb * R + col0;
      const int L = seg.ctx + seg.drafts;
      const int m0 = seg.rt * R + col0;          // first row of this thread's columns
      ok = mbar_wait_warp(&q_full[qb], (si / Lay::kQBufs) & 1, wc, 70) && ok;
      if (tid < kCols) nr[tid] = 0.f;
      bool unset = true;                         // tid < kCols: column tid has no reference yet
      if (tid == 0 && !Lay::kConvert) s_fix[(si & 3) * 4 + grp] = 0;
      // (a wait that gave up: this group goes on to the vote at the item's end)
      ok = named_bar_and(bar_id, 128, ok);
      const bool begun = ok;
      bool force = true;                         // some column has no reference yet
      float sum[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) sum[c] = 0.f;
      const int i_end = i + seg.t1 - seg.t0;
      // (turns: tile i of the CTA belongs to group i % 2)
      int tile = seg.t0;
      if (Lay::kTurns && (i & 1) != grp) {
        ++tile;
        ++i;
      }
      const bool any = tile < seg.t1;            // this group has a tile of the item
      if (!any && lane == 0) mbar_arrive(&q_empty[qb]);
      int last = i;                              // its last one
      for (; begun && tile < seg.t1; tile += kEvery, i += kEvery) {
        last = i;
        const int key = tile * 128 + tid;
        const int u = key - seg.ctx;             // drafted token, negative in the context
        // columns that see this key (only tiles with the end of the sequence
        // or drafted tokens need them)
        const bool edge = tile * 128 + 128 > seg.ctx;
        uint64_t seen = ~0ull;
        if (edge && u >= 0) {
          seen = 0ull;
          const uint8_t* column = p.mask ? p.mask + seg.b * p.mask_stride + u : nullptr;
          if (u < seg.drafts && p.T == 1) {
            if (column == nullptr || column[0] != 0) seen = ~0ull;
          } else if (u < seg.drafts) {
            int t = m0 % p.T;
#pragma unroll 16
            for (int c = 0; c < kCols; ++c) {
              const bool sees = column ? column[static_cast<long long>(t) * p.T] != 0 : u <= t;
              seen |= static_cast<uint64_t>(sees) << c;
              if (++t == p.T) t = 0;
            }
          }
        }
        if (threadIdx.x == 0) FA_TRACE_AT(i, 0);
        if (threadIdx.x == 0) FA_TRACE_AT(i, 1);
        ok = wait_s(i, 72) && ok;  // S(i) is complete, and so are the copies it was made from
        if (threadIdx.x == 0) FA_TRACE_AT(i, 2);
        tc_fence_after();
        // (rows past the sequence have no scales; a V scale that is not a size
        // makes its row's probabilities NaN)
        float sk_now = 1.f, sv_now = 1.f, lv = 0.f;
        if constexpr (E4M3) {
          if (key < L) {
            const float* sc = reinterpret_cast<const float*>(smem + Lay::kScale + i % Lay::kScales * 1024);
            sk_now = sc[tid];
            sv_now = sc[128 + tid];
            if (!(sv_now >= 0.f && sv_now < INFINITY)) sv_now = NAN;
          }
          lv = lg2_approx(fmaxf(sv_now, kTreeMinScale));
        }
        // d: exponent of a probability against its row's reference (without
        // the V scale sv = 2^lv, which multiplies what is stored)
        float d[kCols];
        {
          const uint32_t tS = tmem + lane_off + (i & 1) * Lay::kSCols + col0;
          uint32_t raw[kCols];
          tmem_ld_cols<kCols>(tS, raw);
          if constexpr (Lay::kStackQ) {
#pragma unroll
            for (int t = 1; t < Lay::kTermsQ; ++t) {
              uint32_t more[kCols];
              tmem_ld_cols<kCols>(tS + t * R, more);
#pragma unroll
              for (int c = 0; c < kCols; c += 2) {
                float lo, hi;
                f2unpack(fadd2(f2pack(__uint_as_float(raw[c]), __uint_as_float(raw[c + 1])),
                               f2pack(__uint_as_float(more[c]), __uint_as_float(more[c + 1]))), lo, hi);
                raw[c] = __float_as_uint(lo);
                raw[c + 1] = __float_as_uint(hi);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[i & 1]);
          const unsigned long long f2 = E4M3 ? f2pack(sk_now, sk_now) : f2pack(p.scale_log2, p.scale_log2);
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(nr + c);
            unsigned long long a = f2pack(__uint_as_float(raw[c]), __uint_as_float(raw[c + 1]));
            unsigned long long b = f2pack(__uint_as_float(raw[c + 2]), __uint_as_float(raw[c + 3]));
            if constexpr (E4M3) {
              const float4 q4 = *reinterpret_cast<const float4*>(qs + c);
              a = ffma2(fmul2(a, f2), f2pack(q4.x, q4.y), f2pack(n4.x, n4.y));
              b = ffma2(fmul2(b, f2), f2pack(q4.z, q4.w), f2pack(n4.z, n4.w));
            } else {
              a = ffma2(a, f2, f2pack(n4.x, n4.y));
              b = ffma2(b, f2, f2pack(n4.z, n4.w));
            }
            f2unpack(a, d[c], d[c + 1]);
            f2unpack(b, d[c + 2], d[c + 3]);
          }
        }
        if (tile + kEvery >= seg.t1) {           // nobody of this warp reads Q's scales again
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_empty[qb]);
        }
        if (edge && u >= 0) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (!((seen >> c) & 1)) d[c] = -INFINITY;
        }
        if (E4M3 && !(sv_now == sv_now)) {
          // a V row without a scale makes the rows that see it NaN, and no other
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if ((seen >> c) & 1) d[c] = NAN;
          sv_now = 0.f;
          lv = 0.f;
        }
        float top = d[0];
#pragma unroll
        for (int c = 1; c + 1 < kCols; c += 2) top = fmax3(top, d[c], d[c + 1]);
        top = fmaxf(top, d[kCols - 1]) + lv;
        if (threadIdx.x == 0) FA_TRACE_AT(i, 3);
        if (named_bar_or(bar_id, 128, top > kOver || force || !ok)) {
          // some row's reference moves (or a wait gave up)
          if constexpr (E4M3) {
            // rows of zeros, see the top; their scale is 1.  (O(i - kPBufs) is
            // complete before V(i) is waited for, for the reason given below.)
            const bool maybe = key < L && sv_now == 1.f;
            if (__any_sync(0xffffffffu, maybe)) {
              if (!Lay::kConvert && i >= Lay::kPBufs) ok = wait_o(i - Lay::kPBufs, 80) && ok;
              ok = wait_v(i, 81) && ok;
              if (ok && maybe && tree_zero_row<Lay>(smem, i, tid)) {
                sv_now = 0.f;
                lv = kTreeMinScaleLog2;
              }
            }
          }
          if (!named_bar_and(bar_id, 128, ok)) { ok = false; break; }
          constexpr int kPart = kCols < 32 ? kCols : 32;  // (registers)
#pragma unroll
          for (int part = 0; part < kCols; part += kPart) {
            float m[kPart];
#pragma unroll
            for (int c = 0; c < kPart; ++c) m[c] = d[part + c] + lv;
            reduce_columns<kPart, true>(m, lane, s_warp + warp * kCols + part);
          }
          named_bar_sync(bar_id, 128);
          if (tid < kCols) {
            const float* w = s_warp + grp * 4 * kCols + tid;
            const float m = fmaxf(fmaxf(w[0], w[kCols]), fmaxf(w[2 * kCols], w[3 * kCols]));
            float by = 0.f, factor = 1.f;
            if (m > -INFINITY && (unset || m > kBias)) {
              by = kBias - m;
              // (a row without a key so far has sums of zero)
              if (!unset) factor = exp2f(by);
              unset = false;
            }
            nr[tid] += by;
            move[tid] = by;
            alpha[tid] = factor;
          }
          force = named_bar_or(bar_id, 128, tid < kCols && unset);
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(move + c);
            d[c] += m4.x;
            d[c + 1] += m4.y;
            d[c + 2] += m4.z;
            d[c + 3] += m4.w;
          }
          if (tile - seg.t0 >= kEvery) {
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
              const float4 a4 = *reinterpret_cast<const float4*>(alpha + c);
              sum[c] *= a4.x;
              sum[c + 1] *= a4.y;
              sum[c + 2] *= a4.z;
              sum[c + 3] *= a4.w;
            }
            // O^T: this thread is row d = tid; the products so far have to be complete
            ok = wait_o(i - kEvery, 73);
            if (!named_bar_and(bar_id, 128, ok)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < Lay::kTermsP; ++t) {
#pragma unroll 1
              for (int c = 0; c < kCols; c += 8) {
                const uint32_t at = tO + t * R + col0 + c;
                uint32_t ro[8];
                tmem_ld8(at, ro);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  ro[e] = __float_as_uint(__uint_as_float(ro[e]) * alpha[c + e]);
                tmem_st_n<8>(at, ro);
              }
            }
            tmem_st_wait();
          }
        }
        if (threadIdx.x == 0) FA_TRACE_AT(i, 4);
        // the product that read this P buffer before is complete (so V(i - 2), and
        // with it the slot's round before V(i)'s, is known to have come and gone)
        if (i >= Lay::kPBufs) ok = wait_o(i - Lay::kPBufs, 75) && ok;
        // V rows that the cache does not hold are cleared (0 x NaN is NaN), and
        // drafted rows are searched for values that are not finite (where V is
        // converted, that is done there)
        if (edge && !Lay::kConvert) {
          const int slot = i % kSlotsV;
          ok = wait_v(i, 74) && ok;
          if (ok && u >= 0) {
            uint8_t* row = smem + Lay::kV + slot * Lay::kSlotBytes + tid * 128;
            // A thread has its key's row, or half of it if the groups share the
            // tile.  (The lanes start at different 16-byte chunks: rows are 128
            // bytes apart, so a chunk of 32 rows is in the same banks.  Rarely
            // executed code is kept short: what it costs is fetching it.)
            constexpr int kChunks = Lay::kTurns ? 8 : 4;
            auto chunk = [&](int pn, int ch) {
              const int at = Lay::kTurns ? (ch + tid) & 7 : grp * 4 + ((ch + tid) & 3);
              return reinterpret_cast<uint4*>(row + pn * 16384 + at * 16);
            };
            if (key >= L) {
#pragma unroll
              for (int pn = 0; pn < Lay::kPanels; ++pn)
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) *chunk(pn, ch) = make_uint4(0u, 0u, 0u, 0u);
            } else {
              // elements of a word whose exponent is all ones (e4m3: whose code
              // is NaN) carry into their top bit
              constexpr uint32_t kMask = E4M3 ? 0x7F7F7F7Fu : BF16 ? 0x7F807F80u : 0x7C007C00u;
              constexpr uint32_t kOne = E4M3 ? 0x01010101u : BF16 ? 0x00800080u : 0x04000400u;
              constexpr uint32_t kTop = E4M3 ? 0x80808080u : 0x80008000u;
              uint32_t bad = 0u;
#pragma unroll
              for (int pn = 0; pn < Lay::kPanels; ++pn)
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                  const uint4 v = *chunk(pn, ch);
                  bad |= ((v.x & kMask) + kOne) | ((v.y & kMask) + kOne) | ((v.z & kMask) + kOne) |
                         ((v.w & kMask) + kOne);
                }
              if (bad & kTop) {
                s_fix[(si & 3) * 4 + grp] = 1;
#pragma unroll 1
                for (int e = 0; e < Lay::kPanels * kChunks * 4; ++e) {
                  uint32_t* w = reinterpret_cast<uint32_t*>(chunk(e / (kChunks * 4), e / 4 % kChunks)) + e % 4;
                  uint32_t clear = ((*w & kMask) + kOne) & kTop;  // top bit of each such element
                  clear = E4M3 ? (clear >> 7) * 0xFFu : (clear >> 15) * 0xFFFFu;
                  *w &= ~clear;
                }
              }
            }
          }
        }
        if (threadIdx.x == 0) FA_TRACE_AT(i, 5);
        // probabilities, their sums, and P^T
        uint8_t* prow = smem + Lay::kP + (i % Lay::kPBufs) * Lay::kPBytes + tid * 128;
        const uint32_t swz = tid & 7;
        constexpr int kStep = kCols < 16 ? 8 : 16;
        const unsigned long long sv2 = f2pack(sv_now, sv_now);
#pragma unroll
        for (int c = 0; c < kCols; c += kStep) {
          constexpr int kTerms = Lay::kTermsP;
          uint32_t w[kTerms][kStep / 4];          // e5m2 terms, four columns a word
          uint32_t h[kStep / 2];                  // 16-bit pairs
#pragma unroll
          for (int e = 0; e < kStep; e += 4) {
            float pr[4];
#pragma unroll
            for (int o = 0; o < 4; o += 2) {
              unsigned long long x = f2pack(ex2_approx(d[c + e + o]), ex2_approx(d[c + e + o + 1]));
              const unsigned long long s2 = fadd2(f2pack(sum[c + e + o], sum[c + e + o + 1]), x);
              f2unpack(s2, sum[c + e + o], sum[c + e + o + 1]);
              if (E4M3) x = fmul2(x, sv2);
              f2unpack(x, pr[o], pr[o + 1]);
            }
            if constexpr (Lay::kTerms8) {
              uint32_t q[kTerms];
              e5m2_terms<kTerms>(pr[0], pr[1], pr[2], pr[3], q);
#pragma unroll
              for (int t = 0; t < kTerms; ++t) w[t][e / 4] = q[t];
            } else {
              h[e / 2] = pack2<BF16 && !E4M3>(pr[0], pr[1]);
              h[e / 2 + 1] = pack2<BF16 && !E4M3>(pr[2], pr[3]);
            }
          }
          // kStep columns of the key's row of P^T, in 16-byte chunks swizzled by the row
          auto chunk = [&](int byte) {
            return prow + (byte >> 7) * 16384 + ((((byte >> 4) & 7) ^ swz) << 4) + (byte & 15);
          };
          if constexpr (Lay::kTerms8) {
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
              uint8_t* to = chunk(t * R + col0 + c);
              if constexpr (kStep == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[t][0], w[t][1]);
              else *reinterpret_cast<uint4*>(to) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < kStep / 2; e += 4)
              *reinterpret_cast<uint4*>(chunk(2 * (col0 + c) + 4 * e)) =
                  make_uint4(h[e], h[e + 1], h[e + 2], h[e + 3]);
          }
        }
        if (threadIdx.x == 0) FA_TRACE_AT(i, 6);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i & 1]);
        if (threadIdx.x == 0) FA_TRACE_AT(i, 7);
      }
      // ----------------------------------------------------------- end of the item
      const bool whole = ok && (!any || wait_o(last, 76));
      i = i_end;
      if (!named_bar_and(3, 256, whole)) { ok = false; break; }
      tc_fence_after();
      // sums of the columns over the 128 keys' threads
      reduce_columns<kCols, false>(sum, lane, s_warp + warp * kCols);
      named_bar_sync(3, 256);
      const bool complete = seg.t0 == 0 && seg.t1 == seg.nt;
      float* slot = p.partial + (2 * static_cast<size_t>(blockIdx.x) + (seg.t0 == 0 ? 1 : 0)) * tree_slot_floats<Lay>();
      const long long out0 = (static_cast<long long>(seg.b) * p.Hq + static_cast<long long>(seg.hk) * p.group) * p.T;
      // this group finishes columns e0 .. e0 + R / 2
      const int e0 = grp * (R / 2);
      float stat_l = 0.f, stat_top = 0.f;
      if (tid < R / 2) {
        const int col = e0 + tid;
        auto total = [&](int g, int c) {
          const float* w = s_warp + g * 4 * kCols + c;
          return (w[0] + w[kCols]) + (w[2 * kCols] + w[3 * kCols]);
        };
        float l, top;                            // sum, reference
        if constexpr (Lay::kTurns) {
          const float l0 = total(0, col), l1 = total(1, col);
          const float r0 = -s_nr[col], r1 = -s_nr[kCols + col];
          top = fmaxf(l0 == 0.f ? -INFINITY : r0, l1 == 0.f ? -INFINITY : r1);
          const float w0 = l0 == 0.f ? 0.f : ex2_approx(r0 - top), w1 = l1 == 0.f ? 0.f : ex2_approx(r1 - top);
          l = (l0 == 0.f ? 0.f : w0 * l0) + (l1 == 0.f ? 0.f : w1 * l1);
          const float inv = !complete ? 1.f : l == 0.f ? 0.f : 1.f / l;
          s_weight[col] = w0 * inv;
          s_weight[kCols + col] = w1 * inv;
        } else {
          l = total(grp, tid);
          top = -nr[tid];
          s_weight[grp * kCols + tid] = l == 0.f ? 0.f : complete ? 1.f / l : 1.f;
        }
        stat_l = l;
        stat_top = top;
      }
      named_bar_sync(bar_id, 128);
      const volatile int* found = s_fix + (si & 3) * 4;
      const int fix = found[0] | found[1] | (Lay::kConvert ? found[2] | found[3] : 0);
      constexpr int kOut = Lay::kTurns ? 8 : 16;  // columns at a time
#pragma unroll 1
      for (int c = 0; c < R / 2; c += kOut) {
        if (seg.rt * R + e0 + c >= rows_all) break;  // (no such rows)
        float o[kOut];
        if constexpr (!Lay::kTurns) {
          uint32_t ro[kOut];
          tmem_ld_cols<kOut>(tmem + lane_off + Lay::kTmemO + e0 + c, ro);
#pragma unroll
          for (int e = 0; e < kOut; e += 4) {
            // (weight 0: no key seen)
            const float4 w = *reinterpret_cast<const float4*>(s_weight + e0 + c + e);
            o[e] = w.x == 0.f ? 0.f : w.x * __uint_as_float(ro[e]);
            o[e + 1] = w.y == 0.f ? 0.f : w.y * __uint_as_float(ro[e + 1]);
            o[e + 2] = w.z == 0.f ? 0.f : w.z * __uint_as_float(ro[e + 2]);
            o[e + 3] = w.w == 0.f ? 0.f : w.w * __uint_as_float(ro[e + 3]);
          }
        } else {
#pragma unroll
        for (int e = 0; e < kOut; ++e) o[e] = 0.f;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float og[8];
          tmem_sum8<Lay::kTermsP, R>(
              tmem + lane_off + Lay::kTmemO + g * Lay::kOCols + e0 + c, og);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // (weight 0: no key seen, and maybe nothing written there)
            const float w = s_weight[g * kCols + e0 + c + e];
            o[e] += w == 0.f ? 0.f : w * og[e];
          }
        }
        }
        if (tid >= D) continue;                  // (d = 64: the upper lanes hold nothing)
        const int m = seg.rt * R + e0 + c;       // first of kOut rows
        if (complete) {
          int t = seg.drafts == p.T ? 0 : m % p.T;
          uint16_t* to = reinterpret_cast<uint16_t*>(p.o) + (out0 + m) * D + tid;
#pragma unroll
          for (int e = 0; e < kOut; ++e) {
            if (m + e < rows_all && (seg.drafts == p.T || t < seg.drafts))
              to[e * D] = static_cast<uint16_t>(pack2<BF16>(o[e], 0.f));
            if (++t == p.T) t = 0;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kOut; ++e) slot[(e0 + c + e) * D + tid] = o[e];
        }
      }
      if (fix && tid < D)
        tree_add_not_finite<D, BF16, E4M3>(p, seg.b, seg.hk, seg.ctx, seg.drafts, max(seg.ctx, seg.t0 * 128),
                                           min(L, seg.t1 * 128), seg.rt * R + e0, R / 2, tid,
                                           complete ? nullptr : slot + e0 * D);
      if (tid < R / 2) {
        const int col = e0 + tid, m = seg.rt * R + col;
        if (!complete) {
          reinterpret_cast<float2*>(slot + R * D)[col] = make_float2(stat_top, stat_l);
        } else if (m < rows_all && (seg.drafts == p.T || m % p.T < seg.drafts)) {
          p.lse[out0 + m] = stat_l == 0.f ? -INFINITY : (stat_top + log2f(stat_l)) * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      named_bar_sync(3, 256);                    // O and the statistics are reused
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::kTmemCols);
  }
}

// Adds up the parts of the items that were cut, in the order of the keys.
// Blocks (c, y): the item whose first cut is at the start of CTA c + 1's piece
// (if any).  With ways = 1 a warp adds up a row (8 rows a block); with ways = 8 a
// block does, each warp every 8th part.
constexpr int kTreeJoinWarps = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kTreeJoinWarps * 32) fa_tree_join_kernel(const TreeParams p, int R, int ways) {
  constexpr int kVec = D / 32;                   // columns of a lane
  constexpr int kRounds = kTreeMaxCtas / 32;     // parts of a lane
  __shared__ float s_o[kTreeJoinWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x + 1;
  const int4* heads = reinterpret_cast<const int4*>(p.heads);
  const int4 head = heads[c0];
  const int b = head.x, item = head.y;
  if (b < 0) return;
  // (a CTA whose own first item is the same one did not begin it)
  const int4 before = heads[c0 - 1];
  if (before.x == b && before.y == item) return;
  // parts: of CTA c0 - 1, which began the item, then of those that go on with it
  int parts = 1;
  for (int c = c0; c < p.grid; c += 32) {
    int4 h = make_int4(-1, -1, 0, 0);
    if (c + lane < p.grid) h = heads[c + lane];
    const unsigned other = ~__ballot_sync(0xffffffffu, h.x == b && h.y == item);
    parts += other ? __ffs(other) - 1 : 32;
    if (other) break;
  }
  const int hk = item / p.row_tiles, rt = item - hk * p.row_tiles;
  const int r = ways == 1 ? blockIdx.y * kTreeJoinWarps + warp : blockIdx.y;
  const int m = rt * R + r;
  if (r >= R || m >= p.group * p.T || m % p.T >= head.z) return;  // (ways = 8: the whole block)
  const size_t slot_floats = static_cast<size_t>(R) * (D + 2);
  auto part = [&](int i) {
    return p.partial + (i == 0 ? 2 * static_cast<size_t>(c0 - 1) + 1 : 2 * static_cast<size_t>(c0 + i - 1)) * slot_floats;
  };
  // weight of a part: 2^(its reference - the largest); parts without a key: 0
  float w[kRounds], ref[kRounds], l = 0.f, top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    float2 st = make_float2(0.f, 0.f);
    if (k * 32 + lane < parts) st = reinterpret_cast<const float2*>(part(k * 32 + lane) + R * D)[r];
    ref[k] = st.x;
    w[k] = st.y;
    if (st.y != 0.f) top = fmaxf(top, st.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const float sum = w[k];
    w[k] = sum == 0.f ? 0.f : exp2f(ref[k] - top);
    l += sum == 0.f ? 0.f : w[k] * sum;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float acc[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
  const int way = ways == 1 ? 0 : warp;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
#pragma unroll 4
    for (int j = way; j < 32; j += ways) {
      if (k * 32 + j >= parts) break;
      const float wi = __shfl_sync(0xffffffffu, w[k], j);
      const float* from = part(k * 32 + j) + r * D + lane * kVec;
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc[e] += wi == 0.f ? 0.f : wi * from[e];
    }
  }
  if (ways > 1) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) s_o[warp][lane * kVec + e] = acc[e];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      for (int x = 1; x < kTreeJoinWarps; ++x) acc[e] += s_o[x][lane * kVec + e];
  }
  const long long row = (static_cast<long long>(b) * p.Hq + static_cast<long long>(hk) * p.group) * p.T + m;
  uint32_t* to = reinterpret_cast<uint32_t*>(p.o) + (row * D + lane * kVec) / 2;
#pragma unroll
  for (int e = 0; e < kVec; e += 2)
    to[e / 2] = pack2<BF16>(l == 0.f ? 0.f : acc[e] / l, l == 0.f ? 0.f : acc[e + 1] / l);
  if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
}

template <int D, bool BF16, bool E4M3, int R>
static cudaError_t launch_tree_t(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p,
                                 int device, cudaStream_t stream) {
  using Lay = TreeLayout<D, BF16, E4M3, R>;
  auto kern = fa_tree_kernel<D, BF16, E4M3, R>;
  // once per device: a decoding step is short
  static std::atomic<unsigned long long> ready{0};
  const unsigned long long bit = 1ull << device;
  if ((ready.load(std::memory_order_relaxed) & bit) == 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kSmemBytes);
    if (e != cudaSuccess) return e;
    if constexpr (R == 128) {
      // the register split in the kernel assumes exactly this launch allocation
      cudaFuncAttributes attr;
      e = cudaFuncGetAttributes(&attr, kern);
      if (e != cudaSuccess) return e;
      if (attr.numRegs != kTreeLaunchRegs) return cudaErrorInvalidConfiguration;
    }
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  kern<<<p.grid, kTreeThreads, Lay::kSmemBytes, stream>>>(tmk, tmv, p);
  // items of one tile are never cut
  if (p.grid > 1 && static_cast<long long>(p.c.table_stride) * p.c.page_size > 128)
  {
    // few long items are cut into many parts: a block per row then
    const int rows = std::min(R, p.group * p.T);
    const long long items = static_cast<long long>(p.B) * p.c.Hk * p.row_tiles;
    const int ways = items * kTreeJoinWarps <= p.grid ? kTreeJoinWarps : 1;
    const unsigned ys = ways == 1 ? (rows + kTreeJoinWarps - 1) / kTreeJoinWarps : rows;
    fa_tree_join_kernel<D, BF16><<<dim3(p.grid - 1, ys), kTreeJoinWarps * 32, 0, stream>>>(p, R, ways);
  }
  return cudaGetLastError();
}

cudaError_t launch_tree(int d, bool bf16, bool e4m3, int rows, const CUtensorMap& tmk,
                        const CUtensorMap& tmv, const TreeParams& p, int device, cudaStream_t stream) {
#define FA_TREE_R(DD, BB, EE)                                                     \
  (rows == 16   ? launch_tree_t<DD, BB, EE, 16>(tmk, tmv, p, device, stream)              \
   : rows == 32 ? launch_tree_t<DD, BB, EE, 32>(tmk, tmv, p, device, stream)              \
   : rows == 64 ? launch_tree_t<DD, BB, EE, 64>(tmk, tmv, p, device, stream)              \
                : launch_tree_t<DD, BB, EE, 128>(tmk, tmv, p, device, stream))
  if (d == 128) {
    if (bf16) return e4m3 ? FA_TREE_R(128, true, true) : FA_TREE_R(128, true, false);
    return e4m3 ? FA_TREE_R(128, false, true) : FA_TREE_R(128, false, false);
  }
  if (bf16) return e4m3 ? FA_TREE_R(64, true, true) : FA_TREE_R(64, true, false);
  return e4m3 ? FA_TREE_R(64, false, true) : FA_TREE_R(64, false, false);
#undef FA_TREE_R
}

}  // namespace fa
