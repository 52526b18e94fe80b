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
// tensor core as they are: an 8-bit cache is never converted.  Instead the
// 16-bit operand is cut into 8-bit terms, which one kind::f8f6f4 product sums
// exactly in fp32:
//   * Q, scaled per row by a power of two to [128, 256): e4m3 terms (4
//     significant bits each), 2 for bf16 (8 bits), 3 for fp16 (11 bits); what
//     falls below the last term is at most 2^-17 of the row's largest value;
//   * P: fp16 first (11 bits), then e5m2 terms, whose byte is the high byte of
//     an fp16 value (3 bits each, down to steps of 2^-16 below a reference at
//     2^11, so that small probabilities are not lost beside a large one): 3
//     terms, rounded at the end (9 bits, finer than bf16), or all 4 (exact).
// The scale of a K row multiplies its row of S^T, the scale of a V row its
// row of P^T: both are one thread's.
//
// Softmax.  A thread owns one key and half of the R rows (columns of S^T).
// Rows keep a reference exponent r (shared memory); probabilities are
// 2^(z - r), their sums per thread and column stay in registers until the end
// of the item.  r follows a row's maximum only when a score passes it by a
// factor of 2^4 (2^8 for 16-bit P): the usual tile needs no maximum at all,
// only one vote of the 128 threads that no score did.
//
// Roles (384 threads, one CTA per SM): warps 0-3 and 4-7 softmax of the first
// and second half of the columns, warp 8 loads (TMA), warp 9 issues MMAs, warps
// 10-11 prepare Q.  The pipeline over tiles i is S(0) S(1) [PV(i) S(i+2)]...,
// the loads come in the same order.
//
// Work split.  All key tiles of all items form one line that is cut evenly
// into one piece per CTA, whatever the lengths; an item that is cut leaves
// partial results (unnormalised O, r, sum) in the workspace, and
// fa_tree_join_kernel adds them up in order.
#include "fa_serve.h"

namespace fa {

constexpr int kTreeThreads = 384;
constexpr float kTreeNoRef = 1e30f;   // negated reference of a row without a key yet
constexpr float kTreeMinScale = 0x1p-90f;  // V scales below count as this (keeps sums in range)

template <int D_, bool BF16, bool E4M3, int R_>
struct TreeLayout {
  static constexpr int D = D_, R = R_;
  static constexpr int kCols = R / 2;                       // columns of a softmax thread
  static constexpr int kTermsQ = E4M3 ? (BF16 ? 2 : 3) : 1;
  static constexpr int kTermsP = E4M3 ? (BF16 ? 3 : 4) : 1;
  static constexpr int kPanels = (D * (E4M3 ? 1 : 2) + 127) / 128;  // 128-byte panels of a row
  static constexpr int kPanelElems = E4M3 ? 128 : 64;
  static constexpr int kSlotBytes = kPanels * 16384;
  static constexpr int kSteps = D * (E4M3 ? 1 : 2) / 32;    // MMAs of 32 bytes over d
  // up to 64 rows the terms of P sit side by side (one product of N = terms x R
  // columns, summed at the end); with 128 rows each has its own panel and its
  // own product into the same columns
  static constexpr bool kStack = E4M3 && R < 128;
  static constexpr int kPRow = E4M3 ? kTermsP * R : 2 * R;  // bytes of a key's row of P^T
  static constexpr int kPBytes = (kPRow + 127) / 128 * 16384;
  static constexpr int kPBufs = R == 128 ? 1 : 2;
  static constexpr int kQPanel = R * 128;
  static constexpr int kQBytes = kTermsQ * kPanels * kQPanel;
  static constexpr int kQBufs = R == 128 ? 1 : 2;
  static constexpr int kScales = E4M3 ? 8 : 0;              // ring of tile scales, 1 KB each
  static constexpr int kStatBytes = (kQBufs + 3 + 4) * R * 4;
  static constexpr int kFixed = kPBufs * kPBytes + kQBufs * kQBytes + kScales * 1024 + kStatBytes + 512 + 1024;
  static constexpr int kSlotsFit = (232448 - kFixed) / kSlotBytes;
  static constexpr int kSlots = kSlotsFit < 12 ? kSlotsFit : 12;
  static_assert(kSlots >= 4, "K/V ring");
  static constexpr int kP = kSlots * kSlotBytes;
  static constexpr int kQ = kP + kPBufs * kPBytes;
  static constexpr int kScale = kQ + kQBufs * kQBytes;
  static constexpr int kStat = kScale + kScales * 1024;
  static constexpr int kBar = kStat + kStatBytes;
  static constexpr int kSmemBytes = kBar + 512 + 1024;      // + slack to align to 1024
  static constexpr int kOCols = kStack ? kTermsP * R : R;
  static constexpr int kTmemUsed = 2 * R + kOCols;
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
  const long long room = min(static_cast<long long>(p.c.table_stride) * p.c.page_size, (1ll << 31) - 256);
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

// This CTA's walk over its piece of the line of key tiles, item by item.
struct TreeWalk {
  int b, item, tile, nt;  // next item of sequence b (nt tiles each), first tile in it
  int left;               // tiles left in the piece
  int ctx, drafts;
};
struct TreeSeg {
  int b, hk, rt;          // the item
  int t0, t1, nt;         // its tiles [t0, t1) of nt
  int ctx, drafts;
};
__device__ __forceinline__ bool tree_next(TreeWalk& w, const TreeParams& p, TreeSeg& s) {
  if (w.left <= 0) return false;
  const int items = p.c.Hk * p.row_tiles;
  while (w.item >= items || w.nt == 0) {
    const TreeLens l = tree_lens(p, ++w.b);
    w.nt = tree_tiles(l);
    w.ctx = l.ctx;
    w.drafts = l.drafts;
    w.item = 0;
  }
  s.b = w.b;
  s.hk = w.item / p.row_tiles;
  s.rt = w.item - s.hk * p.row_tiles;
  s.t0 = w.tile;
  s.t1 = min(w.nt, w.tile + w.left);
  s.nt = w.nt;
  s.ctx = w.ctx;
  s.drafts = w.drafts;
  w.left -= s.t1 - s.t0;
  w.tile = 0;
  ++w.item;
  return true;
}

// Position in the load order K0 K1 V0 K2 V1 ... of the K and the V of tile i
// of n.
__device__ __forceinline__ int tree_k_pos(int i) { return i < 2 ? i : 2 * i - 1; }
__device__ __forceinline__ int tree_v_pos(int i, int n) { return min(2 * i + 2, 2 * n - 1); }

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

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// e4m3 bytes back to fp32 (two per call).
__device__ __forceinline__ void unpack_e4m3x2(uint32_t pair, float& lo, float& hi) {
  uint32_t half2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(static_cast<unsigned short>(pair)));
  unpack2<false>(half2, lo, hi);
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

template <int D, bool BF16, bool E4M3, int R>
__global__ void __launch_bounds__(kTreeThreads, 1)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const TreeParams p) {
  using Lay = TreeLayout<D, BF16, E4M3, R>;
  constexpr int kCols = Lay::kCols;
  constexpr int kSlots = Lay::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float* s_qs = reinterpret_cast<float*>(smem + Lay::kStat);  // [kQBufs][R] Q unscale x scale_log2
  float* s_nr = s_qs + Lay::kQBufs * R;                       // [R] negated references
  float* s_alpha = s_nr + R;                                  // [R]
  float* s_sum = s_alpha + R;                                 // [R] 1 / sum, at the end
  float* s_wmax = s_sum + R;                                  // [4][R] per-warp column values
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* kv_full = bars;                     // [kSlots]
  uint64_t* kv_empty = kv_full + kSlots;        // [kSlots]
  uint64_t* sc_full = kv_empty + kSlots;        // [8]
  uint64_t* sc_empty = sc_full + 8;             // [8]
  uint64_t* s_full = sc_empty + 8;              // [2]
  uint64_t* p_full = s_full + 2;                // [2]
  uint64_t* q_full = p_full + 2;                // [2]
  uint64_t* q_empty = q_full + 2;               // [2]
  uint64_t* o_full = q_empty + 2;
  uint64_t* pv_done = o_full + 1;
  uint64_t* drain = pv_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_fix = abort_flag + 1;         // [2 parities][2 groups]
  TreeWalk* s_walk = reinterpret_cast<TreeWalk*>(const_cast<int*>(s_fix + 4));
  long long* s_scan = reinterpret_cast<long long*>(smem + Lay::kStat);  // setup only [12 + 1]
  static_assert(8 * (2 * 12 + 16 + 11) + 4 * 6 + sizeof(TreeWalk) <= 512, "barrier area");
  static_assert(Lay::kStatBytes >= 13 * 8, "scan scratch");
  const WaitCtl wc{abort_flag, p.wait_ns};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(&sc_full[s], 1);
      mbar_init(&sc_empty[s], 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 8);
      mbar_init(&q_full[s], 2);
      mbar_init(&q_empty[s], 9);
    }
    mbar_init(o_full, 1);
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, Lay::kTmemCols);
    tmem_relinquish();
  }
  // ------------------------------------------------- this CTA's piece of the line
  {
    const int per = (p.B + kTreeThreads - 1) / kTreeThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
    const int items = p.c.Hk * p.row_tiles;
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      const TreeLens l = tree_lens(p, b);
      if (l.bad && blockIdx.x == 0) record_error(kErrDeviceSeqlen, 60);
      sum += static_cast<long long>(tree_tiles(l)) * items;
    }
    long long inc = sum;  // inclusive sum over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    long long before = inc - sum, total = 0;
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      const long long x = s_scan[w];
      if (w < warp) before += x;
      total += x;
    }
    const long long lo = total / gridDim.x, rest = total % gridDim.x;
    const long long c = blockIdx.x;
    const long long p0 = lo * c + min(c, rest), p1 = p0 + lo + (c < rest ? 1 : 0);
    if (threadIdx.x == 0 && p1 == p0) s_walk->left = 0;
    if (p1 > p0 && before <= p0 && p0 < before + sum) {  // exactly one thread
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        const TreeLens l = tree_lens(p, b);
        const int nt = tree_tiles(l);
        const long long here = static_cast<long long>(nt) * items;
        if (p0 < at + here) {
          s_walk->b = b;
          s_walk->item = static_cast<int>((p0 - at) / nt);
          s_walk->tile = static_cast<int>((p0 - at) % nt);
          s_walk->nt = nt;
          s_walk->left = static_cast<int>(p1 - p0);
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
  const int n_tiles = walk.left;
  __syncthreads();  // s_scan's memory holds the statistics from here on
  // whether this CTA's first item was begun by an earlier CTA: the join reads it
  if (threadIdx.x == 0) {
    int* head = p.heads + blockIdx.x * 4;
    const bool cont = n_tiles > 0 && walk.tile > 0;
    head[0] = cont ? walk.b : -1;
    head[1] = cont ? walk.item : -1;
    head[2] = cont && walk.tile + n_tiles >= walk.nt;  // it ends here
    head[3] = cont ? walk.drafts : 0;
  }

  if (warp == 8) {
    // ------------------------------------------------------------- loads
    if (lane == 0) {
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmv);
    }
    const int pieces = 128 / p.box;  // lane l < pieces loads keys l box .. of a tile
    TreeSeg seg{};
    bool more = tree_next(walk, p, seg);
    int tile = seg.t0;
    int z[2] = {0, 0}, y[2] = {0, 0};         // tiles i and i - 1
    bool on[2] = {false, false};
    int pos = 0, scales = 0;                  // slots, tile scales loaded
    bool ok = true;
    auto load_slot = [&](bool is_v, int zz, int yy, bool use) {
      const int slot = pos % kSlots;
      ok = mbar_wait_warp(&kv_empty[slot], ((pos / kSlots) & 1) ^ 1, wc, 61);
      if (!ok) return;
      const uint32_t mine = use ? static_cast<uint32_t>(Lay::kPanels * p.box * 128) : 0u;
      const uint32_t all = __reduce_add_sync(0xffffffffu, mine);
      if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], all);
      __syncwarp();
      if (use) {
#pragma unroll
        for (int pn = 0; pn < Lay::kPanels; ++pn)
          tma_load_3d(smem + slot * Lay::kSlotBytes + pn * 16384 + lane * p.box * 128,
                      is_v ? &tmv : &tmk, &kv_full[slot], pn * Lay::kPanelElems, yy, zz);
      }
      __syncwarp();
      ++pos;
    };
    for (int i = 0; i <= n_tiles && ok; ++i) {
      z[1] = z[0];
      y[1] = y[0];
      on[1] = on[0];
      if (i < n_tiles && more) {
        // K of tile i (and the scales of its rows)
        const int L = seg.ctx + seg.drafts;
        const int key = tile * 128 + lane * p.box;
        on[0] = lane < pieces && key < L;
        bool good = false;
        if (on[0]) {
          const int at = key / p.c.page_size;
          const int page = p.c.table ? p.c.table[static_cast<long long>(seg.b) * p.c.table_stride + at] : seg.b;
          good = page >= 0 && page < p.c.num_pages;
          if (!good) record_error(kErrDeviceSeqlen, 62);
          // (a page that is not in the pool: past the map's last slice, read as zeros)
          z[0] = good ? page * p.c.Hk + seg.hk : p.c.num_pages * p.c.Hk;
          y[0] = key - at * p.c.page_size;
        }
        load_slot(false, z[0], y[0], on[0]);
        if (!ok) break;
        if constexpr (E4M3) {
          const int ss = i % Lay::kScales;
          ok = mbar_wait_warp(&sc_empty[ss], ((i / Lay::kScales) & 1) ^ 1, wc, 63);
          if (!ok) break;
          const bool use = on[0] && good;
          const uint32_t all = __reduce_add_sync(0xffffffffu, use ? 8u * p.box : 0u);
          if (lane == 0) mbar_arrive_expect_tx(&sc_full[ss], all);
          __syncwarp();
          if (use) {
            float* dst = reinterpret_cast<float*>(smem + Lay::kScale + ss * 1024) + lane * p.box;
            const long long row = static_cast<long long>(z[0]) * p.c.page_size + y[0];
            bulk_load(dst, p.c.k_scale + row, 4u * p.box, &sc_full[ss]);
            bulk_load(dst + 128, p.c.v_scale + row, 4u * p.box, &sc_full[ss]);
          }
          __syncwarp();
          ++scales;
        }
        if (++tile == seg.t1) {
          more = tree_next(walk, p, seg);
          tile = seg.t0;
        }
      }
      if (i >= 1) load_slot(true, z[1], y[1], on[1]);  // V(i - 1) follows K(i)
    }
    // never leave with copies in flight
    for (int s = 0; s < kSlots; ++s) {
      if (pos > s) {
        const int last = pos - 1 - ((pos - 1 - s) % kSlots);
        mbar_wait_drain(&kv_full[s], (last / kSlots) & 1, 200000000ull);
      }
    }
    if constexpr (E4M3) {
      for (int s = 0; s < Lay::kScales; ++s) {
        if (scales > s) {
          const int last = scales - 1 - ((scales - 1 - s) % Lay::kScales);
          mbar_wait_drain(&sc_full[s], (last / Lay::kScales) & 1, 200000000ull);
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------- MMA issue
    if (lane == 0 && n_tiles > 0) {
      constexpr uint32_t kFormat = E4M3 ? 0u : (BF16 ? 1u : 0u);
      constexpr uint32_t kIdescS = (1u << 4) | (kFormat << 7) | (kFormat << 10) |
                                   (static_cast<uint32_t>(R >> 3) << 17) | (8u << 24);
      // A = V MN-major, B = P^T MN-major; e4m3 caches: B is e5m2 (format 1)
      constexpr int kNPv = Lay::kOCols;
      constexpr uint32_t kIdescO = (1u << 4) | (kFormat << 7) | ((E4M3 ? 1u : kFormat) << 10) |
                                   (1u << 15) | (1u << 16) |
                                   (static_cast<uint32_t>(kNPv >> 3) << 17) | (8u << 24);
      const uint32_t base = smem_addr(smem);
      TreeWalk ws = walk, wo = walk;
      TreeSeg ss{}, so{};
      bool ok = true;
      int s_tile = 0, s_segs = -1;  // tile of the segment of the next S, its index
      auto issue_s = [&](int i) {
        if (s_segs < 0 || s_tile == ss.t1) {
          tree_next(ws, p, ss);
          s_tile = ss.t0;
          ++s_segs;
          ok = mbar_wait(&q_full[s_segs % Lay::kQBufs], (s_segs / Lay::kQBufs) & 1, wc, 64);
          if (!ok) return;
        }
        const int pos = tree_k_pos(i), slot = pos % kSlots;
        ok = mbar_wait(&kv_full[slot], (pos / kSlots) & 1, wc, 65);
        if (!ok) return;
        tc_fence_after();
        const uint32_t a0 = sdesc_lo(base + slot * Lay::kSlotBytes, false);
        const uint32_t b0 = sdesc_lo(base + Lay::kQ + (s_segs % Lay::kQBufs) * Lay::kQBytes, false);
        const uint32_t d = tmem + (i & 1) * R;
#pragma unroll
        for (int t = 0; t < Lay::kTermsQ; ++t) {
#pragma unroll
          for (int k = 0; k < Lay::kSteps; ++k)
            tree_mma<E4M3>(d, a0 + (k >> 2) * 1024 + (k & 3) * 2,
                           b0 + t * (Lay::kPanels * Lay::kQPanel >> 4) + (k >> 2) * (Lay::kQPanel >> 4) +
                               (k & 3) * 2,
                           kIdescS, t + k > 0);
        }
        umma_commit(&s_full[i & 1]);
        umma_commit(&kv_empty[slot]);
        if (++s_tile == ss.t1) umma_commit(&q_empty[s_segs % Lay::kQBufs]);
      };
      int o_tile = 0;
      bool o_begun = false;
      auto issue_o = [&](int i) {
        if (!o_begun || o_tile == so.t1) {
          tree_next(wo, p, so);
          o_tile = so.t0;
          o_begun = true;
        }
        ok = mbar_wait(&p_full[i & 1], (i >> 1) & 1, wc, 66);
        if (!ok) return;
        const int pos = tree_v_pos(i, n_tiles), slot = pos % kSlots;
        ok = mbar_wait(&kv_full[slot], (pos / kSlots) & 1, wc, 67);
        if (!ok) return;
        tc_fence_after();
        const uint32_t a0 = sdesc_lo(base + slot * Lay::kSlotBytes, true);
        const uint32_t b0 = sdesc_lo(base + Lay::kP + (i % Lay::kPBufs) * Lay::kPBytes, true);
        const uint32_t d = tmem + 2 * R;
        constexpr int kKeySteps = E4M3 ? 4 : 8;                  // 32 or 16 keys each
        constexpr uint32_t kKeyStep = E4M3 ? 256u : 128u;        // x 16 bytes
        constexpr int kTerms = E4M3 && !Lay::kStack ? Lay::kTermsP : 1;
        const bool first = o_tile == so.t0;
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
#pragma unroll
          for (int k = 0; k < kKeySteps; ++k)
            tree_mma<E4M3>(d, a0 + k * kKeyStep, b0 + t * 1024 + k * kKeyStep, kIdescO,
                           !first || t + k > 0);
        }
        umma_commit(&kv_empty[slot]);
        umma_commit(pv_done);
        if (++o_tile == so.t1) umma_commit(o_full);
      };
      issue_s(0);
      if (ok && n_tiles > 1) issue_s(1);
      for (int i = 0; i < n_tiles && ok; ++i) {
        issue_o(i);
        if (ok && i + 2 < n_tiles) issue_s(i + 2);
      }
      umma_commit(drain);
      mbar_wait_drain(drain, 0, 200000000ull);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------------------------------------- Q
    constexpr int kLanes = D / 8;                // lanes of a row, 8 values each
    constexpr int kRowsWarp = 32 / kLanes;
    const int rows_all = p.group * p.T;
    TreeSeg seg;
    for (int si = 0; tree_next(walk, p, seg); ++si) {
      const int qb = si % Lay::kQBufs;
      if (!mbar_wait_warp(&q_empty[qb], ((si / Lay::kQBufs) & 1) ^ 1, wc, 68)) break;
      const int sub = lane / kLanes, l = lane % kLanes;
      const long long row0 = (static_cast<long long>(seg.b) * p.Hq + static_cast<long long>(seg.hk) * p.group) * p.T +
                             static_cast<long long>(seg.rt) * R;
      uint8_t* qdst = smem + Lay::kQ + qb * Lay::kQBytes;
#pragma unroll 4
      for (int r0 = (warp - 10) * kRowsWarp; r0 < R; r0 += 2 * kRowsWarp) {
        const int r = r0 + sub;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (seg.rt * R + r < rows_all)
          x = *(reinterpret_cast<const uint4*>(p.q + (row0 + r) * D * 2) + l);
        if constexpr (E4M3) {
          float f[8];
          float amax = abs_max8(x, BF16, 0.f);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
            amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          unpack8<BF16>(x, f);
          // up = 2^(7 - e), e the exponent of amax: amax up in [128, 256)
          const int e = amax > 0.f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23), 8), 253) : 134;
          const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
          const float down = __uint_as_float(static_cast<uint32_t>(e - 7) << 23);
          if (l == 0)
            s_qs[qb * R + r] = amax < INFINITY ? down * p.scale_log2 : __int_as_float(0x7fffffff);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= up;
#pragma unroll
          for (int t = 0; t < Lay::kTermsQ; ++t) {
            uint32_t w[2];
            w[0] = pack_e4m3x4(f[0], f[1], f[2], f[3]);
            w[1] = pack_e4m3x4(f[4], f[5], f[6], f[7]);
            if (t + 1 < Lay::kTermsQ) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float a, b;
                unpack_e4m3x2(w[i >> 1] >> (16 * (i & 1)), a, b);
                f[2 * i] -= a;
                f[2 * i + 1] -= b;
              }
            }
            // 8 bytes at column 8 l of row r: chunk l / 2, swizzled by the row
            const uint32_t at = r * 128 + ((((l >> 1) ^ (r & 7)) << 4) | ((l & 1) << 3));
            *reinterpret_cast<uint2*>(qdst + t * Lay::kQPanel + at) = make_uint2(w[0], w[1]);
          }
        } else {
          const uint32_t at = (l >> 3) * Lay::kQPanel + r * 128 + (((l & 7) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(qdst + at) = x;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qb]);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const int grp = warp >> 2;
    const int tid = threadIdx.x & 127;           // key of the tile = TMEM lane; d at the end
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int col0 = grp * kCols;
    const int bar_id = 1 + grp;
    float* nr = s_nr + col0;
    float* alpha = s_alpha + col0;
    // a row's reference stands for P = 2^kBias, and moves when P would pass
    // 2^kOver.  e5m2 terms reach from 2^15 down to steps of 2^-16: the reference
    // at 2^11 leaves 2^4 above it and 2^-27 below; fp16 has steps of 2^-24.
    constexpr float kBias = E4M3 ? 11.f : BF16 ? 0.f : 7.f;
    constexpr float kOver = E4M3 ? 15.f : kBias + 8.f;
    const int rows_all = p.group * p.T;
    bool ok = true;
    int i = 0;                                   // tile of this CTA
    TreeSeg seg;
    for (int si = 0; tree_next(walk, p, seg); ++si) {
      const int qb = si % Lay::kQBufs;
      const float* qs = s_qs + qb * R + col0;
      const int L = seg.ctx + seg.drafts;
      const int m0 = seg.rt * R + col0;          // first row of this thread's columns
      const int t_first = m0 % p.T;
      ok = mbar_wait_warp(&q_full[qb], (si / Lay::kQBufs) & 1, wc, 69) && ok;
      if (tid < kCols) nr[tid] = kTreeNoRef;
      if (tid == 0) s_fix[(si & 1) * 2 + grp] = 0;
      // (a wait that gave up: this group goes on to the vote at the item's end)
      ok = named_bar_and(bar_id, 128, ok);
      const bool begun = ok;
      float sum[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) sum[c] = 0.f;
      for (int tile = seg.t0; begun && tile < seg.t1; ++tile, ++i) {
        const int key = tile * 128 + tid;
        const int u = key - seg.ctx;             // drafted token, negative in the context
        // columns that see this key (only tiles with the end of the sequence
        // or drafted tokens need them)
        const bool edge = tile * 128 + 128 > seg.ctx;
        uint64_t seen = ~0ull;
        if (edge && u >= 0) {
          seen = 0ull;
          if (u < seg.drafts) {
            int t = t_first;
            for (int c = 0; c < kCols; ++c) {
              if (tree_sees(p, seg.b, t, u)) seen |= 1ull << c;
              if (++t == p.T) t = 0;
            }
          }
        }
        float sk = 1.f, sv = 1.f;
        if constexpr (E4M3) {
          const int ss = i % Lay::kScales;
          ok = mbar_wait_warp(&sc_full[ss], (i / Lay::kScales) & 1, wc, 70) && ok;
          if (key < L) {
            const float* sc = reinterpret_cast<const float*>(smem + Lay::kScale + ss * 1024);
            sk = sc[tid];
            sv = sc[128 + tid];
            // (a scale that is not a size makes its row's probabilities NaN)
            if (!(sv >= kTreeMinScale)) sv = sv >= 0.f ? kTreeMinScale : NAN;
            else if (sv == INFINITY) sv = NAN;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_empty[ss]);
        }
        ok = mbar_wait_warp(&s_full[i & 1], (i >> 1) & 1, wc, 71) && ok;
        tc_fence_after();
        float x[kCols];
        {
          uint32_t raw[kCols];
          tmem_ld_cols<kCols>(tmem + lane_off + (i & 1) * R + col0, raw);
#pragma unroll
          for (int c = 0; c < kCols; ++c) x[c] = __uint_as_float(raw[c]) * (E4M3 ? sk : p.scale_log2);
        }
        if (edge && u >= 0) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (!((seen >> c) & 1)) x[c] = -INFINITY;
        }
        // exponents against the references; z = x qs + log2 sv is the exponent
        // of what is stored
        const float lv = E4M3 ? log2f(sv) : 0.f;
        const float limit = kOver - lv;
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float dd = E4M3 ? fmaf(x[c], qs[c], nr[c]) : x[c] + nr[c];
          top = fmaxf(top, dd);
        }
        if (named_bar_or(bar_id, 128, top > limit || !ok)) {
          // some row's reference moves (or a wait gave up)
          if (!named_bar_and(bar_id, 128, ok)) { ok = false; break; }
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const float z = (E4M3 ? x[c] * qs[c] : x[c]) + lv;
            const float m = warp_max(((seen >> c) & 1) ? z : -INFINITY);
            if (lane == 0) s_wmax[(warp & 3) * R + col0 + c] = m;
          }
          named_bar_sync(bar_id, 128);
          if (tid < kCols) {
            float m = s_wmax[col0 + tid];
#pragma unroll
            for (int w = 1; w < 4; ++w) m = fmaxf(m, s_wmax[w * R + col0 + tid]);
            const float old = nr[tid];
            const float now = m > -INFINITY ? fminf(old, kBias - m) : old;
            nr[tid] = now;
            alpha[tid] = exp2f(now - old);  // 0 for a row that had no key yet
          }
          named_bar_sync(bar_id, 128);
#pragma unroll
          for (int c = 0; c < kCols; ++c) sum[c] *= alpha[c];
          if (tile > seg.t0) {
            // O^T: this thread is row d = tid.  Its products up to tile i - 2 are
            // complete (S(i) was committed after them); PV(i - 1) is waited for.
            ok = mbar_wait_warp(pv_done, (i - 1) & 1, wc, 72);
            if (!named_bar_and(bar_id, 128, ok)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < Lay::kOCols / R; ++t) {
#pragma unroll
              for (int c = 0; c < kCols; c += 8) {
                const uint32_t at = tmem + lane_off + 2 * R + t * R + col0 + c;
                uint32_t ro[8];
                tmem_ld8(at, ro);
#pragma unroll
                for (int e = 0; e < 8; ++e) ro[e] = __float_as_uint(__uint_as_float(ro[e]) * alpha[c + e]);
                tmem_st_n<8>(at, ro);
              }
            }
            tmem_st_wait();
          }
        }
        // V rows that the cache does not hold are cleared (0 x NaN is NaN), and
        // drafted rows are searched for values that are not finite
        if (edge) {
          const int pos = tree_v_pos(i, n_tiles), slot = pos % kSlots;
          ok = mbar_wait_warp(&kv_full[slot], (pos / kSlots) & 1, wc, 73) && ok;
          if (ok && u >= 0) {
            uint8_t* row = smem + slot * Lay::kSlotBytes + tid * 128;
#pragma unroll
            for (int pn = 0; pn < Lay::kPanels; ++pn) {
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                uint4* at = reinterpret_cast<uint4*>(row + pn * 16384 + (grp * 4 + ch) * 16);
                if (key >= L) {
                  *at = make_uint4(0u, 0u, 0u, 0u);
                } else {
                  uint4 v = *at;
                  uint32_t w[4] = {v.x, v.y, v.z, v.w};
                  bool found = false;
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    uint32_t bad;  // all ones in the elements that are not finite
                    if constexpr (E4M3) bad = __vcmpeq4(w[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                    else if constexpr (BF16) bad = __vcmpeq2(w[e] & 0x7F807F80u, 0x7F807F80u);
                    else bad = __vcmpeq2(w[e] & 0x7C007C00u, 0x7C007C00u);
                    found |= bad != 0;
                    w[e] &= ~bad;
                  }
                  if (found) {
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                    s_fix[(si & 1) * 2 + grp] = 1;
                  }
                }
              }
            }
          }
        }
        if (Lay::kPBufs == 1 && i > 0)
          ok = mbar_wait_warp(pv_done, (i - 1) & 1, wc, 74) && ok;
        // probabilities, their sums, and P^T
        uint8_t* prow = smem + Lay::kP + (i % Lay::kPBufs) * Lay::kPBytes + tid * 128;
        const uint32_t swz = tid & 7;
        if constexpr (E4M3) {
          constexpr int kTerms = Lay::kTermsP;
#pragma unroll
          for (int c = 0; c < kCols; c += 8) {
            uint32_t w[2][kTerms];
#pragma unroll
            for (int q4 = 0; q4 < 2; ++q4) {
              float pr[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int cc = c + 4 * q4 + e;
                const float ex = ex2_approx(fmaf(x[cc], qs[cc], nr[cc]));
                sum[cc] += ex;
                pr[e] = ((seen >> cc) & 1) ? ex * sv : 0.f;
              }
              e5m2_terms<kTerms>(pr[0], pr[1], pr[2], pr[3], w[q4]);
            }
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
              const int at = t * R + col0 + c;   // byte of the key's row of P^T
              *reinterpret_cast<uint2*>(prow + (at >> 7) * 16384 + ((((at >> 4) & 7) ^ swz) << 4) + (at & 8)) =
                  make_uint2(w[0][t], w[1][t]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols; c += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = ex2_approx(x[c + 2 * e] + nr[c + 2 * e]);
              const float b = ex2_approx(x[c + 2 * e + 1] + nr[c + 2 * e + 1]);
              sum[c + 2 * e] += a;
              sum[c + 2 * e + 1] += b;
              w[e] = pack2<BF16>(a, b);
            }
            const int at = 2 * (col0 + c);
            *reinterpret_cast<uint4*>(prow + (at >> 7) * 16384 + ((((at >> 4) & 7) ^ swz) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&p_full[i & 1]);
          if (tile + 1 == seg.t1) mbar_arrive(&q_empty[qb]);
        }
      }
      // ----------------------------------------------------------- end of the item
      const bool whole = ok && mbar_wait_warp(o_full, si & 1, wc, 75);
      if (!named_bar_and(3, 256, whole)) { ok = false; break; }
      tc_fence_after();
      // sums of the columns over the 128 keys' threads
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float v = sum[c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s_wmax[(warp & 3) * R + col0 + c] = v;
      }
      named_bar_sync(bar_id, 128);
      const bool complete = seg.t0 == 0 && seg.t1 == seg.nt;
      float* slot = p.partial + (2 * static_cast<size_t>(blockIdx.x) + (seg.t0 == 0 ? 1 : 0)) * tree_slot_floats<Lay>();
      const long long out0 = (static_cast<long long>(seg.b) * p.Hq + static_cast<long long>(seg.hk) * p.group) * p.T;
      if (tid < kCols) {
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) l += s_wmax[w * R + col0 + tid];
        const int m = m0 + tid;
        if (complete) {
          s_sum[col0 + tid] = l == 0.f ? 0.f : 1.f / l;
          if (m < rows_all && m % p.T < seg.drafts)
            p.lse[out0 + m] = l == 0.f ? -INFINITY : (log2f(l) - nr[tid]) * 0.69314718055994531f;
        } else {
          float2* st = reinterpret_cast<float2*>(slot + R * D) + col0 + tid;
          *st = make_float2(-nr[tid], l);
        }
      }
      named_bar_sync(bar_id, 128);
      const int fix = s_fix[(si & 1) * 2] | s_fix[(si & 1) * 2 + 1];
#pragma unroll 1
      for (int c = 0; c < kCols; c += 8) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
        for (int t = 0; t < Lay::kOCols / R; ++t) {
          uint32_t ro[8];
          tmem_ld8(tmem + lane_off + 2 * R + t * R + col0 + c, ro);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += __uint_as_float(ro[e]);
        }
        if (tid >= D) continue;                  // (d = 64: the upper lanes hold nothing)
        if (fix) {
          // drafted V rows with values that are not finite were cleared there:
          // add them for the queries that see them
          for (int key = max(seg.ctx, seg.t0 * 128); key < min(L, seg.t1 * 128); ++key) {
            const long long row = cache_row(p.c, seg.b, seg.hk, key);
            if (row < 0) continue;
            float v, skip;
            if constexpr (E4M3) unpack_e4m3x2(p.c.v[row * D + tid], v, skip);
            else unpack2<BF16>(reinterpret_cast<const uint16_t*>(p.c.v)[row * D + tid], v, skip);
            if (fabsf(v) < INFINITY) continue;
            for (int e = 0; e < 8; ++e)
              if (tree_sees(p, seg.b, (m0 + c + e) % p.T, key - seg.ctx)) o[e] += v;
          }
        }
        if (complete) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int m = m0 + c + e;
            if (m < rows_all && m % p.T < seg.drafts) {
              const float inv = s_sum[col0 + c + e];
              const float y = inv == 0.f ? 0.f : o[e] * inv;
              reinterpret_cast<uint16_t*>(p.o)[(out0 + m) * D + tid] =
                  static_cast<uint16_t>(pack2<BF16>(y, 0.f));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) slot[(col0 + c + e) * D + tid] = o[e];
        }
      }
      tc_fence_before();
      named_bar_sync(bar_id, 128);               // s_sum, s_wmax are reused
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::kTmemCols);
  }
}

// Adds up the parts of the items that were cut.  Block (c, y): the item whose
// first cut is at the start of CTA c's piece (if any), its rows y, y + gridDim.y
// ...; a thread is a column of O.
template <int D, bool BF16>
__global__ void __launch_bounds__(D) fa_tree_join_kernel(const TreeParams p, int R) {
  const int c0 = blockIdx.x + 1;
  const int* head = p.heads + c0 * 4;
  const int b = head[0], item = head[1];
  if (b < 0) return;
  // (a CTA whose own first item is the same one did not begin it)
  if (p.heads[(c0 - 1) * 4] == b && p.heads[(c0 - 1) * 4 + 1] == item) return;
  int last = c0;
  while (!p.heads[last * 4 + 2] && last + 1 < p.grid) ++last;
  const size_t slot_floats = static_cast<size_t>(R) * (D + 2);
  const float* first = p.partial + (2 * static_cast<size_t>(c0 - 1) + 1) * slot_floats;
  const int hk = item / p.row_tiles, rt = item - hk * p.row_tiles;
  const long long out0 = (static_cast<long long>(b) * p.Hq + static_cast<long long>(hk) * p.group) * p.T;
  const int drafts = head[3];
  for (int r = blockIdx.y; r < R; r += gridDim.y) {
    const int m = rt * R + r;
    if (m >= p.group * p.T || m % p.T >= drafts) continue;
    auto part = [&](int c) {
      return c == c0 - 1 ? first : p.partial + 2 * static_cast<size_t>(c) * slot_floats;
    };
    float top = -INFINITY;
    for (int c = c0 - 1; c <= last; ++c) {
      const float2 st = reinterpret_cast<const float2*>(part(c) + R * D)[r];
      if (st.y != 0.f) top = fmaxf(top, st.x);
    }
    float l = 0.f, o = 0.f;
    for (int c = c0 - 1; c <= last; ++c) {
      const float* s = part(c);
      const float2 st = reinterpret_cast<const float2*>(s + R * D)[r];
      const float w = st.y == 0.f ? 0.f : exp2f(st.x - top);
      l += w * st.y;
      o += w == 0.f ? 0.f : w * s[r * D + threadIdx.x];
    }
    const float y = l == 0.f ? 0.f : o / l;
    reinterpret_cast<uint16_t*>(p.o)[(out0 + m) * D + threadIdx.x] =
        static_cast<uint16_t>(pack2<BF16>(y, 0.f));
    if (threadIdx.x == 0)
      p.lse[out0 + m] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
  }
}

template <int D, bool BF16, bool E4M3, int R>
static cudaError_t launch_tree_t(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p,
                                 cudaStream_t stream) {
  using Lay = TreeLayout<D, BF16, E4M3, R>;
  auto kern = fa_tree_kernel<D, BF16, E4M3, R>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<p.grid, kTreeThreads, Lay::kSmemBytes, stream>>>(tmk, tmv, p);
  // items of one tile are never cut
  if (p.grid > 1 && static_cast<long long>(p.c.table_stride) * p.c.page_size > 128)
    fa_tree_join_kernel<D, BF16><<<dim3(p.grid - 1, R < 16 ? R : 16), D, 0, stream>>>(p, R);
  return cudaGetLastError();
}

cudaError_t launch_tree(int d, bool bf16, bool e4m3, int rows, const CUtensorMap& tmk,
                        const CUtensorMap& tmv, const TreeParams& p, cudaStream_t stream) {
#define FA_TREE_R(DD, BB, EE)                                                     \
  (rows == 16   ? launch_tree_t<DD, BB, EE, 16>(tmk, tmv, p, stream)              \
   : rows == 32 ? launch_tree_t<DD, BB, EE, 32>(tmk, tmv, p, stream)              \
   : rows == 64 ? launch_tree_t<DD, BB, EE, 64>(tmk, tmv, p, stream)              \
                : launch_tree_t<DD, BB, EE, 128>(tmk, tmv, p, stream))
  if (d == 128) {
    if (bf16) return e4m3 ? FA_TREE_R(128, true, true) : FA_TREE_R(128, true, false);
    return e4m3 ? FA_TREE_R(128, false, true) : FA_TREE_R(128, false, false);
  }
  if (bf16) return e4m3 ? FA_TREE_R(64, true, true) : FA_TREE_R(64, true, false);
  return e4m3 ? FA_TREE_R(64, false, true) : FA_TREE_R(64, false, false);
#undef FA_TREE_R
}

}  // namespace fa
