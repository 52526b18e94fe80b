// The paged K/V cache: quantising rows as they are written, and reading them
// back (fa.h, "The K/V cache").
//
// HBM-bound copies with a row-wise scale: 16-bit rows are read once and
// written once as e4m3 codes with one fp32 scale each (3 d + 4 bytes a row),
// or the other way round.  One row is one or half a warp's worth of 16-byte
// vectors, so a row's largest magnitude takes 3 or 4 shuffles and the row
// never leaves its registers.  A thread moves the same vector of K and of V.
// 131 us to read one context of 32768 positions and 32 heads back (d 128, 814 MB:
// 6.2 TB/s, 0.95 of a measured copy), 48 us to write a padded batch's prompts
// (256 MB, 5.3 TB/s).
#include "fa_serve.h"

namespace fa {

constexpr int kCacheThreads = 256;
// A block copies kCachePasses x (256 / lanes of a row) rows of one (sequence,
// head); a thread has all its 2 x kCachePasses 16-byte loads in flight at once
// (with one row per thread the chain lengths -> page table -> row -> store left
// the memory half idle: 82 against 60 us for the 256 MB of a padded
// batch's prompts).
constexpr int kCachePasses = 4;

template <int D>
struct CacheBlock {
  static constexpr int kLanes = D / 8;                        // 16-byte vectors of a 16-bit row
  static constexpr int kRows = kCacheThreads / kLanes;        // rows of a pass
  static constexpr int kBlockRows = kCachePasses * kRows;
};

// What this block copies: rows n0 .. of (b, h), below len.
struct CopyPart {
  int b, h, n0, len;
  long long start;
};
template <int D>
__device__ __forceinline__ CopyPart copy_part(const CacheCopyParams& p) {
  const unsigned chunks = (static_cast<unsigned>(p.N) + CacheBlock<D>::kBlockRows - 1) / CacheBlock<D>::kBlockRows;
  const unsigned bh = blockIdx.x / chunks;
  CopyPart c;
  c.n0 = static_cast<int>((blockIdx.x - bh * chunks) * CacheBlock<D>::kBlockRows);
  c.b = static_cast<int>(bh / static_cast<unsigned>(p.c.Hk));
  c.h = static_cast<int>(bh - static_cast<unsigned>(c.b) * static_cast<unsigned>(p.c.Hk));
  c.len = p.lens ? p.lens[c.b] : p.N;
  c.start = p.start ? p.start[c.b] : 0;
  if (c.len < 0 || c.len > p.N) {
    if (threadIdx.x == 0) record_error(kErrDeviceSeqlen, 3);
    c.len = c.len < 0 ? 0 : p.N;
  }
  return c;
}

// Largest magnitude of a row held by kLanes lanes, 8 values each, two at a
// time; NaN propagates.
template <int kLanes, bool BF16>
__device__ __forceinline__ float row_amax(const uint4& v) {
  auto mx = [](uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  };
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t m = mx(mx(v.x & kAbs, v.y & kAbs), mx(v.z & kAbs, v.w & kAbs));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = mx(m, __shfl_xor_sync(0xffffffffu, m, o));
  float lo, hi;
  unpack2<BF16>(m, lo, hi);
  return max_nan(lo, hi);
}

// Slots of a thread's rows n1 + e kRows, -1 for those that are not copied: lane e
// of a row's lanes looks up row e, the others are told.
template <int D>
__device__ __forceinline__ long long copy_slots(const CacheCopyParams& p, const CopyPart& c, int lane, int n1,
                                                long long (&slot)[kCachePasses]) {
  const int n = n1 + (lane & (kCachePasses - 1)) * CacheBlock<D>::kRows;
  const long long mine = n < c.len ? cache_row(p.c, c.b, c.h, c.start + n) : -1;
  if (lane < kCachePasses && n < c.len && mine < 0) record_error(kErrDeviceSeqlen, 4);
#pragma unroll
  for (int e = 0; e < kCachePasses; ++e)
    slot[e] = __shfl_sync(0xffffffffu, mine, e, CacheBlock<D>::kLanes);
  return mine;
}

// The copy is bound by its instructions, not by memory, unless what a row needs
// once is done once: its slot, and the two divisions of its scale, which the
// lanes of a row share out over the 2 x kCachePasses rows that they hold (150
// instructions a vector before, and 60 against 48 us for the 256 MB of a
// padded batch's prompts).
template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_write_kernel(const CacheCopyParams p) {
  constexpr int kLanes = CacheBlock<D>::kLanes, kRows = CacheBlock<D>::kRows;
  const CopyPart c = copy_part<D>(p);
  if (c.n0 >= c.len) return;
  const int lane = threadIdx.x % kLanes, n1 = c.n0 + threadIdx.x / kLanes;
  const uint8_t* k = p.k + 2 * (c.b * p.ks.b + c.h * p.ks.h + n1 * p.ks.n) + 16 * lane;
  const uint8_t* v = p.v + 2 * (c.b * p.vs.b + c.h * p.vs.h + n1 * p.vs.n) + 16 * lane;
  const long long k_step = 2 * kRows * p.ks.n, v_step = 2 * kRows * p.vs.n;
  uint4 x[kCachePasses][2];
#pragma unroll
  for (int e = 0; e < kCachePasses; ++e) {
    x[e][0] = x[e][1] = make_uint4(0u, 0u, 0u, 0u);
    if (n1 + e * kRows < c.len) {
      x[e][0] = __ldcs(reinterpret_cast<const uint4*>(k + e * k_step));
      x[e][1] = __ldcs(reinterpret_cast<const uint4*>(v + e * v_step));
    }
  }
  long long slot[kCachePasses];
  const long long mine = copy_slots<D>(p, c, lane, n1, slot);
  if constexpr (E4M3) {
    // lane l takes row l % 8 of the 8 (pass e, K or V: e = row / 2, w = row % 2);
    // with 16 lanes the first 8 form 448 / top, the others top / 448
    static_assert(2 * kCachePasses == 8, "8 rows for 8 or 16 lanes");
    const int row = lane & 7;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < kCachePasses; ++e)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float m = row_amax<kLanes, BF16>(x[e][w]);
        if (row == 2 * e + w) amax = m;
      }
    const long long at = __shfl_sync(0xffffffffu, mine, row >> 1, kLanes);
    const float top = fmaxf(amax, 448.f * 0x1p-126f);
    float inv, scale;
    if constexpr (kLanes == 16) {
      inv = scale = __fdiv_rn(lane < 8 ? 448.f : top, lane < 8 ? top : 448.f);
    } else {
      inv = __fdiv_rn(448.f, top);
      scale = __fdiv_rn(top, 448.f);
    }
    if (lane >= kLanes - 8 && at >= 0) {
      if (!(amax > 0.f)) scale = 1.f;
      if (!(amax < INFINITY)) {
        scale = __int_as_float(0x7fffffff);  // the row reads back as NaN
        record_error(kErrDeviceScale, 5);
      }
      ((row & 1) ? p.c.v_scale : p.c.k_scale)[at] = scale;
    }
#pragma unroll
    for (int e = 0; e < kCachePasses; ++e)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float f = __shfl_sync(0xffffffffu, inv, 2 * e + w, kLanes);
        if (slot[e] >= 0)
          reinterpret_cast<uint2*>((w ? p.c.v : p.c.k) + slot[e] * D)[lane] = to_e4m3x8(x[e][w], BF16, f);
      }
  } else {
#pragma unroll
    for (int e = 0; e < kCachePasses; ++e)
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (slot[e] >= 0) reinterpret_cast<uint4*>((w ? p.c.v : p.c.k) + slot[e] * D * 2)[lane] = x[e][w];
  }
}

// 8 e4m3 codes times a scale, rounded to 16 bits.
template <bool BF16>
__device__ __forceinline__ uint4 from_e4m3x8(const uint2& codes, float scale) {
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = i < 2 ? codes.x : codes.y;
    const unsigned short pair = static_cast<unsigned short>(word >> (16 * (i & 1)));
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(pair));
    float lo, hi;
    unpack2<false>(half2, lo, hi);
    out[i] = pack2<BF16>(lo * scale, hi * scale);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_read_kernel(const CacheCopyParams p) {
  constexpr int kLanes = CacheBlock<D>::kLanes;
  const CopyPart c = copy_part<D>(p);
  const int clear_end = p.clear ? p.N : 0;       // rows below it are written in any case
  if (c.n0 >= max(c.len, clear_end)) return;
  const int lane = threadIdx.x % kLanes, n1 = c.n0 + threadIdx.x / kLanes;
  long long slot[kCachePasses];
  copy_slots<D>(p, c, lane, n1, slot);
  using Vec = std::conditional_t<E4M3, uint2, uint4>;
  Vec x[kCachePasses][2];
  float scale[kCachePasses][2];
#pragma unroll
  for (int e = 0; e < kCachePasses; ++e) {
    if (slot[e] < 0) continue;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* cache = w ? p.c.v : p.c.k;
      x[e][w] = __ldcs(reinterpret_cast<const Vec*>(cache + slot[e] * (D * (E4M3 ? 1 : 2))) + lane);
      if (E4M3) scale[e][w] = (w ? p.c.v_scale : p.c.k_scale)[slot[e]];
    }
  }
#pragma unroll
  for (int e = 0; e < kCachePasses; ++e) {
    const int n = n1 + e * CacheBlock<D>::kRows;
    if (slot[e] < 0 && n >= clear_end) continue;
    const long long row = (static_cast<long long>(c.b) * p.c.Hk + c.h) * p.N + n;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint4 y = make_uint4(0u, 0u, 0u, 0u);
      if (slot[e] >= 0) {
        if constexpr (E4M3) y = from_e4m3x8<BF16>(x[e][w], scale[e][w]);
        else y = x[e][w];
      }
      __stcs(reinterpret_cast<uint4*>((w ? p.v_out : p.k_out) + row * D * 2) + lane, y);
    }
  }
}

static unsigned cache_grid(int d, const CacheCopyParams& p) {
  const int rows = d == 128 ? CacheBlock<128>::kBlockRows : CacheBlock<64>::kBlockRows;
  return static_cast<unsigned>(static_cast<long long>(p.B) * p.c.Hk * ((p.N + rows - 1) / rows));
}

#define FA_CACHE_LAUNCH(KERNEL)                                                              \
  const unsigned grid = cache_grid(d, p);                                                    \
  if (d == 128) {                                                                            \
    if (bf16) e4m3 ? KERNEL<128, true, true><<<grid, kCacheThreads, 0, stream>>>(p)          \
                   : KERNEL<128, true, false><<<grid, kCacheThreads, 0, stream>>>(p);        \
    else e4m3 ? KERNEL<128, false, true><<<grid, kCacheThreads, 0, stream>>>(p)              \
              : KERNEL<128, false, false><<<grid, kCacheThreads, 0, stream>>>(p);            \
  } else {                                                                                   \
    if (bf16) e4m3 ? KERNEL<64, true, true><<<grid, kCacheThreads, 0, stream>>>(p)           \
                   : KERNEL<64, true, false><<<grid, kCacheThreads, 0, stream>>>(p);         \
    else e4m3 ? KERNEL<64, false, true><<<grid, kCacheThreads, 0, stream>>>(p)               \
              : KERNEL<64, false, false><<<grid, kCacheThreads, 0, stream>>>(p);             \
  }                                                                                          \
  return cudaGetLastError()

cudaError_t launch_cache_write(int d, bool bf16, bool e4m3, const CacheCopyParams& p,
                               cudaStream_t stream) {
  FA_CACHE_LAUNCH(fa_cache_write_kernel);
}

cudaError_t launch_cache_read(int d, bool bf16, bool e4m3, const CacheCopyParams& p,
                              cudaStream_t stream) {
  FA_CACHE_LAUNCH(fa_cache_read_kernel);
}
#undef FA_CACHE_LAUNCH

}  // namespace fa
