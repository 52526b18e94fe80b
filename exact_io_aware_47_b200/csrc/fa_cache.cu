// The paged K/V cache: quantising rows as they are written, and reading them
// back (fa.h, "The K/V cache").
//
// HBM-bound copies with a row-wise scale: 16-bit rows are read once and
// written once as e4m3 codes with one fp32 scale each (3 d + 4 bytes a row),
// or the other way round.  One row is one or half a warp's worth of 16-byte
// vectors, so a row's largest magnitude takes 3 or 4 shuffles and the row
// never leaves its registers.  A thread moves the same vector of K and of V.
#include "fa_serve.h"

namespace fa {

constexpr int kCacheThreads = 256;

// The rows of a copy: (b, h, n) with n fastest, one per kLanes threads.
template <int kLanes>
__device__ __forceinline__ bool copy_row(const CacheCopyParams& p, int& b, int& h, int& n, int& lane) {
  const long long id = static_cast<long long>(blockIdx.x) * kCacheThreads + threadIdx.x;
  lane = static_cast<int>(id % kLanes);
  const long long row = id / kLanes;
  if (row >= static_cast<long long>(p.B) * p.c.Hk * p.N) return false;
  const unsigned r = static_cast<unsigned>(row);  // B Hk N < 2^31
  const unsigned bh = r / static_cast<unsigned>(p.N);
  n = static_cast<int>(r - bh * static_cast<unsigned>(p.N));
  b = static_cast<int>(bh / static_cast<unsigned>(p.c.Hk));
  h = static_cast<int>(bh - static_cast<unsigned>(b) * static_cast<unsigned>(p.c.Hk));
  return true;
}

// Slot of row n of sequence b, -1 for rows that are not copied.
__device__ __forceinline__ long long copy_slot(const CacheCopyParams& p, int b, int h, int n,
                                               bool first) {
  int len = p.lens ? p.lens[b] : p.N;
  if (len < 0 || len > p.N) {
    if (first && n == 0) record_error(kErrDeviceSeqlen, 3);
    len = len < 0 ? 0 : p.N;
  }
  if (n >= len) return -1;
  const long long slot = cache_row(p.c, b, h, (p.start ? static_cast<long long>(p.start[b]) : 0) + n);
  if (slot < 0 && first) record_error(kErrDeviceSeqlen, 4);
  return slot;
}

// amax of a row held by kLanes lanes, 8 values each; NaN propagates.
template <int kLanes, bool BF16>
__device__ __forceinline__ float row_amax(const uint4& v) {
  float m = abs_max8(v, BF16, 0.f);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_write_kernel(const CacheCopyParams p) {
  constexpr int kLanes = D / 8;
  int b = 0, h = 0, n = 0, lane = 0;
  const bool valid = copy_row<kLanes>(p, b, h, n, lane);
  const long long slot = valid ? copy_slot(p, b, h, n, lane == 0) : -1;
  uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (slot >= 0) {
    x[0] = __ldcs(reinterpret_cast<const uint4*>(p.k + 2 * (b * p.ks.b + h * p.ks.h + n * p.ks.n)) + lane);
    x[1] = __ldcs(reinterpret_cast<const uint4*>(p.v + 2 * (b * p.vs.b + h * p.vs.h + n * p.vs.n)) + lane);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint8_t* cache = w ? p.c.v : p.c.k;
    if constexpr (E4M3) {
      const float amax = row_amax<kLanes, BF16>(x[w]);  // whole warps: no lane has left
      if (slot < 0) continue;
      const float top = fmaxf(amax, 448.f * 0x1p-126f);
      float scale = amax > 0.f ? __fdiv_rn(top, 448.f) : 1.f;
      if (!(amax < INFINITY)) {
        scale = __int_as_float(0x7fffffff);  // the row reads back as NaN
        if (lane == 0) record_error(kErrDeviceScale, 5);
      }
      reinterpret_cast<uint2*>(cache + slot * D)[lane] =
          to_e4m3x8(x[w], BF16, __fdiv_rn(448.f, top));
      if (lane == 0) (w ? p.c.v_scale : p.c.k_scale)[slot] = scale;
    } else {
      if (slot >= 0) reinterpret_cast<uint4*>(cache + slot * D * 2)[lane] = x[w];
    }
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
  constexpr int kLanes = D / 8;
  int b, h, n, lane;
  if (!copy_row<kLanes>(p, b, h, n, lane)) return;
  const long long slot = copy_slot(p, b, h, n, lane == 0);
  if (slot < 0) return;
  const long long row = (static_cast<long long>(b) * p.c.Hk + h) * p.N + n;
  uint4 y[2];
  if constexpr (E4M3) {
    const uint2 ck = __ldcs(reinterpret_cast<const uint2*>(p.c.k + slot * D) + lane);
    const uint2 cv = __ldcs(reinterpret_cast<const uint2*>(p.c.v + slot * D) + lane);
    const float sk = p.c.k_scale[slot], sv = p.c.v_scale[slot];
    y[0] = from_e4m3x8<BF16>(ck, sk);
    y[1] = from_e4m3x8<BF16>(cv, sv);
  } else {
    y[0] = __ldcs(reinterpret_cast<const uint4*>(p.c.k + slot * D * 2) + lane);
    y[1] = __ldcs(reinterpret_cast<const uint4*>(p.c.v + slot * D * 2) + lane);
  }
  reinterpret_cast<uint4*>(p.k_out + row * D * 2)[lane] = y[0];
  reinterpret_cast<uint4*>(p.v_out + row * D * 2)[lane] = y[1];
}

static unsigned cache_grid(int d, const CacheCopyParams& p) {
  const long long threads = static_cast<long long>(p.B) * p.c.Hk * p.N * (d / 8);
  return static_cast<unsigned>((threads + kCacheThreads - 1) / kCacheThreads);
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
