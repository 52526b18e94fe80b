// Attention of drafted tokens over the paged cache (fa.h, fa_fwd_tree).
//
// One warp per query row, 32 keys at a time: a lane scores one key, the warp
// keeps the running maximum and sum of the softmax, and each lane accumulates
// its columns of O over the 32 probabilities.
#include "fa_serve.h"

namespace fa {

constexpr int kTreeWarps = 4;

// Lengths of sequence b, clamped into range and reported.
struct TreeLens {
  int ctx, drafts;
};
__device__ __forceinline__ TreeLens tree_lens(const TreeParams& p, int b) {
  const long long room = static_cast<long long>(p.c.table_stride) * p.c.page_size;
  const int n_in = p.draft_lens ? p.draft_lens[b] : p.T;
  const int ctx_in = p.ctx_lens[b];
  const int n_cap = static_cast<int>(min(static_cast<long long>(p.T), room));
  const int n = min(max(n_in, 0), n_cap);
  const int ctx = static_cast<int>(min(static_cast<long long>(max(ctx_in, 0)), room - n));
  if (n != n_in || ctx != ctx_in) record_error(kErrDeviceSeqlen, 6);
  return TreeLens{ctx, n};
}

template <int D, bool BF16, bool E4M3>
__device__ __forceinline__ float cache_value(const uint8_t* cache, const float* scale,
                                             long long row, int col) {
  if constexpr (E4M3) {
    const unsigned short code = cache[row * D + col];
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(code));
    float lo, hi;
    unpack2<false>(half2, lo, hi);
    return lo * scale[row];
  } else {
    float lo, hi;
    unpack2<BF16>(reinterpret_cast<const uint16_t*>(cache)[row * D + col], lo, hi);
    return lo;
  }
}

template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(kTreeWarps * 32) fa_tree_kernel(const TreeParams p) {
  __shared__ float qs[kTreeWarps][D];
  constexpr int kCols = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kTreeWarps + warp;
  if (row >= static_cast<long long>(p.B) * p.Hq * p.T) return;
  const int t = static_cast<int>(row % p.T);
  const int h = static_cast<int>(row / p.T % p.Hq);
  const int b = static_cast<int>(row / p.T / p.Hq);
  const TreeLens len = tree_lens(p, b);
  if (t >= len.drafts) return;
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + row * D;
#pragma unroll
  for (int e = 0; e < kCols; ++e) {
    float lo, hi;
    unpack2<BF16>(q[lane + 32 * e], lo, hi);
    qs[warp][lane + 32 * e] = lo * p.scale_log2;
  }
  __syncwarp();
  float m = -INFINITY, l = 0.f, acc[kCols] = {};
  const int keys = len.ctx + len.drafts;
  for (int j0 = 0; j0 < keys; j0 += 32) {
    const int j = j0 + lane;
    bool seen = j < keys;
    if (seen && j >= len.ctx) {
      const int u = j - len.ctx;
      seen = p.mask ? p.mask[b * p.mask_stride + static_cast<long long>(t) * p.T + u] != 0 : u <= t;
    }
    long long slot = -1;
    float s = -INFINITY;
    if (seen) {
      slot = cache_row(p.c, b, h / p.group, j);
      if (slot < 0) {
        record_error(kErrDeviceSeqlen, 7);
      } else {
        s = 0.f;
        for (int c = 0; c < D; ++c)
          s += qs[warp][c] * cache_value<D, BF16, E4M3>(p.c.k, p.c.k_scale, slot, c);
      }
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m_new = fmaxf(m, mx);
    const float mu = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = exp2f(m - mu);
    const float pr = slot >= 0 ? exp2f(s - mu) : 0.f;
    float sum = pr;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * alpha + sum;
    m = m_new;
#pragma unroll
    for (int e = 0; e < kCols; ++e) acc[e] *= alpha;
    for (int i = 0; i < 32; ++i) {
      const float pi = __shfl_sync(0xffffffffu, pr, i);
      const long long si = __shfl_sync(0xffffffffu, slot, i);
      if (si < 0) continue;  // not seen: its row is not read
#pragma unroll
      for (int e = 0; e < kCols; ++e)
        acc[e] += pi * cache_value<D, BF16, E4M3>(p.c.v, p.c.v_scale, si, lane + 32 * e);
    }
  }
  uint16_t* o = reinterpret_cast<uint16_t*>(p.o) + row * D;
#pragma unroll
  for (int e = 0; e < kCols; ++e) {
    const float y = l == 0.f ? 0.f : acc[e] / l;
    o[lane + 32 * e] = static_cast<uint16_t>(pack2<BF16>(y, 0.f));
  }
  if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

cudaError_t launch_tree(int d, bool bf16, bool e4m3, const TreeParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.Hq * p.T;
  const unsigned grid = static_cast<unsigned>((rows + kTreeWarps - 1) / kTreeWarps);
#define FA_TREE(DD, BB, EE) fa_tree_kernel<DD, BB, EE><<<grid, kTreeWarps * 32, 0, stream>>>(p)
  if (d == 128) {
    if (bf16) e4m3 ? FA_TREE(128, true, true) : FA_TREE(128, true, false);
    else e4m3 ? FA_TREE(128, false, true) : FA_TREE(128, false, false);
  } else {
    if (bf16) e4m3 ? FA_TREE(64, true, true) : FA_TREE(64, true, false);
    else e4m3 ? FA_TREE(64, false, true) : FA_TREE(64, false, false);
  }
#undef FA_TREE
  return cudaGetLastError();
}

}  // namespace fa
