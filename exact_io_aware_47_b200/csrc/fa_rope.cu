// Rotary positions on Q and K in one launch (fa.h, "Rotary positions"), and
// their gradient (the same rotation by the opposite angle).
//
// HBM-bound: every element is read once and written once (4 bytes); the work
// beside it is one sine and cosine per pair and row, which all heads share.
// So a thread owns 16 columns of one row (two 16-byte vectors that hold both
// halves of 8 pairs), computes its 8 angles once, and walks over heads.  86 us for
// 537 MB (B2, 32 + 32 heads, N 8192, d 128): 6.2 TB/s, 0.95 of a measured copy.
//
// Angles.  A position of 10^6 times a frequency near 1 needs more than the 24
// bits of fp32: the angle is formed in turns, p * (f / 2 pi), in fp64, reduced
// to [-1/2, 1/2] there, and only the remainder goes to fp32 (2^-26 turns
// absolute, below the rounding of sine and cosine).
#include "fa_serve.h"

namespace fa {

constexpr int kRopeThreads = 128;
constexpr int kRopeHeads = 4;  // heads in flight per thread: 8 16-byte loads

// The 8 elements of a vector as fp32 and back.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  unpack2<BF16>(v.x, f[0], f[1]);
  unpack2<BF16>(v.y, f[2], f[3]);
  unpack2<BF16>(v.z, f[4], f[5]);
  unpack2<BF16>(v.w, f[6], f[7]);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]),
                    pack2<BF16>(f[6], f[7]));
}

template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads)
    fa_rope_kernel(const RopeParams p, int heads_per_thread, int chunks) {
  constexpr int kUnits = D / 16;  // threads per row
  const long long id = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int u = static_cast<int>(id % kUnits);
  const long long rc = id / kUnits;
  const long long rows = static_cast<long long>(p.B) * p.N;
  const long long row = rc % rows;
  const int chunk = static_cast<int>(rc / rows);
  if (chunk >= chunks) return;
  const int b = static_cast<int>(row / p.N);
  const int n = static_cast<int>(row - static_cast<long long>(b) * p.N);

  // vectors (8 columns each) v0 and v1 of this thread: the first rot / 16
  // units take vector u and its partner rot / 16 further, which holds the
  // other halves of the pairs in the half layout; the rest copy
  const int ru = p.rot / 16;
  const bool rotates = u < ru;
  const int v0 = rotates ? u : 2 * ru + (u - ru);
  const int v1 = rotates ? u + ru : 2 * ru + (u - ru) + (kUnits - ru);
  float cs[8], sn[8];
  if (rotates) {
    const double pos =
        p.positions ? static_cast<double>(p.positions[b * p.pos_stride + n]) : static_cast<double>(n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = INTERLEAVED ? (i < 4 ? 4 * v0 + i : 4 * v1 + i - 4) : 8 * u + i;
      const double turns = pos * (p.inv_freq[pair] * 0.15915494309189533577);  // 1 / (2 pi)
      const float r = static_cast<float>(turns - rint(turns));
      float s, c;
      sincospif(2.f * r, &s, &c);
      cs[i] = p.factor * c;
      sn[i] = p.factor * (p.sign * s);
    }
  }
  const int h_all = p.t[0].heads + p.t[1].heads;
  const int h_begin = chunk * heads_per_thread;
  const int h_end = min(h_begin + heads_per_thread, h_all);
  for (int h0 = h_begin; h0 < h_end; h0 += kRopeHeads) {
    uint4 a[kRopeHeads], c[kRopeHeads];
#pragma unroll
    for (int e = 0; e < kRopeHeads; ++e) {
      if (h0 + e >= h_end) break;
      const int w = h0 + e >= p.t[0].heads;
      const RopeTensor& t = p.t[w];
      const int h = h0 + e - (w ? p.t[0].heads : 0);
      const uint8_t* src = t.x + 2 * (b * t.xs.b + h * t.xs.h + n * t.xs.n);
      a[e] = *reinterpret_cast<const uint4*>(src + 16 * v0);
      c[e] = *reinterpret_cast<const uint4*>(src + 16 * v1);
    }
#pragma unroll
    for (int e = 0; e < kRopeHeads; ++e) {
      if (h0 + e >= h_end) break;
      const int w = h0 + e >= p.t[0].heads;
      const RopeTensor& t = p.t[w];
      const int h = h0 + e - (w ? p.t[0].heads : 0);
      if (rotates) {
        float x[8], y[8];
        unpack8<BF16>(a[e], x);
        unpack8<BF16>(c[e], y);
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
            x[2 * i] = x0 * cs[i] - x1 * sn[i];
            x[2 * i + 1] = x1 * cs[i] + x0 * sn[i];
            y[2 * i] = y0 * cs[i + 4] - y1 * sn[i + 4];
            y[2 * i + 1] = y1 * cs[i + 4] + y0 * sn[i + 4];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x0 = x[i], y0 = y[i];
            x[i] = x0 * cs[i] - y0 * sn[i];
            y[i] = y0 * cs[i] + x0 * sn[i];
          }
        }
        a[e] = pack8<BF16>(x);
        c[e] = pack8<BF16>(y);
      } else if (t.in_place) {
        continue;
      }
      uint8_t* dst = t.y + 2 * (b * t.ys.b + h * t.ys.h + n * t.ys.n);
      *reinterpret_cast<uint4*>(dst + 16 * v0) = a[e];
      *reinterpret_cast<uint4*>(dst + 16 * v1) = c[e];
    }
  }
}

cudaError_t launch_rope(int d, bool bf16, bool interleaved, const RopeParams& p, int num_sms,
                        cudaStream_t stream) {
  const int heads = p.t[0].heads + p.t[1].heads;
  const long long threads_per_chunk = static_cast<long long>(p.B) * p.N * (d / 16);
  // many heads per thread share its angles; with few rows the heads are
  // spread over threads instead, until the device is full (2 x 8192 rows, 64 heads:
  // 86 us, with 4 heads a thread 91, with all 99; 32 rows, 40 heads: 3.6 us, with
  // all heads 12.3)
  const long long full = static_cast<long long>(num_sms) * 2048;
  int hpt = kRopeHeads;
  while (hpt < heads && threads_per_chunk * ((heads + 2 * hpt - 1) / (2 * hpt)) >= full) hpt *= 2;
  const int chunks = (heads + hpt - 1) / hpt;
  const long long blocks = (threads_per_chunk * chunks + kRopeThreads - 1) / kRopeThreads;
  const unsigned grid = static_cast<unsigned>(blocks);
#define FA_ROPE(DD, BB, II) \
  fa_rope_kernel<DD, BB, II><<<grid, kRopeThreads, 0, stream>>>(p, hpt, chunks)
  if (d == 128) {
    if (bf16) interleaved ? FA_ROPE(128, true, true) : FA_ROPE(128, true, false);
    else interleaved ? FA_ROPE(128, false, true) : FA_ROPE(128, false, false);
  } else {
    if (bf16) interleaved ? FA_ROPE(64, true, true) : FA_ROPE(64, true, false);
    else interleaved ? FA_ROPE(64, false, true) : FA_ROPE(64, false, false);
  }
#undef FA_ROPE
  return cudaGetLastError();
}

}  // namespace fa
