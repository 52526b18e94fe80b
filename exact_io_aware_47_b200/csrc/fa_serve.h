// Parameters shared between the host launchers and the kernels of the serving
// operators: rotary positions, the paged K/V cache, attention of drafted
// tokens.
#pragma once

#include "fa_internal.h"

namespace fa {

// Element strides (batch, head, row) of a [B, H, N, d] tensor, d contiguous.
struct Strides3 {
  long long b, h, n;
};

struct RopeTensor {
  const uint8_t* x;
  uint8_t* y;
  Strides3 xs, ys;
  int heads;
  bool in_place;  // same pointer and strides: the columns past rot need no copy
};

struct RopeParams {
  RopeTensor t[2];           // q, k
  const int32_t* positions;  // nullptr: row n is at position n
  long long pos_stride;
  const double* inv_freq;    // [rot / 2]
  int B, N, rot;
  float factor;
  float sign;                // +1: rotate by theta, -1: by -theta (gradient)
};

// A paged cache as one sequence table sees it (fa.h, "The K/V cache").
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;            // e4m3 only
  float* v_scale;
  const int32_t* table;      // nullptr: page b for sequence b
  int table_stride;          // pages per sequence (1 without a table)
  int num_pages, page_size, Hk;
  long long room;            // positions of a sequence: those of the table, below 2^31
  unsigned page_mul, page_shift;  // x / page_size = umulhi(x, page_mul) >> page_shift, x < 2^31
};

// Row index (over [num_pages, Hk, page_size]) of position `pos` of sequence b
// and head h; -1 if the position is past the table or its page is not in the
// pool.
__device__ __forceinline__ long long cache_row(const CacheView& c, int b, int h, long long pos) {
  if (pos < 0 || pos >= c.room) return -1;
  const unsigned at = __umulhi(static_cast<unsigned>(pos), c.page_mul) >> c.page_shift;
  const int row = static_cast<int>(pos - static_cast<long long>(at) * c.page_size);
  const int page = c.table ? c.table[static_cast<long long>(b) * c.table_stride + at] : b;
  if (page < 0 || page >= c.num_pages) return -1;
  return (static_cast<long long>(page) * c.Hk + h) * c.page_size + row;
}

struct CacheCopyParams {
  CacheView c;
  const uint8_t* k;          // write: sources [B, Hk, N, d]
  const uint8_t* v;
  Strides3 ks, vs;
  uint8_t* k_out;            // read: destinations, contiguous
  uint8_t* v_out;
  const int32_t* start;      // nullptr: 0
  const int32_t* lens;       // nullptr: N
  int B, N;
  bool clear;                // read: rows that are not read become zeros
};

struct TreeParams {
  CacheView c;
  const uint8_t* q;          // [B, Hq, T, d]
  uint8_t* o;
  float* lse;
  const int32_t* ctx_lens;
  const int32_t* draft_lens;  // nullptr: T
  const uint8_t* mask;       // nullptr: u <= t
  long long mask_stride;     // T * T, or 0 for a shared mask
  int B, Hq, T, group;       // group = Hq / Hk
  float scale_log2;          // scale * log2(e)
  int row_tiles;             // ceil(group * T / rows of a tile)
  int box, box_log2;         // keys of one TMA load: a power of two that divides page_size
  int grid;                  // CTAs
  int* heads;                // workspace: [grid][4], see fa_tree_kernel
  float* partial;            // workspace: [grid][2] slots
  unsigned long long wait_ns;
};

constexpr int kTreeMaxCtas = 160;

// Rows of a tile, for `rows` query rows per K/V head.
inline int tree_rows(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

cudaError_t launch_rope(int d, bool bf16, bool interleaved, const RopeParams& p, int num_sms,
                        cudaStream_t stream);
cudaError_t launch_cache_write(int d, bool bf16, bool e4m3, const CacheCopyParams& p,
                               cudaStream_t stream);
cudaError_t launch_cache_read(int d, bool bf16, bool e4m3, const CacheCopyParams& p,
                              cudaStream_t stream);
cudaError_t launch_tree(int d, bool bf16, bool e4m3, int rows, const CUtensorMap& tmk,
                        const CUtensorMap& tmv, const TreeParams& p, int device, cudaStream_t stream);

}  // namespace fa
