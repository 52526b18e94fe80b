// C ABI of the serving operators: argument checks and launches.
//
// As in fa_api.cu, every check runs on the host before anything is enqueued.
#include "fa_serve.h"

namespace fa {
namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Strides of a [B, H, N, d] tensor: host int64[3] or nullptr for contiguous.  No
// dimension spans more than 2^40 elements, so extents stay far within 64 bits.
int read_strides(const int64_t* s, int B, int H, int N, int d, Strides3* out) {
  if (s == nullptr) {
    *out = Strides3{static_cast<long long>(H) * N * d, static_cast<long long>(N) * d, d};
    return FA_OK;
  }
  const int n[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] > (1ll << 40) / std::max(n[i] - 1, 1)) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (s[i] % 8 != 0) return FA_ERR_ALIGNMENT;
  *out = Strides3{s[0], s[1], s[2]};
  return FA_OK;
}

// Elements from the first to one past the last.
long long extent(const Strides3& s, int B, int H, int N, int d) {
  return (B - 1) * s.b + (H - 1) * s.h + (N - 1) * s.n + d;
}

// Whether rows of a strided tensor can share memory.  With the dimensions of
// more than one element sorted by stride, each stride has to reach past all
// that the smaller ones span.
bool rows_may_overlap(const Strides3& s, int B, int H, int N, int d) {
  long long st[3] = {s.b, s.h, s.n};
  long long n[3] = {B, H, N};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (st[j] > st[j + 1]) {
        std::swap(st[j], st[j + 1]);
        std::swap(n[j], n[j + 1]);
      }
  long long span = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (st[i] < span) return true;
    span += (n[i] - 1) * st[i];
  }
  return false;
}

bool same_view(const void* x, const Strides3& xs, const void* y, const Strides3& ys, int B, int H,
               int N) {
  return x == y && (B == 1 || xs.b == ys.b) && (H == 1 || xs.h == ys.h) && (N == 1 || xs.n == ys.n);
}

bool ranges_overlap(const void* x, long long nx, const void* y, long long ny) {
  const uint8_t* a = static_cast<const uint8_t*>(x);
  const uint8_t* b = static_cast<const uint8_t*>(y);
  return a < b + 2 * ny && b < a + 2 * nx;
}

// Whether a row of x [B, Hx, N, d] can share memory with one of y [B, Hy, N, d].
// Q, K and V are often slices of one buffer, so address ranges say little: with
// the strides equal, or nearly so, row y - row x = y - x + sum of t_i s_i, where
// t_i is the difference of two indices (of equal strides together), and the rows
// meet if that is within (-d, d).  The largest stride first, each t_i has few
// values from which the smaller strides can still get there; where a search of
// kSteps does not end (strides that no tensor of separate rows has), the answer
// is yes.
struct RowDistance {
  static constexpr int kSteps = 20000;
  struct Term {
    long long stride, lo, hi;  // t_i stride with lo <= t_i <= hi
  };
  Term term[6];
  int terms = 0, steps = 0;
  long long d;

  void add(long long stride, long long lo, long long hi) {
    if (stride == 0 || lo == hi) return;
    int i = 0;
    while (i < terms && term[i].stride > stride) ++i;
    if (i == terms || term[i].stride != stride) {
      for (int j = terms++; j > i; --j) term[j] = term[j - 1];
      term[i] = Term{stride, 0, 0};
    }
    term[i].lo += lo;
    term[i].hi += hi;
  }
  bool reaches(int i, long long at) {
    if (i == terms) return -d < at && at < d;
    long long least = at, most = at;  // of what the smaller strides can add
    for (int j = i + 1; j < terms; ++j) {
      least += term[j].lo * term[j].stride;
      most += term[j].hi * term[j].stride;
    }
    const Term& c = term[i];
    // least + t s < d and most + t s > -d
    auto floor_div = [](long long a, long long b) { return a / b - (a % b < 0 ? 1 : 0); };
    const long long lo = std::max(c.lo, floor_div(-d - most, c.stride) + 1);
    const long long hi = std::min(c.hi, floor_div(d - 1 - least, c.stride));
    for (long long t = lo; t <= hi; ++t) {
      if (++steps > kSteps) return true;
      if (reaches(i + 1, at + t * c.stride)) return true;
    }
    return false;
  }
};
bool rows_may_meet(const void* x, const Strides3& xs, int Hx, const void* y, const Strides3& ys, int Hy,
                   int B, int N, int d) {
  if (!ranges_overlap(x, extent(xs, B, Hx, N, d), y, extent(ys, B, Hy, N, d))) return false;
  RowDistance r;
  r.d = d;
  const long long x_st[3] = {xs.b, xs.h, xs.n}, y_st[3] = {ys.b, ys.h, ys.n};
  const int nx[3] = {B, Hx, N}, ny[3] = {B, Hy, N};
  for (int i = 0; i < 3; ++i) {
    r.add(x_st[i], 1 - nx[i], 0);
    r.add(y_st[i], 0, ny[i] - 1);
  }
  const auto bytes = static_cast<long long>(reinterpret_cast<intptr_t>(y) - reinterpret_cast<intptr_t>(x));
  return r.reaches(0, bytes / 2);
}

int rope_tensor(const void* x, const int64_t* xs, void* y, const int64_t* ys, int B, int H, int N,
                int d, int dtype, RopeTensor* t) {
  if (!x || !y) return FA_ERR_INVALID_ARG;
  int st = check_common(B, H, N, d, 1.f, dtype);
  if (st != FA_OK) return st;
  if (!aligned(x, 16) || !aligned(y, 16)) return FA_ERR_ALIGNMENT;
  t->x = static_cast<const uint8_t*>(x);
  t->y = static_cast<uint8_t*>(y);
  t->heads = H;
  if ((st = read_strides(xs, B, H, N, d, &t->xs)) != FA_OK) return st;
  if ((st = read_strides(ys, B, H, N, d, &t->ys)) != FA_OK) return st;
  if (rows_may_overlap(t->ys, B, H, N, d)) return FA_ERR_INVALID_ARG;
  t->in_place = same_view(x, t->xs, y, t->ys, B, H, N);
  if (!t->in_place &&
      ranges_overlap(x, extent(t->xs, B, H, N, d), y, extent(t->ys, B, H, N, d)))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

int rope_core(const void* q, const int64_t* qs, void* qo, const int64_t* qos, int Hq,
              const void* k, const int64_t* ks, void* ko, const int64_t* kos, int Hk,
              const int32_t* positions, int64_t positions_stride, const double* inv_freq, int B,
              int N, int d, int rot, int interleaved, float factor, int dtype, float sign,
              void* stream) {
  if (!inv_freq || positions_stride < 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(factor) && factor > 0.f)) return FA_ERR_INVALID_ARG;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  int st = rope_tensor(q, qs, qo, qos, B, Hq, N, d, dtype, &p.t[0]);
  if (st != FA_OK) return st;
  if (k == nullptr) {
    if (Hk != 0 || ko != nullptr) return FA_ERR_INVALID_ARG;
  } else {
    st = rope_tensor(k, ks, ko, kos, B, Hk, N, d, dtype, &p.t[1]);
    if (st != FA_OK) return st;
    const RopeTensor &tq = p.t[0], &tk = p.t[1];
    if (rows_may_meet(qo, tq.ys, Hq, ko, tk.ys, Hk, B, N, d) ||
        rows_may_meet(qo, tq.ys, Hq, k, tk.xs, Hk, B, N, d) ||
        rows_may_meet(q, tq.xs, Hq, ko, tk.ys, Hk, B, N, d))
      return FA_ERR_INVALID_ARG;
  }
  if (rot < 16 || rot > d || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  if ((positions && !aligned(positions, 4)) || !aligned(inv_freq, 8)) return FA_ERR_ALIGNMENT;
  p.positions = positions;
  p.pos_stride = positions_stride;
  p.inv_freq = inv_freq;
  p.B = B;
  p.N = N;
  p.rot = rot;
  p.factor = factor;
  p.sign = sign;
  DeviceInfo di;
  st = current_device_info(&di);
  if (st != FA_OK) return st;
  const cudaError_t e = launch_rope(d, dtype == FA_BF16, interleaved != 0, p, di.num_sms,
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Checks shared by everything that takes a cache; fills the view.
int cache_view(const void* k_cache, const void* v_cache, const float* k_scale,
               const float* v_scale, const int32_t* table, int table_stride, int B, int Hk, int d,
               int num_pages, int page_size, int format, CacheView* c) {
  if (!k_cache || !v_cache || k_cache == v_cache) return FA_ERR_INVALID_ARG;
  if (format != FA_CACHE_16 && format != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (format == FA_CACHE_E4M3 && (!k_scale || !v_scale || k_scale == v_scale))
    return FA_ERR_INVALID_ARG;
  if (Hk < 1 || num_pages < 1 || page_size < 1) return FA_ERR_INVALID_ARG;
  if (table ? table_stride < 1 : num_pages < B) return FA_ERR_INVALID_ARG;
  if (page_size % 16 != 0 || static_cast<long long>(num_pages) * Hk >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || (table && !aligned(table, 4)) ||
      (format == FA_CACHE_E4M3 && (!aligned(k_scale, 16) || !aligned(v_scale, 16))))
    return FA_ERR_ALIGNMENT;
  c->k = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  c->v = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  c->k_scale = const_cast<float*>(k_scale);
  c->v_scale = const_cast<float*>(v_scale);
  c->table = table;
  c->table_stride = table ? table_stride : 1;
  c->num_pages = num_pages;
  c->page_size = page_size;
  c->Hk = Hk;
  c->room = std::min(static_cast<long long>(c->table_stride) * page_size, (1ll << 31) - 1);
  // 2^(s - 1) < page_size <= 2^s: with m = ceil(2^(31 + s) / page_size) < 2^32 the
  // error of x m / 2^(31 + s) is below x / 2^(31 + s) < 1 / page_size for x < 2^31
  int s = 1;
  while ((1ll << s) < page_size) ++s;
  c->page_mul = static_cast<unsigned>(((1ull << (31 + s)) + page_size - 1) / page_size);
  c->page_shift = static_cast<unsigned>(s - 1);
  return FA_OK;
}

// [num_pages * Hk, page_size, d] view of a cache; box = 128 bytes x box rows,
// 128-byte swizzle.  e4m3 rows of d = 64 are filled with zeros to 128 bytes.
int make_map_cache(CUtensorMap* map, const void* ptr, const CacheView& c, int d, int box_rows,
                   int format, int dtype) {
  const bool e4m3 = format == FA_CACHE_E4M3;
  const cuuint64_t row = static_cast<cuuint64_t>(d) * (e4m3 ? 1 : 2);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.num_pages) * c.Hk};
  const cuuint64_t strides[2] = {row, row * c.page_size};
  const cuuint32_t box[3] = {e4m3 ? 128u : 64u, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(map,
                              e4m3               ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                              : dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              3, const_cast<void*>(ptr), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

int check_tree(int B, int Hq, int Hk, int T, int d, float scale, int dtype) {
  const int st = check_common(B, Hq, T, d, scale, dtype);
  if (st != FA_OK) return st;
  if (Hk < 1 || Hq % Hk != 0) return FA_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(Hq / Hk) * T;
  if (static_cast<long long>(B) * Hk * ((rows + 15) / 16) >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" int fa_rope(const void* q, const int64_t* q_strides, void* q_out,
                       const int64_t* q_out_strides, int Hq, const void* k,
                       const int64_t* k_strides, void* k_out, const int64_t* k_out_strides, int Hk,
                       const int32_t* positions, int64_t positions_stride, const double* inv_freq,
                       int B, int N, int d, int rot, int interleaved, float factor, int dtype,
                       void* stream) {
  return rope_core(q, q_strides, q_out, q_out_strides, Hq, k, k_strides, k_out, k_out_strides, Hk,
                   positions, positions_stride, inv_freq, B, N, d, rot, interleaved, factor, dtype,
                   1.f, stream);
}

extern "C" int fa_rope_bwd(const void* dq, const int64_t* dq_strides, void* dq_in,
                           const int64_t* dq_in_strides, int Hq, const void* dk,
                           const int64_t* dk_strides, void* dk_in, const int64_t* dk_in_strides,
                           int Hk, const int32_t* positions, int64_t positions_stride,
                           const double* inv_freq, int B, int N, int d, int rot, int interleaved,
                           float factor, int dtype, void* stream) {
  return rope_core(dq, dq_strides, dq_in, dq_in_strides, Hq, dk, dk_strides, dk_in, dk_in_strides,
                   Hk, positions, positions_stride, inv_freq, B, N, d, rot, interleaved, factor,
                   dtype, -1.f, stream);
}

extern "C" int fa_cache_write(const void* k, const int64_t* k_strides, const void* v,
                              const int64_t* v_strides, void* k_cache, void* v_cache,
                              float* k_scale, float* v_scale, const int32_t* block_table,
                              int table_stride, const int32_t* start, const int32_t* lens, int B,
                              int Hk, int N, int d, int num_pages, int page_size, int format,
                              int dtype, void* stream) {
  if (!k || !v) return FA_ERR_INVALID_ARG;
  int st = check_common(B, Hk, N, d, 1.f, dtype);
  if (st != FA_OK) return st;
  CacheCopyParams p;
  std::memset(&p, 0, sizeof(p));
  st = cache_view(k_cache, v_cache, k_scale, v_scale, block_table, table_stride, B, Hk, d,
                  num_pages, page_size, format, &p.c);
  if (st != FA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || (start && !aligned(start, 4)) ||
      (lens && !aligned(lens, 4)))
    return FA_ERR_ALIGNMENT;
  if ((st = read_strides(k_strides, B, Hk, N, d, &p.ks)) != FA_OK) return st;
  if ((st = read_strides(v_strides, B, Hk, N, d, &p.vs)) != FA_OK) return st;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.start = start;
  p.lens = lens;
  p.B = B;
  p.N = N;
  DeviceInfo di;
  st = current_device_info(&di);
  if (st != FA_OK) return st;
  const cudaError_t e = launch_cache_write(d, dtype == FA_BF16, format == FA_CACHE_E4M3, p,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" int fa_cache_read(const void* k_cache, const void* v_cache, const float* k_scale,
                             const float* v_scale, void* k_out, void* v_out,
                             const int32_t* block_table, int table_stride, const int32_t* start,
                             const int32_t* lens, int B, int Hk, int N, int d, int num_pages,
                             int page_size, int format, int dtype, void* stream) {
  if (!k_out || !v_out || k_out == v_out) return FA_ERR_INVALID_ARG;
  int st = check_common(B, Hk, N, d, 1.f, dtype);
  if (st != FA_OK) return st;
  CacheCopyParams p;
  std::memset(&p, 0, sizeof(p));
  p.clear = (format & FA_CACHE_CLEAR) != 0;
  format &= ~FA_CACHE_CLEAR;
  st = cache_view(k_cache, v_cache, k_scale, v_scale, block_table, table_stride, B, Hk, d,
                  num_pages, page_size, format, &p.c);
  if (st != FA_OK) return st;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || (start && !aligned(start, 4)) ||
      (lens && !aligned(lens, 4)))
    return FA_ERR_ALIGNMENT;
  p.k_out = static_cast<uint8_t*>(k_out);
  p.v_out = static_cast<uint8_t*>(v_out);
  p.start = start;
  p.lens = lens;
  p.B = B;
  p.N = N;
  DeviceInfo di;
  st = current_device_info(&di);
  if (st != FA_OK) return st;
  const cudaError_t e = launch_cache_read(d, dtype == FA_BF16, format == FA_CACHE_E4M3, p,
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" size_t fa_fwd_tree_workspace_size(int B, int Hq, int Hk, int T, int d) {
  if (check_tree(B, Hq, Hk, T, d, 1.f, FA_BF16) != FA_OK) return 0;
  // per CTA: what it continues (4 ints) and two partial results of a tile's
  // rows (fp32 O, reference and sum)
  const size_t slot = static_cast<size_t>(tree_rows(static_cast<long long>(Hq / Hk) * T)) * (d + 2) * sizeof(float);
  return round256(kTreeMaxCtas * 4 * sizeof(int)) + round256(kTreeMaxCtas * 2 * slot);
}

extern "C" int fa_fwd_tree(const void* q, const void* k_cache, const void* v_cache,
                           const float* k_scale, const float* v_scale, void* o, float* lse,
                           void* workspace, size_t workspace_bytes, const int32_t* block_table,
                           int table_stride, const int32_t* ctx_lens, const int32_t* draft_lens,
                           const uint8_t* tree_mask, int mask_per_batch, int B, int Hq, int Hk,
                           int T, int d, int num_pages, int page_size, float scale, int format,
                           int dtype, void* stream) {
  if (!q || !o || !lse || !ctx_lens) return FA_ERR_INVALID_ARG;
  int st = check_tree(B, Hq, Hk, T, d, scale, dtype);
  if (st != FA_OK) return st;
  TreeParams p;
  std::memset(&p, 0, sizeof(p));
  st = cache_view(k_cache, v_cache, k_scale, v_scale, block_table, table_stride, B, Hk, d,
                  num_pages, page_size, format, &p.c);
  if (st != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(ctx_lens, 4) ||
      (draft_lens && !aligned(draft_lens, 4)))
    return FA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < fa_fwd_tree_workspace_size(B, Hq, Hk, T, d))
    return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGNMENT;
  p.q = static_cast<const uint8_t*>(q);
  p.o = static_cast<uint8_t*>(o);
  p.lse = lse;
  p.ctx_lens = ctx_lens;
  p.draft_lens = draft_lens;
  p.mask = tree_mask;
  p.mask_stride = mask_per_batch ? static_cast<long long>(T) * T : 0;
  p.B = B;
  p.Hq = Hq;
  p.T = T;
  p.group = Hq / Hk;
  p.scale_log2 = scale * 1.4426950408889634f;
  const long long rows_all = static_cast<long long>(p.group) * T;
  const int rows = tree_rows(rows_all);
  p.row_tiles = static_cast<int>((rows_all + rows - 1) / rows);
  // (a CTA counts its piece of all key tiles in 32 bits)
  const long long most = static_cast<long long>(B) * Hk * p.row_tiles * ((p.c.room + 127) / 128);
  if (most >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  p.box_log2 = 7;
  while (page_size % (1 << p.box_log2) != 0) --p.box_log2;  // (page_size is a multiple of 16)
  p.box = 1 << p.box_log2;
  p.heads = static_cast<int*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                       round256(kTreeMaxCtas * 4 * sizeof(int)));
  p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  DeviceInfo di;
  st = current_device_info(&di);
  if (st != FA_OK) return st;
  p.grid = di.num_sms < kTreeMaxCtas ? di.num_sms : kTreeMaxCtas;
  if (most < p.grid) p.grid = static_cast<int>(most);
  CUtensorMap tmk, tmv;
  if (make_map_cache(&tmk, k_cache, p.c, d, p.box, format, dtype) != FA_OK ||
      make_map_cache(&tmv, v_cache, p.c, d, p.box, format, dtype) != FA_OK)
    return FA_ERR_CUDA;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return FA_ERR_CUDA;  // (< kMaxDevices, checked above)
  const cudaError_t e = launch_tree(d, dtype == FA_BF16, format == FA_CACHE_E4M3, rows, tmk, tmv, p,
                                    device, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
