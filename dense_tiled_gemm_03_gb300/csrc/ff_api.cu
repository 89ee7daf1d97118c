// ff_api.cu -- the C ABI of include/feed_forward.h: checks, the choice of a
// kernel, tensor maps and launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "feed_forward.h"
#include "ff_internal.h"
#include "ff_pad.h"

namespace gemm_tn_impl {
namespace {

using gemm_tn_dev::FfArgs;

constexpr int64_t kMost = int64_t{1} << 30;    // sizes below this: twice one stays in 32 bits
constexpr int64_t kMostPitch = int64_t{1} << 32;

bool size_ok(int64_t x) { return x >= 0 && x < kMost; }
bool pitch_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMostPitch; }

// The bytes of a [rows, cols] matrix.
struct Span {
  uintptr_t from, to;
};
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if (p == nullptr || rows == 0 || cols == 0) return {at, at};
  return {at, at + static_cast<uintptr_t>(((rows - 1) * ld + cols) * size)};
}
bool overlap(const Span& a, const Span& b) { return a.from < b.to && b.from < a.to; }

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

// The tensor-memory-access engine's demands on 16-bit operands.
bool addressable(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// A row-major [rows, cols] matrix moved in boxes of box_cols x box_rows; outside it reads as zero.
int encode_box(CUtensorMap* map, CUtensorMapDataType type, int size, const void* p, int64_t rows, int64_t cols, int64_t ld,
               int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  auto fn = encoder();
  if (fn == nullptr) return api_fail(GEMM_TN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(size)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = fn(map, type, 2, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS) return GEMM_TN_OK;
  char text[96];
  std::snprintf(text, sizeof(text), "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
  return api_fail(GEMM_TN_ERR_CUDA, text);
}
// The operands' boxes: 128-byte rows with the swizzle that the MMA's descriptors name.
int encode(CUtensorMap* map, CUtensorMapDataType type, int size, const void* p, int64_t rows, int64_t cols, int64_t ld,
           int box_rows) {
  return encode_box(map, type, size, p, rows, cols, ld, 128 / size, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}
int encode16(CUtensorMap* map, bool bf16, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p, rows, cols, ld,
                box_rows);
}
int encode8(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p, rows, cols, ld, box_rows);
}

// A [rows, cols] fp32 matrix of scales moved in boxes of box_cols x box_rows.
int encode_scales(CUtensorMap* map, const float* p, int64_t rows, int64_t cols, int64_t ld, int box_cols, int box_rows) {
  return encode_box(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p, rows, cols, ld, box_cols, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE);
}
// Whether it can be moved so: unit stride along its columns, and rows of whole 16 bytes.
bool scales_addressable(const float* p, int64_t rows, int64_t cols, int64_t s_i, int64_t s_j) {
  return aligned(p, 16) && (s_j == 1 || cols == 1) && (rows == 1 || (s_i % 4 == 0 && s_i >= cols));
}

// ---------------------------------------------------------------- the choice of a kernel

// Time of a tile of each shape, relative to the first's, where tiles abound
// (smaller tiles read more from L2 for their work). Measured, us: gated 8192 x
// 16384 x 4096 1061, 1512 and 1790; nt 16384 x 4096 x 8192 638, 771 and 900;
// e4m3 8192^3 374, 437 and 443, with a scale for every row of B 547, 580 and 560.
constexpr double kTileTime[4][kNumFfTiles] = {
    {1.0, 0.71, 0.84}, {1.0, 0.60, 0.70}, {1.0, 0.585, 0.59}, {1.0, 0.53, 0.51}};

constexpr int64_t kMostFew = 1024;   // rows of A up to which the skinny kernel (128 to a tile) is looked at

// Blocks of K that a product has at least to be cut, that a part has at least,
// and the most parts. 512 x 512 over 8192 tokens 29.4 us whole and 12.3 cut, over
// 4096 16.6 and 11.4; over 2048 cutting it would cost 0.7.
constexpr int64_t kLeastCut = 64, kLeastPart = 16, kMostParts = 8;

struct Choice {
  int rows = 0, splits = 0;   // skinny (rows != 0)
  int tile = 0;               // whole tiles
  int grid = 0;
};

// Clusters that run at once on the current device: of skinny CTAs by log2 of their number, and pairs of whole tiles.
struct Resident {
  bool known = false;
  int splits[4] = {}, pairs = 0;
};
Resident resident_on(int sms) {
  static std::mutex mutex;
  static Resident devices[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return Resident{};
  std::lock_guard<std::mutex> lock(mutex);
  Resident& r = devices[dev & 63];
  if (!r.known) {
    for (int i = 0; i < 4; ++i) r.splits[i] = ff_resident_clusters(1 << i, sms);
    r.pairs = ff_resident_pairs(sms);
    r.known = r.pairs > 0;
  }
  return r;
}

// GEMM_TN_FF_KERNEL (pair256, pair128, single128, skinny1, skinny2, skinny4 or
// skinny8) runs that kernel wherever it can run (measurements and tests).
struct Forced {
  int tile = -1, splits = 0;
};
Forced forced() {
  Forced f;
  const char* s = std::getenv("GEMM_TN_FF_KERNEL");
  if (s == nullptr) return f;
  const char* names[kNumFfTiles] = {"pair256", "pair128", "single128"};
  for (int t = 0; t < kNumFfTiles; ++t)
    if (std::strcmp(s, names[t]) == 0) f.tile = t;
  for (int splits = 1; splits <= 8; splits *= 2)
    if (std::strncmp(s, "skinny", 6) == 0 && std::atoi(s + 6) == splits) f.splits = splits;
  return f;
}

// The kernel for args' sizes, and args' tile counts. A status.
int choose(int kind, FfArgs& a, int sms, Choice* to) {
  const int64_t out_n = kind == kFfGated ? 2 : 1;   // columns of the product for one of C
  const Forced force = forced();
  const Resident at_once = resident_on(sms);
  if (kind != kFfNt && a.m <= kMostFew && force.tile < 0) {
    const int rows = a.m <= 16 ? 16 : a.m <= 32 ? 32 : a.m <= 64 ? 64 : 128;
    const int64_t m_tiles = (a.m + rows - 1) / rows, n_tiles = (static_cast<int64_t>(a.n) * out_n + 127) / 128;
    const int64_t tiles = m_tiles * n_tiles;
    // K is cut while all clusters run at once and every CTA has a few blocks of K
    int splits = 1;
    for (int i = 1; i < 4; ++i)
      if (tiles <= at_once.splits[i] && a.num_k_blocks >= 4 << i) splits = 1 << i;
    if (force.splits > 0 && a.num_k_blocks >= force.splits) splits = force.splits;
    if (ff_skinny_has(kind, rows, splits) && (force.splits > 0 || ff_skinny_pays(kind, rows, splits, a.num_k_blocks))) {
      if (tiles * splits > INT32_MAX) return api_fail(GEMM_TN_ERR_INVALID_VALUE, "too many output tiles");
      to->rows = rows;
      to->splits = splits == 1 && tiles > sms ? 0 : splits;   // 0: two CTAs to an SM
      to->grid = static_cast<int>(tiles * splits);
      a.num_m_tiles = static_cast<int32_t>(m_tiles);
      a.num_n_tiles = static_cast<int32_t>(n_tiles);
      a.num_tiles = static_cast<int32_t>(tiles);
      return GEMM_TN_OK;
    }
  }
  const int pairs = at_once.pairs;
  if (pairs <= 0) return api_fail(GEMM_TN_ERR_CUDA, "kernel cannot be resident on this device (occupancy query)");
  // the shape with the least time: waves times the time of one of its tiles
  const double* tile_time = kTileTime[kind];
  double best = 0;
  for (int t = 0; t < kNumFfTiles; ++t) {
    const FfTileInfo& f = kFfTiles[t];
    const int64_t mt = (a.m + f.tile_m - 1) / f.tile_m;
    const int64_t nt = (static_cast<int64_t>(a.n) * out_n + f.block_n - 1) / f.block_n;
    if (mt * nt > INT32_MAX || (force.tile >= 0 && t != force.tile)) continue;
    const int64_t slots = f.cta_group == 2 ? pairs : sms;
    const double cost = static_cast<double>((mt * nt + slots - 1) / slots) * tile_time[t];
    if (to->grid == 0 || cost < best) {
      best = cost;
      to->tile = t;
      to->grid = static_cast<int>(std::min(mt * nt, slots)) * f.cta_group;
      a.num_m_tiles = static_cast<int32_t>(mt);
      a.num_n_tiles = static_cast<int32_t>(nt);
      a.num_tiles = static_cast<int32_t>(mt * nt);
      a.group_m = static_cast<int32_t>(std::min<int64_t>(mt, f.cta_group == 2 ? 8 : 16));
    }
  }
  if (to->grid == 0) return api_fail(GEMM_TN_ERR_INVALID_VALUE, "too many output tiles");
  a.splits = 1;
  if (kind == kFfNt) {
    // Few tiles and a long K (a small weight's gradient over many tokens): K is
    // cut into parts that run at once, joined by a second kernel.
    const int64_t slots = kFfTiles[to->tile].cta_group == 2 ? pairs : sms;
    const int64_t parts = std::min<int64_t>({slots / a.num_tiles, a.num_k_blocks / kLeastPart, kMostParts});
    if (parts > 1 && a.num_k_blocks >= kLeastCut) {
      a.splits = static_cast<int32_t>(parts);
      a.num_tiles *= a.splits;
      to->grid *= a.splits;
    }
  }
  return GEMM_TN_OK;
}

// Copies of operands that the engine cannot address, where they need one; freed in stream order.
struct Padded {
  void* workspace = nullptr;
  cudaStream_t stream;
  explicit Padded(cudaStream_t s) : stream(s) {}
  int copy(const void** a, int64_t* lda, int64_t a_rows, int64_t a_cols, const void** b, int64_t* ldb, int64_t b_rows,
           int64_t b_cols) {
    // (one row's pitch is never stepped over)
    if (a_rows == 1) *lda = (a_cols + 7) / 8 * 8;
    if (b_rows == 1) *ldb = (b_cols + 7) / 8 * 8;
    const bool pad_a = !addressable(*a, *lda), pad_b = !addressable(*b, *ldb);
    if (!pad_a && !pad_b) return GEMM_TN_OK;
    const int64_t la = gemm_tn_dev::ff::pad_pitch(a_cols), lb = gemm_tn_dev::ff::pad_pitch(b_cols);
    const size_t a_bytes = pad_a ? static_cast<size_t>((a_rows * la * 2 + 255) / 256 * 256) : 0;
    const size_t b_bytes = pad_b ? static_cast<size_t>(b_rows * lb * 2) : 0;
    cudaError_t e = api_workspace(a_bytes + b_bytes, stream, &workspace);
    if (e != cudaSuccess) {
      workspace = nullptr;
      return api_fail_cuda(e, "workspace");
    }
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const RepackRequest req[2] = {{*a, *lda, w, la, pad_a ? a_rows : 0, a_cols},
                                  {*b, *ldb, w + a_bytes, lb, pad_b ? b_rows : 0, b_cols}};
    e = api_counted(launch_pad_rows(req, stream));
    if (e != cudaSuccess) return api_fail_cuda(e, "padding launch");
    if (pad_a) {
      *a = w;
      *lda = la;
    }
    if (pad_b) {
      *b = w + a_bytes;
      *ldb = lb;
    }
    return GEMM_TN_OK;
  }
  cudaError_t free() {
    void* w = workspace;
    workspace = nullptr;
    return w != nullptr ? cudaFreeAsync(w, stream) : cudaSuccess;
  }
  ~Padded() { free(); }
};

int finish(cudaError_t e) { return e == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(e, "kernel launch"); }

int zero(void* c, int64_t ldc, int64_t rows, int64_t cols, int64_t size, cudaStream_t stream) {
  const cudaError_t e = cudaMemset2DAsync(c, static_cast<size_t>(ldc * size), 0, static_cast<size_t>(cols * size),
                                          static_cast<size_t>(rows), stream);
  return e == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(e, "cudaMemset2DAsync");
}

bool gate_activation(int a) { return a == GEMM_TN_ACT_RELU || a == GEMM_TN_ACT_GELU || a == GEMM_TN_ACT_SILU; }

int refuse(const char* what) { return api_fail(GEMM_TN_ERR_INVALID_VALUE, what); }

}  // namespace
}  // namespace gemm_tn_impl

using namespace gemm_tn_impl;

int gemm_tn_gated(int dtype, int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const void* b, int64_t ldb,
                  void* h, int64_t ldh, void* pre, int64_t ldp, int activation, int* d_status, gemm_tn_stream_t stream) {
  api_begin();
  if (dtype != GEMM_TN_F16 && dtype != GEMM_TN_BF16) return api_fail(GEMM_TN_ERR_UNSUPPORTED_DTYPE, "dtype");
  if (!size_ok(m) || !size_ok(n) || !size_ok(k)) return refuse("sizes must be in [0, 2^30)");
  if (!gate_activation(activation)) return refuse("activation must be relu, gelu or silu");
  if (m == 0 || n == 0) return GEMM_TN_OK;
  if (h == nullptr) return refuse("H is NULL");
  if (!pitch_ok(ldh, n)) return refuse("ldh < n");
  if (pre != nullptr && !pitch_ok(ldp, 2 * n)) return refuse("ldp < 2n");
  if (!aligned(h, 2) || !aligned(pre, 2)) return api_fail(GEMM_TN_ERR_MISALIGNED, "H or pre is not 2-byte aligned");
  const Span sh = span(h, m, n, ldh, 2), sp = span(pre, m, 2 * n, ldp, 2);
  if (overlap(sh, sp)) return refuse("H overlaps pre");
  if (k > 0) {
    if (a == nullptr || b == nullptr) return refuse("A or B is NULL");
    if (!pitch_ok(lda, k) || !pitch_ok(ldb, k)) return refuse("lda or ldb < k");
    if (!aligned(a, 2) || !aligned(b, 2)) return api_fail(GEMM_TN_ERR_MISALIGNED, "A or B is not 2-byte aligned");
    const Span sa = span(a, m, k, lda, 2), sb = span(b, 2 * n, k, ldb, 2);
    if (overlap(sh, sa) || overlap(sh, sb) || overlap(sp, sa) || overlap(sp, sb)) return refuse("H or pre overlaps A or B");
  }
  int sms = 0;
  int st = api_device(&sms);
  if (st != GEMM_TN_OK) return st;
  if (k == 0) {   // act(0) * 0
    st = zero(h, ldh, m, n, 2, stream);
    return st == GEMM_TN_OK && pre != nullptr ? zero(pre, ldp, m, 2 * n, 2, stream) : st;
  }
  const bool bf16 = dtype == GEMM_TN_BF16;
  alignas(64) FfArgs args{};
  args.c = h;
  args.ldc = ldh;
  args.pre = pre;
  args.ldp = ldp;
  args.m = static_cast<int32_t>(m);
  args.n = static_cast<int32_t>(n);
  args.num_k_blocks = static_cast<int32_t>((k + 63) / 64);
  args.activation = activation;
  args.out_kind = bf16 ? GEMM_TN_ELEM_BF16 : GEMM_TN_ELEM_F16;
  args.status = d_status;
  args.timeout_ns = api_watchdog_ns();
  args.drop_load_kb = api_drop_load();
  Choice pick;
  st = choose(kFfGated, args, sms, &pick);
  if (st != GEMM_TN_OK) return st;
  Padded padded(stream);
  st = padded.copy(&a, &lda, m, k, &b, &ldb, 2 * n, k);
  if (st != GEMM_TN_OK) return st;
  st = encode16(&args.tmap_a, bf16, a, m, k, lda, pick.rows ? pick.rows : 128);
  if (st == GEMM_TN_OK) st = encode16(&args.tmap_b, bf16, b, 2 * n, k, ldb, pick.rows ? 64 : kFfTiles[pick.tile].block_n / 2);
  if (st != GEMM_TN_OK) return st;
  args.alone = padded.workspace != nullptr;
  cudaError_t e = api_counted(pick.rows ? launch_ff_skinny(kFfGated, bf16, pick.rows, pick.splits, args, pick.grid, stream)
                                        : launch_ff_gated(pick.tile, bf16, args, pick.grid, stream));
  const cudaError_t freed = padded.free();
  return finish(e == cudaSuccess ? freed : e);
}

int gated_grad(int dtype, int64_t m, int64_t n, const void* grad, int64_t ldg, const void* pre, int64_t ldp, void* out,
               int64_t ldo, int activation, gemm_tn_stream_t stream) {
  api_begin();
  if (dtype != GEMM_TN_F16 && dtype != GEMM_TN_BF16) return api_fail(GEMM_TN_ERR_UNSUPPORTED_DTYPE, "dtype");
  if (!size_ok(m) || !size_ok(n)) return refuse("sizes must be in [0, 2^30)");
  if (!gate_activation(activation)) return refuse("activation must be relu, gelu or silu");
  if (m == 0 || n == 0) return GEMM_TN_OK;
  if (grad == nullptr || pre == nullptr || out == nullptr) return refuse("grad, pre or out is NULL");
  if (!pitch_ok(ldg, n) || !pitch_ok(ldp, 2 * n) || !pitch_ok(ldo, 2 * n)) return refuse("ldg < n, or ldp or ldo < 2n");
  if (!aligned(grad, 2) || !aligned(pre, 2) || !aligned(out, 2))
    return api_fail(GEMM_TN_ERR_MISALIGNED, "grad, pre or out is not 2-byte aligned");
  const Span so = span(out, m, 2 * n, ldo, 2);
  if (overlap(so, span(grad, m, n, ldg, 2))) return refuse("out overlaps grad");
  if (!(out == pre && ldo == ldp) && overlap(so, span(pre, m, 2 * n, ldp, 2)))
    return refuse("out overlaps pre without being pre");
  int sms = 0;
  const int st = api_device(&sms);
  if (st != GEMM_TN_OK) return st;
  const gemm_tn_dev::GatedGradArgs args{grad, pre, out, ldg, ldp, ldo, m, n, activation};
  return finish(api_counted(launch_gated_grad(dtype == GEMM_TN_BF16, args, sms, stream)));
}

int gemm_nt(int dtype, int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const void* b, int64_t ldb, void* c,
            int64_t ldc, int out_dtype, int accumulate, int* d_status, gemm_tn_stream_t stream) {
  api_begin();
  if (dtype != GEMM_TN_F16 && dtype != GEMM_TN_BF16) return api_fail(GEMM_TN_ERR_UNSUPPORTED_DTYPE, "dtype");
  if (out_dtype != GEMM_TN_OUT_INPUT && out_dtype != GEMM_TN_OUT_F32)
    return api_fail(GEMM_TN_ERR_UNSUPPORTED_DTYPE, "out_dtype must be the input's or fp32");
  if (accumulate != 0 && out_dtype != GEMM_TN_OUT_F32) return refuse("accumulate needs an fp32 C");
  if (!size_ok(m) || !size_ok(n) || !size_ok(k)) return refuse("sizes must be in [0, 2^30)");
  if (m == 0 || n == 0) return GEMM_TN_OK;
  const int64_t size = out_dtype == GEMM_TN_OUT_F32 ? 4 : 2;
  if (c == nullptr) return refuse("C is NULL");
  if (!pitch_ok(ldc, n)) return refuse("ldc < n");
  if (!aligned(c, size)) return api_fail(GEMM_TN_ERR_MISALIGNED, "C is not aligned to its element");
  if (k > 0) {
    if (a == nullptr || b == nullptr) return refuse("A or B is NULL");
    if (!pitch_ok(lda, m) || !pitch_ok(ldb, n)) return refuse("lda < m or ldb < n");
    if (!aligned(a, 2) || !aligned(b, 2)) return api_fail(GEMM_TN_ERR_MISALIGNED, "A or B is not 2-byte aligned");
    const Span sc = span(c, m, n, ldc, size);
    if (overlap(sc, span(a, k, m, lda, 2)) || overlap(sc, span(b, k, n, ldb, 2))) return refuse("C overlaps A or B");
  }
  int sms = 0;
  int st = api_device(&sms);
  if (st != GEMM_TN_OK) return st;
  if (k == 0) return accumulate != 0 ? GEMM_TN_OK : zero(c, ldc, m, n, size, stream);
  const bool bf16 = dtype == GEMM_TN_BF16;
  alignas(64) FfArgs args{};
  args.c = c;
  args.ldc = ldc;
  args.m = static_cast<int32_t>(m);
  args.n = static_cast<int32_t>(n);
  args.num_k_blocks = static_cast<int32_t>((k + 63) / 64);
  args.out_kind = size == 4 ? GEMM_TN_ELEM_F32 : bf16 ? GEMM_TN_ELEM_BF16 : GEMM_TN_ELEM_F16;
  args.accumulate = accumulate != 0;
  args.status = d_status;
  args.timeout_ns = api_watchdog_ns();
  args.drop_load_kb = api_drop_load();
  Choice pick;
  st = choose(kFfNt, args, sms, &pick);
  if (st != GEMM_TN_OK) return st;
  Padded padded(stream);
  st = padded.copy(&a, &lda, k, m, &b, &ldb, k, n);
  if (st == GEMM_TN_OK) st = encode16(&args.tmap_a, bf16, a, k, m, lda, 64);
  if (st == GEMM_TN_OK) st = encode16(&args.tmap_b, bf16, b, k, n, ldb, 64);
  if (st != GEMM_TN_OK) return st;
  // (with parts to join it is followed by its own join, which no workspace's end precedes)
  args.alone = padded.workspace != nullptr && args.splits == 1;
  Padded parts(stream);   // (workspace alone)
  JoinRequest join{};
  if (args.splits > 1) {
    const int64_t pitch = (n + 3) / 4 * 4;
    const cudaError_t e = api_workspace(static_cast<size_t>(args.splits * m * pitch * 4), stream, &parts.workspace);
    if (e != cudaSuccess) {
      parts.workspace = nullptr;
      return api_fail_cuda(e, "workspace");
    }
    join = {static_cast<const float*>(parts.workspace), pitch, m * pitch, args.splits, c, ldc, m, n, args.out_kind, args.accumulate};
    args.c = parts.workspace;
    args.ldc = pitch;
    args.part_stride = join.part_stride;
    args.out_kind = GEMM_TN_ELEM_F32;
    args.accumulate = 0;
  }
  cudaError_t e = api_counted(launch_ff_nt(pick.tile, bf16, args, pick.grid, stream));
  if (e == cudaSuccess && args.splits > 1) e = api_counted(launch_join_parts(join, sms, stream));
  const cudaError_t freed = padded.free(), freed_parts = parts.free();
  return finish(e != cudaSuccess ? e : freed != cudaSuccess ? freed : freed_parts);
}

int quantize_e4m3(int src_type, int64_t rows, int64_t cols, const void* x, int64_t ldx, void* q, int64_t ldq,
                  float* scale, int64_t s_line, int64_t s_blk, int block_lines, int transpose, gemm_tn_stream_t stream) {
  api_begin();
  if (src_type < GEMM_TN_ELEM_F16 || src_type > GEMM_TN_ELEM_F32)
    return api_fail(GEMM_TN_ERR_UNSUPPORTED_DTYPE, "src_type must be fp16, bf16 or fp32");
  if (!size_ok(rows) || !size_ok(cols)) return refuse("sizes must be in [0, 2^30)");
  if (block_lines != 1 && block_lines != 128) return refuse("block_lines must be 1 or 128");
  if (rows == 0 || cols == 0) return GEMM_TN_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return refuse("x, q or scale is NULL");
  const int64_t lines = transpose ? cols : rows, along = transpose ? rows : cols;
  if (!pitch_ok(ldx, cols) || !pitch_ok(ldq, along)) return refuse("ldx < cols, or ldq shorter than a line");
  const int64_t size = src_type == GEMM_TN_ELEM_F32 ? 4 : 2;
  if (!aligned(x, size) || !aligned(scale, 4)) return api_fail(GEMM_TN_ERR_MISALIGNED, "x or scale is not aligned to its element");
  const int64_t s_lines = (lines + block_lines - 1) / block_lines, s_blocks = (along + 127) / 128;
  // the scales of different blocks lie at different places: one stride spans the other's extent
  if (s_line < 1 || s_blk < 1 || s_line > kMostPitch || s_blk > kMostPitch ||
      !(s_blocks == 1 || s_lines == 1 || s_line >= (s_blocks - 1) * s_blk + 1 || s_blk >= (s_lines - 1) * s_line + 1))
    return refuse("s_line and s_blk must be positive and keep the scales apart");
  const Span sx = span(x, rows, cols, ldx, size), sq = span(q, lines, along, ldq, 1);
  const Span ss = span(scale, 1, (s_lines - 1) * s_line + (s_blocks - 1) * s_blk + 1, 0, 4);
  if (overlap(sx, sq) || overlap(sx, ss) || overlap(sq, ss)) return refuse("x, q and scale overlap");
  if (((rows + 127) / 128) * ((cols + 127) / 128) > INT32_MAX) return refuse("too many blocks");
  int sms = 0;
  const int st = api_device(&sms);
  if (st != GEMM_TN_OK) return st;
  const gemm_tn_dev::QuantizeArgs args{x, ldx, static_cast<uint8_t*>(q), ldq, scale, s_line, s_blk, rows, cols};
  return finish(api_counted(launch_quantize(src_type, block_lines, transpose != 0, args, stream)));
}

int gemm_tn_e4m3(int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const float* a_scale, int64_t as_row,
                 int64_t as_blk, const void* b, int64_t ldb, const float* b_scale, int64_t bs_row, int64_t bs_blk,
                 int b_block_rows, void* c, int64_t ldc, int out_type, int accumulate, int* d_status,
                 gemm_tn_stream_t stream) {
  api_begin();
  if (out_type < GEMM_TN_ELEM_F16 || out_type > GEMM_TN_ELEM_F32)
    return api_fail(GEMM_TN_ERR_UNSUPPORTED_DTYPE, "out_type must be fp16, bf16 or fp32");
  if (accumulate != 0 && out_type != GEMM_TN_ELEM_F32) return refuse("accumulate needs an fp32 C");
  if (!size_ok(m) || !size_ok(n) || !size_ok(k)) return refuse("sizes must be in [0, 2^30)");
  if (b_block_rows != 1 && b_block_rows != 128) return refuse("b_block_rows must be 1 or 128");
  if (m == 0 || n == 0) return GEMM_TN_OK;
  const int64_t size = out_type == GEMM_TN_ELEM_F32 ? 4 : 2;
  if (c == nullptr) return refuse("C is NULL");
  if (!pitch_ok(ldc, n)) return refuse("ldc < n");
  if (!aligned(c, size)) return api_fail(GEMM_TN_ERR_MISALIGNED, "C is not aligned to its element");
  const int64_t blocks = (k + 127) / 128;
  if (k > 0) {
    if (a == nullptr || b == nullptr || a_scale == nullptr || b_scale == nullptr)
      return refuse("A, B or their scales are NULL");
    if (!pitch_ok(lda, k) || !pitch_ok(ldb, k)) return refuse("lda or ldb < k");
    if (!aligned(a, 16) || !aligned(b, 16) || lda % 16 != 0 || ldb % 16 != 0)
      return api_fail(GEMM_TN_ERR_MISALIGNED, "e4m3 operands need 16-byte-aligned bases and pitches");
    if (!aligned(a_scale, 4) || !aligned(b_scale, 4)) return api_fail(GEMM_TN_ERR_MISALIGNED, "a scale is not 4-byte aligned");
    for (int64_t s : {as_row, as_blk, bs_row, bs_blk})
      if (s < 0 || s > kMostPitch) return refuse("a scale's stride is negative or too large");
    const Span sc = span(c, m, n, ldc, size);
    const int64_t b_lines = (n + b_block_rows - 1) / b_block_rows;
    if (overlap(sc, span(a, m, k, lda, 1)) || overlap(sc, span(b, n, k, ldb, 1)) ||
        overlap(sc, span(a_scale, 1, (m - 1) * as_row + (blocks - 1) * as_blk + 1, 0, 4)) ||
        overlap(sc, span(b_scale, 1, (b_lines - 1) * bs_row + (blocks - 1) * bs_blk + 1, 0, 4)))
      return refuse("C overlaps A, B or their scales");
  }
  int sms = 0;
  int st = api_device(&sms);
  if (st != GEMM_TN_OK) return st;
  if (k == 0) return accumulate != 0 ? GEMM_TN_OK : zero(c, ldc, m, n, size, stream);
  alignas(64) FfArgs args{};
  args.c = c;
  args.ldc = ldc;
  args.a_scale = a_scale;
  args.b_scale = b_scale;
  args.as_row = as_row;
  args.as_blk = as_blk;
  args.bs_row = bs_row;
  args.bs_blk = bs_blk;
  args.b_block_rows = b_block_rows;
  args.m = static_cast<int32_t>(m);
  args.n = static_cast<int32_t>(n);
  args.num_k_blocks = static_cast<int32_t>(blocks);
  args.out_kind = out_type;
  args.accumulate = accumulate != 0;
  args.status = d_status;
  args.timeout_ns = api_watchdog_ns();
  args.drop_load_kb = api_drop_load();
  Choice pick;
  st = choose(b_block_rows == 1 ? kFfE4m3Rows : kFfE4m3, args, sms, &pick);
  if (st != GEMM_TN_OK) return st;
  const FfTileInfo& tile = kFfTiles[pick.tile];
  st = encode8(&args.tmap_a, a, m, k, lda, pick.rows ? pick.rows : 128);
  if (st == GEMM_TN_OK) st = encode8(&args.tmap_b, b, n, k, ldb, pick.rows ? 128 : tile.block_n / tile.cta_group);
  if (st != GEMM_TN_OK) return st;
  if (pick.rows)
    return finish(api_counted(launch_ff_skinny(kFfE4m3, false, pick.rows, pick.splits, args, pick.grid, stream)));

  // Whole tiles take the scales through the TMA too: A's as [block][row], B's
  // likewise or, of 128 rows, as [row / 128][block]. Others are copied first
  // (a 128th of the operands' bytes).
  const int64_t b_lines = (n + b_block_rows - 1) / b_block_rows;
  struct Scales {
    const float* p;
    int64_t rows, cols, s_i, s_j;
  };
  Scales scales[2] = {{a_scale, blocks, m, as_blk, as_row},
                      b_block_rows == 1 ? Scales{b_scale, blocks, n, bs_blk, bs_row}
                                        : Scales{b_scale, b_lines, blocks, bs_row, bs_blk}};
  PackRequest pack[2] = {};
  size_t bytes[2] = {};
  for (int x = 0; x < 2; ++x) {
    const Scales& s = scales[x];
    if (scales_addressable(s.p, s.rows, s.cols, s.s_i, s.s_j)) continue;
    const int64_t pitch = (s.cols + 3) / 4 * 4;
    pack[x] = {s.p, nullptr, s.rows, s.cols, s.s_i, s.s_j, pitch};
    bytes[x] = static_cast<size_t>((s.rows * pitch * 4 + 255) / 256 * 256);
  }
  Padded copies(stream);
  if (bytes[0] + bytes[1] > 0) {
    cudaError_t e = api_workspace(bytes[0] + bytes[1], stream, &copies.workspace);
    if (e != cudaSuccess) {
      copies.workspace = nullptr;
      return api_fail_cuda(e, "workspace");
    }
    uint8_t* to = static_cast<uint8_t*>(copies.workspace);
    for (int x = 0; x < 2; ++x) {
      if (bytes[x] == 0) continue;
      pack[x].dst = reinterpret_cast<float*>(to);
      to += bytes[x];
      scales[x].p = pack[x].dst;
      scales[x].s_i = pack[x].pitch;
    }
    e = api_counted(launch_pack_scales(pack, stream));
    if (e != cudaSuccess) return api_fail_cuda(e, "scales launch");
  }
  auto pitch_of = [](const Scales& s) { return s.rows > 1 ? s.s_i : (s.cols + 3) / 4 * 4; };
  st = encode_scales(&args.tmap_as, scales[0].p, blocks, m, pitch_of(scales[0]), 128, 1);
  if (st == GEMM_TN_OK)
    st = b_block_rows == 1
             ? encode_scales(&args.tmap_bs, scales[1].p, blocks, n, pitch_of(scales[1]), tile.block_n, 1)
             : encode_scales(&args.tmap_bs, scales[1].p, b_lines, blocks, pitch_of(scales[1]), 4, tile.block_n / 128);
  if (st != GEMM_TN_OK) return st;
  args.alone = copies.workspace != nullptr;
  const cudaError_t e = api_counted(launch_ff_e4m3(pick.tile, b_block_rows == 1, args, pick.grid, stream));
  const cudaError_t freed = copies.free();
  return finish(e == cudaSuccess ? freed : e);
}
