// kv_cache_api.cu -- the C ABI declared in include/kv_cache.h: argument checks,
// tensor maps over the page pools, workspaces and the launches of
// sm103_tree_attn.cu, sm103_cache_weigh.cu and kv_cache_ops.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kv_cache.h"
#include "kv_cache_internal.h"

namespace gemm_tn_impl {

namespace {

constexpr int64_t kMax31 = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxStride = int64_t{1} << 39;   // elements: tensor-map strides stay under 2^40 bytes

int invalid(const char* what) { return api_fail(GEMM_TN_ERR_INVALID_VALUE, what); }

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_common(int dtype, int64_t batch, const kv_cache* c) {
  if (dtype != GEMM_TN_F16 && dtype != GEMM_TN_BF16) return api_fail(GEMM_TN_ERR_UNSUPPORTED_DTYPE, "dtype");
  if (c == nullptr) return invalid("cache is NULL");
  if (batch < 0 || batch > kMax31) return invalid("batch must be in [0, 2^31)");
  if (c->head_dim != 64 && c->head_dim != 128) return invalid("head_dim must be 64 or 128");
  if (c->kv_heads < 1 || c->kv_heads > kMax31) return invalid("kv_heads must be in [1, 2^31)");
  const int64_t ps = c->page_size;
  if (!(ps == 8 || ps == 16 || ps == 32 || ps == 64 || (ps >= 128 && ps % 128 == 0 && ps <= (1 << 20))))
    return invalid("page_size must be 8, 16, 32, 64 or a multiple of 128 up to 2^20");
  if (c->num_pages < 1 || c->num_pages > kMax31 - 1) return invalid("num_pages must be in [1, 2^31 - 1)");
  if (c->max_pages < 1 || c->max_pages > (kMax31 - 256) / ps) return invalid("max_pages * page_size must be in [1, 2^31 - 256]");
  if (batch > 1 && c->table_stride < c->max_pages) return invalid("table_stride < max_pages");
  if (batch > 0 && c->kv_heads > kMax31 / batch) return invalid("batch * kv_heads must be below 2^31");
  for (const int64_t s : {c->page_stride, c->slot_stride, c->head_stride})
    if (s < 0 || s >= kMaxStride || s % 8 != 0) return invalid("pool strides must be multiples of 8 elements in [0, 2^39)");
  if ((c->num_pages > 1 && c->page_stride < c->head_dim) || c->slot_stride < c->head_dim ||
      (c->kv_heads > 1 && c->head_stride < c->head_dim))
    return invalid("pool strides must be at least head_dim");
  if (batch == 0) return GEMM_TN_OK;
  if (c->k == nullptr || c->v == nullptr || c->page_table == nullptr || c->lens == nullptr)
    return invalid("the cache's k, v, page_table or lens is NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return api_fail(GEMM_TN_ERR_MISALIGNED, "pool not 16-byte aligned");
  for (const void* p : {static_cast<const void*>(c->page_table), static_cast<const void*>(c->lens),
                        static_cast<const void*>(c->weight), static_cast<const void*>(c->pos),
                        static_cast<const void*>(c->seen)})
    if (!aligned(p, 4)) return api_fail(GEMM_TN_ERR_MISALIGNED, "cache array not 4-byte aligned");
  return GEMM_TN_OK;
}

int check_rows(const kv_rows* r, int64_t batch, int64_t tokens, int64_t heads, int64_t dim) {
  if (r == nullptr || r->data == nullptr) return invalid("q, k_new or v_new is NULL");
  if (!aligned(r->data, 16)) return api_fail(GEMM_TN_ERR_MISALIGNED, "q, k_new or v_new not 16-byte aligned");
  const int64_t strides[3] = {r->batch_stride, r->token_stride, r->head_stride}, sizes[3] = {batch, tokens, heads};
  for (int i = 0; i < 3; ++i)
    if (sizes[i] > 1 && (strides[i] < dim || strides[i] >= kMaxStride || strides[i] % 8 != 0))
      return invalid("strides of q, k_new and v_new must be multiples of 8 elements, at least head_dim and below 2^39");
  return GEMM_TN_OK;
}

struct Range {
  uintptr_t begin, end;
};
bool overlap(const Range& a, const Range& b) {
  return a.begin < a.end && b.begin < b.end && a.begin < b.end && b.begin < a.end;
}
Range pool_range(const void* p, const kv_cache* c) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + 2 * static_cast<uintptr_t>((c->num_pages - 1) * c->page_stride + (c->page_size - 1) * c->slot_stride +
                                             (c->kv_heads - 1) * c->head_stride + c->head_dim)};
}
Range rows_range(const kv_rows* r, int64_t batch, int64_t tokens, int64_t heads, int64_t dim) {   // empty for NULL
  const uintptr_t b = r != nullptr ? reinterpret_cast<uintptr_t>(r->data) : 0;
  if (b == 0) return {0, 0};
  return {b, b + 2 * static_cast<uintptr_t>((batch - 1) * (batch > 1 ? r->batch_stride : 0) + (tokens - 1) * (tokens > 1 ? r->token_stride : 0) +
                                             (heads - 1) * (heads > 1 ? r->head_stride : 0) + dim)};
}

Range words_range(const void* p, int64_t count) {   // of 4 bytes; empty for NULL
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, p != nullptr ? b + 4 * static_cast<uintptr_t>(count) : b};
}
Range table_range(const kv_cache* c, int64_t batch) {
  return words_range(c->page_table, (batch - 1) * (batch > 1 ? c->table_stride : 0) + c->max_pages);
}

// The cache's arrays, also those that the call at hand does not use.
struct CacheRanges {
  Range k, v, table, lens, weight, pos, seen;
};
CacheRanges cache_ranges(const kv_cache* c, int64_t batch) {
  const int64_t slots = batch * c->kv_heads * c->max_pages * c->page_size;
  return {pool_range(c->k, c),         pool_range(c->v, c),           table_range(c, batch),     words_range(c->lens, batch),
          words_range(c->weight, slots), words_range(c->pos, slots), words_range(c->seen, batch)};
}

// An array that a call writes, and the input that it replaces and may be, exactly.
struct Output {
  Range at, own;
};
using Outputs = std::initializer_list<Output>;
using Inputs = std::initializer_list<Range>;   // but for those that outputs replace
// Whether an array lies in one of these, in what they replace, or in an input.
bool meets(const Range& a, Outputs outs, Inputs ins, const Output* but = nullptr) {
  for (const Output& x : outs)
    if (&x != but && (overlap(a, x.at) || overlap(a, x.own))) return true;
  return std::any_of(ins.begin(), ins.end(), [&](const Range& in) { return overlap(a, in); });
}
// Whether an output lies in another array, which other blocks may still read or
// write when it is written.
bool clash(Outputs outs, Inputs ins) {
  return std::any_of(outs.begin(), outs.end(), [&](const Output& o) {
    return meets(o.at, outs, ins, &o) || (o.at.begin != o.own.begin && overlap(o.at, o.own));
  });
}

// Whether a row of the K pool and a row of the V pool share elements; the pools'
// address ranges may interleave (K and V of a page, or of a slot, side by side). The
// rows are `apart` elements plus multiples of the three strides apart: one stride
// after the other, the longest first, only the two multiples next to what is left can
// bring it within the shorter strides' reach. Where a stride is shorter than that
// reach (rows that share elements within one pool) any touching of the ranges counts.
bool pools_overlap(const kv_cache* c) {
  if (!overlap(pool_range(c->k, c), pool_range(c->v, c))) return false;
  struct Dim {
    int64_t stride, count;
  };
  Dim dims[3] = {{c->page_stride, c->num_pages}, {c->slot_stride, c->page_size}, {c->head_stride, c->kv_heads}};
  std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return (a.count > 1 ? a.stride : 0) > (b.count > 1 ? b.stride : 0); });
  int64_t reach = c->head_dim;   // elements from the first to past the last of the dims after the one at hand
  for (int i = 2; i >= 0; --i) {
    if (dims[i].count == 1) continue;
    if (dims[i].stride < reach) return true;
    reach += dims[i].stride * (dims[i].count - 1);
  }
  const int64_t bytes = static_cast<int64_t>(reinterpret_cast<uintptr_t>(c->v) - reinterpret_cast<uintptr_t>(c->k));
  int64_t left[8] = {bytes / 2};   // the pools start on 16-byte boundaries
  int n = 1;
  for (const Dim& d : dims) {
    if (d.count == 1) continue;
    int64_t next[8];
    int m = 0;
    for (int i = 0; i < n; ++i) {
      const int64_t down = left[i] / d.stride - (left[i] % d.stride < 0 ? 1 : 0);
      for (int64_t q = down; q <= down + 1; ++q)
        if (q > -d.count && q < d.count) next[m++] = left[i] - q * d.stride;
    }
    n = m;
    std::copy(next, next + m, left);
  }
  return std::any_of(left, left + n, [&](int64_t x) { return x > -c->head_dim && x < c->head_dim; });
}

// {dim, kv heads, page_size, num_pages}; moved in boxes of 64 elements of one
// head by min(page_size, 128) rows of one page. Page num_pages reads as zeros.
int encode_pool(CUtensorMap* map, bool bf16, const void* pool, const kv_cache* c) {
  const int64_t dims[4] = {c->head_dim, c->kv_heads, c->page_size, c->num_pages};
  const int64_t strides[3] = {c->kv_heads > 1 ? c->head_stride : c->head_dim, c->slot_stride,
                              c->num_pages > 1 ? c->page_stride : c->head_dim};
  const int box[4] = {64, 1, static_cast<int>(std::min<int64_t>(c->page_size, 128)), 1};
  return api_encode_4d(map, bf16, pool, dims, strides, box);
}

// {dim, heads, tokens, batch}
int encode_rows(CUtensorMap* map, bool bf16, const kv_rows* r, int64_t batch, int64_t tokens, int64_t heads, int64_t dim,
                int box_heads, int box_tokens) {
  const int64_t dims[4] = {dim, heads, tokens, batch};
  const int64_t strides[3] = {heads > 1 ? r->head_stride : dim, tokens > 1 ? r->token_stride : dim,
                              batch > 1 ? r->batch_stride : dim};
  const int box[4] = {64, box_heads, box_tokens, 1};
  return api_encode_4d(map, bf16, r->data, dims, strides, box);
}

// log2(e) times the softmax scale
float scale_log2(float softmax_scale, int64_t dim) {
  const double scale = softmax_scale > 0.0f ? static_cast<double>(softmax_scale) : 1.0 / std::sqrt(static_cast<double>(dim));
  return static_cast<float>(scale * 1.4426950408889634);
}

int check_queries(const kv_cache* c, int64_t batch, int64_t tokens, int64_t heads, float softmax_scale) {
  if (tokens < 0 || heads < 0 || tokens > kMax31 || heads > kMax31) return invalid("tokens and heads must be in [0, 2^31)");
  if (heads % c->kv_heads != 0 || heads / c->kv_heads > 128)
    return invalid("heads must be a multiple of kv_heads, at most 128 times it");
  if (!(softmax_scale >= 0.0f) || !std::isfinite(softmax_scale))
    return invalid("softmax_scale must be finite and non-negative");
  if (batch > 0 && tokens > 0 && heads > 0 &&
      (tokens > (int64_t{1} << 40) / batch || batch * tokens > (int64_t{1} << 40) / heads))
    return invalid("batch * tokens * heads must be at most 2^40");
  return GEMM_TN_OK;
}

gemm_tn_dev::CacheView view_of(const kv_cache* c, int64_t batch) {
  gemm_tn_dev::CacheView v{};
  v.k = static_cast<uint4*>(c->k);
  v.v = static_cast<uint4*>(c->v);
  v.page_stride = c->page_stride / 8;
  v.slot_stride = c->slot_stride / 8;
  v.head_stride = c->head_stride / 8;
  v.page_table = c->page_table;
  v.table_stride = c->table_stride;
  v.batch = static_cast<int>(batch);
  v.kv_heads = static_cast<int>(c->kv_heads);
  v.vec = static_cast<int>(c->head_dim / 8);
  v.page_size = static_cast<int>(c->page_size);
  v.num_pages = static_cast<int>(c->num_pages);
  v.capacity = static_cast<int>(c->max_pages * c->page_size);
  return v;
}

// Least key tiles per CTA of the attention.
constexpr int kMinChunk = 2;

// Key tiles that a CTA could walk in the time that it takes to finish one item
// and begin another: items are laid out that far apart before they are cut into
// chunks. GB300, us a call with no gap and with 2 (3 where an item is 256 rows
// wide): 63 tokens of 16 heads over 2 KV heads, 4 sequences of up to 32768
// slots 65.8 and 62.7; 26 tokens of 32 heads over 8, 8 sequences of up to 4096
// 35.0 and 34.2; one token, 2 sequences of 8192 24.2 and 22.5, 64 of up to 8192
// 190.5 and 190.0.
int change_tiles(int units) { return units + 1; }
constexpr int kMaxChange = 8;   // of this and of weigh_change_tiles

// The same for the accumulated weights. Up to 128 query rows are gathered ahead;
// more of them between the items (past 256 a tile is walked once per 256, and the
// change is worth fewer of them: 2 and 4 do the same there). GB300, us a call with
// gaps of 0, 2, 4 and 8: 1 token of 4 heads per KV head, 32 sequences of up to
// 2048 slots 23.4, 22.9, 23.4 and 24.4; 128 rows, 8 of up to 16384 44.3, 43.8, 44.0
// and 44.8, 2 of 8192 14.5, 13.5, 13.9 and 13.9; 256 rows, 8 of up to 8192 47.2,
// 46.2, 44.8 and 41.8; 700 rows, 2 of up to 4000 39.2, 39.1, 39.1 and 41.4.
int weigh_change_tiles(int64_t rows) { return rows <= 128 ? 2 : (rows <= 256 ? 8 : 4); }

// CTAs of a cluster that share each of `items` items of `tiles` key tiles, one
// row tile wide: as many as the tiles keep busy and as find room at once (15
// clusters of 8, 36 of 4 or 76 of 2 on a GB300; 16 of 8 took two rounds, 17.3 us
// for 9.0). GB300, us a call with clusters of 1, 2, 4 and 8, 32 heads over 8 KV
// heads: one token, 1 sequence of 100 slots 8.3, 8.9, 8.8 and 9.1, of 512 10.8,
// 10.4, 9.4 and 9.2, of 2048 21.7, 15.9, 12.1 and 10.5; 4 of 1024 14.7, 12.3 and
// 11.1; 7 of 1024 15.1 and 12.7. 26 tokens, whose joins are larger: 1 of 256
// 10.8, 14.4, 11.4 and 11.3, of 1024 18.3, 18.3, 14.2 and 12.8; 4 of 1024 18.7,
// 18.6 and 15.0 (16.6 cut); 8 of 1024 20.0 and 19.9.
int spread_of(bool decode, int64_t items, int64_t tiles, int sms) {
  if (tiles < (decode ? 4 : 5)) return 1;
  if (tiles > 4 && items * 8 <= sms * 4 / 5) return 8;
  if (items * 4 <= sms * 7 / 8) return 4;
  return decode && items * 2 <= sms * 15 / 16 ? 2 : 1;
}

// Blocks of a cluster that select from one of `lists` lists of at most `slots`
// slots: as many as find room at once, where the lists are long enough for their
// half a dozen meetings. GB300, us a call (with the moves) with clusters of 1, 2,
// 4 and 8, 8 lists a sequence, cut to half: 1 sequence of 8192 slots 17.6, 19.5,
// 19.7 and 22.8, of 32768 50.4, 42.2, 35.9 and 36.7; 2 of 16384 36.9, 34.9 and
// 33.8; 8 of 16384 66.3 and 65.5. Past 40960 slots the keys of a list lie in the
// shared memory of several blocks, of one they do not: 2 of 60000 180, 87 and 75.
int evict_spread(int64_t lists, int64_t slots, int sms) {
  if (slots < 16384) return 1;
  if (lists * 4 <= sms * 7 / 8) return 4;
  return lists * 2 <= sms * 15 / 16 || slots > evict_smem_keys(1 << 30) ? 2 : 1;
}

// Whether the attention's items stay whole, with no workspace and no second
// kernel: one item per CTA, or per cluster of `spread`, where there are no more
// of those than SMs (2), else each CTA takes the items that begin in its chunk
// (1). Cutting them balances the CTAs to a tile and costs a second segment per
// CTA, the parts' way through memory and the join: as much as walking 6 more
// tiles (5 where an item is 256 rows wide, 4 more than a cluster's join). With
// items no more than SMs the longest item decides, `tiles` / spread against
// items * tiles / sms; with more, a chunk overruns by half an item on average.
// Long items are always cut (the host knows what the page table can hold, not
// how ragged the lengths are). GB300, us a call, one token of 32 heads over 8
// KV heads, lengths from three quarters of the stated slots, cut and whole: 1
// sequence of 1024 slots 12.7 and 9.6, of 4096 14.4 and 12.3, of 8192 17.1 and
// 16.7; 2 of 2048 14.0 and 12.2, of 4096 16.0 and 16.9; 16 of 1024 22.8 and
// 18.1, of 3008 39.5 and 35.8; 24 of 500 23.6 and 20.5, of 1000 28.8 and 29.1,
// of 1500 33.2 and 38.6. 26 tokens: 1 of 1024 15.0 and 12.8, of 4096 18.3 and
// 16.7, of 8192 21.9 and 22.9; 4 of 2048 19.5 and 18.4. 60 tokens: 1 of 512 16.6 and 16.1, of 768 17.0 and
// 19.2; 32 of 256 35.6 and 29.6, of 1000 56.8 and 58.5.
int keep_whole(int64_t items, int64_t tiles, int units, int spread, int sms) {
  const int64_t allowance = spread > 1 ? 4 : (units == 2 ? 5 : 6);
  if (tiles > (spread > 1 ? 12 * spread : 32)) return sms == 1 ? 1 : 0;
  if (items <= sms) return tiles * (sms - items * spread) <= allowance * sms * spread ? 2 : 0;
  return tiles <= allowance ? 1 : 0;
}

// The kernels count key tiles in 32 bits, rounded up to whole chunks (one per SM):
// an upper bound of their number, from what the cache and the inputs can hold.
int check_tiles(const kv_cache* c, int64_t batch, int64_t row_units, int64_t tokens) {
  const int64_t per_item = (c->max_pages * c->page_size + 127) / 128 + (tokens + 127) / 128 + 1 + kMaxChange;
  const int64_t items = batch * c->kv_heads;   // below 2^31
  constexpr int64_t kMost = kMax31 - (1 << 16);
  if (row_units > kMost / items || per_item > kMost / (items * row_units))
    return invalid("too many key tiles: batch * kv_heads * tokens * capacity is too large");
  return GEMM_TN_OK;
}

}  // namespace

}  // namespace gemm_tn_impl

using namespace gemm_tn_impl;

extern "C" {

int tree_attn_fwd(int dtype, int64_t batch, int64_t tokens, int64_t heads, const kv_cache* cache, const kv_rows* q,
                  const kv_rows* k_new, const kv_rows* v_new, const uint64_t* mask, const int32_t* token_lens, void* o,
                  float* lse, float softmax_scale, int* d_status, gemm_tn_stream_t stream) {
  api_begin();
  int st = check_common(dtype, batch, cache);
  if (st == GEMM_TN_OK) st = check_queries(cache, batch, tokens, heads, softmax_scale);
  if (st != GEMM_TN_OK) return st;
  if (batch == 0 || tokens == 0 || heads == 0) return GEMM_TN_OK;
  const int64_t dim = cache->head_dim, kv_heads = cache->kv_heads;
  if ((st = check_rows(q, batch, tokens, heads, dim)) != GEMM_TN_OK) return st;
  if ((k_new == nullptr) != (v_new == nullptr)) return invalid("k_new and v_new come together");
  const bool has_new = k_new != nullptr;
  if (!has_new && mask != nullptr) return invalid("a mask needs k_new and v_new");
  if (has_new) {
    if ((st = check_rows(k_new, batch, tokens, kv_heads, dim)) != GEMM_TN_OK) return st;
    if ((st = check_rows(v_new, batch, tokens, kv_heads, dim)) != GEMM_TN_OK) return st;
  }
  if (o == nullptr) return invalid("o is NULL");
  if (!aligned(o, 16) || !aligned(lse, 4) || !aligned(mask, 8) || !aligned(token_lens, 4))
    return api_fail(GEMM_TN_ERR_MISALIGNED, "o, lse, mask or token_lens is not aligned to its element (o: 16 bytes)");
  const CacheRanges r = cache_ranges(cache, batch);
  const Range none = {0, 0};
  if (clash({{words_range(o, batch * tokens * heads * (dim / 2)), none},
             {words_range(lse, batch * tokens * heads), none},
             {words_range(d_status, 1), none}},
            {rows_range(q, batch, tokens, heads, dim), rows_range(k_new, batch, tokens, kv_heads, dim),
             rows_range(v_new, batch, tokens, kv_heads, dim), words_range(mask, 2 * batch * tokens * ((tokens + 63) / 64)),
             words_range(token_lens, batch), r.k, r.v, r.table, r.lens, r.weight, r.pos, r.seen}))
    return invalid("o, lse or the status word overlaps another array of the call");
  alignas(64) gemm_tn_dev::TreeArgs args{};
  args.group = static_cast<int>(heads / kv_heads);
  const bool decode = tokens * args.group <= decode_attn_rows();
  args.tile_tokens = decode ? static_cast<int>(tokens) : tree_attn_tile_rows() / args.group;
  const int64_t row_tiles = (tokens + args.tile_tokens - 1) / args.tile_tokens;
  args.units = row_tiles > 1 ? 2 : 1;
  args.part_rows = decode ? decode_attn_part_rows(static_cast<int>(tokens) * args.group) : args.units * tree_attn_tile_rows();
  args.row_units = static_cast<int>((row_tiles + args.units - 1) / args.units);
  if ((st = check_tiles(cache, batch, args.row_units, tokens)) != GEMM_TN_OK) return st;
  int sms = 0;
  if ((st = api_device(&sms)) != GEMM_TN_OK) return st;

  const bool bf16 = dtype == GEMM_TN_BF16;
  if ((st = encode_rows(&args.tmap_q, bf16, q, batch, tokens, heads, dim, args.group, args.tile_tokens)) != GEMM_TN_OK ||
      (st = encode_pool(&args.tmap_k, bf16, cache->k, cache)) != GEMM_TN_OK ||
      (st = encode_pool(&args.tmap_v, bf16, cache->v, cache)) != GEMM_TN_OK)
    return st;
  if (has_new && ((st = encode_rows(&args.tmap_k_new, bf16, k_new, batch, tokens, kv_heads, dim, 1, 128)) != GEMM_TN_OK ||
                  (st = encode_rows(&args.tmap_v_new, bf16, v_new, batch, tokens, kv_heads, dim, 1, 128)) != GEMM_TN_OK))
    return st;
  args.o = o;
  args.lse = lse;
  args.mask = mask;
  args.lens = cache->lens;
  args.token_lens = token_lens;
  args.page_table = cache->page_table;
  args.table_stride = cache->table_stride;
  args.batch = static_cast<int>(batch);
  args.tokens = static_cast<int>(tokens);
  args.heads = static_cast<int>(heads);
  args.kv_heads = static_cast<int>(kv_heads);
  args.page_size = static_cast<int>(cache->page_size);
  args.num_pages = static_cast<int>(cache->num_pages);
  args.capacity = static_cast<int>(cache->max_pages * cache->page_size);
  args.mask_words = static_cast<int>((tokens + 63) / 64);
  args.has_new = has_new ? 1 : 0;
  args.chunks = sms;
  args.min_chunk = kMinChunk;
  args.gap = change_tiles(args.units);
  args.scale_log2 = scale_log2(softmax_scale, dim);
  args.status = d_status;
  args.timeout_ns = api_watchdog_ns();
  args.drop_load_block = api_drop_load();

  const int64_t item_tiles = (static_cast<int64_t>(args.capacity) + 127) / 128 + (has_new ? (tokens + 127) / 128 : 0);
  const int64_t items = batch * kv_heads * args.row_units;
  const int spread = args.units == 1 ? spread_of(decode, items, item_tiles, sms) : 1;
  args.whole = keep_whole(items, item_tiles, args.units, spread, sms);
  args.spread = args.whole == 2 ? spread : 1;
  if (args.whole == 2) args.chunks = static_cast<int>(items);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto launch = [&] {
    return decode ? launch_decode_attn(static_cast<int>(dim), bf16, args, s)
                  : launch_tree_attn(static_cast<int>(dim), bf16, args, s);
  };
  if (args.whole != 0) {
    args.min_chunk = 1;
    args.gap = 0;
    const cudaError_t e = api_counted(launch());
    return e == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(e, "tree attention launch");
  }
  const size_t part_rows = static_cast<size_t>(2 * args.chunks) * static_cast<size_t>(args.part_rows);
  void* workspace = nullptr;
  cudaError_t e = api_workspace(part_rows * static_cast<size_t>(dim * 4 + 8) + static_cast<size_t>(args.chunks) * 32, s, &workspace);
  if (e != cudaSuccess) return api_fail_cuda(e, "workspace");
  args.part_o = static_cast<float*>(workspace);
  args.part_ml = reinterpret_cast<float2*>(args.part_o + part_rows * static_cast<size_t>(dim));
  args.cuts = reinterpret_cast<int32_t*>(args.part_ml + part_rows);
  e = api_counted(launch());
  if (e == cudaSuccess) e = api_counted(launch_tree_attn_join(static_cast<int>(dim), bf16, args, s));
  const cudaError_t freed = cudaFreeAsync(workspace, s);
  if (e != cudaSuccess) return api_fail_cuda(e, "tree attention launch");
  return freed == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(freed, "cudaFreeAsync (workspace)");
}

int kv_cache_append(int dtype, int64_t batch, int64_t tokens, const kv_cache* cache, const kv_rows* k_new,
                    const kv_rows* v_new, const int32_t* rows, const int32_t* counts, int64_t max_rows, int32_t* lens_out,
                    int32_t* seen_out, int* d_status, gemm_tn_stream_t stream) {
  api_begin();
  int st = check_common(dtype, batch, cache);
  if (st != GEMM_TN_OK) return st;
  if (tokens < 0 || tokens > kMax31 || max_rows < 0 || max_rows > kMax31) return invalid("tokens and max_rows must be in [0, 2^31)");
  if (rows == nullptr && max_rows > tokens) return invalid("max_rows > tokens without rows");
  if (batch == 0) return GEMM_TN_OK;
  if (lens_out == nullptr) return invalid("lens_out is NULL");
  if ((seen_out != nullptr) && cache->seen == nullptr) return invalid("seen_out without seen");
  if (!aligned(rows, 4) || !aligned(counts, 4) || !aligned(lens_out, 4) || !aligned(seen_out, 4))
    return api_fail(GEMM_TN_ERR_MISALIGNED, "rows, counts, lens_out or seen_out not 4-byte aligned");
  if (max_rows > 0 && tokens > 0) {
    if ((st = check_rows(k_new, batch, tokens, cache->kv_heads, cache->head_dim)) != GEMM_TN_OK) return st;
    if ((st = check_rows(v_new, batch, tokens, cache->kv_heads, cache->head_dim)) != GEMM_TN_OK) return st;
    if (max_rows > (int64_t{1} << 34) / (batch * cache->kv_heads)) return invalid("batch * max_rows * kv_heads must be at most 2^34");
  } else if (max_rows > 0) {
    return invalid("max_rows > 0 without tokens");
  }
  const CacheRanges r = cache_ranges(cache, batch);
  const Range none = {0, 0};
  const bool copies = max_rows > 0;
  if (pools_overlap(cache)) return invalid("the K and V pools overlap");
  const Outputs outs = {{r.weight, none},
                        {r.pos, none},
                        {words_range(lens_out, batch), r.lens},
                        {words_range(seen_out, batch), r.seen},
                        {words_range(d_status, 1), none}};
  const Inputs ins = {copies ? rows_range(k_new, batch, tokens, cache->kv_heads, cache->head_dim) : none,
                      copies ? rows_range(v_new, batch, tokens, cache->kv_heads, cache->head_dim) : none,
                      words_range(rows, batch * max_rows), words_range(counts, batch), r.table};
  if (clash(outs, ins) || meets(r.k, outs, ins) || meets(r.v, outs, ins))
    return invalid("a pool, weight, pos, lens_out, seen_out or the status word overlaps another array of the call");
  int sms = 0;
  if ((st = api_device(&sms)) != GEMM_TN_OK) return st;
  gemm_tn_dev::AppendArgs args{};
  args.c = view_of(cache, batch);
  if (max_rows > 0) {
    args.k_new = static_cast<const uint4*>(k_new->data);
    args.v_new = static_cast<const uint4*>(v_new->data);
    args.kn_batch = k_new->batch_stride / 8;
    args.kn_token = k_new->token_stride / 8;
    args.kn_head = k_new->head_stride / 8;
    args.vn_batch = v_new->batch_stride / 8;
    args.vn_token = v_new->token_stride / 8;
    args.vn_head = v_new->head_stride / 8;
  }
  args.rows = rows;
  args.counts = counts;
  args.lens = cache->lens;
  args.seen = cache->seen;
  args.lens_out = lens_out;
  args.seen_out = seen_out;
  args.weight = cache->weight;
  args.pos = cache->pos;
  args.tokens = static_cast<int>(tokens);
  args.max_rows = static_cast<int>(max_rows);
  args.status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool in_place = lens_out == cache->lens || (seen_out != nullptr && seen_out == cache->seen);
  cudaError_t e = cudaSuccess;
  if (max_rows > 0) e = api_counted(launch_cache_append(args, s));
  if (e == cudaSuccess && (in_place || max_rows == 0)) e = api_counted(launch_cache_advance(args, s));
  return e == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(e, "cache append launch");
}

int kv_cache_weigh(int dtype, int64_t batch, int64_t tokens, int64_t heads, const kv_cache* cache, const kv_rows* q,
                   const float* lse, const int32_t* rows, const int32_t* counts, int64_t max_rows, int causal,
                   float softmax_scale, float* weight_out, int* d_status, gemm_tn_stream_t stream) {
  api_begin();
  int st = check_common(dtype, batch, cache);
  if (st == GEMM_TN_OK) st = check_queries(cache, batch, tokens, heads, softmax_scale);
  if (st != GEMM_TN_OK) return st;
  if (max_rows < 0 || max_rows > kMax31 / 256) return invalid("max_rows must be in [0, 2^23)");
  if (rows == nullptr && max_rows > tokens) return invalid("max_rows > tokens without rows");
  if (batch == 0) return GEMM_TN_OK;
  if (heads == 0) return invalid("heads must be positive");
  if (cache->weight == nullptr || weight_out == nullptr) return invalid("weight or weight_out is NULL");
  if (max_rows > 0) {
    if (tokens == 0) return invalid("max_rows > 0 without tokens");
    if ((st = check_rows(q, batch, tokens, heads, cache->head_dim)) != GEMM_TN_OK) return st;
    if (lse == nullptr) return invalid("lse is NULL");
  }
  if (!aligned(rows, 4) || !aligned(counts, 4) || !aligned(lse, 4) || !aligned(weight_out, 4))
    return api_fail(GEMM_TN_ERR_MISALIGNED, "rows, counts, lse or weight_out not 4-byte aligned");
  const CacheRanges r = cache_ranges(cache, batch);
  const Range none = {0, 0};
  const int64_t slots = batch * cache->kv_heads * cache->max_pages * cache->page_size;
  if (clash({{words_range(weight_out, slots), r.weight}, {words_range(d_status, 1), none}},
            {max_rows > 0 ? rows_range(q, batch, tokens, heads, cache->head_dim) : none,
             words_range(lse, max_rows > 0 ? batch * tokens * heads : 0), words_range(rows, batch * max_rows),
             words_range(counts, batch), r.k, r.v, r.table, r.lens, r.pos, r.seen}))
    return invalid("weight_out or the status word overlaps another array of the call");
  if ((st = check_tiles(cache, batch, 1, 0)) != GEMM_TN_OK) return st;
  int sms = 0;
  if ((st = api_device(&sms)) != GEMM_TN_OK) return st;
  const bool bf16 = dtype == GEMM_TN_BF16;
  alignas(64) gemm_tn_dev::WeighArgs args{};
  if ((st = encode_pool(&args.tmap_k, bf16, cache->k, cache)) != GEMM_TN_OK) return st;
  if (max_rows > 0) {
    args.q = q->data;
    args.q_batch = q->batch_stride;
    args.q_token = q->token_stride;
    args.q_head = q->head_stride;
  }
  args.lse = lse;
  args.rows = rows;
  args.counts = counts;
  args.lens = cache->lens;
  args.page_table = cache->page_table;
  args.weight = cache->weight;
  args.weight_out = weight_out;
  args.table_stride = cache->table_stride;
  args.batch = static_cast<int>(batch);
  args.tokens = static_cast<int>(tokens);
  args.heads = static_cast<int>(heads);
  args.kv_heads = static_cast<int>(cache->kv_heads);
  args.group = static_cast<int>(heads / cache->kv_heads);
  args.max_rows = static_cast<int>(max_rows);
  args.page_size = static_cast<int>(cache->page_size);
  args.num_pages = static_cast<int>(cache->num_pages);
  args.capacity = static_cast<int>(cache->max_pages * cache->page_size);
  args.block_tokens = 256 / args.group;
  args.chunks = sms;
  args.min_chunk = 1;
  args.gap = weigh_change_tiles(max_rows * args.group);
  args.causal = causal != 0 ? 1 : 0;
  args.scale_log2 = scale_log2(softmax_scale, cache->head_dim);
  args.status = d_status;
  args.timeout_ns = api_watchdog_ns();
  args.drop_load_block = api_drop_load();
  const cudaError_t e = api_counted(
      launch_cache_weigh(static_cast<int>(cache->head_dim), bf16, args, reinterpret_cast<cudaStream_t>(stream)));
  return e == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(e, "cache weigh launch");
}

int kv_cache_evict(int dtype, int64_t batch, const kv_cache* cache, int64_t keep, int64_t recent, float* weight_out,
                   int32_t* pos_out, int32_t* lens_out, int* d_status, gemm_tn_stream_t stream) {
  api_begin();
  int st = check_common(dtype, batch, cache);
  if (st != GEMM_TN_OK) return st;
  if (keep < 0 || keep > kMax31) return invalid("keep must be in [0, 2^31)");
  if (recent < 0 || recent > keep) return invalid("recent must be in [0, keep]");
  // the kernels walk slots and lists in 32 bits, by up to 2^16 at a time
  if (cache->max_pages * cache->page_size > kMax31 + 1 - (1 << 16))
    return invalid("max_pages * page_size must be at most 2^31 - 2^16");
  if (batch > 0 && cache->kv_heads > (int64_t{1} << 30) / batch) return invalid("batch * kv_heads must be at most 2^30");
  if (batch == 0) return GEMM_TN_OK;
  if (cache->weight == nullptr || weight_out == nullptr || lens_out == nullptr)
    return invalid("weight, weight_out or lens_out is NULL");
  if (recent > 0 && (cache->pos == nullptr || cache->seen == nullptr)) return invalid("recent > 0 needs pos and seen");
  if ((pos_out == nullptr) != (cache->pos == nullptr)) return invalid("pos_out goes with the cache's pos");
  if (!aligned(weight_out, 4) || !aligned(pos_out, 4) || !aligned(lens_out, 4))
    return api_fail(GEMM_TN_ERR_MISALIGNED, "weight_out, pos_out or lens_out not 4-byte aligned");
  const CacheRanges r = cache_ranges(cache, batch);
  const Range none = {0, 0};
  const int64_t slots = batch * cache->kv_heads * cache->max_pages * cache->page_size;
  if (pools_overlap(cache)) return invalid("the K and V pools overlap");
  const Outputs outs = {{words_range(weight_out, slots), r.weight},
                        {words_range(pos_out, slots), r.pos},
                        {words_range(lens_out, batch), r.lens},
                        {words_range(d_status, 1), none}};
  const Inputs ins = {r.table, r.seen};
  if (clash(outs, ins) || meets(r.k, outs, ins) || meets(r.v, outs, ins))
    return invalid("a pool, weight_out, pos_out, lens_out or the status word overlaps another array of the call");
  int sms = 0;
  if ((st = api_device(&sms)) != GEMM_TN_OK) return st;
  gemm_tn_dev::EvictArgs args{};
  args.c = view_of(cache, batch);
  args.weight = cache->weight;
  args.weight_out = weight_out;
  args.pos = cache->pos;
  args.pos_out = pos_out;
  args.seen = cache->seen;
  args.lens = cache->lens;
  args.lens_out = lens_out;
  args.keep = static_cast<int>(keep);
  args.recent = static_cast<int>(recent);
  args.max_moves = static_cast<int>(std::max<int64_t>(0, std::min<int64_t>(keep, args.c.capacity - keep)));
  args.smem_keys = evict_smem_keys(args.c.capacity);
  args.spread = 1;
  args.status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // few rows to move: one kernel (which must not write the lens that its other blocks read)
  if (args.max_moves <= evict_fused_moves() && args.smem_keys == args.c.capacity && lens_out != cache->lens) {
    const cudaError_t e = api_counted(launch_cache_select(args, s));
    return e == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(e, "cache evict launch");
  }
  const size_t lists = static_cast<size_t>(batch * cache->kv_heads);
  args.spread = evict_spread(static_cast<int64_t>(lists), args.c.capacity, sms);
  const int per_block = ((args.c.capacity + args.spread - 1) / args.spread + 31) / 32 * 32;
  args.smem_keys = evict_smem_keys(per_block);
  const size_t count_bytes = (lists * 4 + 15) / 16 * 16;
  const size_t move_bytes = lists * static_cast<size_t>(args.max_moves) * 8;
  const size_t word_bytes = args.smem_keys == per_block ? 0 : lists * static_cast<size_t>((args.c.capacity + 31) / 32) * 12;
  void* workspace = nullptr;
  cudaError_t e = api_workspace(count_bytes + move_bytes + word_bytes, s, &workspace);
  if (e != cudaSuccess) return api_fail_cuda(e, "workspace");
  args.counts = static_cast<int32_t*>(workspace);
  args.moves = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + count_bytes);
  args.words = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + count_bytes + move_bytes);
  e = api_counted(launch_cache_select(args, s));
  if (e == cudaSuccess) e = api_counted(launch_cache_move(args, sms, s));
  const cudaError_t freed = cudaFreeAsync(workspace, s);
  if (e != cudaSuccess) return api_fail_cuda(e, "cache evict launch");
  return freed == cudaSuccess ? GEMM_TN_OK : api_fail_cuda(freed, "cudaFreeAsync (workspace)");
}

}  // extern "C"
