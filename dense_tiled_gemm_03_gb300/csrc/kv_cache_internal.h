// kv_cache_internal.h -- host-side interface of the paged cache's operators:
// kernel arguments, launches, and what kv_cache_api.cu shares with
// gemm_tn_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gemm_tn_internal.h"

namespace gemm_tn_dev {

// Kernel arguments of the attention over a paged cache (sm103_tree_attn.cu).
struct TreeArgs {
  CUtensorMap tmap_q;       // {dim, heads, tokens, batch}, boxes {64, group, tile_tokens, 1}
  CUtensorMap tmap_k;       // {dim, kv heads, page_size, num_pages}, boxes {64, 1, min(page_size, 128), 1}
  CUtensorMap tmap_v;
  CUtensorMap tmap_k_new;   // {dim, kv heads, tokens, batch}, boxes {64, 1, 128, 1}
  CUtensorMap tmap_v_new;
  void* o;                  // [batch, tokens, heads, dim]
  float* lse;               // [batch, tokens, heads], or NULL
  const uint64_t* mask;     // [batch, tokens, mask_words] visible new tokens, or NULL: the causal chain
  const int32_t* lens;      // [batch] cached keys
  const int32_t* token_lens;   // [batch] new tokens, or NULL: all
  const int32_t* page_table;   // [batch] rows of page numbers, table_stride apart
  float* part_o;            // workspace: [2 chunks][dim / 4][part_rows][4] unnormalised rows of cut items
  float2* part_ml;          // [2 chunks][part_rows]: their (maximum, sum)
  int32_t* cuts;            // [chunks][8]: the item that each chunk begins inside of
  int64_t table_stride;
  int batch, tokens, heads, kv_heads, group;
  int page_size, num_pages, capacity;   // capacity: cached keys that a page table row can hold
  int mask_words;
  int part_rows;            // rows per item (units * 128; the decode kernel's 16 or 32)
  int tile_tokens;          // tokens per row tile: floor(128 / group) (the decode kernel: all)
  int units;                // row tiles per item: 1 (both units share the rows) or 2
  int row_units;            // items per KV head of a sequence
  int has_new;
  int chunks;               // CTAs (clusters of `spread` CTAs)
  int min_chunk;            // least key tiles per CTA
  int gap;                  // key tiles that the change to another item costs a CTA
  // 1: a chunk takes the items that begin in it whole; 2: it takes one item
  // (at most `chunks` of them); part_o, part_ml and cuts are NULL in both
  int whole;
  int spread;               // CTAs of a cluster that share an item's key tiles (whole == 2 and units == 1; else 1)
  float scale_log2;         // softmax scale * log2(e), > 0
  int* status;
  uint64_t timeout_ns;
  int drop_load_block;      // test hook: tile whose K load the first CTA skips (-1: none)
};

// Kernel arguments of the accumulated attention weights (sm103_cache_weigh.cu).
struct WeighArgs {
  CUtensorMap tmap_k;       // as in TreeArgs
  const void* q;            // [batch][tokens][heads][dim], strides in elements
  int64_t q_batch, q_token, q_head;
  const float* lse;         // [batch, tokens, heads]
  const int32_t* rows;      // [batch, max_rows] tokens to count, or NULL: the first ones
  const int32_t* counts;    // [batch] how many of them, or NULL: max_rows
  const int32_t* lens;
  const int32_t* page_table;
  const float* weight;      // [batch, kv heads, capacity]
  float* weight_out;
  int64_t table_stride;
  int batch, tokens, heads, kv_heads, group, max_rows;
  int page_size, num_pages, capacity;
  int block_tokens;         // tokens per pass: floor(256 / group)
  int chunks, min_chunk, gap;   // as in TreeArgs
  int causal;
  float scale_log2;
  int* status;
  uint64_t timeout_ns;
  int drop_load_block;
};

// Kernel arguments of append and evict (kv_cache_ops.cu). Strides in 16-byte
// units; vec = 16-byte pieces per row of one head.
struct CacheView {
  uint4* k;
  uint4* v;
  int64_t page_stride, slot_stride, head_stride;
  const int32_t* page_table;
  int64_t table_stride;
  int batch, kv_heads, vec;
  int page_size, num_pages, capacity;
};
struct AppendArgs {
  CacheView c;
  const uint4* k_new;
  const uint4* v_new;
  int64_t kn_batch, kn_token, kn_head, vn_batch, vn_token, vn_head;   // 16-byte units
  const int32_t* rows;      // [batch, max_rows], or NULL: the first ones
  const int32_t* counts;    // [batch], or NULL: max_rows
  const int32_t* lens;
  const int32_t* seen;      // may be NULL
  int32_t* lens_out;
  int32_t* seen_out;
  float* weight;            // [batch, kv heads, capacity], may be NULL
  int32_t* pos;             // may be NULL
  int tokens, max_rows;
  int* status;
};
struct EvictArgs {
  CacheView c;
  const float* weight;
  float* weight_out;
  const int32_t* pos;       // may be NULL (recent is 0 then)
  int32_t* pos_out;
  const int32_t* seen;
  const int32_t* lens;
  int32_t* lens_out;
  int32_t* counts;          // workspace: [batch * kv heads] rows to move
  int2* moves;              // workspace: [batch * kv heads][max_moves] slots (from, to); NULL: the selecting blocks move
  uint32_t* words;          // workspace: [batch * kv heads][3][ceil(capacity / 32)] where keys do not fit in shared memory
  int max_moves;
  int keep, recent;
  int smem_keys;            // keys that a block holds in shared memory (none where it has more slots)
  int spread;               // blocks of a cluster that share a list
  int* status;
};

}  // namespace gemm_tn_dev

namespace gemm_tn_impl {

// Launch attributes of the cache's kernels: clusters of `spread` CTAs,
// programmatic dependent launch. Returns their number.
inline unsigned cache_launch_attributes(cudaLaunchAttribute (&attr)[2], int spread) {
  unsigned n = 0;
  if (spread > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(spread);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent_launch_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  return n;
}

// Attention over a paged cache: rows of queries per tile, the kernel, and the
// kernel that joins the items its chunks cut.
int tree_attn_tile_rows();
cudaError_t launch_tree_attn(int head_dim, bool bf16, const gemm_tn_dev::TreeArgs& args, cudaStream_t stream);
// The same for items of at most decode_attn_rows() query rows, with keys on the
// tensor memory's lanes; args.part_rows is decode_attn_part_rows(rows).
int decode_attn_rows();
int decode_attn_part_rows(int rows);
cudaError_t launch_decode_attn(int head_dim, bool bf16, const gemm_tn_dev::TreeArgs& args, cudaStream_t stream);
cudaError_t launch_tree_attn_join(int head_dim, bool bf16, const gemm_tn_dev::TreeArgs& args, cudaStream_t stream);
cudaError_t launch_cache_weigh(int head_dim, bool bf16, const gemm_tn_dev::WeighArgs& args, cudaStream_t stream);
// Copies the rows; lens_out and seen_out are written by it, or (where one of
// them is its input) by a second launch.
cudaError_t launch_cache_append(const gemm_tn_dev::AppendArgs& args, cudaStream_t stream);
cudaError_t launch_cache_advance(const gemm_tn_dev::AppendArgs& args, cudaStream_t stream);
// Chooses the kept slots and lists the moves; then moves the rows.
int evict_smem_keys(int capacity);
int evict_fused_moves();   // most moves per list that the first kernel can make itself (moves NULL, lens_out not lens)
cudaError_t launch_cache_select(const gemm_tn_dev::EvictArgs& args, cudaStream_t stream);
cudaError_t launch_cache_move(const gemm_tn_dev::EvictArgs& args, int num_sms, cudaStream_t stream);

// What the C ABI's translation units share (gemm_tn_api.cu): the thread's error
// state, the launch counter, device facts, the workspace pool, tensor maps and
// the environment's switches.
void api_begin();
int api_fail(int status, const char* what);
int api_fail_cuda(cudaError_t e, const char* what);
cudaError_t api_counted(cudaError_t e);
int api_device(int* num_sms);
cudaError_t api_workspace(size_t bytes, cudaStream_t stream, void** out);
int api_encode_4d(CUtensorMap* map, bool bf16, const void* ptr, const int64_t dims[4], const int64_t strides[3],
                  const int box[4]);
uint64_t api_watchdog_ns();
int api_drop_load();

}  // namespace gemm_tn_impl
