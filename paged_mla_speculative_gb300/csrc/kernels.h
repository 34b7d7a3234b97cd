// Internal launch interface between the C ABI and the kernels.
#pragma once

#include <cuda.h>   // CUtensorMap (a plain struct; the library does not link the driver)
#include <cuda_runtime.h>

#include "common.cuh"
#include "shared.cuh"

namespace mlav {

// Launch with programmatic overlap: the kernel may
// start while the one before it on the stream ends, and waits for it with
// griddepcontrol.wait before it touches memory.  cluster: CTAs per cluster.
template <typename... Args>
cudaError_t launch_overlapping(void (*kernel)(Args...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                               unsigned cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Split-KV partial kernel on warp-level mma.sync.
int partial_mma_smem_bytes();
cudaError_t partial_mma_prepare();
cudaError_t launch_partial_mma(const Params& p, cudaStream_t stream);

// Split-KV partial kernel on tcgen05 tensor cores with TMEM accumulators.
cudaError_t partial_tc_prepare();
// `overlap`: launch with programmatic stream serialisation, so the kernel's
// CTAs may start while the previous kernel on the stream (the pack) runs;
// the kernel then reads each packed block after its ready flags carry the
// call's tag (Params::pack_flags = 1), or after griddepcontrol.wait, which
// waits for the whole pack grid (pack_flags = 0).
cudaError_t launch_partial_tc(const Params& p, cudaStream_t stream, bool overlap);

// Split-KV partial kernel on CTA pairs (cta_group::2), 128 query rows and
// 256 keys per step, over the packed blocks (Params::split_pairs = 1);
// `overlap` as for launch_partial_tc.  The packed buffer is read through two
// TMA tensor maps (make_pack_maps): rows of 128 bytes, boxes of 256 rows (a
// chunk pair) and of 128 rows (one chunk).
struct PackMaps {
  CUtensorMap pair;    // box 64 x 256 fp16
  CUtensorMap chunk;   // box 64 x 128 fp16
};
cudaError_t make_pack_maps(PackMaps* maps, void* packed, size_t packed_bytes);
cudaError_t partial_pair_prepare();
cudaError_t launch_partial_pair(const Params& p, const PackMaps& maps, cudaStream_t stream, bool overlap);

// Per-call gather of the key rows into packed fp16 operand tiles.
size_t packed_block_bytes();
// The whole pack ahead of the attention kernel (Params::pack_flags = 0).
cudaError_t launch_pack_kv(const Params& p, void* packed, int max_blocks, cudaStream_t stream);
// The two-phase pack that overlaps the attention kernel (pack_flags = 1):
// num_ctas persistent CTAs (one per SM); CTAs stay .. num_ctas-1 pack the
// first `wide_positions` blocks of every split and exit, CTAs 0 .. stay-1
// pack the rest.  pack_kv_prepare sets its shared-memory attributes.
cudaError_t pack_kv_prepare();
cudaError_t launch_pack_kv_overlap(const Params& p, void* packed, int max_blocks, int num_ctas,
                                   int wide_positions, int stay, cudaStream_t stream);

// LSE combine of the split partials into out/lse (`overlap`: may be
// scheduled early; it waits for the partial kernel with griddepcontrol.wait).
cudaError_t launch_combine(const Params& p, cudaStream_t stream, bool overlap);

// Up to kMax copies between device-addressable regions (device memory, or
// page-locked host memory mapped into the device's address space) in one
// kernel launch.  Byte counts are multiples of 4.
struct CopyRegions {
  static constexpr int kMax = 8;
  const void* src[kMax];
  void* dst[kMax];
  long long bytes[kMax];
  int n;
};
cudaError_t launch_copy_regions(const CopyRegions& c, cudaStream_t stream);

// Per-step index builder (index_builder.cu).
struct IndexArgs {
  const int32_t* req_to_token;      // [pool_size][stride] cache slot of each token position
  long long stride;                 // entries per table row (>= max_kv_len)
  int pool_size;
  const int32_t* req_pool_indices;  // [batch]
  const int32_t* prefix_lens;       // [batch]
  int batch, T, page_size, max_kv_len;
  long long capacity;               // entries kv_indices holds (<= INT32_MAX)
  int32_t* kv_indices;
  int32_t* kv_indptr;               // [batch + 1]
  int32_t* kv_lens;                 // [batch]
  int* err;
};
cudaError_t launch_build_indices(const IndexArgs& a, int max_kv_len, cudaStream_t stream);

// KV compaction into 64-row pages (compact.cu).
struct CompactArgs {
  const void* kv_src;               // bf16 [src_slots][576]
  long long src_slots;
  const int32_t* kv_indices;        // page_size 1 slot table of the requests
  const int32_t* kv_indptr;         // [batch + 1]
  const int32_t* kv_lens;           // [batch]
  const int32_t* free_pages;        // [num_free_pages] destination page ids, used in order
  long long num_free_pages;
  void* kv_dst;                     // bf16 [dst_slots][576], dst_slots a multiple of 64
  long long dst_slots;
  int32_t* page_table;              // [num_free_pages] out
  int32_t* page_indptr;             // [batch + 1] out
  int batch, max_kv_len;
  int* err;
};
cudaError_t launch_compact_kv(const CompactArgs& a, cudaStream_t stream);

// Attention of groups of requests that share their first rows: the call's
// layout with its packed keys and queries, the persistent attention, the merge
// -- in this order, each of the last two overlapping the tail of the one before.
struct SharedMaps {
  CUtensorMap pair, chunk, q;   // of the packed keys (two planes, one plane) and queries
};
// The driver's tensor map encoder.
cudaError_t tensor_map_encode(void** fn);
cudaError_t make_shared_maps(SharedMaps* maps, void* k16, long long k_plane, void* q16, long long q_plane);
cudaError_t partial_shared_prepare();
cudaError_t launch_shared_prepare(const SharedParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_partial_shared(const SharedParams& p, const SharedMaps& maps, cudaStream_t stream);
cudaError_t launch_shared_join(const SharedParams& p, cudaStream_t stream);
// Attention of chunks of new tokens (SharedParams::q_indptr set): the layout
// with the packed keys, launch_partial_shared with maps.q from
// make_chunk_query_map (the other maps are those of the shared-prefix call),
// the merge.
cudaError_t make_chunk_query_map(CUtensorMap* map, const void* q, long long rows);
cudaError_t launch_chunk_prepare(const SharedParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_chunk_join(const SharedParams& p, cudaStream_t stream);

// The attention weight given to cached rows (weigh_kv.cu).
struct WeighParams {
  const uint16_t* kv;               // bf16 [num_slots][576]
  const int32_t* kv_indices;
  const int32_t* kv_indptr;         // [batch + 1]
  const int32_t* kv_lens;           // [batch]
  const int32_t* q_indptr;          // [batch + 1]
  const float* lse;                 // [num_tokens][H]
  float* weights;                   // [batch] rows, stride floats apart
  long long stride;
  float scale_log2;
  int batch, num_tokens, H, page_size;
  long long num_slots;
  int max_kv_len;
  int clusters;
  float* part;                      // [2 * clusters][256]: sums of a cluster's first and last block
  int fault_rank;                   // testing: the CTA of each pair that gives up in mid-call, -1 for none
  unsigned* arrived;                // [clusters][2], 0 between calls: clusters done with the block that this one shares first
  int* err;
};
struct WeighMaps {
  CUtensorMap kv, q, q_full;        // rows of 576 bf16: the cache (boxes of a page) and the queries (32 and 128 rows)
};
constexpr size_t weigh_workspace_bytes(int clusters) {
  return static_cast<size_t>(clusters) * 2 * 256 * sizeof(float);
}
cudaError_t make_weigh_maps(WeighMaps* maps, const void* kv, long long num_slots, int page_size, const void* q, long long q_rows);
cudaError_t weigh_prepare();
cudaError_t launch_weigh_kv(const WeighParams& p, const WeighMaps& maps, cudaStream_t stream);

// New tokens' cache rows and queries (append_kv.cu).
struct AppendArgs {
  const uint16_t* kv;               // bf16 [num_tokens][576], rows kv_stride elements apart
  long long kv_stride;
  const uint16_t* weight;           // bf16 [512]
  float eps;
  const uint16_t* q_nope;           // bf16 [num_tokens][heads][512] by strides, or null: in q already
  long long nope_stride_n, nope_stride_h;
  const uint16_t* q_pe;             // bf16 [num_tokens][heads][64] by strides, or null: no queries
  long long pe_stride_n, pe_stride_h;
  const float* cos_sin;             // [max_pos][64]: 32 cosines, 32 sines
  long long max_pos;
  const int32_t* positions;         // [num_tokens]
  const int32_t* slots;             // [num_tokens], -1: padding
  long long num_tokens;
  int heads, halves;                // halves: pairs (i, i + 32) instead of (2i, 2i + 1)
  uint16_t* kv_cache;               // bf16 [num_slots][576]
  long long num_slots;
  uint16_t* q;                      // bf16 [num_tokens][heads][576]
  int* err;
};
cudaError_t launch_append_kv(const AppendArgs& a, cudaStream_t stream);

// Forking and freeing requests of a cache with counted pages (page_pool.cu).
constexpr int FORK_MAX_LAYERS = 1 << 16;   // pieces of a copy are counted in 32 bits
struct ForkArgs {
  const int32_t* parents;           // [num_children]
  int num_children, num_parents;
  const int32_t* kv_indices;        // the parents' page tables
  const int32_t* kv_indptr;         // [num_parents + 1]
  const int32_t* kv_lens;           // [num_parents]
  uint16_t* kv_cache;               // bf16 [num_layers][num_pages * 64][576], layers layer_stride elements apart
  int num_layers;
  long long layer_stride;
  int extra, num_pages, max_kv_len;
  int32_t* page_refs;               // [num_pages]
  const int32_t* free_pages;        // [num_pages]
  int32_t* free_count;              // [1]
  int32_t* child_indices;           // [capacity] out
  long long capacity;
  int32_t* child_indptr;            // [num_children + 1] out
  int32_t* child_lens;              // [num_children] out
  unsigned* ticket;                 // plan workspace, 0 between calls
  int* err;
};
cudaError_t page_pool_prepare();
cudaError_t launch_fork_kv(const ForkArgs& a, int num_sms, cudaStream_t stream);
struct FreeArgs {
  const int32_t* kv_indices;
  const int32_t* kv_indptr;         // [batch + 1]
  int batch, num_pages;
  int32_t* page_refs;               // [num_pages]
  int32_t* free_pages;              // [num_pages]
  int32_t* free_count;              // [1]
  unsigned* page_bits;              // plan workspace, one bit per page, 0 between calls
  int* err;
};
// `max_entries`: of the tables, as far as the host can tell.
cudaError_t launch_free_kv(const FreeArgs& a, int max_entries, cudaStream_t stream);

// Eviction of the rows with the smallest weights (evict_kv.cu).
struct EvictArgs {
  const float* weights;             // [batch] rows, stride floats apart
  long long stride;
  int budget, sink, recent, extra;
  int batch, page, max_kv_len;      // page: rows of a page, 1 or 64
  const int32_t* kv_indices;
  const int32_t* kv_indptr;         // [batch + 1]
  const int32_t* kv_lens;           // [batch]
  uint16_t* kv_cache;               // bf16 [num_layers][num_pages * 64][576], layers layer_stride elements apart; pages only
  int num_layers;
  long long layer_stride;
  int num_pages;                    // or slots
  int32_t* page_refs;               // [num_pages]
  int32_t* free_pages;              // [num_pages]
  int32_t* free_count;              // [1]
  int32_t* new_indices;             // [capacity] out
  long long capacity;
  int32_t* new_indptr;              // [batch + 1] out
  int32_t* new_lens;                // [batch] out
  float* new_weights;               // [batch] rows of new_width, new_stride floats apart, out
  long long new_stride, new_width;
  int32_t* kept;                    // plan workspace: [batch][kept_stride] rows that are kept, of evicted requests
  long long kept_stride;
  unsigned* page_bits;              // plan workspace, one bit per page, 0 between calls
  unsigned* ticket;                 // plan workspace: three words, 0 between calls
  int* err;
  // Set by the launch: rows [copy_from, copy_to) of an evicted request's kept
  // ones are copied once all are chosen, the others (protected ones) before.
  int copy_from, copy_to;
};
cudaError_t evict_prepare();
cudaError_t launch_evict_kv(const EvictArgs& a, int num_sms, cudaStream_t stream);

}  // namespace mlav
