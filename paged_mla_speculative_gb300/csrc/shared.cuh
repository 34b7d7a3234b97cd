// Definitions shared by the kernels of the shared-prefix verify attention.
//
// Every call lays its keys out once in a dense packed space: for each group
// its shared rows, then its requests' own rows, one after another.  Query rows
// go in tiles of 128 consecutive rows of one group (a tile may hold several
// requests).  A tile's key sequence is the group's shared range followed by
// the own range of the requests it holds, walked in half blocks of 128 keys,
// two per step; a key of another request of the tile, or of a draft that is
// not an ancestor, is masked by the key's meta word.
#pragma once

#include "common.cuh"

namespace mlav {

constexpr int SH_ROWS = 128;       // query rows per tile
constexpr int SH_HALF = 128;       // keys per half block
constexpr int SH_TAIL = 128;       // zeroed keys behind the packed space: a half block's overhang
// A tile's cost in steps is its steps plus this: what a segment costs beside
// them (queries in, pipeline fill, last O^T, readout: ~8 us against 3.7 us a step).
constexpr int SH_SEGMENT_COST = 2;
// What the merge of cut tiles costs, in steps (~7 us).
constexpr int SH_JOIN_COST = 2;

// Meta word of a packed key.
constexpr int META_MASKED = -1;            // no row sees it
constexpr int META_SHARED = 0;             // every row of the tile sees it
constexpr int META_POISON = 1 << 30;       // holds a value outside fp16: rows that see it become NaN
// own key of request b: draft -1 for a key before the drafts
__host__ __device__ constexpr int meta_own(int b, int draft) { return b * 64 + 2 + draft; }
constexpr int SH_MAX_BATCH = 1 << 24;
constexpr int SH_MAX_CLUSTERS = 128;   // of the attention kernel (an SM pair each)

struct SharedTile {
  int q_row0, nrows;        // query rows
  int prefix_base, prefix_len;
  int own_base, own_len;
  int halves;               // half blocks of the whole sequence
  int steps;                // (halves + 1) / 2
  int seg0, nseg;           // clusters seg0 .. seg0 + nseg - 1 hold its steps
  int pad[2];
};
static_assert(sizeof(SharedTile) == 48, "three 16-byte loads");

__device__ __forceinline__ int prefix_halves(const SharedTile& t) { return (t.prefix_len + SH_HALF - 1) / SH_HALF; }
// First packed key of half block hb of the tile, and the keys it holds.
__device__ __forceinline__ int half_base(const SharedTile& t, int hb, int& count) {
  const int np = prefix_halves(t);
  if (hb < np) {
    count = min(SH_HALF, t.prefix_len - hb * SH_HALF);
    return t.prefix_base + hb * SH_HALF;
  }
  count = min(SH_HALF, t.own_len - (hb - np) * SH_HALF);
  return t.own_base + (hb - np) * SH_HALF;
}

// Position in the work of a call: step `step` of tile `tile`.
struct SharedPos {
  int tile, step;
};
// A cluster's share of the work, and its first tile (so that its kernel need
// not wait for one load to make the next).
struct SharedShare {
  SharedPos from, to;
  SharedTile first;
};
static_assert(sizeof(SharedShare) == 64, "four 16-byte loads");

struct SharedParams {
  const uint16_t* q;            // bf16 [B * R, 576]
  const uint16_t* kv;           // bf16 [num_slots, 576]
  const int32_t* kv_indices;
  const int32_t* kv_indptr;     // [B + 1]
  const int32_t* kv_lens;       // [B]
  const int32_t* draft_parent;  // [B, T]
  const int32_t* group_indptr;  // [G + 1]
  const int32_t* shared_lens;   // [G]
  float scale_log2;
  int batch, groups, T, H, R;
  int page_size;
  int64_t num_slots;
  int max_kv_len;
  int clusters;                 // of the attention kernel
  int cut_clusters;             // of them that may share tiles: those with partials
  int max_tiles;
  void* out;                    // fp32 or bf16 [B * R, 512]
  float* lse;                   // [B * R]
  int out_bf16;
  int* err;
  int fault_rank;               // testing: the CTA of each pair that gives up in mid-call, -1 for none
  // Workspace.
  uint16_t* q16;                // fp16 [9][q_plane rows][64]
  long long q_plane;            // rows per plane
  uint16_t* k16;                // fp16 [9][k_plane keys][64]
  long long k_plane;
  int* meta;                    // [k_plane]
  int* base;                    // [2 B + 1]: packed base of request b's shared part (its group's first request) and own part
  int* source;                  // [max(B, G)]: per group, the request whose table gives the shared rows
  int* own;                     // [B]: its own rows (>= T), 0 when it cannot be served
  uint32_t* anc;                // [B, T] ancestor masks
  int* tile0;                   // [G] first tile of each group
  int* cost;                    // [max_tiles + 1] prefix sum of the tiles' costs
  SharedTile* tiles;            // [max_tiles]
  SharedShare* share;           // [clusters]
  int* totals;                  // [0] packed keys, [1] tiles
  float* part_o;                // [2 * cut_clusters][128][512], none when that is 1
  float* part_lse;              // [2 * cut_clusters][128]
};

// Partial slot of a segment: a cluster holds at most two tiles that others
// hold parts of, its first and its last.
__device__ __forceinline__ int part_slot(int cluster, bool first) { return 2 * cluster + (first ? 0 : 1); }

}  // namespace mlav
