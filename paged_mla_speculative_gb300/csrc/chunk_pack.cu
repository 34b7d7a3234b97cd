// Preparation of the attention of chunks of new tokens, and the merge after it.
//
// chunk_prepare_kernel, two jobs side by side: CTA 0 lays out the call on the
// device (lengths are device data) -- which requests can be served, their
// place in the packed key space, their query-row tiles, and the division of
// all tiles' steps over the attention kernel's clusters, by sums in closed form
// (chunk_steps.h), so that neither the workspace nor the time grows with the
// tokens: even to a step among the clusters that the plan has partials for
// (SharedParams::cut_clusters, by its verify calls' rows, not by a chunk's), by
// whole tiles among the others; the other CTAs gather the requests' rows into
// fp16 planes of 64 dims as shared_pack.cu's do (each scans the lengths itself).
// Queries are not touched here: the attention kernel widens them in place.
// HBM and L2 are the bound: 1152 bytes read and written a row (117000 rows in
// 42 us); for a few thousand rows it is the chain of the layout, 8 us.
//
// A step's cost counts four, a tile's beginning and end four more, a step of a
// request whose keys at most two tiles read five: with all steps alike, one
// chunk beside 23 decoding requests took 515 us, not 479; with eight for a
// tile's ends 2048 first tokens took 305 us, not 293.
//
// chunk_join_kernel: the LSE merge of the tiles that several clusters share.
#include "shared.cuh"
#include "kernels.h"
#include "pack_rows.cuh"

#include <algorithm>

namespace mlav {
namespace {

constexpr int SMALL = 512;     // requests laid out in shared memory

// What totals[2] and the scan say of a call.
constexpr int CHUNK_BAD_REQUEST = 1, CHUNK_BAD_TOKENS = 2;

__device__ __forceinline__ ChunkSteps chunk_steps(int n, int c, int H) {
  const bool cold = static_cast<long long>(c) * H <= CHUNK_COLD_TILES * SH_ROWS;
  return ChunkSteps(n, c, H, cold ? CHUNK_COLD_STEP : CHUNK_STEP, CHUNK_SEGMENT);
}

struct ChunkLayout {
  int base[SMALL + 1], own[SMALL], tile0[SMALL + 1];
  long long cost[SMALL + 1];
};

// By the whole CTA: own[b] = rows of request b if it is served and has new
// tokens, else 0; base[b] its first packed key, tile0[b] its first tile and
// cost[b] the cost of the tiles before it (either may be null).  `most`
// receives the largest cost of a tile.  Returns CHUNK_BAD_*.
__device__ __forceinline__ int scan_chunks(const SharedParams& p, int* base, int* own, int* tile0, long long* cost, void* s_warp,
                                           int* most, bool report) {
  const int tid = threadIdx.x, B = p.batch;
  bool bad = false;
  int n = 0, ip0 = 0, ip1 = 0, q0 = 0, q1 = 0;
  auto load = [&](int b) {
    n = p.kv_lens[b], ip0 = p.kv_indptr[b], ip1 = p.kv_indptr[b + 1], q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
  };
  const int ipn = p.kv_indptr[B];
  for (int b = tid; b < B; b += PACK_THREADS) {
    load(b);
    bad |= q0 < 0 || q1 < q0 || q1 > p.num_tokens;
  }
  const bool tokens_ok = __syncthreads_or(bad) == 0;
  int errs = tokens_ok ? 0 : ERR_INDPTR, largest = 0;
  int keys = 0, tiles = 0;
  long long total = 0;
  for (int b0 = 0; b0 < B; b0 += PACK_THREADS) {
    const int b = b0 + tid;
    int mine = 0, rows = 0;
    long long sum = 0;
    if (b < B) {
      if (B > PACK_THREADS) load(b);
      const int c = q1 - q0;
      const long long need = p.page_size == 1 ? n : (static_cast<long long>(n) + PAGE - 1) / PAGE;
      const bool len_ok = n >= c && n >= 0 && n <= p.max_kv_len;
      const bool ptr_ok = ip0 >= 0 && ip1 >= ip0 && ip1 <= ipn && static_cast<long long>(ip1) - ip0 == need;
      // (A request without new tokens may hold anything: an idle slot of a batch.)
      if (tokens_ok && c > 0 && !(len_ok && ptr_ok)) errs |= len_ok ? ERR_INDPTR : ERR_LEN;
      if (tokens_ok && c > 0 && len_ok && ptr_ok) {
        const ChunkSteps s = chunk_steps(n, c, p.H);
        mine = n;
        rows = static_cast<int>(s.tiles);
        sum = s.total();
        largest = max(largest, static_cast<int>(s.last) * s.unit + CHUNK_SEGMENT);
      }
      own[b] = mine;
    }
    int all;
    const int end = keys + block_scan(mine, static_cast<int*>(s_warp), all);
    if (b < B) base[b] = end - mine;
    keys += all;
    if (tile0) {
      const int tile_end = tiles + block_scan(rows, static_cast<int*>(s_warp), all);
      if (b < B) tile0[b] = tile_end - rows;
      tiles += all;
      long long all_cost;
      const long long cost_end = total + block_scan(sum, static_cast<long long*>(s_warp), all_cost);
      if (b < B) cost[b] = cost_end - sum;
      total += all_cost;
    }
  }
  if (tid == 0) {
    base[B] = keys;
    if (tile0) tile0[B] = tiles, cost[B] = total;
  }
  if (most && largest) atomicMax(most, largest);
  if (report && errs) atomicOr(p.err, errs);
  const bool any = __syncthreads_or(errs) != 0;
  return !tokens_ok ? CHUNK_BAD_TOKENS : any ? CHUNK_BAD_REQUEST : 0;
}

// CTA 0.
__device__ void plan_chunks(const SharedParams& p, ChunkLayout& s, bool small, void* s_warp) {
  __shared__ int s_most;
  const int tid = threadIdx.x, B = p.batch;
  if (tid == 0) s_most = 0;
  int* base = small ? s.base : p.base;
  int* tile0 = small ? s.tile0 : p.tile0;
  long long* cost = small ? s.cost : p.chunk_cost;
  const int bad = scan_chunks(p, base, small ? s.own : p.own, tile0, cost, s_warp, &s_most, true);
  const int tiles = tile0[B];
  const long long total = cost[B];
  if (small)
    for (int b = tid; b <= B; b += PACK_THREADS) {
      p.base[b] = base[b];
      p.tile0[b] = tile0[b];
    }
  if (tid == 0) {
    p.totals[0] = base[B];
    p.totals[1] = tiles;
    p.totals[2] = bad;
  }
  // Even division over as many clusters as get two steps or more each, as far
  // as there are partials: with a plan of few verify rows the last shares are
  // whole tiles, and few long tiles do not fill the clusters (32 tokens of 64 heads
  // behind 32768 rows: 448 us with a plan of one draft, 129 with one of four).
  // Starts lie at least LEAST apart, so no two start in one tile's leading cost
  // or in one step; those of clusters without partials move up to a
  // tile's border (and some clusters may be left without work).  Where every
  // tile can have a cluster of its own and the longest takes no more than an
  // even share, cut tiles starting twice, and the merge, tiles stay whole.
  constexpr int LEAST = CHUNK_SEGMENT + 2 * CHUNK_COLD_STEP;
  const int used = static_cast<int>(max(1LL, min(static_cast<long long>(p.clusters), total / LEAST)));
  const bool whole = tiles <= p.clusters && s_most <= total / p.clusters + CHUNK_SEGMENT + SH_JOIN_COST * CHUNK_STEP;
  // Starts, and the requests of their tiles.
  __shared__ SharedPos s_start[SH_MAX_CLUSTERS + 1];
  __shared__ int s_request[SH_MAX_CLUSTERS + 1];
  for (int c = tid; c <= p.clusters; c += PACK_THREADS) {
    SharedPos at{tiles, 0};
    int request = B;
    if (whole) {
      at.tile = min(c, tiles);
      if (at.tile < tiles) request = last_not_above(tile0, B, at.tile);
    } else if (c < used && total > 0) {
      const long long x = total * c / used;
      request = last_not_above(cost, B, x);
      const int q0 = p.q_indptr[request];
      const ChunkSteps st = chunk_steps(p.kv_lens[request], p.q_indptr[request + 1] - q0, p.H);
      const long long t = st.tile_at(x - cost[request]);
      at.tile = tile0[request] + static_cast<int>(t);
      at.step = static_cast<int>(max(0LL, x - cost[request] - st.before(t) - CHUNK_SEGMENT) / st.unit);
      if (at.step > 0 && c >= p.cut_clusters) {
        at = SharedPos{at.tile + 1, 0};
        request = at.tile < tiles ? last_not_above(tile0, B, at.tile) : B;
      }
    }
    s_start[c] = at;
    s_request[c] = request;
  }
  __syncthreads();
  for (int c = tid; c < p.clusters; c += PACK_THREADS) {
    SharedShare sh{};
    sh.from = s_start[c];
    sh.to = s_start[c + 1];
    const int request = s_request[c];
    if (sh.from.tile < tiles) sh.first = chunk_tile(p, request, sh.from.tile - tile0[request], base[request]);
    p.share[c] = sh;
  }
}

// `plans` CTAs (1 or 0) lay out the call, the others gather keys.
__global__ void __launch_bounds__(PACK_THREADS, 4) chunk_prepare_kernel(const SharedParams p, int plans) {
  __shared__ ChunkLayout s;
  __shared__ long long s_warp[PACK_THREADS / 32];
  __shared__ long long s_row[2][PACK_KEYS];
  __shared__ int s_meta[2][PACK_KEYS], s_bad[2][PACK_KEYS];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const bool small = p.batch <= SMALL;
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) < plans) {
    plan_chunks(p, s, small, s_warp);
    return;
  }
  const int packer = static_cast<int>(blockIdx.x) - plans, packers = static_cast<int>(gridDim.x) - plans;
  const int* base = small ? s.base : p.base;
  const int* own = small ? s.own : p.own;
  const int bad = small ? scan_chunks(p, s.base, s.own, nullptr, nullptr, s_warp, nullptr, false) : p.totals[2];
  const int total = base[p.batch];
  const int chunks = (total + SH_TAIL + PACK_KEYS - 1) / PACK_KEYS;
  // The slot and meta word of each key of a chunk, by the first warp.
  auto look_up = [&](int chunk, int buf) {
    if (tid >= PACK_KEYS) return;
    const int key = chunk * PACK_KEYS + tid;
    long long row = -1;
    int meta = META_MASKED;
    if (key < total) {
      const int b = last_not_above(base, p.batch, key), j = key - base[b];
      meta = META_SHARED;
      const long long entry = p.kv_indices[p.kv_indptr[b] + (p.page_size == 1 ? j : j / PAGE)];
      row = p.page_size == 1 ? entry : entry * PAGE + j % PAGE;
      if (entry < 0 || row >= p.num_slots) {
        atomicOr(p.err, ERR_SLOT);
        row = -1;
        meta = META_MASKED;
      }
    }
    s_row[buf][tid] = row;
    s_meta[buf][tid] = meta;
    s_bad[buf][tid] = 0;
  };
  int buf = 0;
  if (packer < chunks) look_up(packer, 0);
  __syncthreads();
  for (int chunk = packer; chunk < chunks; chunk += packers, buf ^= 1) {
    const int key0 = chunk * PACK_KEYS, rows = min(PACK_KEYS, total + SH_TAIL - key0);
    Rows x;
    load_rows(p.kv, s_row[buf], x);
    if (chunk + packers < chunks) look_up(chunk + packers, buf ^ 1);   // while the rows arrive
    report_range(store_rows(x, s_bad[buf], p.k16, p.k_plane, key0, rows), p.err);
    __syncthreads();
    if (tid < rows) p.meta[key0 + tid] = s_meta[buf][tid] | (s_bad[buf][tid] ? META_POISON : 0);
  }
  if (bad == 0) return;
  // NaN for the tokens of requests that are not served (all tokens, when
  // q_indptr does not divide them).
  const float nan = __int_as_float(0x7fc00000);
  auto fill = [&](long long row0, long long row1) {
    for (long long row = row0 + packer; row < row1; row += packers)
      for (int col = tid; col < D_V / 4; col += PACK_THREADS)
        store_merged(p, row, col, make_float4(nan, nan, nan, nan), nan);
  };
  if (bad == CHUNK_BAD_TOKENS) {
    fill(0, static_cast<long long>(p.num_tokens) * p.H);
    return;
  }
  for (int b = 0; b < p.batch; ++b)
    if (own[b] == 0) fill(static_cast<long long>(p.q_indptr[b]) * p.H, static_cast<long long>(p.q_indptr[b + 1]) * p.H);
}

// Tiles that several clusters hold parts of: CTAs CHUNK_JOIN_CTAS c .. merge
// the tile that cluster c is the first of several to hold, 128 threads per
// row.  Parts were just written and mostly come from L2.
constexpr int JOIN_ROWS = 2;
constexpr int JOIN_CTAS = SH_ROWS / JOIN_ROWS;

__global__ void __launch_bounds__(JOIN_ROWS * 128) chunk_join_kernel(const SharedParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int c = blockIdx.x / JOIN_CTAS;
  const SharedPos from = p.share[c].from, to = p.share[c].to;
  const int tile = to.tile;
  if (to.step == 0 || (from.tile == tile && from.step > 0)) return;   // its last tile is whole, or another cluster's
  int nseg = 1;
  while (c + nseg < p.clusters && p.share[c + nseg].from.tile == tile && p.share[c + nseg].from.step > 0) ++nseg;
  const SharedShare& next = p.share[c + 1];   // starts in the tile: has its record
  const int r = (blockIdx.x % JOIN_CTAS) * JOIN_ROWS + (threadIdx.x >> 7), col = threadIdx.x & 127;
  if (r >= next.first.nrows) return;
  const int slot0 = part_slot(c, from.tile == tile);
  auto at = [&](int s) { return static_cast<size_t>(s ? part_slot(c + s, true) : slot0) * SH_ROWS + r; };
  float4 acc;
  float lse;
  merge_parts(p, nseg, at, col, acc, lse);
  store_merged(p, next.first.q_row0 + r, col, acc, lse);
}

}  // namespace

cudaError_t launch_chunk_prepare(const SharedParams& p, int num_sms, cudaStream_t stream) {
  if (p.clusters > SH_MAX_CLUSTERS) return cudaErrorInvalidValue;
  const long long most = static_cast<long long>(p.batch) * p.max_kv_len + SH_TAIL;
  // Packers: one resident wave (four CTAs per SM).
  const unsigned packers = static_cast<unsigned>(std::min<long long>((most + PACK_KEYS - 1) / PACK_KEYS, 4LL * num_sms - 1));
  if (p.batch <= SMALL) return launch_overlapping(chunk_prepare_kernel, dim3(1 + packers), PACK_THREADS, 0, stream, 1, p, 1);
  const cudaError_t e = launch_overlapping(chunk_prepare_kernel, dim3(1), PACK_THREADS, 0, stream, 1, p, 1);
  return e != cudaSuccess ? e : launch_overlapping(chunk_prepare_kernel, dim3(packers), PACK_THREADS, 0, stream, 1, p, 0);
}

cudaError_t launch_chunk_join(const SharedParams& p, cudaStream_t stream) {
  // (The last cluster's share ends with a tile.)
  const unsigned ctas = static_cast<unsigned>(std::max(1, std::min(p.cut_clusters, p.clusters - 1))) * JOIN_CTAS;
  return launch_overlapping(chunk_join_kernel, dim3(ctas), JOIN_ROWS * 128, 0, stream, 1, p);
}

}  // namespace mlav
