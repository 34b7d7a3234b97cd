// Preparation of the shared-prefix verify attention, and the merge after it.
//
// shared_prepare_kernel, three jobs side by side:
//  * CTA 0 (and 1, the ancestor masks) lays out the call on the device (lengths are device data): which
//    requests can be served, each group's shared range and each request's own
//    range in the packed key space, the query-row tiles, and the division of
//    all tiles' steps over the attention kernel's clusters, even to a step, so
//    that one long prompt or many short ones fill the GPU alike;
//  * some CTAs widen the queries (bf16 to fp16, planes of 64 dims);
//  * the others gather each distinct row once -- shared rows once per group,
//    not once per request -- and widen it into fp16 planes of 64 dims, which
//    the attention kernel reads by TMA (any 128 consecutive keys are one box).
//    Values that have no fp16 counterpart are packed as zero and marked in the
//    key's meta word, so that only rows that see the key are affected.
//  The packers need the packed bases only: each scans the batch's lengths
//  itself (about 2 us, in shared memory) instead of waiting for CTA 0, which
//  took 7 us in a launch of its own.  Batches beyond SMALL requests are
//  planned first and packed by a second launch that reads CTA 0's arrays.
//  HBM and L2 are the bound of the packing: 1152 bytes read and written a row.
//
// shared_join_kernel: the LSE merge of the tiles that several clusters share.
#include "shared.cuh"
#include "kernels.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

namespace mlav {
namespace {

constexpr int THREADS = 256;
constexpr int PACK_KEYS = 32;                                   // rows per CTA iteration
constexpr int PER_THREAD = PACK_KEYS * ROW_CHUNKS / THREADS;    // 9 granules
static_assert(PER_THREAD * THREADS == PACK_KEYS * ROW_CHUNKS, "even split");
constexpr int SMALL = 512;     // requests, groups and tiles laid out in shared memory

// Inclusive block scan; `all` receives the block's total.
__device__ __forceinline__ int block_scan(int x, int* s_warp, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) x += all;
    all += s_warp[w];
  }
  return x;
}

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The groups of a call; when they do not partition the batch: one group, and
// no request is served.
struct Groups {
  const int32_t* indptr;
  const int32_t* shared_lens;
  int n, batch;
  bool ok;
  __device__ __forceinline__ int begin(int g) const { return ok ? indptr[g] : (g ? batch : 0); }
  __device__ __forceinline__ int of(int b) const { return ok ? last_not_above(indptr, n, b) : 0; }
};

// Own rows, packed bases and each group's source request, by the whole CTA;
// returns the packed keys.  `report`: set the error bits of what cannot be served.
// `indptr` and `lens`: copies of the groups' arrays to keep using, or the
// arrays themselves.  (Beside the packers' loads a dependent load takes up to
// 2 us: a small call makes one round of them and goes on in shared memory.)
__device__ __forceinline__ int scan_requests(const SharedParams& p, int* own, int* base, int* source, int* indptr, int* lens,
                                             int* s_warp, Groups& grp, bool report) {
  const int tid = threadIdx.x, B = p.batch;
  bool bad = false;
  // The first round's loads go out before the groups are known.
  int n = 0, ip0 = 0, ip1 = 0;
  const int ipn = p.kv_indptr[B];
  if (tid < B) n = p.kv_lens[tid], ip0 = p.kv_indptr[tid], ip1 = p.kv_indptr[tid + 1];
  for (int g = tid; g < p.groups; g += THREADS) {
    const int a = p.group_indptr[g], z = p.group_indptr[g + 1];
    bad |= z < a || (g == 0 && a != 0) || (g == p.groups - 1 && z != B);
    source[g] = INT_MAX;
    if (indptr) {
      indptr[g] = a;
      lens[g] = p.shared_lens[g];
      if (g == p.groups - 1) indptr[g + 1] = z;
    }
  }
  const bool groups_ok = __syncthreads_or(bad) == 0;
  grp = Groups{indptr ? indptr : p.group_indptr, indptr ? lens : p.shared_lens, groups_ok ? p.groups : 1, B, groups_ok};
  int errs = groups_ok ? 0 : ERR_INDPTR;
  for (int b = tid; b < B; b += THREADS) {
    const int g = grp.of(b);
    if (b >= THREADS) n = p.kv_lens[b], ip0 = p.kv_indptr[b], ip1 = p.kv_indptr[b + 1];
    const long long need = p.page_size == 1 ? n : (static_cast<long long>(n) + PAGE - 1) / PAGE;
    const int S = groups_ok ? grp.shared_lens[g] : 0;
    const bool len_ok = n >= p.T && n <= p.max_kv_len && S >= 0 && S <= n - p.T;
    const bool ptr_ok = ip0 >= 0 && ip1 >= ip0 && ip1 <= ipn && static_cast<long long>(ip1) - ip0 == need;
    const bool ok = groups_ok && len_ok && ptr_ok;
    if (!len_ok) errs |= ERR_LEN;
    else if (!ptr_ok) errs |= ERR_INDPTR;
    own[b] = ok ? n - S : 0;           // at least T
    if (ok) atomicMin(source + g, b);
  }
  if (report && errs) atomicOr(p.err, errs);
  __syncthreads();
  int before = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + tid;
    int prefix = 0, mine = 0;
    if (b < B) {
      const int g = grp.of(b);
      mine = own[b];
      if (b == grp.begin(g) && *static_cast<volatile int*>(source + g) != INT_MAX) prefix = grp.shared_lens[g];
    }
    int all;
    const int end = before + block_scan(prefix + mine, s_warp, all);
    if (b < B) {
      base[2 * b] = end - mine - prefix;
      base[2 * b + 1] = end - mine;
    }
    before += all;
  }
  if (tid == 0) base[2 * B] = before;
  __syncthreads();
  return before;
}

struct Layout {
  int own[SMALL], base[2 * SMALL + 1], source[SMALL], indptr[SMALL + 1], lens[SMALL];
};
struct PlanLayout {
  Layout l;
  int tile0[SMALL], cost[SMALL + 1];
  SharedTile tiles[SMALL];
  SharedPos start[SH_MAX_CLUSTERS + 1];
};

// CTA 1.  Ancestor masks: a warp holds a request's parents and walks them by
// shuffles (walking them in global memory took a load per level).
__device__ __forceinline__ void plan_ancestors(const SharedParams& p) {
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < p.batch; b += THREADS / 32) {
    const int par = lane < p.T ? p.draft_parent[static_cast<size_t>(b) * p.T + lane] : -1;
    if (par < -1 || par >= lane + (lane < p.T ? 0 : 1)) atomicOr(p.err, ERR_PARENT);
    const int up = par >= lane ? -1 : par;
    uint32_t mask = 1u << lane;
    int cur = up;
    for (int it = 1; it < p.T; ++it) {
      if (cur >= 0) mask |= 1u << cur;
      const int next = __shfl_sync(0xffffffffu, up, max(cur, 0));
      cur = cur >= 0 ? next : -1;
    }
    if (lane < p.T) p.anc[static_cast<size_t>(b) * p.T + lane] = mask;
  }
}

// CTA 0.  Arrays that others read go to the workspace; the ones used here
// only, and those of a small call, are in shared memory.
__device__ void plan_call(const SharedParams& p, PlanLayout& s, bool small, int* s_warp) {
  __shared__ int s_max;
  const int tid = threadIdx.x, B = p.batch, lane = tid & 31;
  if (tid == 0) s_max = 0;
  int* own = small ? s.l.own : p.own;
  int* base = small ? s.l.base : p.base;
  Groups grp;
  const int keys = scan_requests(p, own, base, small ? s.l.source : p.source, small ? s.l.indptr : nullptr, s.l.lens, s_warp, grp,
                                 true);
  if (small)
    for (int b = tid; b < B; b += THREADS) p.own[b] = own[b];
  // Tiles of each group.
  const int G = grp.n;
  int* tile0 = small ? s.tile0 : p.tile0;
  int tiles = 0;
  for (int g0 = 0; g0 < G; g0 += THREADS) {
    const int g = g0 + tid;
    int n = 0;
    if (g < G) n = static_cast<int>((static_cast<long long>(grp.begin(g + 1) - grp.begin(g)) * p.R + SH_ROWS - 1) / SH_ROWS);
    int all;
    const int end = tiles + block_scan(n, s_warp, all);
    if (g < G) tile0[g] = end - n;
    tiles += all;
  }
  if (tid == 0) {
    p.totals[0] = keys;
    p.totals[1] = tiles;
  }
  __syncthreads();
  // Tile records and the prefix sum of their costs.
  int* cost = tiles <= SMALL ? s.cost : p.cost;
  SharedTile* recs = tiles <= SMALL ? s.tiles : p.tiles;
  int total = 0, most = 0;
  for (int t0 = 0; t0 < tiles; t0 += THREADS) {
    const int t = t0 + tid;
    SharedTile rec{};
    int c = 0;
    if (t < tiles) {
      const int g = last_not_above(tile0, G, t);
      const int first = grp.begin(g) * p.R, rows = grp.begin(g + 1) * p.R - first;
      const int off = (t - tile0[g]) * SH_ROWS;
      rec.q_row0 = first + off;
      rec.nrows = min(SH_ROWS, rows - off);
      const int b0 = rec.q_row0 / p.R, b1 = (rec.q_row0 + rec.nrows - 1) / p.R;
      rec.own_base = base[2 * b0 + 1];
      rec.own_len = base[2 * b1 + 1] + own[b1] - rec.own_base;
      if (rec.own_len > 0) {       // some request of the tile is served
        rec.prefix_base = base[2 * grp.begin(g)];
        rec.prefix_len = grp.shared_lens[g];
        rec.halves = prefix_halves(rec) + (rec.own_len + SH_HALF - 1) / SH_HALF;
        rec.steps = (rec.halves + 1) / 2;
        c = rec.steps + SH_SEGMENT_COST;
      }
    }
    most = max(most, c);
    int all;
    const int end = total + block_scan(c, s_warp, all);
    if (t < tiles) {
      recs[t] = rec;
      cost[t] = end - c;
    }
    total += all;
  }
  for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) atomicMax(&s_max, most);
  if (tid == 0) cost[tiles] = total;
  __syncthreads();
  // Even division over as many clusters as get two steps or more each.
  // Starts lie at least SH_SEGMENT_COST + 2 apart, so no used cluster is
  // empty and no two start in one tile's leading cost.  Where every tile can
  // have a cluster of its own and the longest takes no more than an even
  // share, cut tiles starting twice, and the merge, tiles stay whole.
  int used = max(1, min(p.cut_clusters, total / (SH_SEGMENT_COST + 2)));
  const bool whole = tiles <= p.clusters && s_max <= total / p.clusters + SH_SEGMENT_COST + SH_JOIN_COST;
  if (whole) used = tiles;
  for (int c = tid; c <= p.clusters; c += THREADS) {
    SharedPos at{tiles, 0};
    if (whole) {
      at.tile = min(c, tiles);
    } else if (c < used && total > 0) {
      const int x = static_cast<int>(static_cast<long long>(total) * c / used);
      at.tile = last_not_above(cost, tiles, x);
      at.step = max(0, x - cost[at.tile] - SH_SEGMENT_COST);
    }
    s.start[c] = at;
  }
  __syncthreads();
  for (int c = tid; c < p.clusters; c += THREADS) {
    SharedShare sh{};
    sh.from = s.start[c];
    sh.to = s.start[c + 1];
    if (sh.from.tile < tiles) sh.first = recs[sh.from.tile];
    p.share[c] = sh;
  }
  // Which clusters hold each tile.
  for (int t = tid; t < tiles; t += THREADS) {
    const int c = cost[t + 1] - cost[t];
    SharedTile rec = recs[t];
    if (c > 0) {
      // Last cluster that starts at or before step `step` of the tile.
      auto last_before = [&](int step) {
        int lo = 0, hi = used;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          const SharedPos at = s.start[mid];
          if (at.tile < t || (at.tile == t && at.step <= step)) lo = mid;
          else hi = mid;
        }
        return lo;
      };
      rec.seg0 = whole ? t : last_before(0);
      rec.nseg = whole ? 1 : last_before(c - SH_SEGMENT_COST - 1) - rec.seg0 + 1;
    }
    p.tiles[t] = rec;
  }
}

struct Rows {
  uint4 v[PER_THREAD];
};
// A granule that the call reads once.  (No read-only load: those are for
// memory that nothing writes while the kernel runs, and this one is launched
// while the kernel before it may still write its inputs.)
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
// Row r of 32 (each THREADS / 8 granules apart) at src + s_row[r] * 576, or
// zeros where s_row is negative.
__device__ __forceinline__ void load_rows(const uint16_t* src, const long long* s_row, Rows& x) {
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * THREADS;
    const int r = e / ROW_CHUNKS, c = e - r * ROW_CHUNKS;
    const long long row = s_row[r];
    x.v[u] = row >= 0 ? load_once(reinterpret_cast<const uint4*>(src + row * D_QK) + c) : make_uint4(0, 0, 0, 0);
  }
}
// Widened into the planes at plane rows row0 .. row0 + rows - 1.  A value
// outside fp16 is packed as zero and sets s_bad of its row; returns whether
// this thread met one.
__device__ __forceinline__ bool store_rows(const Rows& x, int* s_bad, uint16_t* dst, long long plane, long long row0, int rows) {
  bool any = false;
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * THREADS;
    const int r = e / ROW_CHUNKS, c = e - r * ROW_CHUNKS;
    bool bad = false;
    uint4 w = widen_bf16x8(x.v[u], bad);
    if (bad) {
      any = true;
      s_bad[r] = 1;
      uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((h[k] & 0x7c00u) == 0x7c00u) h[k] &= 0xffff0000u;
        if ((h[k] & 0x7c000000u) == 0x7c000000u) h[k] &= 0x0000ffffu;
      }
      w = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (r < rows) *reinterpret_cast<uint4*>(dst + ((c >> 3) * plane + row0 + r) * 64 + (c & 7) * 8) = w;
  }
  return any;
}

// `packers` CTAs (the last of the grid) gather keys, those before them widen
// queries, the first `plans` (2 or 0) lay out the call.
__global__ void __launch_bounds__(THREADS, 4) shared_prepare_kernel(const SharedParams p, int plans, int packers) {
  __shared__ PlanLayout s;
  __shared__ int s_warp[THREADS / 32];
  __shared__ long long s_row[2][PACK_KEYS];
  __shared__ int s_meta[2][PACK_KEYS], s_bad[2][PACK_KEYS];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const bool small = p.batch <= SMALL && p.groups <= SMALL;
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) < plans) {
    if (blockIdx.x == 0) plan_call(p, s, small, s_warp);
    else plan_ancestors(p);
    return;
  }
  const int packer = static_cast<int>(blockIdx.x) - (static_cast<int>(gridDim.x) - packers);
  if (packer < 0) {
    // Queries: 32 rows per CTA, nine granules per thread.
    const long long rows = static_cast<long long>(p.batch) * p.R;
    const long long row0 = static_cast<long long>(static_cast<int>(blockIdx.x) - plans) * PACK_KEYS;
    bool bad = false;
    uint4 v[PER_THREAD];
#pragma unroll
    for (int u = 0; u < PER_THREAD; ++u) {
      const int e = tid + u * THREADS;
      const long long row = row0 + e / ROW_CHUNKS;
      v[u] = row < rows ? load_once(reinterpret_cast<const uint4*>(p.q + row * D_QK) + e % ROW_CHUNKS) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < PER_THREAD; ++u) {
      const int e = tid + u * THREADS;
      const long long row = row0 + e / ROW_CHUNKS;
      const int c = e % ROW_CHUNKS;
      if (row < rows)
        *reinterpret_cast<uint4*>(p.q16 + ((c >> 3) * p.q_plane + row) * 64 + (c & 7) * 8) = widen_bf16x8(v[u], bad);
    }
    report_range(bad, p.err);
    return;
  }
  int total;
  Groups grp;
  if (small) {
    total = scan_requests(p, s.l.own, s.l.base, s.l.source, s.l.indptr, s.l.lens, s_warp, grp, false);
  } else {
    total = p.totals[0];
    grp = Groups{p.group_indptr, p.shared_lens, p.groups, p.batch, true};   // (no key of a group that is none is packed)
  }
  const int* own = small ? s.l.own : p.own;
  const int* base = small ? s.l.base : p.base;
  const int* source = small ? s.l.source : p.source;
  const int chunks = (total + SH_TAIL + PACK_KEYS - 1) / PACK_KEYS;
  // The slot and meta word of each key of a chunk, by the first warp.
  auto look_up = [&](int chunk, int buf) {
    if (tid >= PACK_KEYS) return;
    const int key = chunk * PACK_KEYS + tid;
    long long row = -1;
    int meta = META_MASKED;
    if (key < total) {
      const int part = last_not_above(base, 2 * p.batch, key);
      int b = part >> 1, j = key - base[part];
      if (part & 1) {
        const int n = p.kv_lens[b];
        j += n - own[b];                            // behind the shared rows
        meta = meta_own(b, max(-1, j - (n - p.T)));
      } else {
        b = source[grp.of(b)];
        meta = META_SHARED;
      }
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
}

// Rows of tiles that several clusters hold parts of (or none: no request of
// the tile is served): 128 threads per row, a float4 of each part per thread,
// up to JOIN_FLIGHT parts loaded before any is used.  A row's parts were just
// written and mostly come from L2; the launch and one round trip are the time.
constexpr int JOIN_ROWS = 2;
constexpr int JOIN_FLIGHT = 8;
constexpr int JOIN_MAX = SH_MAX_CLUSTERS / 32;   // parts per lane

__global__ void __launch_bounds__(JOIN_ROWS * 128) shared_join_kernel(const SharedParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int tile = blockIdx.x / (SH_ROWS / JOIN_ROWS);
  if (tile >= p.totals[1]) return;
  const SharedTile t = p.tiles[tile];
  const int lane = threadIdx.x & 31, col = threadIdx.x & 127;
  const int r = (blockIdx.x % (SH_ROWS / JOIN_ROWS)) * JOIN_ROWS + (threadIdx.x >> 7);
  if (t.nseg == 1 || r >= t.nrows) return;
  const int row = t.q_row0 + r;
  const float nan = __int_as_float(0x7fc00000);
  float4 acc = make_float4(nan, nan, nan, nan);
  float lse = nan;
  if (t.nseg > 1 && p.own[row / p.R] > 0) {
    // The first part is its cluster's first segment if the cluster starts
    // with the tile; the others begin inside it, hence with it.
    const SharedPos from = p.share[t.seg0].from;
    const int slot0 = part_slot(t.seg0, from.tile == tile);
    auto at = [&](int s) { return static_cast<size_t>(s ? part_slot(t.seg0 + s, true) : slot0) * SH_ROWS + r; };
    float L[JOIN_MAX], mx = -INFINITY;
    bool any_nan = false;
#pragma unroll
    for (int k = 0; k < JOIN_MAX; ++k) {
      L[k] = 32 * k + lane < t.nseg ? p.part_lse[at(32 * k + lane)] : -INFINITY;
      any_nan |= L[k] != L[k];
      mx = fmaxf(mx, L[k]);
    }
    any_nan = __any_sync(0xffffffffu, any_nan);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float top = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < JOIN_MAX; ++k) {
      L[k] = ex2((L[k] - top) * kLog2e);
      sum += L[k];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // Every key masked (bad slots): weight 0 everywhere.
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < JOIN_MAX; ++k) {
      for (int s0 = 32 * k; s0 < min(t.nseg, 32 * k + 32); s0 += JOIN_FLIGHT) {
        float4 x[JOIN_FLIGHT];
#pragma unroll
        for (int f = 0; f < JOIN_FLIGHT; ++f)
          if (s0 + f < t.nseg) x[f] = __ldcs(reinterpret_cast<const float4*>(p.part_o + at(s0 + f) * D_V) + col);
#pragma unroll
        for (int f = 0; f < JOIN_FLIGHT; ++f) {
          const float w = __shfl_sync(0xffffffffu, L[k], (s0 + f) & 31) * inv;
          if (s0 + f >= t.nseg || w == 0.f) continue;   // (a part of weight 0 may hold anything)
          acc.x += w * x[f].x;
          acc.y += w * x[f].y;
          acc.z += w * x[f].z;
          acc.w += w * x[f].w;
        }
      }
    }
    lse = sum > 0.f ? top + logf(sum) : -INFINITY;
    if (any_nan) {
      acc = make_float4(nan, nan, nan, nan);
      lse = nan;
    }
  }
  const size_t at = static_cast<size_t>(row) * (D_V / 4) + col;
  if (p.out_bf16) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
    reinterpret_cast<uint2*>(p.out)[at] = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  } else {
    reinterpret_cast<float4*>(p.out)[at] = acc;
  }
  if (col == 0) p.lse[row] = lse;
}

}  // namespace

cudaError_t launch_shared_prepare(const SharedParams& p, int num_sms, cudaStream_t stream) {
  if (p.clusters > SH_MAX_CLUSTERS) return cudaErrorInvalidValue;
  auto grid = [](long long ctas) { return dim3(static_cast<unsigned>(ctas)); };
  const long long rows = static_cast<long long>(p.batch) * p.R;
  const long long query_ctas = (rows + PACK_KEYS - 1) / PACK_KEYS;
  const long long most = static_cast<long long>(p.batch) * p.max_kv_len + SH_TAIL;
  // Packers: what the query CTAs leave of one resident wave (four CTAs per
  // SM), so that none starts when the others are done.
  const long long wave = std::max(2LL * num_sms, 4LL * num_sms - 2 - query_ctas);
  const int packers = static_cast<int>(std::min<long long>((most + PACK_KEYS - 1) / PACK_KEYS, wave));
  if (p.batch <= SMALL && p.groups <= SMALL)
    return launch_overlapping(shared_prepare_kernel, grid(2 + query_ctas + packers), THREADS, 0, stream, 1, p, 2, packers);
  const cudaError_t e = launch_overlapping(shared_prepare_kernel, grid(2 + query_ctas), THREADS, 0, stream, 1, p, 2, 0);
  return e != cudaSuccess ? e : launch_overlapping(shared_prepare_kernel, grid(packers), THREADS, 0, stream, 1, p, 0, packers);
}

cudaError_t launch_shared_join(const SharedParams& p, cudaStream_t stream) {
  const unsigned ctas = static_cast<unsigned>(p.max_tiles) * (SH_ROWS / JOIN_ROWS);
  return launch_overlapping(shared_join_kernel, dim3(ctas), JOIN_ROWS * 128, 0, stream, 1, p);
}

}  // namespace mlav
