// Planning and packing of the shared-prefix verify attention.
//
// shared_plan_kernel: CTA 0 lays out the call on the device (lengths are
// device data): which requests can be served, each group's shared range and
// each request's own range in the packed key space, the query-row tiles, and
// the division of all tiles' steps over the attention kernel's clusters, even
// to a step, so that one long prompt or many short ones fill the GPU alike.
// The other CTAs widen the queries meanwhile (bf16 to fp16, planes of 64 dims).
//
// shared_pack_kernel: gathers each distinct row once -- shared rows once per
// group, not once per request -- and widens it into fp16 planes of 64 dims,
// which the attention kernel reads by TMA (any 128 consecutive keys are one
// box).  Values that have no fp16 counterpart are packed as zero and marked in
// the key's meta word, so that only rows that see the key are affected.
//
// shared_join_kernel: the LSE merge of the tiles that several clusters share.
#include "shared.cuh"
#include "kernels.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

namespace mlav {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PACK_THREADS = 256;
constexpr int PACK_KEYS = 32;                                        // rows per CTA iteration
constexpr int PER_THREAD = PACK_KEYS * ROW_CHUNKS / PACK_THREADS;    // 9 granules
static_assert(PER_THREAD * PACK_THREADS == PACK_KEYS * ROW_CHUNKS, "even split");

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
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return x + (warp ? before : 0);
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

__device__ void plan_call(const SharedParams& p) {
  __shared__ int s_warp[PLAN_THREADS / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, B = p.batch;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  int bad = 0;
  for (int g = tid; g < p.groups; g += PLAN_THREADS) {
    if (p.group_indptr[g + 1] < p.group_indptr[g]) bad = 1;
    if (g == 0 && (p.group_indptr[0] != 0 || p.group_indptr[p.groups] != B)) bad = 1;
  }
  if (bad) s_bad = 1;
  for (int b = tid; b < max(B, p.groups); b += PLAN_THREADS) p.source[b] = INT_MAX;
  __syncthreads();
  // Groups that do not partition the batch: one group, no request served.
  const bool groups_ok = s_bad == 0;
  const int G = groups_ok ? p.groups : 1;
  auto group_begin = [&](int g) { return groups_ok ? p.group_indptr[g] : (g ? B : 0); };
  if (!groups_ok && tid == 0) atomicOr(p.err, ERR_INDPTR);

  // Requests: can each be served?
  int errs = 0;
  for (int b = tid; b < B; b += PLAN_THREADS) {
    const int g = groups_ok ? last_not_above(p.group_indptr, G, b) : 0;
    const int n = p.kv_lens[b], ip0 = p.kv_indptr[b], ip1 = p.kv_indptr[b + 1], ipn = p.kv_indptr[B];
    const long long need = p.page_size == 1 ? n : (static_cast<long long>(n) + PAGE - 1) / PAGE;
    const int S = groups_ok ? p.shared_lens[g] : 0;
    const bool len_ok = n >= p.T && n <= p.max_kv_len && S >= 0 && S <= n - p.T;
    const bool ptr_ok = ip0 >= 0 && ip1 >= ip0 && ip1 <= ipn && static_cast<long long>(ip1) - ip0 == need;
    const bool ok = groups_ok && len_ok && ptr_ok;
    if (!len_ok) errs |= ERR_LEN;
    else if (!ptr_ok) errs |= ERR_INDPTR;
    p.group_of[b] = g;
    p.own[b] = ok ? n - S : 0;         // at least T
    if (ok) atomicMin(p.source + g, b);
  }
  if (errs) atomicOr(p.err, errs);
  for (int i = tid; i < B * p.T; i += PLAN_THREADS)
    p.anc[i] = ancestor_mask(p.draft_parent + static_cast<size_t>(i / p.T) * p.T, i % p.T, p.err);
  __syncthreads();

  // Packed bases, in request order.
  int before = 0;
  for (int b0 = 0; b0 < B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    int prefix = 0, own = 0;
    if (b < B) {
      const int g = p.group_of[b];
      own = p.own[b];
      if (b == group_begin(g) && __ldcg(p.source + g) != INT_MAX) prefix = p.shared_lens[g];
    }
    int all;
    const int end = before + block_scan(prefix + own, s_warp, all);
    if (b < B) {
      p.base[2 * b] = end - own - prefix;
      p.base[2 * b + 1] = end - own;
    }
    before += all;
  }
  if (tid == 0) {
    p.base[2 * B] = before;
    p.totals[0] = before;
  }
  // Tiles of each group.
  int tiles = 0;
  for (int g0 = 0; g0 < G; g0 += PLAN_THREADS) {
    const int g = g0 + tid;
    int n = 0;
    if (g < G) n = static_cast<int>((static_cast<long long>(group_begin(g + 1) - group_begin(g)) * p.R + SH_ROWS - 1) / SH_ROWS);
    int all;
    const int end = tiles + block_scan(n, s_warp, all);
    if (g < G) p.tile0[g] = end - n;
    tiles += all;
  }
  if (tid == 0) p.totals[1] = tiles;
  __syncthreads();
  // Tile records and the prefix sum of their costs.
  int cost = 0;
  for (int t0 = 0; t0 < tiles; t0 += PLAN_THREADS) {
    const int t = t0 + tid;
    SharedTile rec{};
    int c = 0;
    if (t < tiles) {
      const int g = last_not_above(p.tile0, G, t);
      const int first = group_begin(g) * p.R, rows = group_begin(g + 1) * p.R - first;
      const int off = (t - p.tile0[g]) * SH_ROWS;
      rec.q_row0 = first + off;
      rec.nrows = min(SH_ROWS, rows - off);
      rec.b0 = rec.q_row0 / p.R;
      const int b1 = (rec.q_row0 + rec.nrows - 1) / p.R;
      rec.own_base = p.base[2 * rec.b0 + 1];
      rec.own_len = p.base[2 * b1 + 1] + p.own[b1] - rec.own_base;
      if (rec.own_len > 0) {       // some request of the tile is served
        rec.prefix_base = p.base[2 * group_begin(g)];
        rec.prefix_len = p.shared_lens[g];
        rec.halves = prefix_halves(rec) + (rec.own_len + SH_HALF - 1) / SH_HALF;
        rec.steps = (rec.halves + 1) / 2;
        c = rec.steps + SH_SEGMENT_COST;
      }
    }
    int all;
    const int end = cost + block_scan(c, s_warp, all);
    if (t < tiles) {
      p.tiles[t] = rec;
      p.cost[t] = end - c;
    }
    cost += all;
  }
  if (tid == 0) p.cost[tiles] = cost;
  __syncthreads();
  // Even division over as many clusters as get two steps or more each.
  // Starts lie at least SH_SEGMENT_COST + 2 apart, so no used cluster is
  // empty and no two start in one tile's leading cost.
  const int used = max(1, min(p.clusters, cost / (SH_SEGMENT_COST + 2)));
  for (int c = tid; c <= p.clusters; c += PLAN_THREADS) {
    SharedPos at{tiles, 0};
    if (c < used && cost > 0) {
      const int x = static_cast<int>(static_cast<long long>(cost) * c / used);
      at.tile = last_not_above(p.cost, tiles, x);
      at.step = max(0, x - p.cost[at.tile] - SH_SEGMENT_COST);
    }
    p.start[c] = at;
  }
  __syncthreads();
  // Which clusters hold each tile.
  for (int t = tid; t < tiles; t += PLAN_THREADS) {
    const int steps = p.tiles[t].steps;
    if (steps == 0) continue;
    // Last cluster that starts at or before step `step` of the tile.
    auto last_before = [&](int step) {
      int lo = 0, hi = used;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        const SharedPos s = p.start[mid];
        if (s.tile < t || (s.tile == t && s.step <= step)) lo = mid;
        else hi = mid;
      }
      return lo;
    };
    const int a = last_before(0), z = last_before(steps - 1);
    p.tiles[t].seg0 = a;
    p.tiles[t].nseg = z - a + 1;
  }
}

// 32 rows of a 576-wide bf16 array, row r at src + s_row[r] * 576 (negative:
// zeros), widened into the planes at plane rows row0 .. row0 + rows - 1.  A
// value outside fp16 is packed as zero and sets s_bad of its row; returns
// whether this thread met one.
__device__ __forceinline__ bool pack_rows(const uint16_t* src, const long long* s_row, int* s_bad, uint16_t* dst,
                                          long long plane, long long row0, int rows) {
  uint4 v[PER_THREAD];
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * PACK_THREADS;
    const int r = e / ROW_CHUNKS, c = e - r * ROW_CHUNKS;
    const long long row = s_row[r];
    v[u] = make_uint4(0, 0, 0, 0);
    if (row >= 0)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                   : "=r"(v[u].x), "=r"(v[u].y), "=r"(v[u].z), "=r"(v[u].w)
                   : "l"(reinterpret_cast<const uint4*>(src + row * D_QK) + c));
  }
  bool any = false;
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * PACK_THREADS;
    const int r = e / ROW_CHUNKS, c = e - r * ROW_CHUNKS;
    bool bad = false;
    uint4 w = widen_bf16x8(v[u], bad);
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

__global__ void __launch_bounds__(PLAN_THREADS) shared_plan_kernel(const SharedParams p) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (blockIdx.x == 0) {
    plan_call(p);
    return;
  }
  // Queries: 128 rows per CTA, nine granules per thread.
  const long long rows = static_cast<long long>(p.batch) * p.R;
  const long long row0 = static_cast<long long>(blockIdx.x - 1) * (PACK_KEYS * (PLAN_THREADS / PACK_THREADS));
  bool bad = false;
  uint4 v[PER_THREAD];
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * PLAN_THREADS;
    const long long row = row0 + e / ROW_CHUNKS;
    v[u] = make_uint4(0, 0, 0, 0);
    if (row < rows) v[u] = __ldg(reinterpret_cast<const uint4*>(p.q + row * D_QK) + e % ROW_CHUNKS);
  }
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * PLAN_THREADS;
    const long long row = row0 + e / ROW_CHUNKS;
    const int c = e % ROW_CHUNKS;
    if (row < rows)
      *reinterpret_cast<uint4*>(p.q16 + ((c >> 3) * p.q_plane + row) * 64 + (c & 7) * 8) = widen_bf16x8(v[u], bad);
  }
  report_range(bad, p.err);
}

__global__ void __launch_bounds__(PACK_THREADS, 4) shared_pack_kernel(const SharedParams p) {
  __shared__ long long s_row[PACK_KEYS];
  __shared__ int s_meta[PACK_KEYS], s_bad[PACK_KEYS];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int total = p.totals[0], tid = threadIdx.x;
  const int chunks = (total + SH_TAIL + PACK_KEYS - 1) / PACK_KEYS;
  for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int key0 = chunk * PACK_KEYS, rows = min(PACK_KEYS, total + SH_TAIL - key0);
    if (tid < PACK_KEYS) {
      const int key = key0 + tid;
      long long row = -1;
      int meta = META_MASKED;
      if (key < total) {
        const int part = last_not_above(p.base, 2 * p.batch, key);
        int b = part >> 1, j = key - p.base[part];
        if (part & 1) {
          j += p.kv_lens[b] - p.own[b];               // behind the shared rows
          meta = meta_own(b, max(-1, j - (p.kv_lens[b] - p.T)));
        } else {
          b = p.source[p.group_of[b]];
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
      s_row[tid] = row;
      s_meta[tid] = meta;
      s_bad[tid] = 0;
    }
    __syncthreads();
    report_range(pack_rows(p.kv, s_row, s_bad, p.k16, p.k_plane, key0, rows), p.err);
    __syncthreads();
    if (tid < rows) p.meta[key0 + tid] = s_meta[tid] | (s_bad[tid] ? META_POISON : 0);
  }
}

// Rows of tiles that several clusters hold parts of (or none: no request of
// the tile is served), one warp per row, four rows per CTA.
constexpr int JOIN_ROWS = 4;

__global__ void __launch_bounds__(JOIN_ROWS * 32) shared_join_kernel(const SharedParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int tile = blockIdx.x / (SH_ROWS / JOIN_ROWS);
  if (tile >= p.totals[1]) return;
  const SharedTile t = p.tiles[tile];
  const int lane = threadIdx.x & 31;
  const int r = (blockIdx.x % (SH_ROWS / JOIN_ROWS)) * JOIN_ROWS + (threadIdx.x >> 5);
  if (t.nseg == 1 || r >= t.nrows) return;
  const int row = t.q_row0 + r;
  const float nan = __int_as_float(0x7fc00000);
  float4 acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
  float lse = nan;
  if (t.nseg > 1 && p.own[row / p.R] > 0) {
    const SharedPos s0 = p.start[t.seg0];
    auto slot = [&](int s) { return part_slot(t.seg0 + s, s > 0 || (s0.tile == tile && s0.step == 0)); };
    float mx = -INFINITY, sum = 0.f;
    bool any_nan = false;
    for (int s = lane; s < t.nseg; s += 32) {
      const float L = p.part_lse[static_cast<size_t>(slot(s)) * SH_ROWS + r];
      any_nan |= L != L;
      mx = fmaxf(mx, L);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    any_nan = __any_sync(0xffffffffu, any_nan);
    const float base = mx == -INFINITY ? 0.f : mx;
    for (int s = 0; s < t.nseg; ++s) {
      const size_t at = static_cast<size_t>(slot(s)) * SH_ROWS + r;
      const float w = ex2((p.part_lse[at] - base) * kLog2e);
      sum += w;
      if (w == 0.f) continue;
      const float4* o = reinterpret_cast<const float4*>(p.part_o + at * D_V) + lane;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const float4 x = __ldcs(o + 32 * f);
        acc[f].x += w * x.x;
        acc[f].y += w * x.y;
        acc[f].z += w * x.z;
        acc[f].w += w * x.w;
      }
    }
    // Every key masked (bad slots): weight 0 everywhere.
    const float inv = any_nan ? nan : sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = make_float4(acc[f].x * inv, acc[f].y * inv, acc[f].z * inv, acc[f].w * inv);
    lse = any_nan ? nan : sum > 0.f ? base + logf(sum) : -INFINITY;
  } else {
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = make_float4(nan, nan, nan, nan);
  }
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const size_t at = static_cast<size_t>(row) * D_V / 4 + lane + 32 * f;
    if (p.out_bf16) {
      __nv_bfloat162 lo = __floats2bfloat162_rn(acc[f].x, acc[f].y), hi = __floats2bfloat162_rn(acc[f].z, acc[f].w);
      reinterpret_cast<uint2*>(p.out)[at] = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    } else {
      reinterpret_cast<float4*>(p.out)[at] = acc[f];
    }
  }
  if (lane == 0) p.lse[row] = lse;
}

cudaError_t launch(void (*kernel)(const SharedParams), long long grid, unsigned block, const SharedParams& p,
                   cudaStream_t stream, bool overlap) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.batch) * p.R;
  const int per_cta = PACK_KEYS * (PLAN_THREADS / PACK_THREADS);
  return launch(shared_plan_kernel, 1 + (rows + per_cta - 1) / per_cta, PLAN_THREADS, p, stream, false);
}

cudaError_t launch_shared_pack(const SharedParams& p, int num_sms, cudaStream_t stream) {
  const long long most = static_cast<long long>(p.batch) * p.max_kv_len + SH_TAIL;
  const long long chunks = (most + PACK_KEYS - 1) / PACK_KEYS;
  return launch(shared_pack_kernel, std::min<long long>(chunks, 6LL * num_sms), PACK_THREADS, p, stream, true);
}

cudaError_t launch_shared_join(const SharedParams& p, cudaStream_t stream) {
  return launch(shared_join_kernel, static_cast<long long>(p.max_tiles) * (SH_ROWS / JOIN_ROWS), JOIN_ROWS * 32, p, stream, true);
}

}  // namespace mlav
