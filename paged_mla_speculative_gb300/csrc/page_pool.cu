// Forking and freeing requests of a paged cache with counted pages.
//
// The pool is three arrays the caller owns: page_refs[page] (how many tables
// hold the page; 0 when it is free), free_pages (a stack) and free_count (its
// height, on the device, so that both calls can be captured).
//
// Fork, child c of parent p with n = kv_lens[p] rows, in child order:
//   entries     ceil((n + extra) / 64); the first n / 64 are the parent's own
//               pages (page_refs + 1), the rest are fresh: the j-th page that
//               the call takes is free_pages[free_count - 1 - j], page_refs 1;
//   partial     the n % 64 rows of the parent's page n / 64 are copied into
//               the child's first fresh page, in every layer;
//   outputs     child_lens = n + extra, child_indptr the prefix sum of the
//               entry counts, child_indices the entries, free_count lowered.
//   The longest leading run of children whose entries fit the capacity and
//   whose fresh pages fit the stack is forked, later ones get length 0
//   (ERR_CAPACITY); a parent that is out of range (ERR_POOL), whose length is
//   outside [0, max_kv_len - extra] (ERR_LEN) or whose table does not hold n
//   rows (ERR_INDPTR) gives its child length 0.
// Free: every entry of the tables lowers its page's count; pages whose count
// falls to 0 are pushed in ascending order, whatever the order in which the
// counts fell.  A count that is not positive already (a page freed twice) is
// left as it is (ERR_REF).
// A page id outside the cache is reported (ERR_SLOT) and touches nothing; a
// partial page outside the cache is copied as zeros.
#include "common.cuh"
#include "kernels.h"

#include <cooperative_groups.h>

namespace mlav {
namespace {

constexpr int FORK_THREADS = 256;
constexpr int FORK_CHUNK = 4 * FORK_THREADS;                       // table entries per CTA
constexpr int COPY_PER_THREAD = PAGE * ROW_CHUNKS / FORK_THREADS;  // 18 granules

// Rows and entries of child i, or zero entries with the error bit that says why.
struct Child {
  int parent, n;
  long long total, fresh;   // entries, of them fresh
  int bad;
};
__device__ __forceinline__ Child load_child(const ForkArgs& a, int i) {
  Child c{};
  c.parent = a.parents[i];
  if (c.parent < 0 || c.parent >= a.num_parents) {
    c.bad = ERR_POOL;
    return c;
  }
  c.n = a.kv_lens[c.parent];
  const long long p0 = a.kv_indptr[c.parent], p1 = a.kv_indptr[c.parent + 1], pn = a.kv_indptr[a.num_parents];
  if (c.n < 0 || static_cast<long long>(c.n) + a.extra > a.max_kv_len) {
    c.bad = ERR_LEN;
  } else if (p0 < 0 || p1 > pn || p1 - p0 < (static_cast<long long>(c.n) + PAGE - 1) / PAGE) {
    c.bad = ERR_INDPTR;
  } else {
    c.total = (static_cast<long long>(c.n) + a.extra + PAGE - 1) / PAGE;
    c.fresh = c.total - c.n / PAGE;
  }
  if (c.bad) c.n = 0;
  return c;
}

struct Sums {
  long long total, fresh;
};
__device__ __forceinline__ Sums block_scan(Sums x, Sums* s_warp, Sums& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, x.total, o), f = __shfl_up_sync(0xffffffffu, x.fresh, o);
    if (lane >= o) x.total += t, x.fresh += f;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  all = Sums{0, 0};
  for (int w = 0; w < FORK_THREADS / 32; ++w) {
    if (w == warp) x.total += all.total, x.fresh += all.fresh;
    all.total += s_warp[w].total;
    all.fresh += s_warp[w].fresh;
  }
  // x: inclusive, with the warps before this one.
  return x;
}

// grid (table chunks + layers, children).  Every CTA scans all children's
// counts itself (a few loads per thread), which gives its child's offsets and
// the capacity cut without a second launch; the last CTA to have read
// free_count lowers it.
__global__ void __launch_bounds__(FORK_THREADS) fork_kv_kernel(const ForkArgs a, int table_parts) {
  __shared__ Sums s_warp[FORK_THREADS / 32];
  __shared__ Sums s_mine, s_fit;
  __shared__ unsigned long long s_last[2];
  const int c = blockIdx.y, tid = threadIdx.x;
  const long long left = max(0, min(*a.free_count, a.num_pages));
  if (tid < 2) s_last[tid] = 0;
  if (tid == 0) s_mine = Sums{0, 0};
  Sums before{0, 0};
  for (int base = 0; base < a.num_children; base += FORK_THREADS) {
    const int i = base + tid;
    Sums x{0, 0};
    if (i < a.num_children) {
      const Child ch = load_child(a, i);
      x = Sums{ch.total, ch.fresh};
    }
    Sums all;
    const Sums own = x;
    x = block_scan(x, s_warp, all);
    x.total += before.total;
    x.fresh += before.fresh;
    if (i < a.num_children) {
      if (x.total <= a.capacity && x.fresh <= left) {   // ends never fall: the largest that fits
        if (i <= c) atomicMax(&s_last[0], static_cast<unsigned long long>(x.total));
        atomicMax(&s_last[1], static_cast<unsigned long long>(x.fresh));
      }
      if (i == c) {
        s_mine = Sums{x.total - own.total, x.fresh - own.fresh};
        s_fit = x;
      }
    }
    before.total += all.total;
    before.fresh += all.fresh;
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const unsigned ctas = gridDim.x * gridDim.y;
    if (atomicAdd(a.ticket, 1u) == ctas - 1) {
      *a.ticket = 0;
      *a.free_count = static_cast<int32_t>(left - static_cast<long long>(s_last[1]));
    }
  }
  const Child ch = load_child(a, c);
  const bool fits = s_fit.total <= a.capacity && s_fit.fresh <= left;
  if (blockIdx.x == 0 && tid == 0) {
    if (ch.bad) atomicOr(a.err, ch.bad);
    if (!fits && ch.total > 0) atomicOr(a.err, ERR_CAPACITY);
    a.child_lens[c] = fits && !ch.bad ? ch.n + a.extra : 0;
    a.child_indptr[c + 1] = static_cast<int32_t>(s_last[0]);
    if (c == 0) a.child_indptr[0] = 0;
  }
  if (!fits || ch.total == 0) return;
  const int full = ch.n / PAGE, partial = ch.n % PAGE;
  const int32_t* held = a.kv_indices + a.kv_indptr[ch.parent];
  // The page at entry j >= full.
  auto fresh = [&](long long j) { return a.free_pages[left - 1 - (s_mine.fresh + j - full)]; };

  if (static_cast<int>(blockIdx.x) < table_parts) {
    int bad = 0;
    for (long long j = static_cast<long long>(blockIdx.x) * FORK_CHUNK + tid;
         j < min(ch.total, static_cast<long long>(blockIdx.x + 1) * FORK_CHUNK); j += FORK_THREADS) {
      const int32_t page = j < full ? held[j] : fresh(j);
      a.child_indices[s_mine.total + j] = page;
      if (page < 0 || page >= a.num_pages) {
        bad |= ERR_SLOT;
      } else if (j < full) {
        if (atomicAdd(a.page_refs + page, 1) <= 0) bad |= ERR_REF;
      } else if (atomicExch(a.page_refs + page, 1) != 0) {
        bad |= ERR_REF;   // the stack held a page that is in use
      }
    }
    if (bad) atomicOr(a.err, bad);
    return;
  }
  if (partial == 0) return;
  const long long from = held[full], to = fresh(full);
  if (to < 0 || to >= a.num_pages) return;             // reported with the table
  const bool src_ok = from >= 0 && from < a.num_pages;
  if (!src_ok && tid == 0) atomicOr(a.err, ERR_SLOT);
  uint16_t* layer = a.kv_cache + static_cast<long long>(blockIdx.x - table_parts) * a.layer_stride;
  const uint4* src = reinterpret_cast<const uint4*>(layer + from * PAGE * D_QK);
  uint4* dst = reinterpret_cast<uint4*>(layer + to * PAGE * D_QK);
  uint4 v[COPY_PER_THREAD];
#pragma unroll
  for (int u = 0; u < COPY_PER_THREAD; ++u) {
    const int e = tid + u * FORK_THREADS;
    v[u] = make_uint4(0, 0, 0, 0);
    if (src_ok && e < partial * ROW_CHUNKS) v[u] = src[e];
  }
#pragma unroll
  for (int u = 0; u < COPY_PER_THREAD; ++u) {
    const int e = tid + u * FORK_THREADS;
    if (e < partial * ROW_CHUNKS) dst[e] = v[u];
  }
}

// One cluster: counts lowered (the one thread that takes a count from 1 to 0
// marks the page in a bit map), then the bit map read in order, so the pushed
// pages ascend whatever order the counts fell in, and cleared for the next call.
constexpr int FREE_THREADS = 1024;
constexpr int FREE_CTAS = 8;

__global__ void __launch_bounds__(FREE_THREADS) free_kv_kernel(const FreeArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int s_warp[FREE_THREADS / 32];
  __shared__ int s_total, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // Tables that are not one run of entries are refused as a whole.
  const long long first = a.kv_indptr[0], end = a.kv_indptr[a.batch];
  bool bad_table = first < 0;
  for (int b = tid; b < a.batch; b += FREE_THREADS) bad_table |= a.kv_indptr[b + 1] < a.kv_indptr[b];
  if (bad_table) s_bad = 1;
  const long long count = *a.free_count;
  __syncthreads();
  const bool refused = s_bad != 0, count_ok = count >= 0 && count <= a.num_pages;
  if (rank == 0 && tid == 0 && (refused || !count_ok)) atomicOr(a.err, (refused ? ERR_INDPTR : 0) | (count_ok ? 0 : ERR_CAPACITY));
  if (refused || !count_ok) return;   // the same in every CTA of the cluster
  int bad = 0;
  for (long long i = first + static_cast<long long>(rank) * FREE_THREADS + tid; i < end;
       i += static_cast<long long>(ctas) * FREE_THREADS) {
    const int page = a.kv_indices[i];
    if (page < 0 || page >= a.num_pages) {
      bad |= ERR_SLOT;
      continue;
    }
    const int had = atomicSub(a.page_refs + page, 1);
    if (had == 1) {
      atomicOr(a.page_bits + (page >> 5), 1u << (page & 31));
    } else if (had <= 0) {   // never raises a count to 1, so "1 to 0" stays unique
      atomicAdd(a.page_refs + page, 1);
      bad |= ERR_REF;
    }
  }
  if (bad) atomicOr(a.err, bad);
  cluster.sync();
  // This CTA's words of the bit map, in order: `per` consecutive ones per thread.
  const int words = (a.num_pages + 31) / 32;
  const int per = (words + ctas * FREE_THREADS - 1) / (ctas * FREE_THREADS);
  const long long w0 = (static_cast<long long>(rank) * FREE_THREADS + tid) * per;
  int mine = 0;
  for (int k = 0; k < per; ++k)
    if (w0 + k < words) mine += __popc(__ldcg(a.page_bits + w0 + k));
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < FREE_THREADS / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  if (tid == 0) s_total = total;
  cluster.sync();
  long long at = count + before + x - mine, all = 0;
  for (int r = 0; r < ctas; ++r) {
    const int t = *cluster.map_shared_rank(&s_total, r);
    if (r < rank) at += t;
    all += t;
  }
  if (mine)
    for (int k = 0; k < per; ++k) {
      if (w0 + k >= words) break;
      unsigned w = __ldcg(a.page_bits + w0 + k);
      if (w) a.page_bits[w0 + k] = 0;
      while (w) {
        const int bit = __ffs(static_cast<int>(w)) - 1;
        w &= w - 1;
        if (at < a.num_pages) a.free_pages[at] = static_cast<int32_t>((w0 + k) * 32 + bit);
        ++at;
      }
    }
  if (rank == 0 && tid == 0) {
    if (count + all > a.num_pages) atomicOr(a.err, ERR_CAPACITY);
    *a.free_count = static_cast<int32_t>(min(count + all, static_cast<long long>(a.num_pages)));
  }
  cluster.sync();   // no CTA leaves while another reads its total
}

}  // namespace

cudaError_t launch_fork_kv(const ForkArgs& a, cudaStream_t stream) {
  const int entries = (a.max_kv_len + PAGE - 1) / PAGE;
  const int table_parts = (entries + FORK_CHUNK - 1) / FORK_CHUNK;
  const dim3 grid(table_parts + a.num_layers, a.num_children);
  fork_kv_kernel<<<grid, FORK_THREADS, 0, stream>>>(a, table_parts);
  return cudaGetLastError();
}

cudaError_t launch_free_kv(const FreeArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(FREE_CTAS);
  cfg.blockDim = dim3(FREE_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = FREE_CTAS;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, free_kv_kernel, a);
}

}  // namespace mlav
