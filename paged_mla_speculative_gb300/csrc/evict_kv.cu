// Eviction: requests cut down to the rows that were given most attention.
//
// A request of n rows that is over the budget keeps its first `sink` rows, its
// last `recent` rows and, of the others, those with the largest weights, the
// lowest index first among equals, `budget` in all and in their order.
//
// evict_select_kernel, a cluster of CTAs per request: the weights as ordered
// 32-bit keys in shared memory; the key of the last row that is kept by three
// histograms (11, 11 and 10 bits) that the cluster's CTAs add up through
// distributed shared memory; then one scan gives every kept row its new place
// (rows above that key, rows equal to it, both in order).  Every CTA scans all
// requests' lengths itself for its place in the new tables and on the stack of
// free pages, as fork_kv does: how many entries stay follows from the lengths
// alone.  Pages of 64: those that hold protected leading rows alone stay, the
// kept rows behind them go to fresh pages (so that pages shared with other
// requests are not written, and no row is read after it was overwritten), all
// others of the table are given back.  Single slots: kept slots stay, no row
// moves.
// evict_copy_kernel: the kept rows of every layer into the fresh pages.
// evict_push_kernel: pages whose count fell to 0, in ascending order.
//
// The copies are bound by HBM (1152 bytes read and written a row and layer);
// the rest is a chain of dependent loads and cluster barriers.
#include "common.cuh"
#include "kernels.h"
#include "page_pool.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace mlav {
namespace {

namespace cg = cooperative_groups;

constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int MAX_CTAS = 8;                // per request
constexpr int MAX_CACHED = 24576;          // keys that a CTA holds in shared memory

// Larger weights have larger keys; -0 is 0, NaN is below every number.
__device__ __forceinline__ unsigned ordered(float w) {
  if (w != w) return 0;
  const unsigned u = __float_as_uint(w == 0.f ? 0.f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A request's rows and entries; nothing, with the error bit that says why, for
// one that is out of order.
struct Item {
  int n, m, ip0, entries;     // rows, kept rows, the table
  int stay;                   // entries that stay, in order: the first ones (pages), the kept ones (slots)
  long long total, fresh;     // entries of the new table, of them fresh
  int bad;
};
__device__ __forceinline__ Item load_item(const EvictArgs& a, int b) {
  Item x{};
  x.n = a.kv_lens[b];
  x.ip0 = a.kv_indptr[b];
  const long long p1 = a.kv_indptr[b + 1], pn = a.kv_indptr[a.batch];
  if (x.n < 0 || x.n > a.max_kv_len || static_cast<long long>(min(x.n, a.budget)) + a.extra > a.max_kv_len) {
    x.bad = ERR_LEN;
  } else if (x.ip0 < 0 || p1 > pn || (p1 - x.ip0) * a.page < x.n) {
    x.bad = ERR_INDPTR;
  } else {
    x.entries = static_cast<int>(p1 - x.ip0);
    x.m = min(x.n, a.budget);
    x.stay = a.page == 1 ? x.m : x.n <= a.budget ? (x.n + a.page - 1) / a.page : a.sink / a.page;
    x.total = (static_cast<long long>(x.m) + a.extra + a.page - 1) / a.page;
    x.fresh = x.total - x.stay;
  }
  if (x.bad) x.n = 0;
  return x;
}

struct Sums {
  long long total, fresh;
};
__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// Inclusive scan over the CTA's threads; `all` receives the total.
__device__ __forceinline__ long long cta_scan(long long x, long long* s_warp, long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_scan(x, lane);
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  all = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) x += all;
    all += s_warp[w];
  }
  return x;
}

// grid: `ctas` CTAs (a cluster) per request.
__global__ void __launch_bounds__(THREADS, 1) evict_select_kernel(const EvictArgs a, int cached) {
  extern __shared__ unsigned s_keys[];
  __shared__ int s_hist[BINS];
  __shared__ long long s_warp[WARPS];
  __shared__ Sums s_mine, s_fit;
  __shared__ unsigned long long s_last[2];
  __shared__ Item s_item;
  __shared__ int s_bin, s_above;
  __shared__ long long s_count;
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int b = blockIdx.x / ctas, tid = threadIdx.x;
  const int height = *a.free_count;
  const bool height_ok = height >= 0 && height <= a.num_pages;
  const long long left = height_ok ? height : -1;   // a stack that is out of order serves nobody
  if (tid < 2) s_last[tid] = 0;
  Sums before{0, 0};
  for (int base = 0; base < a.batch; base += THREADS) {
    const int i = base + tid;
    Sums x{0, 0};
    if (i < a.batch) {
      const Item it = load_item(a, i);
      x = Sums{it.total, it.fresh};
      if (i == b) s_item = it;
    }
    const Sums own = x;
    Sums all;
    x.total = before.total + cta_scan(x.total, s_warp, all.total);
    x.fresh = before.fresh + cta_scan(x.fresh, s_warp, all.fresh);
    if (i < a.batch) {
      if (x.total <= a.capacity && x.fresh <= left) {   // ends never fall: the largest that fits
        if (i <= b) atomicMax(&s_last[0], static_cast<unsigned long long>(x.total));
        atomicMax(&s_last[1], static_cast<unsigned long long>(x.fresh));
      }
      if (i == b) {
        s_mine = Sums{x.total - own.total, x.fresh - own.fresh};
        s_fit = x;
      }
    }
    before.total += all.total;
    before.fresh += all.fresh;
  }
  __syncthreads();
  if (tid == 0) {   // the last CTA that has read the height lowers it
    __threadfence();
    if (atomicAdd(a.ticket, 1u) == gridDim.x - 1) {
      *a.ticket = 0;
      if (height_ok) *a.free_count = static_cast<int32_t>(left - static_cast<long long>(s_last[1]));
      else atomicOr(a.err, ERR_CAPACITY);
    }
  }
  const Item it = s_item;
  const bool fits = s_fit.total <= a.capacity && s_fit.fresh <= left;
  const bool served = fits && !it.bad;
  if (rank == 0 && tid == 0) {
    if (it.bad) atomicOr(a.err, it.bad);
    if (!it.bad && !fits && (it.total > 0 || it.entries > 0)) atomicOr(a.err, ERR_CAPACITY);
    a.new_lens[b] = served ? it.m + a.extra : 0;
    a.new_indptr[b + 1] = static_cast<int32_t>(s_last[0]);
    if (b == 0) a.new_indptr[0] = 0;
  }
  const long long all_threads = static_cast<long long>(ctas) * THREADS, me = static_cast<long long>(rank) * THREADS + tid;
  float* new_row = a.new_weights + b * a.new_stride;
  // Behind the kept rows: 0.
  for (long long j = (served ? it.m : 0) + me; j < a.new_width; j += all_threads) new_row[j] = 0.f;
  if (!served) return;   // the whole cluster

  const int n = it.n;
  const bool over = n > a.budget;
  const float* row = a.weights + b * a.stride;
  const int32_t* held = a.kv_indices + it.ip0;
  int32_t* table = a.new_indices + s_mine.total;
  const int lo = a.sink, hi = n - a.recent;    // rows lo .. hi - 1 are chosen among, when the request is over the budget
  // This CTA's rows: `per` consecutive ones per thread (an odd number, so that
  // a warp's keys lie in different banks).
  const int per = static_cast<int>((n + all_threads - 1) / all_threads) | 1;
  const long long first = static_cast<long long>(rank) * THREADS * per;
  const int count = static_cast<int>(max(0LL, min(static_cast<long long>(THREADS) * per, n - first)));
  const int j0 = static_cast<int>(min(first, static_cast<long long>(n)));
  const bool in_smem = count <= cached;
  int k = a.budget - a.sink - a.recent;        // to be chosen
  unsigned cut = 0xffffffffu;                  // the key of the last one chosen
  int equal = 0;                               // of the rows with that key, how many
  if (over) {
    auto key_at = [&](int i) { return in_smem ? s_keys[i] : ordered(row[j0 + i]); };
    if (in_smem)
      for (int i = tid; i < count; i += THREADS) s_keys[i] = ordered(row[j0 + i]);
    if (k > 0) {
      unsigned prefix = 0;
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < BINS; i += THREADS) s_hist[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < count; i0 += THREADS) {
          const int i = i0 + tid, j = j0 + i;
          bool mine = i < count && j >= lo && j < hi;
          const unsigned key = mine ? key_at(i) : 0;
          mine = mine && (pass == 0 || (key >> (shift + bits)) == prefix);
          const int bin = mine ? static_cast<int>((key >> shift) & ((1u << bits) - 1)) : -1;
          int same;
          __match_all_sync(0xffffffffu, bin, &same);
          if (same) {   // (many rows of one weight: one addition for the warp)
            if (bin >= 0 && (tid & 31) == 0) atomicAdd(s_hist + bin, 32);
          } else if (bin >= 0) {
            atomicAdd(s_hist + bin, 1);
          }
        }
        cluster.sync();
        // The bin, from the top, in which the k-th row lies: two bins per thread.
        const int top = BINS - 1 - 2 * tid;
        int h0 = 0, h1 = 0;
        for (int r = 0; r < ctas; ++r) {
          const int* h = cluster.map_shared_rank(s_hist, r);
          h0 += h[top];
          h1 += h[top - 1];
        }
        long long all;
        const long long end = cta_scan(h0 + h1, s_warp, all), start = end - h0 - h1;
        if (start < k && k <= end) {
          const bool upper = k <= start + h0;
          s_bin = upper ? top : top - 1;
          s_above = static_cast<int>(upper ? start : start + h0);
        }
        cluster.sync();   // histograms are read, s_bin is set
        prefix = (prefix << bits) | static_cast<unsigned>(s_bin);
        k -= s_above;
      }
      cut = prefix;
      equal = k;
    }
    __syncthreads();
  }
  // Rows above the cut (or protected) and rows equal to it, before each
  // thread's, in order: its kept rows' new places.
  int above = 0, ties = 0;
  const int t0 = min(tid * per, count), t1 = min(t0 + per, count);
  auto kind = [&](int i) {   // 1: kept, 2: kept while there are fewer than `equal`, 0: not
    const int j = j0 + i;
    if (!over || j < lo || j >= hi) return 1;
    const unsigned key = in_smem ? s_keys[i] : ordered(row[j]);
    return equal > 0 && key == cut ? 2 : equal > 0 && key > cut ? 1 : 0;
  };
  for (int i = t0; i < t1; ++i) {
    const int x = kind(i);
    above += x == 1;
    ties += x == 2;
  }
  long long all;
  const long long mine = static_cast<long long>(above) << 32 | static_cast<unsigned>(ties);
  long long place = cta_scan(mine, s_warp, all) - mine;
  if (tid == 0) s_count = all;
  cluster.sync();
  for (int r = 0; r < rank; ++r) place += *cluster.map_shared_rank(&s_count, r);
  int a0 = static_cast<int>(place >> 32), e0 = static_cast<int>(place & 0xffffffffll), errs = 0;
  for (int i = t0; i < t1; ++i) {
    const int x = kind(i), j = j0 + i;
    const bool kept = x == 1 || (x == 2 && e0 < equal);
    const int to = a0 + min(e0, equal);
    if (kept) {
      new_row[to] = row[j];
      if (a.page > 1) {
        if (over) a.kept[b * a.kept_stride + to] = j;
      } else {
        const int slot = held[j];
        table[to] = slot;
        if (slot < 0 || slot >= a.num_pages) errs |= ERR_SLOT;
      }
    } else if (a.page == 1) {
      errs |= release_page(held[j], a.num_pages, a.page_refs, a.page_bits);
    }
    a0 += x == 1;
    e0 += x == 2;
  }
  // Entries: those that stay, fresh ones, and those that are left.
  for (long long e = (a.page == 1 ? it.stay : 0) + me; e < it.total; e += all_threads) {
    int page;
    if (e < it.stay) {
      page = held[e];
      if (page < 0 || page >= a.num_pages) errs |= ERR_SLOT;
    } else {
      page = a.free_pages[left - 1 - (s_mine.fresh + e - it.stay)];
      if (page < 0 || page >= a.num_pages) errs |= ERR_SLOT;
      else if (atomicExch(a.page_refs + page, 1) != 0) errs |= ERR_REF;   // the stack held a page that is in use
    }
    table[e] = page;
  }
  for (long long e = (a.page == 1 ? n : it.stay) + me; e < it.entries; e += all_threads)
    errs |= release_page(held[e], a.num_pages, a.page_refs, a.page_bits);
  if (errs) atomicOr(a.err, errs);
  cluster.sync();   // no CTA leaves while another reads its count
}

// Rows of an evicted request, COPY_ROWS at a time, in some of the layers: nine
// 16-byte granules in flight per lane (a warp takes four rows).
constexpr int COPY_THREADS = 256, COPY_ROWS = COPY_THREADS / 32 * 4;

__global__ void __launch_bounds__(COPY_THREADS) evict_copy_kernel(const EvictArgs a, int layers_each) {
  __shared__ long long s_src[COPY_ROWS], s_dst[COPY_ROWS];
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  const int tid = threadIdx.x;
  const int stay = a.sink / PAGE;
  const int i0 = stay * PAGE + static_cast<int>(blockIdx.x) * COPY_ROWS;
  for (int b = blockIdx.y; b < a.batch; b += gridDim.y) {
    // (A request that is not served has length 0; a length of 0 has no rows.)
    if (a.new_lens[b] == 0 || a.kv_lens[b] <= a.budget) continue;
    const int rows = min(COPY_ROWS, a.budget - i0);
    if (rows <= 0) continue;
    __syncthreads();
    if (tid < COPY_ROWS) {
      long long src = -1, dst = -1;
      if (tid < rows) {
        const int i = i0 + tid, j = a.kept[b * a.kept_stride + i];
        const int from = a.kv_indices[a.kv_indptr[b] + j / PAGE], to = a.new_indices[a.new_indptr[b] + i / PAGE];
        if (to >= 0 && to < a.num_pages) dst = static_cast<long long>(to) * PAGE + i % PAGE;
        if (from >= 0 && from < a.num_pages) src = static_cast<long long>(from) * PAGE + j % PAGE;
        else atomicOr(a.err, ERR_SLOT);   // no such page: zeros
      }
      s_src[tid] = src;
      s_dst[tid] = dst;
    }
    __syncthreads();
    const int lane = tid & 31, r0 = (tid >> 5) * 4;
    for (int l = blockIdx.z * layers_each; l < min(a.num_layers, static_cast<int>(blockIdx.z + 1) * layers_each); ++l) {
      uint16_t* layer = a.kv_cache + static_cast<long long>(l) * a.layer_stride;
      uint4 v[9];
#pragma unroll
      for (int u = 0; u < 9; ++u) {
        const int e = lane + 32 * u, r = e / ROW_CHUNKS;
        const long long src = s_src[r0 + r];
        v[u] = src >= 0 ? *(reinterpret_cast<const uint4*>(layer + src * D_QK) + e % ROW_CHUNKS) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 9; ++u) {
        const int e = lane + 32 * u, r = e / ROW_CHUNKS;
        const long long dst = s_dst[r0 + r];
        if (dst >= 0) *(reinterpret_cast<uint4*>(layer + dst * D_QK) + e % ROW_CHUNKS) = v[u];
      }
    }
  }
}

// One cluster.
__global__ void __launch_bounds__(POOL_THREADS) evict_push_kernel(const EvictArgs a) {
  __shared__ int s_warp[POOL_THREADS / 32];
  __shared__ int s_total;
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  const long long count = *a.free_count;
  if (count < 0 || count > a.num_pages) return;   // (reported, and nothing was given back)
  cg::this_cluster().sync();                      // (every CTA has read the height)
  push_marked(a.page_bits, a.num_pages, count, a.free_pages, a.free_count, a.err, s_warp, s_total);
}

}  // namespace

cudaError_t evict_prepare() {
  return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_CACHED * 4);
}

cudaError_t launch_evict_kv(const EvictArgs& a, int num_sms, cudaStream_t stream) {
  // CTAs per request: while they fill no SM twice and have two rows per thread.
  int ctas = 1;
  while (ctas < MAX_CTAS && 2LL * ctas * a.batch <= num_sms && a.max_kv_len > 2LL * THREADS * ctas) ctas *= 2;
  const long long slice = ((a.max_kv_len + static_cast<long long>(ctas) * THREADS - 1) / (static_cast<long long>(ctas) * THREADS) | 1) * THREADS;
  const int cached = static_cast<int>(std::min<long long>(slice, MAX_CACHED));
  cudaError_t e = launch_overlapping(evict_select_kernel, dim3(static_cast<unsigned>(ctas) * a.batch), THREADS,
                                     static_cast<size_t>(cached) * 4, stream, static_cast<unsigned>(ctas), a, cached);
  const int moved = std::min(a.budget, a.max_kv_len) - a.sink / PAGE * PAGE;
  if (e == cudaSuccess && a.page > 1 && moved > 0) {
    const unsigned parts = static_cast<unsigned>((moved + COPY_ROWS - 1) / COPY_ROWS);
    const unsigned requests = static_cast<unsigned>(std::min(a.batch, 65535));
    // A CTA's rows are looked up once for several layers, where enough CTAs are left.
    const long long ctas_of_a_layer = static_cast<long long>(parts) * requests;
    const int each = std::max(static_cast<int>(std::clamp<long long>(ctas_of_a_layer * a.num_layers / (16LL * num_sms), 1, 16)),
                              (a.num_layers + 65534) / 65535);
    const unsigned z = static_cast<unsigned>((a.num_layers + each - 1) / each);
    e = launch_overlapping(evict_copy_kernel, dim3(parts, requests, z), COPY_THREADS, 0, stream, 1, a, each);
  }
  if (e != cudaSuccess) return e;
  unsigned push = 1;
  while (push < 8 && a.num_pages / 32 > 4LL * POOL_THREADS * push) push *= 2;
  return launch_overlapping(evict_push_kernel, dim3(push), POOL_THREADS, 0, stream, push, a);
}

}  // namespace mlav
