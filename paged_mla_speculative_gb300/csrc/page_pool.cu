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
#include "copy_ring.h"
#include "kernels.h"
#include "page_pool.cuh"
#include "tc_ptx.cuh"

#include <algorithm>

namespace mlav {
namespace {

constexpr int FORK_THREADS = 256;
constexpr int FORK_CHUNK = 4 * FORK_THREADS;     // table entries per CTA
// Partial pages are copied through shared memory by bulk copies, two pieces of
// half a page in turn: the rows of a partial page are one run of bytes.
constexpr int PIECE = PAGE / 2 * ROW_BYTES;
constexpr int COPY_SMEM = 2 * PIECE;
constexpr int COPY_CTAS_PER_SM = 3;
constexpr long long COPY_LIMIT = 1LL << 31;      // cycles before a wait gives up

// Rows and entries of child i, or zero entries with the error bit that says why.
struct Child {
  int parent, n, ip0;
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
  c.ip0 = a.kv_indptr[c.parent];
  const long long p1 = a.kv_indptr[c.parent + 1], pn = a.kv_indptr[a.num_parents];
  if (c.n < 0 || static_cast<long long>(c.n) + a.extra > a.max_kv_len) {
    c.bad = ERR_LEN;
  } else if (c.ip0 < 0 || p1 > pn || p1 - c.ip0 < (static_cast<long long>(c.n) + PAGE - 1) / PAGE) {
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

// The copy of `bytes` from page `from` to page `to` in each layer l0, l0 +
// step, .., by one thread: the pieces of copy_through_two.
struct LayerCopy {
  const ForkArgs& a;
  uint32_t buf, mbar;
  long long from, to;
  int bytes, l0, step;

  __device__ __forceinline__ int pieces() const { return (bytes + PIECE - 1) / PIECE; }   // of a layer
  __device__ __forceinline__ int total() const { return (a.num_layers - l0 + step - 1) / step * pieces(); }
  // Piece i's first byte in the layer's page `page`, and its size.
  __device__ __forceinline__ uint8_t* at(int i, long long page, int& size) const {
    const int off = i % pieces() * PIECE;
    size = min(PIECE, bytes - off);
    return reinterpret_cast<uint8_t*>(a.kv_cache + static_cast<long long>(l0 + i / pieces() * step) * a.layer_stride) +
           page * PAGE * ROW_BYTES + off;
  }
  __device__ __forceinline__ void load(int i) {
    int size;
    const uint8_t* src = at(i, from, size);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(mbar + 8 * (i & 1)), "r"(size) : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     buf + (i & 1) * PIECE),
                 "l"(src), "r"(size), "r"(mbar + 8 * (i & 1))
                 : "memory");
  }
  __device__ __forceinline__ bool landed(int i) { return tc::mbar_try(mbar + 8 * (i & 1), (i >> 1) & 1); }
  __device__ __forceinline__ void store(int i) {
    int size;
    uint8_t* dst = at(i, to, size);
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\ncp.async.bulk.commit_group;\n" ::"l"(dst),
                 "r"(buf + (i & 1) * PIECE), "r"(size)
                 : "memory");
  }
  __device__ __forceinline__ void drain() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
  __device__ __forceinline__ long long now() { return clock64(); }
  __device__ __forceinline__ void late() { atomicOr(a.err, ERR_TIMEOUT); }
};

// grid (table_parts + copy_parts, children).  Every CTA scans all children's
// counts itself (a few loads per thread), which gives its child's offsets and
// the capacity cut without a second launch; the last CTA to have read
// free_count lowers it.  Copy part k of a child takes layers k, k +
// copy_parts, ..; as many parts as fill the SMs once, so that the scan (about
// 3 us of dependent loads) is paid once per SM slot and not once per layer.
__global__ void __launch_bounds__(FORK_THREADS) fork_kv_kernel(const ForkArgs a, int table_parts) {
  extern __shared__ __align__(128) uint8_t s_copy[];
  __shared__ Sums s_warp[FORK_THREADS / 32];
  __shared__ Sums s_mine, s_fit;
  __shared__ Child s_child;
  __shared__ unsigned long long s_last[2];
  __shared__ __align__(8) uint64_t s_mbar[2];
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  const int c = blockIdx.y, tid = threadIdx.x;
  const int height = *a.free_count;
  const bool height_ok = height >= 0 && height <= a.num_pages;
  const long long left = height_ok ? height : 0;
  if (tid < 2) s_last[tid] = 0;
  if (tid == 0) {
    tc::mbar_init(smem_u32(s_mbar), 1);
    tc::mbar_init(smem_u32(s_mbar + 1), 1);
    tc::mbar_fence_init();
  }
  Sums before{0, 0};
  for (int base = 0; base < a.num_children; base += FORK_THREADS) {
    const int i = base + tid;
    Sums x{0, 0};
    if (i < a.num_children) {
      const Child ch = load_child(a, i);
      x = Sums{ch.total, ch.fresh};
      if (i == c) s_child = ch;
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
      if (height_ok) *a.free_count = static_cast<int32_t>(left - static_cast<long long>(s_last[1]));
      else atomicOr(a.err, ERR_CAPACITY);
    }
  }
  const Child ch = s_child;
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
  const int32_t* held = a.kv_indices + ch.ip0;
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
  const int part = static_cast<int>(blockIdx.x) - table_parts, parts = static_cast<int>(gridDim.x) - table_parts;
  if (from >= 0 && from < a.num_pages) {
    if (tid == 0) {
      LayerCopy copy{a, smem_u32(s_copy), smem_u32(s_mbar), from, to, partial * ROW_BYTES, part, parts};
      copy_through_two(copy, copy.total(), COPY_LIMIT);
      asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
    }
    return;
  }
  if (tid == 0) atomicOr(a.err, ERR_SLOT);
  for (int l = part; l < a.num_layers; l += parts) {   // no such page: zeros
    uint4* dst = reinterpret_cast<uint4*>(a.kv_cache + static_cast<long long>(l) * a.layer_stride + to * PAGE * D_QK);
    for (int e = tid; e < partial * ROW_CHUNKS; e += FORK_THREADS) dst[e] = make_uint4(0, 0, 0, 0);
  }
}

// One cluster: counts lowered (the one thread that takes a count from 1 to 0
// marks the page in a bit map), then the bit map read in order, so the pushed
// pages ascend whatever order the counts fell in, and cleared for the next call.
constexpr int FREE_THREADS = POOL_THREADS;
constexpr int FREE_MAX_CTAS = 8;

__global__ void __launch_bounds__(FREE_THREADS) free_kv_kernel(const FreeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int s_warp[FREE_THREADS / 32];
  __shared__ int s_total, s_bad;
  const int tid = threadIdx.x;
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
       i += static_cast<long long>(ctas) * FREE_THREADS)
    bad |= release_page(a.kv_indices[i], a.num_pages, a.page_refs, a.page_bits);
  if (bad) atomicOr(a.err, bad);
  cluster.sync();
  push_marked(a.page_bits, a.num_pages, count, a.free_pages, a.free_count, a.err, s_warp, s_total);
}

}  // namespace

cudaError_t page_pool_prepare() {
  return cudaFuncSetAttribute(fork_kv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, COPY_SMEM);
}

cudaError_t launch_fork_kv(const ForkArgs& a, int num_sms, cudaStream_t stream) {
  const int entries = (a.max_kv_len + PAGE - 1) / PAGE;
  const int table_parts = (entries + FORK_CHUNK - 1) / FORK_CHUNK;
  const int slots = COPY_CTAS_PER_SM * num_sms;
  const int copy_parts = std::max(1, std::min(a.num_layers, slots / a.num_children));
  const dim3 grid(table_parts + copy_parts, a.num_children);
  return launch_overlapping(fork_kv_kernel, grid, FORK_THREADS, COPY_SMEM, stream, 1, a, table_parts);
}

cudaError_t launch_free_kv(const FreeArgs& a, int max_entries, cudaStream_t stream) {
  // One CTA while it has at most four entries and four bit-map words per
  // thread; the cluster's barriers cost about 1 us.
  const long long work = std::max<long long>(max_entries, a.num_pages / 32);
  unsigned ctas = 1;
  while (ctas < FREE_MAX_CTAS && work > 4LL * FREE_THREADS * ctas) ctas *= 2;
  return launch_overlapping(free_kv_kernel, dim3(ctas), FREE_THREADS, 0, stream, ctas, a);
}

}  // namespace mlav
