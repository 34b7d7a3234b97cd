// What freeing and evicting have in common: counts of pages that fall, and a bit
// map of the pages that reach 0, pushed on the pool's stack in ascending order
// (by push_marked in freeing; evict_kv.cu, whose pools of single slots have
// larger maps, has a push of its own).
#pragma once

#include "common.cuh"

#include <cooperative_groups.h>

namespace mlav {

constexpr int POOL_THREADS = 1024;

// What follows when a page's count fell from `had`: the one thread that took
// it from 1 to 0 marks the page in the bit map.  Returns the error bits.
__device__ __forceinline__ int mark_released(int page, int had, int32_t* page_refs, unsigned* page_bits) {
  if (had == 1) {
    atomicOr(page_bits + (page >> 5), 1u << (page & 31));
  } else if (had <= 0) {   // never raises a count to 1, so "1 to 0" stays unique
    atomicAdd(page_refs + page, 1);
    return ERR_REF;
  }
  return 0;
}
// One count less for `page`.
__device__ __forceinline__ int release_page(int page, int num_pages, int32_t* page_refs, unsigned* page_bits) {
  if (page < 0 || page >= num_pages) return ERR_SLOT;
  return mark_released(page, atomicSub(page_refs + page, 1), page_refs, page_bits);
}

// By a whole cluster of CTAs of POOL_THREADS: the marked pages, in order, on
// the stack of height `count`, and the bit map cleared for the next call.
__device__ __forceinline__ void push_marked(unsigned* page_bits, int num_pages, long long count, int32_t* free_pages,
                                            int32_t* free_count, int* err, int* s_warp, int& s_total) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  // (Volatile: the words were set by other SMs' atomics.)
  const volatile unsigned* bits = page_bits;
  // This CTA's words of the bit map, in order: `per` consecutive ones per thread.
  const int words = num_pages / 32 + (num_pages % 32 != 0);
  const int per = (words + ctas * POOL_THREADS - 1) / (ctas * POOL_THREADS);
  const long long w0 = (static_cast<long long>(rank) * POOL_THREADS + tid) * per;
  int mine = 0;
  for (int k = 0; k < per; ++k)
    if (w0 + k < words) mine += __popc(bits[w0 + k]);
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < POOL_THREADS / 32; ++w) {
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
      unsigned w = bits[w0 + k];
      if (w) page_bits[w0 + k] = 0;
      while (w) {
        const int bit = __ffs(static_cast<int>(w)) - 1;
        w &= w - 1;
        if (at < num_pages) free_pages[at] = static_cast<int32_t>((w0 + k) * 32 + bit);
        ++at;
      }
    }
  if (rank == 0 && tid == 0) {
    if (count + all > num_pages) atomicOr(err, ERR_CAPACITY);
    *free_count = static_cast<int32_t>(min(count + all, static_cast<long long>(num_pages)));
  }
  cluster.sync();   // no CTA leaves while another reads its total
}

}  // namespace mlav
