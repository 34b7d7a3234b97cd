// Eviction: requests cut down to the rows that were given most attention.
//
// A request of n rows that is over the budget keeps its first `sink` rows, its
// last `recent` rows and, of the others, those with the largest weights, the
// lowest index first among equals, `budget` in all and in their order.
//
// evict_select_kernel, a cluster of CTAs per request: the weights as ordered
// 32-bit keys in shared memory; the key of the last row that is kept by three
// histograms (11, 11 and 10 bits) that the cluster's CTAs add up through
// distributed shared memory; then one scan of the warps' counts gives every kept
// row its new place (rows above that key, rows equal to it, both in order).  Every CTA scans all
// requests' lengths itself for its place in the new tables and on the stack of
// free pages, as fork_kv does: how many entries stay follows from the lengths
// alone.  Pages of 64: those that hold protected leading rows alone stay, the
// kept rows behind them go to fresh pages (so that pages shared with other
// requests are not written, and no row is read after it was overwritten), all
// others of the table are given back.  Single slots: kept slots stay, no row
// moves.
// With pages, CTAs of evict_select_kernel that no request needs copy the protected
// rows meanwhile: those stay whatever the weights, and their places, too, follow
// from the lengths.
// evict_copy_kernel: the other kept rows of every layer into the fresh pages, and
// beside it the pages whose count fell to 0, in ascending order, onto the stack
// (evict_push_kernel where nothing is copied).
//
// The copies are bound by HBM (1152 bytes read and written a row and layer): 16
// requests cut to 2048 rows in 16 layers, 1.2 GB, take 193 us, 6.3 TB/s, with 256
// protected rows copied while the others are chosen (206 behind the choosing,
// which takes 24: 450 to 500 instructions a row on an SM per request, half of
// what it can issue in that time, barriers between; a cluster of two for these
// was no faster, its barriers taking what it gained).
// Single slots: 32 requests of 16 to 32 thousand take 55 us, the choosing 41 and
// the push 14.  The atomics on 655000 scattered counts and bits are 14 of the 55.
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
constexpr int ROWS_PER_CTA = 12288;        // from which a request gets another CTA, where SMs are left: a cluster barrier is ~1 us
constexpr int MAX_CACHED = 24576;          // keys that a CTA holds in shared memory
constexpr int GROUP = 32;                  // strips of THREADS rows placed by one scan
constexpr int FLIGHT = 6;                  // strips whose loads and atomics are under way together

// Larger weights have larger keys; -0 is 0, NaN is below every number.
__device__ __forceinline__ unsigned ordered(float w) {
  if (w != w) return 0;
  const unsigned u = __float_as_uint(w == 0.f ? 0.f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr unsigned PROTECTED = 0xffffffffu;   // no weight's key
// The weight of a key (a NaN for NaN, 0 for -0).
__device__ __forceinline__ float weight_of(unsigned key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }

// A request's rows and entries; nothing, with the error bit that says why, for
// one that is out of order.
struct Item {
  int n, m, ip0, entries;     // rows, kept rows, the table
  int stay;                   // entries that stay, in order: the first ones (pages), the kept ones (slots)
  int total, fresh;           // entries of the new table, of them fresh
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
    x.total = static_cast<int>((static_cast<long long>(x.m) + a.extra + a.page - 1) / a.page);
    x.fresh = x.total - x.stay;
  }
  if (x.bad) x.n = 0;
  return x;
}

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// Inclusive scan over a CTA of T threads; `all` receives the total.
template <int T>
__device__ __forceinline__ long long cta_scan(long long x, long long* s_warp, long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_scan(x, lane);
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  const long long y = warp_scan(lane < T / 32 ? s_warp[lane] : 0, lane);   // (by every warp: no third barrier)
  all = __shfl_sync(0xffffffffu, y, T / 32 - 1);
  const long long before = __shfl_sync(0xffffffffu, y, max(warp - 1, 0));
  return x + (warp ? before : 0);
}
// Two counts below 2^32 in one word.
__device__ __forceinline__ long long pair_of(int hi, int lo) { return static_cast<long long>(hi) << 32 | static_cast<unsigned>(lo); }
__device__ __forceinline__ long long high(long long x) { return x >> 32; }
__device__ __forceinline__ long long low(long long x) { return x & 0xffffffffll; }

// A warp's share, warp `w` of `warps`, of the protected rows of an evicted
// request that are copied early: those in its first fresh page before copy_from,
// and its kept rows from copy_to on, four rows of
// a layer at a time (with four layers, whose pages are looked up once, 16
// requests took 199 us, not 193).  `top` is the first of its fresh pages on the
// stack, the others lie below.
constexpr int EARLY_FLIGHT = 5;
constexpr long long EARLY_LEAST = 8192;   // rows, in all layers, that make up for the CTAs (260 made a call 2 us slower, 4160 gained nothing)
constexpr long long EARLY_MOST = 65536;   // that can be copied while rows are chosen: 151 MB (1536 recent ones, all early 205 us, up to here 193)
__device__ __noinline__ void copy_protected(const EvictArgs& a, int n, const int32_t* held, const int32_t* top, int w, int warps) {
  const int lane = threadIdx.x & 31, from = a.sink / PAGE * PAGE, lead = a.copy_from - from, rows = lead + a.budget - a.copy_to;
  const int quads = (rows + 3) / 4;
  const long long tasks = static_cast<long long>(quads) * a.num_layers;
  // Lane q, for row 4 quad + q % 4: its old and new page (-1: none), and the rows in them.
  int src = -1, dst = -1, places = 0;
  auto look_up = [&](long long task) {
    const int r = 4 * static_cast<int>(task % quads) + (lane & 3);
    src = dst = -1;
    if (task >= tasks || r >= rows) return;
    const int i = r < lead ? from + r : a.copy_to + r - lead, j = r < lead ? i : n - a.budget + i;
    const int old_page = held[j / PAGE], new_page = top[from / PAGE - i / PAGE];
    places = j % PAGE << 8 | i % PAGE;
    if (new_page >= 0 && new_page < a.num_pages) dst = new_page;
    if (old_page >= 0 && old_page < a.num_pages) src = old_page;
    else if (lane < 4) atomicOr(a.err, ERR_SLOT);   // no such page: zeros
  };
  look_up(w);
  for (long long task = w; task < tasks; task += warps) {
    uint16_t* layer = a.kv_cache + task / quads * a.layer_stride;
#pragma unroll
    for (int u0 = 0; u0 < 9; u0 += EARLY_FLIGHT) {
      uint4 v[EARLY_FLIGHT];
#pragma unroll
      for (int u = u0; u < min(u0 + EARLY_FLIGHT, 9); ++u) {
        const int e = lane + 32 * u, q = e / ROW_CHUNKS;
        const int page = __shfl_sync(0xffffffffu, src, q), row = __shfl_sync(0xffffffffu, places, q) >> 8;
        v[u - u0] = page >= 0 ? *(reinterpret_cast<const uint4*>(layer + (static_cast<long long>(page) * PAGE + row) * D_QK) + e % ROW_CHUNKS)
                              : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = u0; u < min(u0 + EARLY_FLIGHT, 9); ++u) {
        const int e = lane + 32 * u, q = e / ROW_CHUNKS;
        const int page = __shfl_sync(0xffffffffu, dst, q), row = __shfl_sync(0xffffffffu, places, q) & 255;
        if (page >= 0) *(reinterpret_cast<uint4*>(layer + (static_cast<long long>(page) * PAGE + row) * D_QK) + e % ROW_CHUNKS) = v[u - u0];
      }
    }
    look_up(task + warps);
  }
}

// grid: `ctas` CTAs (a cluster) per request, then CTAs that copy protected rows,
// as many for each request.  (The sums of all requests' entries stay below
// 2^31: so does max_batch * max_kv_len.)  EARLY: whether there are such CTAs (as
// one kernel, calls without them took 1 to 2 us longer).
template <bool EARLY>
__global__ void __launch_bounds__(THREADS, 1) evict_select_kernel(const __grid_constant__ EvictArgs a, int cached) {
  extern __shared__ unsigned s_keys[];
  __shared__ __align__(8) int s_hist[BINS];
  __shared__ int s_bins[WARPS];
  __shared__ long long s_warp[WARPS], s_place[GROUP * WARPS];
  __shared__ long long s_mine, s_fit, s_count;
  __shared__ unsigned long long s_last[2];
  __shared__ Item s_item;
  __shared__ int s_bin, s_above;
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  auto sync = [&]() {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int copier = EARLY ? static_cast<int>(blockIdx.x) - ctas * a.batch : -1;   // 0 and above: one that copies
  const int b = copier >= 0 ? copier % a.batch : static_cast<int>(blockIdx.x) / ctas;
  const float* row = a.weights + b * a.stride;
  const int height = *a.free_count;
  Item item{};
  if (tid < a.batch) item = load_item(a, tid);
  // A CTA that has the request alone loads the weights before it knows how many.
  const bool alone = ctas == 1 && a.max_kv_len <= cached && copier < 0;
  if (alone) {
#pragma unroll 8
    for (int i = tid; i < a.max_kv_len; i += THREADS) s_keys[i] = ordered(row[i]);
  }
  const bool height_ok = height >= 0 && height <= a.num_pages;
  const long long left = height_ok ? height : -1;   // a stack that is out of order serves nobody
  if (tid < 2) s_last[tid] = 0;
  long long before = 0;                             // entries, of them fresh
  for (int base = 0; base < a.batch; base += THREADS) {
    const int i = base + tid;
    if (base > 0) item = i < a.batch ? load_item(a, i) : Item{};
    if (i == b) s_item = item;
    const long long own = pair_of(item.total, item.fresh);
    long long all;
    const long long x = before + cta_scan<THREADS>(own, s_warp, all);
    if (i < a.batch) {
      if (high(x) <= a.capacity && low(x) <= left) {   // ends never fall: the largest that fits
        if (i <= b) atomicMax(&s_last[0], static_cast<unsigned long long>(high(x)));
        atomicMax(&s_last[1], static_cast<unsigned long long>(low(x)));
      }
      if (i == b) {
        s_mine = x - own;
        s_fit = x;
      }
    }
    before += all;
  }
  __syncthreads();
  const Item it = s_item;
  const bool fits = high(s_fit) <= a.capacity && low(s_fit) <= left;
  const bool served = fits && !it.bad;
  if (rank == 0 && tid == 0 && copier < 0) {
    if (it.bad) atomicOr(a.err, it.bad);
    if (!it.bad && !fits && (it.total > 0 || it.entries > 0)) atomicOr(a.err, ERR_CAPACITY);
    a.new_lens[b] = served ? it.m + a.extra : 0;
    a.new_indptr[b + 1] = static_cast<int32_t>(s_last[0]);
    if (b == 0) a.new_indptr[0] = 0;
  }
  const long long all_threads = static_cast<long long>(ctas) * THREADS, me = static_cast<long long>(rank) * THREADS + tid;
  float* new_row = a.new_weights + b * a.new_stride;
  // Behind the kept rows: 0.
  if (copier < 0)
    for (long long j = (served ? it.m : 0) + me; j < a.new_width; j += all_threads) new_row[j] = 0.f;
  // The last CTA that has read the height lowers it.
  auto lower = [&]() {
    if (tid != 0) return;
    if (gridDim.x > 1) {
      __threadfence();
      if (atomicAdd(a.ticket, 1u) != gridDim.x - 1) return;
      *a.ticket = 0;
    }
    if (height_ok) *a.free_count = static_cast<int32_t>(left - static_cast<long long>(s_last[1]));
    else atomicOr(a.err, ERR_CAPACITY);
  };
  if (!served || (copier >= 0 && it.n <= a.budget)) {   // the whole cluster
    lower();
    return;
  }

  const int n = it.n;
  const bool over = n > a.budget;
  const int32_t* held = a.kv_indices + it.ip0;
  int32_t* table = a.new_indices + high(s_mine);
  int errs = 0;
  // Entries: those that stay (pages), fresh ones, and those that are left.  Each
  // thread's first of both kinds is loaded here, and used at the end.
  const long long e0 = (a.page == 1 ? it.stay : 0) + me, l0 = (a.page == 1 ? n : it.stay) + me;
  auto entry_at = [&](long long e) { return e < it.stay ? held[e] : a.free_pages[left - 1 - (low(s_mine) + e - it.stay)]; };
  if (copier >= 0) {
    lower();
    const int part = copier / a.batch, parts = (static_cast<int>(gridDim.x) - ctas * a.batch) / a.batch;
    copy_protected(a, n, held, a.free_pages + (left - 1 - low(s_mine)), part * WARPS + warp, parts * WARPS);
    return;
  }
  const int first_entry = e0 < it.total ? entry_at(e0) : 0, first_left = l0 < it.entries ? held[l0] : 0;

  // This CTA's rows: strips of THREADS rows.
  const int strips_each = static_cast<int>((n + all_threads - 1) / all_threads);
  const int j0 = static_cast<int>(min(static_cast<long long>(rank) * strips_each * THREADS, static_cast<long long>(n)));
  const int count = min(strips_each * THREADS, n - j0), strips = (count + THREADS - 1) / THREADS;
  const bool in_smem = count <= cached;
  // A request over the budget: the `budget` rows with the largest keys are
  // kept, protected rows having a key above all others.  (The places behind
  // the last row have the lowest: the rows before them are more than enough.)
  const int lo = a.sink - j0, hi = n - a.recent - j0;   // rows before lo and from hi on are protected
  auto key_of = [&](int i) { return i >= count ? 0u : i < lo || i >= hi ? PROTECTED : ordered(row[j0 + i]); };
  auto key_at = [&](int i) { return in_smem ? s_keys[i] : key_of(i); };
  int k = a.budget;
  unsigned cut = PROTECTED;                    // the key of the last row that is kept
  int equal = 0;                               // of the rows with that key, how many
  if (over && k > 0) {
    if (alone) {
      for (int i = count + tid; i < strips * THREADS; i += THREADS) s_keys[i] = 0;
      for (int i = tid; i < lo; i += THREADS) s_keys[i] = PROTECTED;
      for (int i = hi + tid; i < count; i += THREADS) s_keys[i] = PROTECTED;
    } else if (in_smem) {
#pragma unroll 8
      for (int i = tid; i < strips * THREADS; i += THREADS) s_keys[i] = key_of(i);
    }
    unsigned prefix = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < BINS; i += THREADS) s_hist[i] = 0;
      __syncthreads();
      const unsigned mask = (1u << bits) - 1;
#pragma unroll 4
      for (int s = 0; s < strips; ++s) {
        const unsigned key = key_at(s * THREADS + tid);
        const bool mine = pass == 0 || key >> (shift + bits) == prefix;
        const unsigned bin = key >> shift & mask;
        // (Many rows of one weight: one addition for the warp.)
        if (__all_sync(0xffffffffu, mine) && __all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
          if (lane == 0) atomicAdd(s_hist + bin, 32);
        } else if (mine) {
          atomicAdd(s_hist + bin, 1);
        }
      }
      sync();
      // The bin, from the top, in which the k-th row lies: two bins per thread.
      const int top = BINS - 1 - 2 * tid;
      int h0 = 0, h1 = 0;
      if (ctas == 1) {
        const int2 h = *reinterpret_cast<const int2*>(s_hist + top - 1);
        h0 = h.y, h1 = h.x;
      } else {
#pragma unroll
        for (int r = 0; r < MAX_CTAS; ++r) {
          if (r >= ctas) continue;
          const int2 h = *reinterpret_cast<const int2*>(cluster.map_shared_rank(s_hist, r) + top - 1);
          h0 += h.y, h1 += h.x;
        }
      }
      // (The warp in which it lies, by every warp; the lane, by that one.)
      const int warp_sum = __reduce_add_sync(0xffffffffu, h0 + h1);
      if (lane == 0) s_bins[warp] = warp_sum;
      __syncthreads();
      int upto = s_bins[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int at = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, upto >= k))) - 1;
      const int earlier = at > 0 ? __shfl_sync(0xffffffffu, upto, max(at - 1, 0)) : 0;
      if (warp == at) {
        int end = h0 + h1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += y;
        }
        end += earlier;
        const int start = end - h0 - h1;
        if (start < k && k <= end) {
          const bool upper = k <= start + h0;
          s_bin = upper ? top : top - 1;
          s_above = upper ? start : start + h0;
        }
      }
      sync();   // histograms are read, s_bin is set
      prefix = (prefix << bits) | static_cast<unsigned>(s_bin);
      k -= s_above;
    }
    cut = prefix;
    equal = k;
  }
  // (Each thread's first entries: their counts answer while rows are placed.)
  auto put_entry = [&](long long e, int page) {   // the count that a fresh entry had
    table[e] = page;
    if (page < 0 || page >= a.num_pages) errs |= ERR_SLOT;
    else if (e >= it.stay) return atomicExch(a.page_refs + page, 1);
    return 0;
  };
  const int exchanged = e0 < it.total ? put_entry(e0, first_entry) : 0;
  int left_had = 2;
  if (l0 < it.entries) {
    if (first_left < 0 || first_left >= a.num_pages) errs |= ERR_SLOT;
    else left_had = atomicSub(a.page_refs + first_left, 1);
  }
  // Rows above the cut (or protected) and rows equal to it that lie before the
  // CTA's, then before each strip's and warp's: the kept rows' new places.
  long long base = 0;
  if (ctas > 1) {
    int above = 0, ties = 0;
#pragma unroll 4
    for (int s = 0; s < strips; ++s) {
      const int i = s * THREADS + tid;
      const unsigned key = over ? key_at(i) : 0;
      above += over ? key > cut : i < count;
      ties += over && key == cut;
    }
    long long all;
    cta_scan<THREADS>(pair_of(above, ties), s_warp, all);
    if (tid == 0) s_count = all;
    cluster.sync();
    for (int r = 0; r < rank; ++r) base += *cluster.map_shared_rank(&s_count, r);
  }
  for (int g0 = 0; g0 < strips; g0 += GROUP) {
    const int g1 = min(strips, g0 + GROUP), entries = (g1 - g0) * WARPS;
    // Rows that are kept (above the cut), and those with the cut's key, of
    // which the first `equal` are.
    auto strip = [&](int s, unsigned& key, unsigned& above, unsigned& ties) {
      const int i = s * THREADS + tid;
      key = over ? key_at(i) : 0;
      above = __ballot_sync(0xffffffffu, over ? key > cut : i < count);
      ties = __ballot_sync(0xffffffffu, over && key == cut);
    };
    __syncthreads();
#pragma unroll 4
    for (int s = g0; s < g1; ++s) {
      unsigned key, above, ties;
      strip(s, key, above, ties);
      if (lane == 0) s_place[(s - g0) * WARPS + warp] = pair_of(__popc(above), __popc(ties));
    }
    __syncthreads();
    const long long mine = tid < entries ? s_place[tid] : 0;
    long long all;
    const long long end = cta_scan<THREADS>(mine, s_warp, all);
    if (tid < entries) s_place[tid] = base + end - mine;
    base += all;
    __syncthreads();
    for (int s0 = g0; s0 < g1; s0 += FLIGHT) {
      int to[FLIGHT], slot[FLIGHT], had[FLIGHT];   // to: the new place, -1 dropped, -2 no row
      float w[FLIGHT];
#pragma unroll
      for (int u = 0; u < FLIGHT; ++u) {
        const int s = s0 + u, i = s * THREADS + tid;
        to[u] = -2;
        w[u] = 0.f;
        if (s < g1) {
          unsigned key, above, ties;
          strip(s, key, above, ties);
          const long long place = s_place[(s - g0) * WARPS + warp];
          const unsigned lower = (1u << lane) - 1;
          const int e = static_cast<int>(low(place)) + __popc(ties & lower);
          if (i < count)
            to[u] = (above >> lane & 1) || ((ties >> lane & 1) && e < equal)
                        ? static_cast<int>(high(place)) + __popc(above & lower) + min(e, equal)
                        : -1;
          if (to[u] >= 0) w[u] = over && key != PROTECTED ? weight_of(key) : row[j0 + i];
        }
        slot[u] = a.page == 1 && to[u] != -2 ? held[j0 + i] : 0;
      }
      if (a.page > 1) {
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u)
          if (to[u] >= 0) {
            new_row[to[u]] = w[u];
            if (over) a.kept[b * a.kept_stride + to[u]] = j0 + (s0 + u) * THREADS + tid;
          }
        continue;
      }
#pragma unroll
      for (int u = 0; u < FLIGHT; ++u) {
        had[u] = 2;
        if (to[u] == -2) continue;
        if (slot[u] < 0 || slot[u] >= a.num_pages) errs |= ERR_SLOT;
        else if (to[u] == -1) had[u] = atomicSub(a.page_refs + slot[u], 1);
        if (to[u] >= 0) {
          new_row[to[u]] = w[u];
          table[to[u]] = slot[u];
        }
      }
#pragma unroll
      for (int u = 0; u < FLIGHT; ++u) errs |= mark_released(slot[u], had[u], a.page_refs, a.page_bits);
    }
  }
  if (exchanged != 0) errs |= ERR_REF;   // the stack held a page that is in use
  for (long long e = e0 + all_threads; e < it.total; e += all_threads)
    if (put_entry(e, entry_at(e)) != 0) errs |= ERR_REF;
  errs |= mark_released(first_left, left_had, a.page_refs, a.page_bits);
  for (long long e = l0 + all_threads; e < it.entries; e += all_threads)
    errs |= release_page(held[e], a.num_pages, a.page_refs, a.page_bits);
  if (errs) atomicOr(a.err, errs);
  lower();
  if (ctas > 1) cluster.sync();   // no CTA leaves while another reads its count
}

// By `parts` CTAs of T threads: the marked pages, in order, on the stack of
// height `count`.  Each CTA adds up the words before its own; the last one
// done clears the bit map for the next call and raises the height.
template <int T>
__device__ __forceinline__ void push_marked_part(const EvictArgs& a, int part, int parts, long long count, long long* s_warp, int& s_done) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = a.num_pages / 32 + (a.num_pages % 32 != 0);
  const int each = ((words + parts - 1) / parts + T - 1) / T * T;
  const int w0 = static_cast<int>(min(static_cast<long long>(part) * each, static_cast<long long>(words))), w1 = min(words, w0 + each);
  int sum = 0;
#pragma unroll 8
  for (int w = 4 * tid; w < w0; w += 4 * T) {   // (w0 is a multiple of four)
    const uint4 x = __ldcg(reinterpret_cast<const uint4*>(a.page_bits + w));
    sum += __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w);
  }
  long long before = 0, all = 0;
  if (part > 0) cta_scan<T>(sum, s_warp, before);
  for (int w = w0; w < w1; w += T) {
    const unsigned word = w + tid < w1 ? __ldcg(a.page_bits + w + tid) : 0;
    const int mine = __popc(word);
    long long these;
    const long long at = count + before + all + cta_scan<T>(mine, s_warp, these) - mine;
    all += these;
    // A warp writes out its 32 words one by one, a lane per bit.
    const long long warp_at = __shfl_sync(0xffffffffu, at, 0);
    const int off = static_cast<int>(at - warp_at);
    auto put = [&](int k) {
      const unsigned x = __shfl_sync(0xffffffffu, word, k);
      const long long to = warp_at + __shfl_sync(0xffffffffu, off, k) + __popc(x & ((1u << lane) - 1));
      if ((x >> lane & 1u) && to < a.num_pages) a.free_pages[to] = (w + warp * 32 + k) * 32 + lane;
    };
    unsigned some = __ballot_sync(0xffffffffu, word != 0);
    if (__popc(some) > 8) {
#pragma unroll 8
      for (int k = 0; k < 32; ++k) put(k);
    } else {
      for (; some; some &= some - 1) put(__ffs(static_cast<int>(some)) - 1);
    }
  }
  __syncthreads();
  if (tid == 0) {
    int done = 1;
    if (parts > 1) {
      atomicAdd(a.ticket + 2, static_cast<unsigned>(all));
      __threadfence();
      done = atomicAdd(a.ticket + 1, 1u) == static_cast<unsigned>(parts) - 1;
      __threadfence();
    }
    s_done = done;
    if (done) {
      const long long pushed = parts > 1 ? static_cast<long long>(atomicExch(a.ticket + 2, 0u)) : all;
      a.ticket[1] = 0;
      if (count + pushed > a.num_pages) atomicOr(a.err, ERR_CAPACITY);
      *a.free_count = static_cast<int32_t>(min(count + pushed, static_cast<long long>(a.num_pages)));
    }
  }
  __syncthreads();
  if (s_done)
    for (int w = 4 * tid; w < words; w += 4 * T)   // (the map is padded to 16 bytes)
      *reinterpret_cast<uint4*>(a.page_bits + w) = make_uint4(0, 0, 0, 0);
}

// Rows of an evicted request, COPY_ROWS at a time, in some of the layers: nine
// 16-byte granules in flight per lane (a warp takes four rows).
constexpr int COPY_THREADS = 256, COPY_ROWS = COPY_THREADS / 32 * 4;

// The grid's last column in x pushes the marked pages while the others copy.
__global__ void __launch_bounds__(COPY_THREADS) evict_copy_kernel(const EvictArgs a, int layers_each) {
  __shared__ long long s_src[COPY_ROWS], s_dst[COPY_ROWS];
  __shared__ long long s_warp[COPY_THREADS / 32];
  __shared__ int s_done;
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  const int tid = threadIdx.x;
  if (blockIdx.x == gridDim.x - 1) {
    const long long count = *a.free_count;
    if (blockIdx.y == 0 && blockIdx.z == 0 && count >= 0 && count <= a.num_pages)   // (else reported, and nothing was given back)
      push_marked_part<COPY_THREADS>(a, 0, 1, count, s_warp, s_done);
    return;
  }
  const int i0 = a.copy_from + static_cast<int>(blockIdx.x) * COPY_ROWS;
  for (int b = blockIdx.y; b < a.batch; b += gridDim.y) {
    // (A request that is not served has length 0; a length of 0 has no rows.)
    if (a.new_lens[b] == 0 || a.kv_lens[b] <= a.budget) continue;
    const int rows = min(COPY_ROWS, a.copy_to - i0);
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

__global__ void __launch_bounds__(THREADS) evict_push_kernel(const EvictArgs a) {
  __shared__ long long s_warp[WARPS];
  __shared__ int s_done;
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  const long long count = *a.free_count;
  if (count < 0 || count > a.num_pages) return;   // (reported, and nothing was given back)
  push_marked_part<THREADS>(a, blockIdx.x, gridDim.x, count, s_warp, s_done);
}

}  // namespace

cudaError_t evict_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_CACHED * 4);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_CACHED * 4);
}

cudaError_t launch_evict_kv(const EvictArgs& args, int num_sms, cudaStream_t stream) {
  EvictArgs a = args;
  // CTAs per request: more for long ones, while they fill no SM twice.
  int ctas = 1;
  while (ctas < MAX_CTAS && 2LL * ctas * a.batch <= num_sms && a.max_kv_len > ROWS_PER_CTA * ctas) ctas *= 2;
  const long long strips = (a.max_kv_len + static_cast<long long>(ctas) * THREADS - 1) / (static_cast<long long>(ctas) * THREADS);
  const int cached = static_cast<int>(std::min<long long>(strips * THREADS, MAX_CACHED));
  // The SMs that are left copy protected rows, where those are enough.
  a.copy_from = a.sink / PAGE * PAGE;
  a.copy_to = std::min(a.budget, a.max_kv_len);
  int copiers = 0;
  if (a.page > 1 && a.budget < a.max_kv_len) {
    const long long each = static_cast<long long>(a.batch) * a.num_layers;   // rows of the call per row of a request
    const int lead = a.sink - a.copy_from, early = lead + static_cast<int>(std::min<long long>(a.recent, EARLY_MOST / each));
    const long long tasks = (early + 3LL) / 4 * a.num_layers, enough = ((tasks + WARPS - 1) / WARPS + ctas - 1) / ctas * ctas;
    if (early * each >= EARLY_LEAST)
      copiers = static_cast<int>(std::clamp<long long>((num_sms - ctas * a.batch) / a.batch / ctas * ctas, 0, enough));
    if (copiers > 0) a.copy_from = a.sink, a.copy_to -= early - lead;
  }
  cudaError_t e = launch_overlapping(copiers > 0 ? evict_select_kernel<true> : evict_select_kernel<false>,
                                     dim3(static_cast<unsigned>(ctas + copiers) * a.batch), THREADS, static_cast<size_t>(cached) * 4,
                                     stream, static_cast<unsigned>(ctas), a, cached);
  if (e != cudaSuccess) return e;
  const int moved = a.copy_to - a.copy_from;
  if (a.page > 1 && moved > 0) {
    const unsigned parts = static_cast<unsigned>((moved + COPY_ROWS - 1) / COPY_ROWS);
    const unsigned requests = static_cast<unsigned>(std::min(a.batch, 65535));
    // A CTA's rows are looked up once for several layers, where enough CTAs are left.
    const long long ctas_of_a_layer = static_cast<long long>(parts) * requests;
    const int each = std::max(static_cast<int>(std::clamp<long long>(ctas_of_a_layer * a.num_layers / (16LL * num_sms), 1, 16)),
                              (a.num_layers + 65534) / 65535);
    const unsigned z = static_cast<unsigned>((a.num_layers + each - 1) / each);
    return launch_overlapping(evict_copy_kernel, dim3(parts + 1, requests, z), COPY_THREADS, 0, stream, 1, a, each);
  }
  // A word per thread, as long as the words before a CTA's are soon added up.
  const unsigned push = static_cast<unsigned>(std::clamp((a.num_pages / 32 + THREADS - 1) / THREADS, 1, 128));
  return launch_overlapping(evict_push_kernel, dim3(push), THREADS, 0, stream, 1, a);
}

}  // namespace mlav
