// The attention weight that new tokens give to each cached row, added up.
//
// For request b with n rows and c new tokens (the last rows), key j:
//     weights[b][j] += sum over tokens i >= j - (n - c) and heads h of
//                      exp(scale * dot(q[i][h], k_j) - lse[i][h])
// with the log-sum-exp that the attention of these tokens left: one pass, no
// maxima, and a sum over the query rows, not over the keys.
//
// weigh_kernel: a persistent kernel on CTA pairs (tcgen05 cta_group::2).  A
// block of 256 keys (128 a CTA) stays in shared memory while the request's
// query rows pass it in tiles of 256:
//     S^T[key, row] = K_block[256 x 576] . Q_tile[256 x 576]^T   in bf16, fp32 sums
// so a key is a lane of tensor memory and its weight a sum in a thread's
// register: no shuffles, no atomics, one order.  Keys come straight from the
// cache (TMA boxes of a page, or 16-byte copies of single slots' rows), in nine slots
// of 64 dims of which each is refilled as soon as the block's last tile has
// read it; queries come through a ring of four slots of 64 dims.  bf16
// products are exact and nothing is widened, so no value is out of range.
// The steps (a tile against a block) of all requests are divided evenly over
// the clusters in closed form (weigh_steps.h), by every CTA for itself.
//
// Where clusters share a block, the last of them to be done adds up all sums,
// in cluster order (a launch for that took 2.5 us).
//
// What bounds it: with many query rows the tensor cores and the queries' way
// from L2 (16 KB a slot and CTA for 256 x 256 x 64 products): 256 tokens of 64
// heads on 33000 rows take 328 us, 1.89 PFLOP/s, a step 2.85 us.  One load of
// 16 KB per slot: with four of 4 KB they took 449 us, a step 3.9.  With few rows it is
// the keys' bytes: 16 decoding requests on 160000 rows take 43 us, 4.3 TB/s,
// of which some 10 us are the launch, the division and the first block.
//
// Roles (24 warps per CTA): warps 0-15 take the scores, warp 16 issues MMAs
// (even CTA), warp 17 loads queries, warps 18 and 19 keys, warps 20-23 hand
// gathered keys over.  Every wait is bounded; a
// pair whose wait runs out leaves NaN in all of its blocks.
#include "kernels.h"
#include "pair_common.cuh"
#include "weigh_steps.h"

#include <algorithm>

namespace mlav {
namespace {

constexpr int KEYS = 256, TILE = 256;       // keys of a block, query rows of a tile
constexpr int HKEYS = KEYS / 2;             // keys of a CTA
constexpr int SCORE_WARPS = 16, MMA_WARP = 16, Q_WARP = 17, K_WARP = 18;
constexpr int K_WARPS = 2;                  // that gather slots; a page's boxes are loaded by the first
constexpr int RELAY_WARP = K_WARP + K_WARPS, RELAYS = 4;   // that hand gathered chunks over
constexpr int NWARPS = RELAY_WARP + RELAYS, NTHREADS = NWARPS * 32;
constexpr int NCHUNK = 9;                   // chunks of 64 dims
constexpr int K_SLOT = HKEYS * 128;         // 16 KB: 128 keys x 64 dims
constexpr int Q_SLOT = (TILE / 2) * 128;    // 16 KB: 128 rows x 64 dims
constexpr int NQ = 4;
constexpr int Q_BOX = 32, Q_FULL = TILE / 2;   // rows of a query load: of part of a tile's half, of all of it
constexpr int OFF_K = 0;
constexpr int OFF_Q = OFF_K + NCHUNK * K_SLOT;
constexpr int OFF_LSE = OFF_Q + NQ * Q_SLOT;                // float [16 warps][64] log-sum-exps of a warp's columns
constexpr int OFF_SUM = OFF_LSE + SCORE_WARPS * 64 * 4;     // float [2][4][128] a block's sums by column group
constexpr int OFF_MBAR = OFF_SUM + 2 * 4 * HKEYS * 4;
constexpr int MB_KF = 0;     // [9] even CTA: key slot landed in both CTAs (see MB_KL)
constexpr int MB_KE = 9;     // [9] key slot read by its block's last MMAs
constexpr int MB_QF = 18;    // [4] even CTA: query slot landed in both CTAs
constexpr int MB_QE = 22;    // [4] query slot read
constexpr int MB_SF = 26;    // [2] scores of a step done
constexpr int MB_SE = 28;    // [2] even CTA: scores of a step read by both CTAs' warps
constexpr int MB_DONE = 30;  // after an abort: every MMA issued is done
constexpr int MB_KL = 31;    // [9] gathered keys: the slot's copies landed in this CTA (MB_KF: in the odd one)
constexpr int NMBAR = 40;
constexpr int OFF_MISC = OFF_MBAR + NMBAR * 8;              // tmem base, abort flag, the peer's, "the last to be done"
constexpr int OFF_PLAN = OFF_MISC + 16;                     // Cursor: the start of the share
constexpr int OFF_SCAN = OFF_PLAN + 128;                    // long long [warps]
constexpr int SMEM_TOTAL = OFF_SCAN + 32 * 8;
static_assert(SMEM_TOTAL <= 232448, "shared memory budget");
static_assert(OFF_MISC % 16 == 0 && OFF_PLAN % 16 == 0, "alignment");
constexpr int TMEM_COLS = 512;              // two buffers of 256 columns
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride 1024 bytes, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFF) | (16u >> 4) << 16; }

// Testing: the query slot before which WeighParams::fault_rank's CTA gives up
// (in the second step of its share).
constexpr int FAULT_SLOT = NCHUNK + 3;

// A request as every role derives it.
struct Request {
  int n, c, cached, ip0, q0;
  WeighSteps s;
};
// False (and no steps) for a request that cannot be served or has no new
// tokens; `errs` receives why.
__device__ __forceinline__ bool load_request(const WeighParams& p, int b, Request& r, int& errs) {
  r.n = p.kv_lens[b];
  r.ip0 = p.kv_indptr[b];
  r.q0 = p.q_indptr[b];
  const int ip1 = p.kv_indptr[b + 1], ipn = p.kv_indptr[p.batch], q1 = p.q_indptr[b + 1];
  r.c = q1 - r.q0;
  r.cached = r.n - r.c;
  r.s = WeighSteps();
  const long long need = p.page_size == 1 ? r.n : (static_cast<long long>(r.n) + PAGE - 1) / PAGE;
  if (r.q0 < 0 || q1 < r.q0 || q1 > p.num_tokens) {
    errs |= ERR_INDPTR;
  } else if (r.c == 0) {   // may hold anything: an idle slot of a batch
    return false;
  } else if (r.n < r.c || r.n < 0 || r.n > p.max_kv_len) {
    errs |= ERR_LEN;
  } else if (r.ip0 < 0 || ip1 < r.ip0 || ip1 > ipn || static_cast<long long>(ip1) - r.ip0 != need) {
    errs |= ERR_INDPTR;
  } else {
    r.s = WeighSteps(r.n, r.c, p.H);
    return true;
  }
  return false;
}

// Where a role is: tile `t` of block `kb` of request `b`, whose first tile for
// this cluster was t0.
struct Cursor {
  Request r;
  long long left;   // steps, this one among them; 0: the cluster has none
  long long done, total;   // steps of the call before t0, and all
  int b, kb, t, t0;
  // Tiles of this block that are the cluster's: t0 .. end - 1.
  __device__ __forceinline__ int end() const {
    return static_cast<int>(min(r.s.tiles, static_cast<long long>(t) + left));
  }
  // To the next block (the tiles up to end() are done); false at the end.
  __device__ __forceinline__ bool next_block(const WeighParams& p) {
    const int tiles = end() - t;
    left -= tiles;
    done += tiles;
    if (left <= 0) return false;
    if (++kb == r.s.blocks) {
      int errs = 0;
      do {
        if (++b >= p.batch) return false;   // (there is one: `left` says so)
      } while (!load_request(p, b, r, errs));
      kb = 0;
    }
    t = t0 = static_cast<int>(r.s.first(kb));
    return true;
  }
};
static_assert(sizeof(Cursor) <= OFF_SCAN - OFF_PLAN, "shared memory");

__device__ __forceinline__ uint32_t idesc(int rows) {   // bf16, both K-major
  return tc::idesc_f16(KEYS, 0, 1, 0, 0) | static_cast<uint32_t>(rows >> 3) << 17;
}
// Columns of a tile: 32 at a time, as a pair's MMA takes them.
__device__ __forceinline__ int tile_columns(const Request& r, int H, int t) {
  return static_cast<int>(min(static_cast<long long>(TILE), (static_cast<long long>(r.c) * H - static_cast<long long>(t) * TILE + 31) / 32 * 32));
}

// The division: every CTA adds up all requests' steps itself (one round of
// loads per NTHREADS requests) and takes its cluster's even share.
__device__ __forceinline__ void plan_share(const WeighParams& p, int cluster, Cursor* start, long long* s_warp, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Request r;
  int errs = 0;
  long long own = 0;
  auto load = [&](int b) {
    own = 0;
    if (b < p.batch && load_request(p, b, r, errs)) own = r.s.total();
  };
  // The cluster's share starts in request b, `sum` - own steps of the call
  // before it: one thread's.
  auto place = [&](int b, long long sum, long long total) {
    const long long used = min(static_cast<long long>(p.clusters), total);
    if (cluster >= used) return;
    const long long from = total * cluster / used, to = total * (cluster + 1) / used;
    if (own == 0 || sum - own > from || from >= sum) return;
    Cursor c;
    c.r = r;
    c.left = to - from;
    c.done = from;
    c.total = total;
    c.b = b;
    const long long step = from - (sum - own);
    c.kb = static_cast<int>(r.s.block_at(step));
    c.t = c.t0 = static_cast<int>(r.s.first(c.kb) + step - r.s.before(c.kb));
    *start = c;
  };
  if (p.batch <= 32) {   // a warp's work, and no barrier
    if (warp != 0) return;
    load(lane);
    if (lane == 0) start->left = 0;
    const bool undivided = lane < p.batch && (r.q0 < 0 || r.c < 0 || r.q0 > p.num_tokens - r.c);
    if (__any_sync(0xffffffffu, undivided)) {
      if (report && lane == 0) atomicOr(p.err, ERR_INDPTR);
      return;
    }
    if (report && errs) atomicOr(p.err, errs);
    long long sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    place(lane, sum, __shfl_sync(0xffffffffu, sum, 31));
    return;
  }
  // Inclusive sum over the CTA's threads.
  auto scan = [&](long long x, long long& all) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    all = 0;
    for (int w = 0; w < NWARPS; ++w) {
      if (w == warp) x += all;
      all += s_warp[w];
    }
    return x;
  };
  load(tid);
  // (tokens that are not divided: nothing is weighed)
  bool bad = false;
  for (int b = tid; b < p.batch; b += NTHREADS) {
    const int q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
    bad |= q0 < 0 || q1 < q0 || q1 > p.num_tokens;
  }
  if (tid == 0) start->left = 0;
  if (__syncthreads_or(bad)) {
    if (report && tid == 0) atomicOr(p.err, ERR_INDPTR);
    return;
  }
  long long all, total, sum = scan(own, total);
  for (int b0 = NTHREADS; b0 < p.batch; b0 += NTHREADS) {
    load(b0 + tid);
    scan(own, all);
    total += all;
  }
  if (report && errs) atomicOr(p.err, errs);
  long long before = 0;
  for (int b0 = 0; b0 < p.batch; b0 += NTHREADS) {
    if (p.batch > NTHREADS) {
      load(b0 + tid);
      sum = before + scan(own, all);
      before += all;
    }
    place(b0 + tid, sum, total);
  }
}

// Bounded wait of a warp; PEER: for barriers that the peer's threads arrive on.
template <bool PEER>
__device__ __forceinline__ void wait_bar(uint32_t mbar, uint32_t parity, volatile int* abort, int* err) {
  if (!(PEER ? tc::mbar_try_cluster(mbar, parity) : tc::mbar_try(mbar, parity))) {
    const long long t0 = clock64();
    while (!(PEER ? tc::mbar_try_cluster(mbar, parity) : tc::mbar_try(mbar, parity))) {
      if (*abort) break;
      if (clock64() - t0 > WAIT_LIMIT) {
        *abort = 1;
        atomicOr(err, ERR_TIMEOUT);
        break;
      }
    }
  }
  __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    weigh_kernel(const WeighParams p, const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_q_full) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t rank = tc::cluster_rank(), peer = rank ^ 1u;
  const int cluster = blockIdx.x >> 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  volatile int* s_last = reinterpret_cast<volatile int*>(smem + OFF_MISC + 12);
  Cursor* s_start = reinterpret_cast<Cursor*>(smem + OFF_PLAN);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t mbar0 = sbase + OFF_MBAR;
  auto mbar = [&](int i) { return mbar0 + 8u * static_cast<uint32_t>(i); };
  if (tid == 0) {
    for (int i = 0; i < NMBAR; ++i)
      tc::mbar_init(mbar(i), i == MB_SE || i == MB_SE + 1 ? 2 * SCORE_WARPS : i >= MB_KL ? K_WARPS * 32 : i < MB_KF + NCHUNK && p.page_size == 1 ? 2 : 1);
    tc::mbar_fence_init();
    s_abort[0] = s_abort[1] = 0;
  }
  if (warp == MMA_WARP) tc::tmem_alloc_pair<TMEM_COLS>(smem_u32(s_tmem));
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync_relaxed();   // the peer's barriers exist and the pair's TMEM is allocated
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const uint32_t even_mbar0 = tc::peer_addr(mbar0, 0);
  auto even_mbar = [&](int i) { return even_mbar0 + 8u * static_cast<uint32_t>(i); };
  // Everything read from here on may have been written by the kernel before.
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  plan_share(p, cluster, s_start, reinterpret_cast<long long*>(smem + OFF_SCAN), blockIdx.x == 0);
  __syncthreads();
  Cursor at = *s_start;
  const bool working = at.left > 0 && !(sbase & 1023);
  if (sbase & 1023 && tid == 0) {   // the swizzled tiles need it (uniform over the pair)
    atomicOr(p.err, ERR_INTERNAL);
    *s_abort = 1;
  }

  if (working) {
    if (warp == Q_WARP) {
      int n = 0;   // slots filled
      do {
        const int end = at.end();
#pragma unroll 1
        for (int t = at.t; t < end && !*s_abort; ++t) {
          const int half = tile_columns(at.r, p.H, t) / 2, boxes = (half + Q_BOX - 1) / Q_BOX;
          const int row0 = at.r.q0 * p.H + t * TILE + static_cast<int>(rank) * half;
#pragma unroll 1
          for (int c = 0; c < NCHUNK; ++c, ++n) {
            const int slot = n % NQ;
            if (n >= NQ) wait_bar<false>(mbar(MB_QE + slot), static_cast<uint32_t>((n / NQ - 1) & 1), s_abort, p.err);
            if (n == FAULT_SLOT && p.fault_rank == static_cast<int>(rank)) *s_abort = 1;   // (testing)
            if (*s_abort) break;
            if (rank == 0) {
              if (lane == 0) tc::mbar_arrive_expect(mbar(MB_QF + slot), 2 * boxes * Q_BOX * 128);
              __syncwarp();
            }
            if (half == Q_FULL)
              tc::tma_load_2d_pair(sbase + OFF_Q + slot * Q_SLOT, &tm_q_full, 64 * c, row0, even_mbar(MB_QF + slot));
            else
              for (int x = 0; x < boxes; ++x)
                tc::tma_load_2d_pair(sbase + OFF_Q + slot * Q_SLOT + x * Q_BOX * 128, &tm_q, 64 * c, row0 + x * Q_BOX,
                                     even_mbar(MB_QF + slot));
          }
        }
      } while (!*s_abort && at.next_block(p));
    } else if (warp >= RELAY_WARP) {
      // Gathered chunks, once they landed, to the even CTA's MMA warp, in turn.
      // The fence that shows ordinary writes to the tensor cores takes some
      // 1500 cycles beside copies under way: by the MMA warp itself, chunk by
      // chunk, it was the bound (16 decoding requests 80 us).
      if (p.page_size == 1) {
        int n = warp - RELAY_WARP;   // the chunk in the cluster's share
        int blk = 0;
        do {
          for (; n < (blk + 1) * NCHUNK && !*s_abort; n += RELAYS) {
            const int c = n % NCHUNK;
            wait_bar<false>(mbar(MB_KL + c), static_cast<uint32_t>(blk & 1), s_abort, p.err);
            tc::fence_async_smem();
            if (lane == 0 && *s_abort == 0) tc::mbar_arrive_cluster(even_mbar(MB_KF + c));
            __syncwarp();
          }
          ++blk;
        } while (!*s_abort && at.next_block(p));
      }
    } else if (warp >= K_WARP && p.page_size == 1) {
      // Slots, gathered by 16-byte copies: a warp has 64 of the CTA's 128 keys,
      // eight lanes a row of 128 bytes, four rows at a time.  (tile::gather4,
      // four rows an instruction, took 80 cycles each: 12 us a block.)  A
      // thread's copies arrive on the slot's barrier by themselves.
      constexpr int ROWS = HKEYS / K_WARPS, COPIES = ROWS / 4;
      static_assert(ROWS == 64, "two rows per lane");
      const int kw = warp - K_WARP, r4 = lane >> 3, col = lane & 7;
      int next[2];   // the slots of the block's rows kw * 64 + lane, + 32
      auto look_up = [&](const Cursor& c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = c.kb * KEYS + static_cast<int>(rank) * HKEYS + kw * ROWS + 32 * i + lane;
          next[i] = j < c.r.n ? p.kv_indices[c.r.ip0 + j] : 0;
        }
      };
      look_up(at);
      int blk = 0;
      bool more = true;
      while (more) {
        // Rows behind the request's last and bad slots: row 0, whose scores
        // nobody takes.
        const bool bad0 = next[0] < 0 || next[0] >= p.num_slots, bad1 = next[1] < 0 || next[1] >= p.num_slots;
        if (__any_sync(0xffffffffu, bad0 || bad1) && lane == 0) atomicOr(p.err, ERR_SLOT);
        if (bad0) next[0] = 0;
        if (bad1) next[1] = 0;
        int slot[COPIES];   // of rows 4 i + r4
#pragma unroll
        for (int i = 0; i < COPIES; ++i) slot[i] = __shfl_sync(0xffffffffu, next[i >= COPIES / 2], (4 * i + r4) & 31);
        more = at.next_block(p);
        if (more) look_up(at);   // (arrives while this block's rows are on their way)
#pragma unroll 1
        for (int c = 0; c < NCHUNK; ++c) {
          if (blk > 0) wait_bar<false>(mbar(MB_KE + c), static_cast<uint32_t>((blk - 1) & 1), s_abort, p.err);
          if (*s_abort) break;
          // Rows 4 i + r4: their swizzle alternates.
          const uint32_t dst = sbase + OFF_K + c * K_SLOT + kw * ROWS * 128 + r4 * 128;
          const uint32_t even = (col ^ r4) << 4, odd = (col ^ (r4 + 4)) << 4;
          const uint16_t* src = p.kv + 64 * c + 8 * col;
#pragma unroll
          for (int i = 0; i < COPIES; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst + i * 512 + (i & 1 ? odd : even)),
                         "l"(src + static_cast<long long>(slot[i]) * D_QK)
                         : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(mbar(MB_KL + c)) : "memory");
        }
        if (*s_abort) break;
        ++blk;
      }
      asm volatile("cp.async.wait_all;\n" ::: "memory");
    } else if (warp == K_WARP) {
      // Pages: two boxes a chunk.  Pages behind the request's last and bad
      // ones: page 0, whose scores nobody takes.
      int blk = 0, next;   // the block's page, of lanes 0 and 1
      auto look_up = [&](const Cursor& c) {
        const int j = c.kb * KEYS + static_cast<int>(rank) * HKEYS + (lane & 1) * PAGE;
        next = j < c.r.n ? p.kv_indices[c.r.ip0 + j / PAGE] : 0;
      };
      look_up(at);
      bool more = true;
      while (more) {
        const bool bad = next < 0 || next >= p.num_slots / PAGE;
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err, ERR_SLOT);
        const int row = bad ? 0 : next * PAGE;
        const int row0 = __shfl_sync(0xffffffffu, row, 0), row1 = __shfl_sync(0xffffffffu, row, 1);
        more = at.next_block(p);
        if (more) look_up(at);
#pragma unroll 1
        for (int c = 0; c < NCHUNK; ++c) {
          if (c == 1 && more) {   // the next block's pages into L2, a lane per 1/9 of one
            const int page = __shfl_sync(0xffffffffu, next, lane >= NCHUNK ? 1 : 0);
            if (lane < 2 * NCHUNK && page >= 0 && page < p.num_slots / PAGE)
              tc::prefetch_l2(p.kv + static_cast<long long>(page) * PAGE * D_QK + (lane % NCHUNK) * (PAGE * 64), PAGE * 128);
            __syncwarp();
          }
          if (blk > 0) wait_bar<false>(mbar(MB_KE + c), static_cast<uint32_t>((blk - 1) & 1), s_abort, p.err);
          if (*s_abort) break;
          if (rank == 0) {
            if (lane == 0) tc::mbar_arrive_expect(mbar(MB_KF + c), 2 * K_SLOT);
            __syncwarp();
          }
          const uint32_t dst = sbase + OFF_K + c * K_SLOT;
          tc::tma_load_2d_pair(dst, &tm_kv, 64 * c, row0, even_mbar(MB_KF + c));
          tc::tma_load_2d_pair(dst + K_SLOT / 2, &tm_kv, 64 * c, row1, even_mbar(MB_KF + c));
        }
        if (*s_abort) break;
        ++blk;
      }
    } else if (warp == MMA_WARP && rank == 0) {
      int n = 0, g = 0, blk = 0;   // query slots, steps, blocks so far
      do {
        const int end = at.end();
#pragma unroll 1
        for (int t = at.t; t < end && !*s_abort; ++t, ++g) {
          const uint32_t d = tmem + 256u * static_cast<uint32_t>(g & 1), shape = idesc(tile_columns(at.r, p.H, t));
          if (g >= 2) wait_bar<true>(mbar(MB_SE + (g & 1)), static_cast<uint32_t>((g / 2 - 1) & 1), s_abort, p.err);
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < NCHUNK; ++c, ++n) {
            const int slot = n % NQ;
            if (t == at.t) wait_bar<true>(mbar(MB_KF + c), static_cast<uint32_t>(blk & 1), s_abort, p.err);
            wait_bar<false>(mbar(MB_QF + slot), static_cast<uint32_t>((n / NQ) & 1), s_abort, p.err);
            if (*s_abort) break;
            tc::fence_after_sync();
            if (tc::elect_one()) {
              const uint32_t a = desc_lo(sbase + OFF_K + c * K_SLOT), b = desc_lo(sbase + OFF_Q + slot * Q_SLOT);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_pair_one(d, a + 2 * kk, b + 2 * kk, DESC_HI, shape, (c > 0 || kk > 0) ? 1u : 0u);
              tc::commit_pair_one(mbar(MB_QE + slot));
              if (t == end - 1) tc::commit_pair_one(mbar(MB_KE + c));
              if (c == NCHUNK - 1) tc::commit_pair_one(mbar(MB_SF + (g & 1)));
            }
            __syncwarp();
          }
        }
        ++blk;
      } while (!*s_abort && at.next_block(p));
    } else if (warp < SCORE_WARPS) {
      const int quad = warp & 3, grp = warp >> 2;   // TMEM lanes 32 quad .., columns 64 grp ..
      float* s_lse = reinterpret_cast<float*>(smem + OFF_LSE) + warp * 64;
      const int key = quad * 32 + lane;             // of the CTA's 128
      const float scale = p.scale_log2;
      int g = 0, blk = 0;
      do {
        const int end = at.end(), H = p.H;
        const int j = at.kb * KEYS + static_cast<int>(rank) * HKEYS + key;
        // Rows of the request before this one do not see the key.
        const int sees = max(0, min(j, at.r.n - 1) - at.r.cached) * H;
        const int warp_sees = __reduce_max_sync(0xffffffffu, sees);
        const int rows = at.r.c * H;
        const float* lse = p.lse + static_cast<long long>(at.r.q0) * H;
        // Only keys in the cache are given anything.
        bool valid = false;
        float had = 0.f;
        float* weight = p.weights + static_cast<long long>(at.b) * p.stride + j;
        const bool whole = at.t0 == at.r.s.first(at.kb) && end == at.r.s.tiles;
        if (grp == 0 && j < at.r.n) {
          const long long s = p.kv_indices[at.r.ip0 + (p.page_size == 1 ? j : j / PAGE)];
          valid = s >= 0 && s < (p.page_size == 1 ? p.num_slots : p.num_slots / PAGE);
          if (whole) had = *weight;
        }
        float sum = 0.f;
#pragma unroll 1
        for (int t = at.t; t < end; ++t, ++g) {
          const int cols = tile_columns(at.r, H, t), c0 = grp * 64, row0 = t * TILE + c0;
          // The columns' log-sum-exps as powers of two; rows that give
          // nothing (past the request's, or not finite): +inf.
          bool odd = row0 + 64 > rows || row0 < warp_sees;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = row0 + lane + 32 * i;
            const float l = r < rows ? lse[r] : INFINITY;
            const bool none = !(fabsf(l) < INFINITY);
            s_lse[lane + 32 * i] = none ? INFINITY : l * kLog2e;
            odd |= none;
          }
          odd = __any_sync(0xffffffffu, odd);
          __syncwarp();
          const uint32_t sb = static_cast<uint32_t>(g & 1);
          wait_bar<false>(mbar(MB_SF + sb), static_cast<uint32_t>((g >> 1) & 1), s_abort, p.err);
          tc::fence_after_sync();
          float part = 0.f;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (c0 + 32 * h >= cols) break;
            float x[32];
            tc::tmem_ld32f(tmem + (static_cast<uint32_t>(quad * 32) << 16) + 256u * sb + c0 + 32 * h, x);
            tc::tmem_wait_ld();
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            if (!odd) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 l4 = *reinterpret_cast<const float4*>(s_lse + 32 * h + 4 * i);
                y[0] += ex2(fmaf(x[4 * i], scale, -l4.x));
                y[1] += ex2(fmaf(x[4 * i + 1], scale, -l4.y));
                y[2] += ex2(fmaf(x[4 * i + 2], scale, -l4.z));
                y[3] += ex2(fmaf(x[4 * i + 3], scale, -l4.w));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float l = s_lse[32 * h + i];
                const float e = ex2(fmaf(x[i], scale, -l));
                y[i & 3] += l < INFINITY && row0 + 32 * h + i >= sees ? e : 0.f;
              }
            }
            part += (y[0] + y[1]) + (y[2] + y[3]);
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0 && *s_abort == 0) tc::mbar_arrive_cluster(even_mbar(MB_SE + sb));
          sum += part;
        }
        // The block's sums over the four column groups.
        float* s_sum = reinterpret_cast<float*>(smem + OFF_SUM) + (blk & 1) * 4 * HKEYS;
        s_sum[grp * HKEYS + key] = sum;
        named_sync(1, SCORE_WARPS * 32);
        if (grp == 0) {
          float v = (s_sum[key] + s_sum[HKEYS + key]) + (s_sum[2 * HKEYS + key] + s_sum[3 * HKEYS + key]);
          if (*s_abort != 0) v = __int_as_float(0x7fc00000);
          if (whole) {
            if (valid) *weight = had + v;
          } else {
            // The block's steps are s0 .. s1 - 1 of the call: clusters first ..
            // last have some of them, each in its first block, but the first
            // of them in its last.
            const long long s0 = at.done - (at.t0 - at.r.s.first(at.kb)), s1 = s0 + at.r.s.tiles - at.r.s.first(at.kb);
            const long long used = min(static_cast<long long>(p.clusters), at.total);
            const int first = static_cast<int>(((s0 + 1) * used - 1) / at.total), last = static_cast<int>((s1 * used - 1) / at.total);
            const bool own = at.total * first / used < s0;   // it has another block before this one
            float* part = p.part + static_cast<int>(rank) * HKEYS + key;
            part[(2 * cluster + (blk > 0 ? 1 : 0)) * KEYS] = v;
            __threadfence();
            named_sync(2, HKEYS);
            if (key == 0) *s_last = atomicAdd(p.arrived + 2 * first + rank, 1u) == static_cast<unsigned>(last - first);
            named_sync(2, HKEYS);
            if (*s_last) {
              __threadfence();
              float sum = __ldcg(part + (2 * first + (own ? 1 : 0)) * KEYS);
              for (int c = first + 1; c <= last; ++c) sum += __ldcg(part + 2 * c * KEYS);
              if (valid) *weight += sum;
              if (key == 0) p.arrived[2 * first + rank] = 0;
            }
          }
        }
        ++blk;
      } while (at.next_block(p));
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0 && s_abort[0] != 0)
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(tc::peer_addr(smem_u32(s_tmem + 2), peer)), "r"(1) : "memory");
  // Neither CTA leaves while the peer may signal its barriers or read its operands.
  tc::cluster_sync();
  tc::fence_after_sync();
  if (s_abort[0] != 0 || s_abort[1] != 0) {   // the same in both CTAs
    settle(1LL << 22);                        // copies under way land within microseconds
    if (warp == MMA_WARP) {
      if (rank == 0) tc::commit_pair(mbar(MB_DONE));
      wait_drain(mbar(MB_DONE), 0, p.err);
    }
    if (working && tid < HKEYS) {
      const float nan = __int_as_float(0x7fc00000);
      Cursor c = *s_start;
      do {
        const int j = c.kb * KEYS + static_cast<int>(rank) * HKEYS + tid;
        if (c.t0 == c.r.s.first(c.kb) && c.end() == c.r.s.tiles && j < c.r.n)   // (shared blocks have it from their sums)
          p.weights[static_cast<long long>(c.b) * p.stride + j] = nan;
      } while (c.next_block(p));
    }
    tc::cluster_sync();
    tc::fence_after_sync();
  }
  if (warp == MMA_WARP) tc::tmem_dealloc_pair<TMEM_COLS>(tmem);
}

}  // namespace

cudaError_t make_weigh_maps(WeighMaps* maps, const void* kv, long long num_slots, int page_size, const void* q, long long q_rows) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  void* fn = nullptr;
  const cudaError_t e = tensor_map_encode(&fn);
  if (e != cudaSuccess) return e;
  auto rows_of = [&](CUtensorMap* map, const void* base, long long rows, cuuint32_t box_rows) {
    const cuuint64_t dims[2] = {D_QK, static_cast<cuuint64_t>(rows)}, strides[1] = {ROW_BYTES};
    const cuuint32_t box[2] = {64, box_rows}, estrides[2] = {1, 1};
    return reinterpret_cast<Encode>(fn)(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estrides,
                                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  // (slots are gathered without a map)
  if (rows_of(&maps->kv, kv, num_slots, page_size == 1 ? 1 : PAGE) != CUDA_SUCCESS ||
      rows_of(&maps->q, q, q_rows, Q_BOX) != CUDA_SUCCESS || rows_of(&maps->q_full, q, q_rows, Q_FULL) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

cudaError_t weigh_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(weigh_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(weigh_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

cudaError_t launch_weigh_kv(const WeighParams& p, const WeighMaps& maps, cudaStream_t stream) {
  return launch_overlapping(weigh_kernel, dim3(2 * p.clusters), NTHREADS, SMEM_TOTAL, stream, 1, p, maps.kv, maps.q, maps.q_full);
}

}  // namespace mlav
