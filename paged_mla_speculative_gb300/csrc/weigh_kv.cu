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
// cache (TMA boxes of a page, or tile::gather4 of four slots), in nine slots
// of 64 dims of which each is refilled as soon as the block's last tile has
// read it; queries come through a ring of four slots of 64 dims.  bf16
// products are exact and nothing is widened, so no value is out of range.
// The steps (a tile against a block) of all requests are divided evenly over
// the clusters in closed form (weigh_steps.h), by every CTA for itself.
//
// Where clusters share a block their sums meet in weigh_join_kernel, in
// cluster order.
//
// What bounds it: with many query rows the tensor cores and the queries' way
// from L2 (16 KB a slot and CTA for 256 x 256 x 64 products), with few the
// keys' bytes.
//
// Roles (19 warps per CTA): warps 0-15 take the scores, warp 16 issues MMAs
// (even CTA), warp 17 loads queries, warp 18 keys.  Every wait is bounded; a
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
constexpr int NTHREADS = 19 * 32;
constexpr int NCHUNK = 9;                   // chunks of 64 dims
constexpr int K_SLOT = HKEYS * 128;         // 16 KB: 128 keys x 64 dims
constexpr int Q_SLOT = (TILE / 2) * 128;    // 16 KB: 128 rows x 64 dims
constexpr int NQ = 4;
constexpr int Q_BOX = 32;                   // rows of a query load
constexpr int OFF_K = 0;
constexpr int OFF_Q = OFF_K + NCHUNK * K_SLOT;
constexpr int OFF_LSE = OFF_Q + NQ * Q_SLOT;                // float [16 warps][64] log-sum-exps of a warp's columns
constexpr int OFF_SUM = OFF_LSE + SCORE_WARPS * 64 * 4;     // float [2][4][128] a block's sums by column group
constexpr int OFF_MBAR = OFF_SUM + 2 * 4 * HKEYS * 4;
constexpr int MB_KF = 0;     // [9] even CTA: key slot landed in both CTAs
constexpr int MB_KE = 9;     // [9] key slot read by its block's last MMAs
constexpr int MB_QF = 18;    // [4] even CTA: query slot landed in both CTAs
constexpr int MB_QE = 22;    // [4] query slot read
constexpr int MB_SF = 26;    // [2] scores of a step done
constexpr int MB_SE = 28;    // [2] even CTA: scores of a step read by both CTAs' warps
constexpr int MB_DONE = 30;  // after an abort: every MMA issued is done
constexpr int NMBAR = 31;
constexpr int OFF_MISC = OFF_MBAR + NMBAR * 8 + 8;          // tmem base, abort flag, the peer's
constexpr int OFF_PLAN = OFF_MISC + 16;                     // start of the share
constexpr int SMEM_TOTAL = OFF_PLAN + 32 + 32 * 8;
static_assert(SMEM_TOTAL <= 232448, "shared memory budget");
static_assert(OFF_MISC % 16 == 0 && OFF_PLAN % 16 == 0, "alignment");
constexpr int TMEM_COLS = 512;              // two buffers of 256 columns
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride 1024 bytes, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFF) | (16u >> 4) << 16; }

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
  } else if (r.n < r.c || r.n < 0 || r.n > p.max_kv_len) {
    errs |= ERR_LEN;
  } else if (r.ip0 < 0 || ip1 < r.ip0 || ip1 > ipn || static_cast<long long>(ip1) - r.ip0 != need) {
    errs |= ERR_INDPTR;
  } else {
    r.s = WeighSteps(r.n, r.c, p.H);
    return r.c > 0;
  }
  return false;
}

// A share of the work: `steps` steps from step `step` of the requests' steps
// from request `request` on.
struct Share {
  long long step, steps;
  int request;
};

// Where a role is: tile `t` of block `kb` of request `b`, whose first tile for
// this cluster was t0.
struct Cursor {
  Request r;
  long long left;   // steps, this one among them
  int b, kb, t, t0;
  // Moves to the request that has steps at or after b.
  __device__ __forceinline__ void start(const WeighParams& p, const Share& sh) {
    b = sh.request;
    left = sh.steps;
    if (left <= 0) return;
    int errs = 0;
    load_request(p, b, r, errs);
    kb = static_cast<int>(r.s.block_at(sh.step));
    t = t0 = static_cast<int>(r.s.first(kb) + sh.step - r.s.before(kb));
  }
  // Tiles of this block that are the cluster's: t0 .. end - 1.
  __device__ __forceinline__ int end() const {
    return static_cast<int>(min(r.s.tiles, static_cast<long long>(t) + left));
  }
  // To the next block (the tiles up to end() are done); false at the end.
  __device__ __forceinline__ bool next_block(const WeighParams& p) {
    left -= end() - t;
    if (left <= 0) return false;
    if (++kb == r.s.blocks) {
      int errs = 0;
      do ++b;
      while (b < p.batch - 1 && !load_request_at(p, errs));
      if (b == p.batch - 1) load_request(p, b, r, errs);
      kb = 0;
    }
    t = t0 = static_cast<int>(r.s.first(kb));
    return true;
  }
  __device__ __forceinline__ bool load_request_at(const WeighParams& p, int& errs) { return load_request(p, b, r, errs); }
};

__device__ __forceinline__ uint32_t idesc(int rows) {   // bf16, both K-major
  return tc::idesc_f16(KEYS, 0, 1, 0, 0) | static_cast<uint32_t>(rows >> 3) << 17;
}
// Columns of a tile: 32 at a time, as a pair's MMA takes them.
__device__ __forceinline__ int tile_columns(const Request& r, int H, int t) {
  return static_cast<int>(min(static_cast<long long>(TILE), (static_cast<long long>(r.c) * H - static_cast<long long>(t) * TILE + 31) / 32 * 32));
}

// The division: every CTA adds up all requests' steps itself (a few loads per
// thread) and takes its cluster's even share.
__device__ void plan_share(const WeighParams& p, int cluster, Share* share, long long* s_warp, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long total = 0, from = 0, to = 0;
  int errs = 0;
  // (tokens that are not divided: nothing is weighed)
  bool bad = false;
  for (int b = tid; b < p.batch; b += NTHREADS) {
    const int q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
    bad |= q0 < 0 || q1 < q0 || q1 > p.num_tokens;
  }
  if (tid == 0) *share = Share{0, 0, 0};
  if (__syncthreads_or(bad)) {
    if (report && tid == 0) atomicOr(p.err, ERR_INDPTR);
    return;
  }
  for (int pass = 0; pass < 2; ++pass) {   // the total, then the place of `from` in it
    long long before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += NTHREADS) {
      const int b = b0 + tid;
      long long x = 0;
      if (b < p.batch) {
        Request r;
        if (load_request(p, b, r, errs)) x = r.s.total();
      }
      const long long own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) s_warp[warp] = x;
      __syncthreads();
      long long all = 0;
      for (int w = 0; w < NTHREADS / 32; ++w) {
        if (w == warp) x += all;
        all += s_warp[w];
      }
      if (pass == 0) total += all;
      x += before;   // inclusive
      if (pass == 1 && own > 0 && x - own <= from && from < x) *share = Share{from - (x - own), to - from, b};
      before += all;
    }
    if (pass == 0) {
      const long long used = min(static_cast<long long>(p.clusters), total);
      if (cluster >= used) break;
      from = total * cluster / used;
      to = total * (cluster + 1) / used;
    }
  }
  if (report && errs) atomicOr(p.err, errs);
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
    weigh_kernel(const WeighParams p, const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t rank = tc::cluster_rank(), peer = rank ^ 1u;
  const int cluster = blockIdx.x >> 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  Share* s_share = reinterpret_cast<Share*>(smem + OFF_PLAN);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t mbar0 = sbase + OFF_MBAR;
  auto mbar = [&](int i) { return mbar0 + 8u * static_cast<uint32_t>(i); };
  if (tid == 0) {
    for (int i = 0; i < NMBAR; ++i) tc::mbar_init(mbar(i), i == MB_SE || i == MB_SE + 1 ? 2 * SCORE_WARPS : 1);
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
  plan_share(p, cluster, s_share, reinterpret_cast<long long*>(smem + OFF_PLAN + 32), blockIdx.x == 0);
  __syncthreads();
  Share share = *s_share;
  if (sbase & 1023) {   // the swizzled tiles need it (uniform over the pair)
    if (tid == 0) {
      atomicOr(p.err, ERR_INTERNAL);
      *s_abort = 1;
    }
    __syncthreads();
    share.steps = 0;
  }
  Cursor at;
  at.start(p, share);

  if (share.steps > 0) {
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
            if (*s_abort) break;
            if (rank == 0) {
              if (lane == 0) tc::mbar_arrive_expect(mbar(MB_QF + slot), 2 * boxes * Q_BOX * 128);
              __syncwarp();
            }
            for (int x = 0; x < boxes; ++x)
              tc::tma_load_2d_pair(sbase + OFF_Q + slot * Q_SLOT + x * Q_BOX * 128, &tm_q, 64 * c, row0 + x * Q_BOX,
                                   even_mbar(MB_QF + slot));
          }
        }
      } while (!*s_abort && at.next_block(p));
    } else if (warp == K_WARP) {
      int blk = 0;
      // Lane i's rows: four slots (page size 1), or its page's first (lanes 0
      // and 1).  Rows behind the request's last and bad slots: row 0, whose
      // scores nobody takes.
      do {
        int row[4];
        const int j0 = at.kb * KEYS + static_cast<int>(rank) * HKEYS;
        bool bad = false;
        if (p.page_size == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + 4 * lane + i;
            long long s = j < at.r.n ? p.kv_indices[at.r.ip0 + j] : 0;
            if (s < 0 || s >= p.num_slots) {
              bad = true;
              s = 0;
            }
            row[i] = static_cast<int>(s);
          }
        } else {
          const int j = j0 + (lane & 1) * PAGE;
          long long s = j < at.r.n ? p.kv_indices[at.r.ip0 + j / PAGE] : 0;
          if (s < 0 || s >= p.num_slots / PAGE) {
            bad = true;
            s = 0;
          }
          row[0] = static_cast<int>(s) * PAGE;
          row[1] = row[2] = row[3] = 0;
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err, ERR_SLOT);
        const int page0 = __shfl_sync(0xffffffffu, row[0], 0), page1 = __shfl_sync(0xffffffffu, row[0], 1);
#pragma unroll 1
        for (int c = 0; c < NCHUNK; ++c) {
          if (blk > 0) wait_bar<false>(mbar(MB_KE + c), static_cast<uint32_t>((blk - 1) & 1), s_abort, p.err);
          if (*s_abort) break;
          if (rank == 0) {
            if (lane == 0) tc::mbar_arrive_expect(mbar(MB_KF + c), 2 * K_SLOT);
            __syncwarp();
          }
          const uint32_t dst = sbase + OFF_K + c * K_SLOT;
          if (p.page_size == 1) {
            tc::tma_gather4_pair(dst + lane * 512, &tm_kv, 64 * c, row[0], row[1], row[2], row[3], even_mbar(MB_KF + c));
            __syncwarp();
          } else {
            tc::tma_load_2d_pair(dst, &tm_kv, 64 * c, page0, even_mbar(MB_KF + c));
            tc::tma_load_2d_pair(dst + K_SLOT / 2, &tm_kv, 64 * c, page1, even_mbar(MB_KF + c));
          }
        }
        ++blk;
      } while (!*s_abort && at.next_block(p));
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
            if (t == at.t) wait_bar<false>(mbar(MB_KF + c), static_cast<uint32_t>(blk & 1), s_abort, p.err);
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
          const float v = (s_sum[key] + s_sum[HKEYS + key]) + (s_sum[2 * HKEYS + key] + s_sum[3 * HKEYS + key]);
          if (!whole)
            p.part[(2 * cluster + (blk > 0 ? 1 : 0)) * KEYS + static_cast<int>(rank) * HKEYS + key] = valid ? v : 0.f;
          else if (valid)
            *weight = had + v;
        }
        ++blk;
      } while (at.next_block(p));
    }
  }

  // Which blocks the cluster shares with others, for the merge.
  if (rank == 0 && tid == 0) {
    WeighCut cut{};
    if (share.steps > 0) {
      Cursor c;
      c.start(p, share);
      cut.first_request = c.b;
      cut.first_block = c.kb;
      cut.continues = c.t0 > c.r.s.first(c.kb);
      int blocks = 0;
      do {
        cut.last_request = c.b;
        cut.last_block = c.kb;
        cut.goes_on = c.end() < c.r.s.tiles;
        cut.last_slot = blocks > 0;
        blocks = 1;
      } while (c.next_block(p));
    }
    p.cut[cluster] = cut;
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
    if (share.steps > 0 && tid < HKEYS) {
      const float nan = __int_as_float(0x7fc00000);
      Cursor c;
      c.start(p, share);
      int blk = 0;
      do {
        const int j = c.kb * KEYS + static_cast<int>(rank) * HKEYS + tid;
        if (c.t0 != c.r.s.first(c.kb) || c.end() != c.r.s.tiles)
          p.part[(2 * cluster + (blk > 0 ? 1 : 0)) * KEYS + static_cast<int>(rank) * HKEYS + tid] = nan;
        else if (j < c.r.n)
          p.weights[static_cast<long long>(c.b) * p.stride + j] = nan;
        ++blk;
      } while (c.next_block(p));
    }
    tc::cluster_sync();
    tc::fence_after_sync();
  }
  if (warp == MMA_WARP) tc::tmem_dealloc_pair<TMEM_COLS>(tmem);
}

// CTA c adds up the parts of the block that cluster c is the first of several
// to hold, in cluster order; a thread per key.
__global__ void __launch_bounds__(KEYS) weigh_join_kernel(const WeighParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int c = blockIdx.x, key = threadIdx.x;
  const WeighCut cut = p.cut[c];
  if (!cut.goes_on || (cut.continues && !cut.last_slot)) return;
  const int b = cut.last_request, j = cut.last_block * KEYS + key;
  float sum = p.part[(2 * c + cut.last_slot) * KEYS + key];
  for (int i = c + 1; i < p.clusters; ++i) {
    const WeighCut next = p.cut[i];
    if (!next.continues || next.first_request != b || next.first_block != cut.last_block) break;
    sum += p.part[2 * i * KEYS + key];
  }
  if (j < p.kv_lens[b]) p.weights[static_cast<long long>(b) * p.stride + j] += sum;
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
  // (tile::gather4: the box is one row high)
  if (rows_of(&maps->kv, kv, num_slots, page_size == 1 ? 1 : PAGE) != CUDA_SUCCESS ||
      rows_of(&maps->q, q, q_rows, Q_BOX) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

cudaError_t weigh_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(weigh_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(weigh_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

cudaError_t launch_weigh_kv(const WeighParams& p, const WeighMaps& maps, cudaStream_t stream) {
  const cudaError_t e = launch_overlapping(weigh_kernel, dim3(2 * p.clusters), NTHREADS, SMEM_TOTAL, stream, 1, p, maps.kv, maps.q);
  return e != cudaSuccess ? e : launch_overlapping(weigh_join_kernel, dim3(p.clusters), KEYS, 0, stream, 1, p);
}

}  // namespace mlav
