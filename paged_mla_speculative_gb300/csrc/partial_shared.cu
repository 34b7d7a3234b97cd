// Attention of groups of requests that share their first rows: a persistent
// kernel on CTA pairs (tcgen05 cta_group::2) over the packed planes of
// shared_pack.cu.
//
// A tile of 128 query rows of a group -- of one request, or of several -- is
// scored against the group's shared keys once and then against its requests'
// own keys, in one softmax: every shared row is read once per 128 query rows
// of the group, not once per request.  The products, the softmax and the
// exchange between the two CTAs of a pair are those of partial_pair.cu:
//     S^T[key, row] = K_pair[256 x 576] . Q_tile[128 x 576]^T
//     O^T[dim, row] += V_pair^T[512 x 256] . P^T[256 x 128]
// with the running maximum and sum in fp32, P in fp16 (rounded once, 2^-11 of
// every weight down to 2^-29 of the row's largest; see P_SHIFT), the bf16 keys
// and queries in fp16 (exact from 2^-14 to 65504, off by less than 2^-25 below),
// O^T in tensor memory, split by value dim over the two CTAs.
//
// What differs is the schedule.  The grid is one cluster per SM pair; cluster
// c walks the steps from start[c] to start[c + 1] of the list of all tiles'
// steps, so every pair works to the end whatever the lengths.  It runs as one
// continuous pipeline over its segments (a segment: consecutive steps of one
// tile): the ring of key chunks, the score buffers and all barrier phases
// carry on over the border, the next tile's queries are loaded as soon as the
// last S^T of the current one is done, and its first products are issued while
// the softmax warps still read out the finished O^T.
//
// A tile that one cluster holds whole is normalised and stored directly;
// otherwise the segment's partial goes to the workspace for shared_join_kernel.
//
// Roles (20 warps per CTA): warps 0-15 softmax, warp 16 MMA issue (even CTA)
// or P^T hand-off (odd CTA), warps 17-19 the key ring (17 the queries too).
// Every wait is bounded.  A CTA whose wait runs out arms and sends nothing any
// more, so its peer's waits run out too or its peer is done; the two tell each
// other at the end, and all of the cluster's rows are NaN.
#include "shared.cuh"
#include "kernels.h"
#include "pair_common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace mlav {
namespace {

constexpr int ROWS = SH_ROWS;       // query rows per pair: MMA N
constexpr int HROWS = ROWS / 2;     // rows of the B operands a CTA holds
constexpr int BN = SH_HALF;         // keys per CTA per step
constexpr int SOFTMAX_WARPS = 16, MMA_WARP = 16, COPY_WARP = 17;
constexpr int NCOPY = 3;            // copy warp k fills ring slot k
constexpr int NWARPS = COPY_WARP + NCOPY;
constexpr int NTHREADS = NWARPS * 32;
constexpr int CHUNK = BN * 128;          // 16 KB: 128 keys x 64 dims fp16
constexpr int Q_CHUNK = HROWS * 128;     // 8 KB: 64 rows x 64 dims
constexpr int Q_PLANES = 3;              // planes per query load
constexpr int NSLOT = NCOPY;
constexpr int OFF_Q = 0;
constexpr int OFF_P = OFF_Q + 9 * Q_CHUNK;            // P^T [key half][128 keys][64 rows] fp16
constexpr int OFF_RING = OFF_P + 2 * CHUNK;
constexpr int OFF_ROPE = OFF_RING + NSLOT * 2 * CHUNK;
constexpr int OFF_RED = OFF_ROPE + CHUNK;             // float [2][128 rows][4 quads] this CTA's row maxima of the step
constexpr int OFF_XRED = OFF_RED + 2 * ROWS * 4 * 4;  // the same of the peer (st.async)
constexpr int OFF_XSUM = OFF_XRED + 2 * ROWS * 4 * 4; // float [128] the peer's row sums
constexpr int OFF_M = OFF_XSUM + ROWS * 4;            // float [2][128] running row max less P_SHIFT (0: none yet); 1 / row sum at the end
constexpr int OFF_ROW = OFF_M + 2 * ROWS * 4;             // int2 [128] request of the row (-1: not served), ancestor mask
constexpr int OFF_MBAR = OFF_ROW + ROWS * 8;
constexpr int NMBAR = 28;
constexpr int OFF_MISC = OFF_MBAR + NMBAR * 8;        // tmem base, P-complete word, absent-unit word, abort flag, the peer's
constexpr int SMEM_TOTAL = OFF_MISC + 32;
static_assert(SMEM_TOTAL <= 232448, "shared memory budget");
static_assert(OFF_P % 1024 == 0 && OFF_RING % 1024 == 0 && OFF_ROPE % 1024 == 0,
              "swizzled tiles need 1024-byte alignment");

// mbarrier indices (same offsets in both CTAs)
constexpr int MB_FULL = 0;     // [3] even CTA: ring slot landed in both CTAs (bytes of both)
constexpr int MB_EMPTY = 3;    // [3] ring slot read by its MMAs (commit to both CTAs)
constexpr int MB_RFULL = 6;    // even CTA: rope slot landed in both CTAs
constexpr int MB_REMPTY = 7;   // rope slot read
constexpr int MB_S = 8;        // [2] S^T buffer done
constexpr int MB_P = 10;       // this CTA's softmax warps wrote their P^T and rescaled O^T
constexpr int MB_PX = 11;      // the peer's half of this CTA's P^T landed (st.async bytes)
constexpr int MB_PF = 12;      // even CTA: the odd CTA's P^T is complete (st.async word)
constexpr int MB_OT = 13;      // O^T of a step done
constexpr int MB_Q = 14;       // even CTA: both halves of a segment's queries landed
constexpr int MB_QE = 15;      // the segment's last S^T is done: its queries can go
constexpr int MB_X = 20;       // [2][4] the peer's row maxima of the step and row group landed (st.async bytes)
constexpr int MB_XS = 16;      // the peer's row sums landed (st.async bytes)
constexpr int MB_DONE = 17;    // after an abort: every MMA issued is done

constexpr int TMEM_COLS = 512;
constexpr uint32_t TM_S = 256;                  // S^T buffer u at 256 + 128u; O^T tile t at 128t

constexpr uint32_t IDESC_S = tc::idesc_f16(256, ROWS, 0, 0, 0);   // fp16, both K-major
constexpr uint32_t IDESC_O = tc::idesc_f16(256, ROWS, 0, 1, 1);   // fp16, both MN-major

// Shared-memory descriptors (tc::desc_sw128): the low word is the address and
// the leading offset, the high word (stride 1024 bytes, 128-byte swizzle) is one.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3FFF) | (lbo >> 4) << 16; }

constexpr int FEW_MOVED = 4;

// Weights are taken relative to 2^-P_SHIFT of the row's largest, so the
// largest is 2^15 in fp16.  Relative to the largest itself, those below 2^-14
// of it would be subnormal and those below 2^-25 zero, though the fp32 row sum
// counts them: where one key without value led by 17 nats, the outputs were
// 16 % too small.  The shift moves that to 2^-29 and 2^-40 and costs nothing
// per score: row sums and O^T carry the same factor.
constexpr float P_SHIFT = 15.f, P_LARGEST = 32768.f;
// Scores (as powers of two) up to which half an ulp is a quarter at most.
constexpr float FUSED_LIMIT = 8388608.f;
// Bounded waits of a warp.  wait_own: for barriers that TMA, tcgen05.commit
// and this CTA's threads complete; wait_peer: for those that the peer's
// st.async complete, acquiring its stores into this CTA's shared memory.
// (pair_common.cuh's waits acquire all memory at cluster scope, which drops
// the SM's L1 lines, spilled registers among them, every step.)
template <bool PEER>
__device__ __noinline__ void wait_longer(uint32_t mbar, uint32_t parity, volatile int* abort, int* err) {
  const long long t0 = clock64();
  while (!(PEER ? tc::mbar_try_cluster_relaxed(mbar, parity) : tc::mbar_try(mbar, parity))) {
    if (*abort) return;
    if (clock64() - t0 > WAIT_LIMIT) {
      *abort = 1;
      atomicOr(err, ERR_TIMEOUT);
      return;
    }
  }
}
template <bool PEER>
__device__ __forceinline__ void wait_bounded(uint32_t mbar, uint32_t parity, volatile int* abort, int* err) {
  if (!(PEER ? tc::mbar_try_cluster_relaxed(mbar, parity) : tc::mbar_try(mbar, parity)))
    wait_longer<PEER>(mbar, parity, abort, err);
  if (PEER) tc::fence_acquire_shared_cluster();
  __syncwarp();
}
__device__ __forceinline__ void wait_own(uint32_t mbar, uint32_t parity, volatile int* abort, int* err) {
  wait_bounded<false>(mbar, parity, abort, err);
}
__device__ __forceinline__ void wait_peer(uint32_t mbar, uint32_t parity, volatile int* abort, int* err) {
  wait_bounded<true>(mbar, parity, abort, err);
}

// Row maxima (or sums) of a warp: lane t starts with eight rows' values over
// its own keys, y[2i + e] of row 8i + 2 (t % 4) + e, and ends with the result
// of row 16 b4 + 8 b3 + 2 (t % 4) + b2 (b: the bits of t).
template <bool SUM>
__device__ __forceinline__ float reduce_rows(float (&y)[8], int lane) {
#pragma unroll
  for (int w = 16, n = 4; n >= 1; w >>= 1, n >>= 1) {
    const bool upper = (lane & w) != 0;
#pragma unroll
    for (int c = 0; c < n; ++c) {
      const float send = upper ? y[c] : y[c + n];
      const float keep = upper ? y[c + n] : y[c];
      const float got = __shfl_xor_sync(0xffffffffu, send, w);
      y[c] = SUM ? keep + got : fmaxf(keep, got);
    }
  }
  return y[0];
}

// Testing: the ring unit before which SharedParams::fault_rank's CTA gives up
// (the first of a second step's O^T, so that a step of scores is done).
constexpr int SH_FAULT_UNIT = 12;
constexpr uint32_t ABSENT_BYTES = 4;   // the odd CTA's signal for a unit it has no half block for

struct Segment {
  SharedTile t;
  int tile, sa, steps;   // steps sa .. sa + steps - 1 of the tile
  bool first, whole;     // the cluster's first segment; the tile's only one
};
// (Plain loads of what the kernel before wrote, here and below: a read-only
// load with an address known early may be moved above griddepcontrol.wait.)
__device__ __forceinline__ SharedTile load_tile(const SharedTile* rec) {
  const int4* q = reinterpret_cast<const int4*>(rec);
  const int4 a = q[0], b = q[1], c = q[2];
  return SharedTile{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, {0, 0}};
}
// The cluster's next segment at or after tile `tile`; false when there is none.
__device__ __forceinline__ bool next_segment(const SharedParams& p, const SharedShare* share, const SharedPos& from,
                                             const SharedPos& to, int tile, Segment& s) {
  for (; tile < to.tile || (tile == to.tile && to.step > 0); ++tile) {
    s.first = tile == from.tile;
    s.t = load_tile(s.first ? &share->first : p.tiles + tile);
    s.tile = tile;
    s.sa = s.first ? from.step : 0;
    const bool ends = tile == to.tile;
    s.steps = (ends ? to.step : s.t.steps) - s.sa;
    s.whole = s.sa == 0 && !ends;
    if (s.steps > 0) return true;
  }
  return false;
}

__device__ __forceinline__ void st_peer(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(cluster_addr), "r"(v) : "memory");
}

// NaN for every row of the segment (a pair that gave up), in the places that
// this CTA's readout writes: value dims 256 t + 128 rank .., lse of its 64 rows.
__device__ __forceinline__ void write_nan_segment(const SharedParams& p, const Segment& s, int cluster, uint32_t rank, int tid) {
  const float nan = __int_as_float(0x7fc00000);
  const size_t row0 = s.whole ? static_cast<size_t>(s.t.q_row0) : static_cast<size_t>(part_slot(cluster, s.first)) * ROWS;
  for (int i = tid; i < s.t.nrows * 256; i += NTHREADS) {
    const int r = i >> 8, c = i & 255;
    const size_t at = (row0 + r) * D_V + (c >> 7) * 256 + rank * 128 + (c & 127);
    if (!s.whole) p.part_o[at] = nan;
    else if (p.out_bf16) reinterpret_cast<uint16_t*>(p.out)[at] = 0x7fc0;
    else reinterpret_cast<float*>(p.out)[at] = nan;
    if (c == 0 && (r >> 6) == static_cast<int>(rank)) (s.whole ? p.lse : p.part_lse)[row0 + r] = nan;
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    partial_shared_kernel(const SharedParams p, const __grid_constant__ CUtensorMap tm_pair,
                          const __grid_constant__ CUtensorMap tm_chunk, const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t rank = tc::cluster_rank();
  const uint32_t peer = rank ^ 1u;
  const int cluster = blockIdx.x >> 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3;            // TMEM lanes 32*quad .. +32 are this warp's
  const int grp = warp >> 2;            // softmax: rows 32*grp .. +32

  float* s_red = reinterpret_cast<float*>(smem + OFF_RED);
  float* s_xred = reinterpret_cast<float*>(smem + OFF_XRED);
  float* s_xsum = reinterpret_cast<float*>(smem + OFF_XSUM);
  float* s_m = reinterpret_cast<float*>(smem + OFF_M);
  int2* s_row = reinterpret_cast<int2*>(smem + OFF_ROW);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + OFF_MISC + 12);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t mbar0 = sbase + OFF_MBAR;
  auto mbar = [&](int i) { return mbar0 + 8u * static_cast<uint32_t>(i); };

  if (tid == 0) {
    for (int i = 0; i < NMBAR; ++i) tc::mbar_init(mbar(i), i == MB_P ? SOFTMAX_WARPS : 1);
    tc::mbar_fence_init();
    s_abort[0] = s_abort[1] = 0;
  }
  if (warp == MMA_WARP) tc::tmem_alloc_pair<TMEM_COLS>(smem_u32(s_tmem));
  tc::fence_before_sync();
  __syncthreads();
  // The peer's barriers exist and the pair's TMEM is allocated.
  tc::cluster_sync_relaxed();
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const uint32_t even_mbar0 = tc::peer_addr(mbar0, 0);   // the even CTA's barriers
  const uint32_t peer_mbar0 = tc::peer_addr(mbar0, peer);
  auto even_mbar = [&](int i) { return even_mbar0 + 8u * static_cast<uint32_t>(i); };
  auto peer_mbar = [&](int i) { return peer_mbar0 + 8u * static_cast<uint32_t>(i); };
  // Everything read from here on was written by the kernel before.
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const SharedShare* share = p.share + cluster;
  const int4 range = *reinterpret_cast<const int4*>(share);
  const SharedPos from{range.x, range.y};
  SharedPos to{range.z, range.w};
  if (sbase & 1023) {   // the swizzled tiles need it (uniform over the pair)
    if (tid == 0) {
      atomicOr(p.err, ERR_INTERNAL);
      *s_abort = 1;
    }
    __syncthreads();
    to = from;
  }
  Segment s;

  if (warp >= COPY_WARP) {
    // ========================= key chunk producers ==========================
    // As in partial_pair.cu: unit n goes to slot n % 3, one warp per slot; the
    // rope chunks go with slot 2; a half block the odd CTA does not have is
    // signalled by ABSENT_BYTES, so that no CTA's barriers run ahead.
    const int cw = warp - COPY_WARP;
    const uint32_t absent_word = tc::peer_addr(smem_u32(s_tmem + 2), 0);
    int n = 0, g0 = 0, k = 0;   // units and segments so far, steps of the segments before
#pragma unroll 1
    for (int tile = from.tile; next_segment(p, share, from, to, tile, s) && !*s_abort; tile = s.tile + 1, g0 += s.steps, ++k) {
      if (cw == 0) {
        // The tile's queries, once the last S^T of the segment before is done
        // (its O^T units, already under way, come after it).  Rows past the
        // tile are the next tile's (or zeros past the batch): their columns
        // of S^T and O^T are not stored.
        if (k > 0) wait_own(mbar(MB_QE), static_cast<uint32_t>((k - 1) & 1), s_abort, p.err);
        if (*s_abort) break;
        if (rank == 0) {
          if (lane == 0) tc::mbar_arrive_expect(mbar(MB_Q), 2 * 9 * Q_CHUNK);
          __syncwarp();
        }
#pragma unroll
        for (int z = 0; z < 9; z += Q_PLANES)
          tc::tma_load_3d_pair(sbase + OFF_Q + z * Q_CHUNK, &tm_q, 0, s.t.q_row0 + static_cast<int>(rank) * HROWS, z,
                               even_mbar(MB_Q));
      }
#pragma unroll 1
      for (int f = 0; f < 2 * s.steps && !*s_abort; ++f) {
        bool is_s;
        int i;
        phase_of(f, s.steps, is_s, i);
        const int hb0 = 2 * (s.sa + i);
        int count;
#pragma unroll 1
        for (int u = 0; u < 4; ++u, ++n) {
          const int slot = n % NSLOT;
          if (slot != cw) continue;
          // S units: the own half block (the peer loads its own); O units:
          // half block h in both CTAs.
          const int h = is_s ? static_cast<int>(rank) : (u & 1);
          const int pair_idx = is_s ? u : 2 * (u >> 1) + static_cast<int>(rank);
          const bool mine = hb0 + h < s.t.halves;
          const bool peers = is_s ? hb0 + static_cast<int>(peer) < s.t.halves : mine;
          if (n >= NSLOT) wait_own(mbar(MB_EMPTY + slot), static_cast<uint32_t>((n / NSLOT - 1) & 1), s_abort, p.err);
          if (n == SH_FAULT_UNIT && p.fault_rank == static_cast<int>(rank)) *s_abort = 1;   // (testing)
          if (*s_abort) break;
          if (rank == 0) {
            if (lane == 0)
              tc::mbar_arrive_expect(mbar(MB_FULL + slot), (mine ? 2 * CHUNK : 0) + (peers ? 2 * CHUNK : ABSENT_BYTES));
            __syncwarp();
          }
          if (mine) {
            tc::tma_load_3d_pair(sbase + OFF_RING + slot * 2 * CHUNK, &tm_pair, 0, half_base(s.t, hb0 + h, count), 2 * pair_idx,
                                 even_mbar(MB_FULL + slot));
          } else if (rank == 1) {
            if (lane == 0) tc::st_async_b32(absent_word, 0, even_mbar(MB_FULL + slot));
            __syncwarp();
          }
        }
        if (*s_abort) break;
        if (is_s && cw == NCOPY - 1) {
          const int g = g0 + i;
          const bool mine = hb0 + static_cast<int>(rank) < s.t.halves, peers = hb0 + static_cast<int>(peer) < s.t.halves;
          if (g > 0) wait_own(mbar(MB_REMPTY), static_cast<uint32_t>((g - 1) & 1), s_abort, p.err);
          if (*s_abort) break;
          if (rank == 0) {
            if (lane == 0) tc::mbar_arrive_expect(mbar(MB_RFULL), (mine ? CHUNK : 0) + (peers ? CHUNK : ABSENT_BYTES));
            __syncwarp();
          }
          if (mine) {
            tc::tma_load_3d_pair(sbase + OFF_ROPE, &tm_chunk, 0, half_base(s.t, hb0 + static_cast<int>(rank), count), 8,
                                 even_mbar(MB_RFULL));
          } else if (rank == 1) {
            if (lane == 0) tc::st_async_b32(absent_word, 0, even_mbar(MB_RFULL));
            __syncwarp();
          }
        }
      }
    }
  } else if (warp == MMA_WARP && rank == 1) {
    // =================== odd CTA: P^T complete -> even CTA ==================
    uint32_t* s_word = s_tmem + 1;
    const uint32_t even_word = tc::peer_addr(smem_u32(s_word), 0);
    int g = 0;
#pragma unroll 1
    for (int tile = from.tile; next_segment(p, share, from, to, tile, s) && !*s_abort; tile = s.tile + 1) {
#pragma unroll 1
      for (int i = 0; i < s.steps && !*s_abort; ++i, ++g) {
        if (lane == 0) tc::mbar_arrive_expect(mbar(MB_PX), CHUNK);
        __syncwarp();
        wait_own(mbar(MB_P), static_cast<uint32_t>(g & 1), s_abort, p.err);
        wait_peer(mbar(MB_PX), static_cast<uint32_t>(g & 1), s_abort, p.err);
        if (*s_abort) break;
        tc::fence_async_smem();   // the st.async bytes are read by the tensor core next
        if (lane == 0) tc::st_async_b32(even_word, static_cast<uint32_t>(g), even_mbar(MB_PF));
        __syncwarp();
      }
    }
  } else if (warp == MMA_WARP) {
    // ======================= MMA issuer (even CTA) ==========================
    int n = 0, g0 = 0, k = 0;
#pragma unroll 1
    for (int tile = from.tile; next_segment(p, share, from, to, tile, s) && !*s_abort; tile = s.tile + 1, g0 += s.steps, ++k) {
      wait_own(mbar(MB_Q), static_cast<uint32_t>(k & 1), s_abort, p.err);
      tc::fence_after_sync();
#pragma unroll 1
      for (int f = 0; f < 2 * s.steps && !*s_abort; ++f) {
        bool is_s;
        int i;
        phase_of(f, s.steps, is_s, i);
        const int g = g0 + i;
        if (is_s) {
          const uint32_t d = tmem + TM_S + 128u * static_cast<uint32_t>(g & 1);
#pragma unroll 1
          for (int u = 0; u < 4; ++u, ++n) {
            const int slot = n % NSLOT;
            wait_own(mbar(MB_FULL + slot), static_cast<uint32_t>((n / NSLOT) & 1), s_abort, p.err);
            tc::fence_after_sync();
            if (tc::elect_one()) {
              const uint32_t a = desc_lo(sbase + OFF_RING + slot * 2 * CHUNK, 16);
              const uint32_t bq = desc_lo(sbase + OFF_Q + u * 2 * Q_CHUNK, 16);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)   // 16-dim steps of the chunk pair
                tc::mma_pair_one(d, a + (((kk >> 2) * CHUNK + (kk & 3) * 32) >> 4),
                                 bq + (((kk >> 2) * Q_CHUNK + (kk & 3) * 32) >> 4), DESC_HI, IDESC_S, (u > 0 || kk > 0) ? 1u : 0u);
              tc::commit_pair_one(mbar(MB_EMPTY + slot));
            }
            __syncwarp();
          }
          wait_own(mbar(MB_RFULL), static_cast<uint32_t>(g & 1), s_abort, p.err);
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint32_t a = desc_lo(sbase + OFF_ROPE, 16), bq = desc_lo(sbase + OFF_Q + 8 * Q_CHUNK, 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc::mma_pair_one(d, a + 2 * kk, bq + 2 * kk, DESC_HI, IDESC_S, 1);
            tc::commit_pair_one(mbar(MB_REMPTY));
            tc::commit_pair_one(mbar(MB_S + (g & 1)));
            if (i == s.steps - 1) tc::commit_pair_one(mbar(MB_QE));
          }
          __syncwarp();
        } else {
          // P^T of the step: this CTA's softmax warps, the odd CTA's st.async
          // bytes, and the odd CTA's word that its own half is complete.
          if (*s_abort) break;
          if (lane == 0) {
            tc::mbar_arrive_expect(mbar(MB_PX), CHUNK);
            tc::mbar_arrive_expect(mbar(MB_PF), 4);
          }
          __syncwarp();
          wait_own(mbar(MB_P), static_cast<uint32_t>(g & 1), s_abort, p.err);
          wait_peer(mbar(MB_PX), static_cast<uint32_t>(g & 1), s_abort, p.err);
          wait_peer(mbar(MB_PF), static_cast<uint32_t>(g & 1), s_abort, p.err);
          tc::fence_async_smem();
          tc::fence_after_sync();
#pragma unroll 1
          for (int u = 0; u < 4; ++u, ++n) {
            const int t = u >> 1, h = u & 1;
            const int slot = n % NSLOT;
            wait_own(mbar(MB_FULL + slot), static_cast<uint32_t>((n / NSLOT) & 1), s_abort, p.err);
            tc::fence_after_sync();
            if (tc::elect_one()) {
              if (2 * (s.sa + i) + h < s.t.halves) {
                const uint32_t a = desc_lo(sbase + OFF_RING + slot * 2 * CHUNK, CHUNK);
                const uint32_t bp = desc_lo(sbase + OFF_P + h * CHUNK, CHUNK);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)   // 16-key steps of the key half
                  tc::mma_pair_one(tmem + 128u * static_cast<uint32_t>(t), a + kk * (2048 >> 4), bp + kk * (2048 >> 4), DESC_HI,
                                   IDESC_O, (i > 0 || h > 0 || kk > 0) ? 1u : 0u);
              }
              tc::commit_pair_one(mbar(MB_EMPTY + slot));
              if (u == 3) tc::commit_pair_one(mbar(MB_OT));
            }
            __syncwarp();
          }
        }
      }
    }
  } else {
    // ============================= softmax =================================
    // The four warps of a row group (32 rows; a warp has 32 keys of each) meet
    // at the group's named barrier; they never leave the loops early, and
    // after an abort their waits return at once.
    // A warp's 32 keys x 32 rows are spread over its lanes as MMA accumulators
    // are: lane t holds keys t / 4 + 8k (k < 4) and, of each, rows 8i + 2 (t %
    // 4) + e (i < 4, e < 2), so that a row's maximum and sum over the warp's
    // keys take three operations in the lane and seven shuffles for all rows
    // (with a key per lane they took 31), and P^T goes out by stmatrix.
    const int c0 = grp * 32;            // pair rows c0 .. c0+31
    const int key = lane >> 2, pair = 2 * (lane & 3);
    const int j = quad * 32 + lane;     // the key whose meta word this lane loads
    // The row whose maximum and sum this lane ends up with.
    const int row = c0 + (lane & 16) + (lane & 8) + pair + ((lane >> 2) & 1);
    const float scale2 = p.scale_log2;
    auto group_sync = [&]() { named_sync(1 + grp, 128); };
    // P^T (key half = rank) goes to the CTA that holds the group's rows: by
    // stmatrix here, or by st.async into the peer with its MB_PX.  Keys k * 8
    // of the warp: + 1024 k bytes.
    const bool p_local = (grp >> 1) == static_cast<int>(rank);
    const uint32_t p_warp = sbase + OFF_P + rank * CHUNK + quad * 32 * 128;
    const uint32_t p_matrix = p_warp + (lane & 7) * 128 + ((((grp & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
    const uint32_t p_peer = tc::peer_addr(p_warp + key * 128 + ((((grp & 1) * 4 + (lane & 3)) ^ key) << 4), peer);
    const uint32_t red_off = (row * 4 + quad) * 4;   // this warp's maximum of the lane's row
    const uint32_t xred_peer = tc::peer_addr(sbase + OFF_XRED + red_off, peer);
    int g = 0, k = 0;   // steps and segments so far
#pragma unroll 1
    for (int tile = from.tile; next_segment(p, share, from, to, tile, s); tile = s.tile + 1, ++k) {
      // This CTA's half block of each step: h0, h0 + 2, ..  Its keys' meta
      // words start at meta0 + 128 hb, those of the own range meta_gap behind.
      const int h0 = 2 * s.sa + static_cast<int>(rank), np = prefix_halves(s.t);
      const int prefix_len = s.t.prefix_len, own_len = s.t.own_len + np * BN;
      const int* meta0 = p.meta + s.t.prefix_base + j;
      const int meta_gap = s.t.own_base - np * BN - s.t.prefix_base;
      const int nsteps = s.steps;
      auto load_meta = [&](int step) {
        const int key = (h0 + 2 * step) * BN;
        const bool shared = key < np * BN;
        if (step >= nsteps || key + j >= (shared ? prefix_len : own_len)) return META_MASKED;
        return meta0[key + (shared ? 0 : meta_gap)];
      };
      int meta = load_meta(0);
      group_sync();   // the previous segment's rows are read
      if (quad == 0) {
        int2 of = make_int2(-1, 0);
        if (c0 + lane < s.t.nrows) {
          const int q = s.t.q_row0 + c0 + lane, b = q / p.R;
          if (p.own[b] > 0) of = make_int2(b, static_cast<int>(p.anc[b * p.T + (q - b * p.R) / p.H]));
        }
        s_row[c0 + lane] = of;
      }
      group_sync();
      float mrow = -INFINITY;             // the lane's row's running max less P_SHIFT, the same in the group's warps of both CTAs
      float lrun = 0.f;                   // its sum over this warp's keys so far
#pragma unroll 1
      for (int it = 0; it < nsteps; ++it, ++g) {
        // After an abort no barrier may be armed before its last phase is over,
        // and no bytes sent that nobody arms for.
        const bool alive = *s_abort == 0;
        // Decided while S^T is computed: do all rows see all of the warp's
        // keys?  If not, which: bit 8k + 2i + e for key k and row (i, e).
        const bool plain = __all_sync(0xffffffffu, meta == META_SHARED);
        uint32_t vis = 0xffffffffu, poison = 0;
        if (!plain) {
          vis = 0;
#pragma unroll 1
          for (int k8 = 0; k8 < 4; ++k8) {
            const int m = __shfl_sync(0xffffffffu, meta, key + 8 * k8);
            if (m < 0) continue;
            poison |= m & META_POISON ? 1u << k8 : 0u;
            const int w = m & ~META_POISON, b = w >> 6, d = (w & 63) - 2;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int2 r = s_row[c0 + 8 * (c >> 1) + pair + (c & 1)];
              const bool v = w == META_SHARED || (r.x == b && (d < 0 || ((static_cast<uint32_t>(r.y) >> d) & 1u)));
              vis |= (v ? 1u : 0u) << (8 * k8 + c);
            }
          }
        }
        meta = load_meta(it + 1);
        const uint32_t sb = static_cast<uint32_t>(g & 1);
        wait_own(mbar(MB_S + sb), static_cast<uint32_t>((g >> 1) & 1), s_abort, p.err);
        tc::fence_after_sync();
        // x[16 hh + 4 i + 2 h + e]: key 8 (2 hh + h), row (i, e).
        const uint32_t s_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + TM_S + 128u * sb + c0;
        float x[32];
        tc::tmem_ld16x32f(s_addr, x);
        tc::tmem_ld16x32f(s_addr + (16u << 16), x + 16);
        tc::tmem_wait_ld();
        float mul = scale2;   // still to be applied to x
        if (!plain || scale2 < 0.f) {
          mul = 1.f;
#pragma unroll
          for (int k8 = 0; k8 < 4; ++k8) {
            const float f = (poison >> k8) & 1u ? __int_as_float(0x7fc00000) : scale2;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float& v = x[16 * (k8 >> 1) + 4 * (c >> 1) + 2 * (k8 & 1) + (c & 1)];
              v = (vis >> (8 * k8 + c)) & 1u ? v * f : -INFINITY;
            }
          }
        }
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int n = 4 * (c >> 1) + (c & 1);
          y[c] = fmaxf(fmaxf(x[n], x[n + 2]), fmaxf(x[n + 16], x[n + 18]));
        }
        const float wmax = mul * reduce_rows<false>(y, lane);
        // Every warp gives its 32 maxima to the group here and in the peer,
        // and takes the maximum of the eight itself.
        s_red[sb * ROWS * 4 + row * 4 + quad] = wmax;
        if (alive) {
          tc::st_async_b32(xred_peer + sb * ROWS * 16, __float_as_uint(wmax), peer_mbar(MB_X + 4 * sb + grp));
          if (quad == 0 && lane == 0) tc::mbar_arrive_expect(mbar(MB_X + 4 * sb + grp), 32 * 16);
        }
        group_sync();
        wait_peer(mbar(MB_X + 4 * sb + grp), static_cast<uint32_t>((g >> 1) & 1), s_abort, p.err);
        float alpha = 1.f;
        {
          const float4 o4 = *reinterpret_cast<const float4*>(s_red + sb * ROWS * 4 + row * 4);
          const float4 p4 = *reinterpret_cast<const float4*>(s_xred + sb * ROWS * 4 + row * 4);
          const float top = fmaxf(fmaxf(fmaxf(o4.x, o4.y), fmaxf(o4.z, o4.w)), fmaxf(fmaxf(p4.x, p4.y), fmaxf(p4.z, p4.w)));
          // (Scores beyond 2^24 may round the difference to 16 or more, which
          // fp16 does not hold: no shift there.)
          float bm = top - P_SHIFT;
          if (top - bm > P_SHIFT + 0.5f) bm = top;
          if (bm > mrow) {
            if (mrow != -INFINITY) alpha = ex2(mrow - bm);
            mrow = bm;
          }
          // A fully masked row: p = ex2(-inf - 0) = 0.  (The group's warps
          // write the same values; the other half of s_m is free until the
          // group has met again.)
          s_m[sb * ROWS + row] = mrow == -INFINITY ? 0.f : mrow;
          s_m[(sb ^ 1u) * ROWS + row] = alpha;
        }
        __syncwarp();
        // The fused product below is exact, the maximum a rounded one, half an
        // ulp of the score away at most.  Weights and row sum share whatever it
        // is, but where it is 1 and more the largest weight would leave fp16:
        // there the scores are rounded as the maximum was.  (All warps of the
        // group decide alike: they hold the same maxima.)
        if (__any_sync(0xffffffffu, fabsf(mrow) > FUSED_LIMIT)) {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] *= mul;
          mul = 1.f;
        }
        // P^T in fp16: the largest weight is 2^15, those from 2^-14 on lose
        // 2^-11 at most, smaller ones 2^-25 (2^-40 of the largest).
        uint32_t pk[16];   // word 4 k8 + i: rows (i, 0) and (i, 1) of key 8 k8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 m2 = *reinterpret_cast<const float2*>(s_m + sb * ROWS + c0 + 8 * i + pair);
          y[2 * i] = y[2 * i + 1] = 0.f;
#pragma unroll
          for (int k8 = 0; k8 < 4; ++k8) {
            const int n = 16 * (k8 >> 1) + 4 * i + 2 * (k8 & 1);
            const float p0 = ex2(fmaf(x[n], mul, -m2.x)), p1 = ex2(fmaf(x[n + 1], mul, -m2.y));
            y[2 * i] += p0;
            y[2 * i + 1] += p1;
            const __half2 hh = __floats2half2_rn(p0, p1);
            pk[4 * k8 + i] = *reinterpret_cast<const uint32_t*>(&hh);
          }
        }
        // O^T of the step before done: the P^T buffers (here and in the peer)
        // are free and O^T can be rescaled.  (A segment's first step: the
        // readout waited for it.)
        if (it > 0) {
          wait_own(mbar(MB_OT), static_cast<uint32_t>((g - 1) & 1), s_abort, p.err);
          tc::fence_after_sync();
          const uint32_t moved = __ballot_sync(0xffffffffu, alpha != 1.f);   // by lane
          if (moved != 0) {
            const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c0;
            const int cnt = __popc(moved);
            if (cnt <= FEW_MOVED) {
              uint32_t m = moved;
              for (int q = 0; q < cnt; ++q) {
                const int l = __ffs(m) - 1;
                m &= m - 1;
                const int c = __shfl_sync(0xffffffffu, row, l) - c0;
                const float a = __shfl_sync(0xffffffffu, alpha, l);
                const uint32_t v0 = tc::tmem_ld1(lane_base + c);
                const uint32_t v1 = tc::tmem_ld1(lane_base + 128 + c);
                tc::tmem_wait_ld();
                tc::tmem_st1(lane_base + c, __float_as_uint(__uint_as_float(v0) * a));
                tc::tmem_st1(lane_base + 128 + c, __float_as_uint(__uint_as_float(v1) * a));
              }
            } else {
              const float* s_alpha = s_m + (sb ^ 1u) * ROWS + c0;
#pragma unroll 1
              for (int t = 0; t < 4; ++t) {   // 16 columns at a time
                const uint32_t at = lane_base + 128u * (t >> 1) + 16u * (t & 1);
                uint32_t v[16];
                tc::tmem_ld16(at, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float4 a4 = *reinterpret_cast<const float4*>(s_alpha + 16 * (t & 1) + 4 * q);
                  v[4 * q] = __float_as_uint(__uint_as_float(v[4 * q]) * a4.x);
                  v[4 * q + 1] = __float_as_uint(__uint_as_float(v[4 * q + 1]) * a4.y);
                  v[4 * q + 2] = __float_as_uint(__uint_as_float(v[4 * q + 2]) * a4.z);
                  v[4 * q + 3] = __float_as_uint(__uint_as_float(v[4 * q + 3]) * a4.w);
                }
                tc::tmem_st16(at, v);
              }
            }
            tc::tmem_wait_st();
          }
        }
        // Eight rows (one i) are a 16-byte granule of the key's swizzled row.
        if (p_local) {
#pragma unroll
          for (int k8 = 0; k8 < 4; ++k8) tc::stmatrix4(p_matrix + k8 * 1024, pk + 4 * k8);
        } else {
          // Lane t takes row granule t % 4 of its key from the four lanes
          // that hold its row pairs (a 4 x 4 transpose, four shuffles a key):
          // four 16-byte stores went out in half the time of sixteen words.
          const bool odd = lane & 1, high = lane & 2;
#pragma unroll
          for (int k8 = 0; k8 < 4; ++k8) {
            const uint32_t* w = pk + 4 * k8;
            const uint32_t r01 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
            const uint32_t r23 = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
            const uint32_t u0 = odd ? r01 : w[0], u1 = odd ? w[1] : r01, v0 = odd ? r23 : w[2], v1 = odd ? w[3] : r23;
            const uint32_t g0 = __shfl_xor_sync(0xffffffffu, high ? u0 : v0, 2);
            const uint32_t g1 = __shfl_xor_sync(0xffffffffu, high ? u1 : v1, 2);
            if (alive) tc::st_async_v4(p_peer + k8 * 1024, high ? make_uint4(g0, g1, v0, v1) : make_uint4(u0, u1, g0, g1), peer_mbar(MB_PX));
          }
        }
        if (p_local) tc::fence_async_smem();   // (the peer's MMA warp fences the st.async bytes)
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(mbar(MB_P));
        // The step's row sums over this warp's 32 keys, off the way to O^T.
        lrun = lrun * alpha + reduce_rows<true>(y, lane);
      }
      // ---- the segment's end: row sums over the group's warps, then the peer's
      const int eb = (g & 1) * ROWS;   // the halves of s_red and s_m that the last step did not use
      s_red[(eb + row) * 4 + quad] = lrun;
      group_sync();
      float* s_l = s_m + eb;
      const size_t part0 = static_cast<size_t>(part_slot(cluster, s.first)) * ROWS;
      if (quad == 0) {
        const float4 q4 = *reinterpret_cast<const float4*>(s_red + (eb + row) * 4);
        const float ls = (q4.x + q4.y) + (q4.z + q4.w);
        if (*s_abort == 0) {
          tc::st_async_b32(tc::peer_addr(sbase + OFF_XSUM + row * 4, peer), __float_as_uint(ls), peer_mbar(MB_XS));
          if (tid == 0) tc::mbar_arrive_expect(mbar(MB_XS), ROWS * 4);
        }
        wait_peer(mbar(MB_XS), static_cast<uint32_t>(k & 1), s_abort, p.err);
        // Both CTAs add the two halves in the same order.
        const float lo = rank == 0 ? ls : s_xsum[row];
        const float hi = rank == 0 ? s_xsum[row] : ls;
        const float l = lo + hi;
        const int r = row;
        const float nan = __int_as_float(0x7fc00000);
        // A row that is not served, or saw a value outside fp16: NaN.
        const bool lost = l != l || s_row[r].x < 0;
        s_l[r] = lost ? nan : l > 0.f ? 1.f / l : 0.f;
        if (r < s.t.nrows && (r >> 6) == static_cast<int>(rank)) {
          const float lse = lost ? nan : l > 0.f ? ((mrow + P_SHIFT) + log2f(l / P_LARGEST)) * kLn2 : -INFINITY;
          if (s.whole) p.lse[s.t.q_row0 + r] = lse;
          else p.part_lse[part0 + r] = lse;
        }
      }
      group_sync();
      // ---- O^T out of TMEM; thread = value dim, each warp store 32
      // consecutive dims of a row.
      wait_own(mbar(MB_OT), static_cast<uint32_t>((g - 1) & 1), s_abort, p.err);
      tc::fence_after_sync();
      const int rows = s.t.nrows - c0;
      const size_t out0 = (s.whole ? static_cast<size_t>(s.t.q_row0) : part0) + c0;
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        float v[32];
        tc::tmem_ld32f(tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128u * t + c0, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 i4 = *reinterpret_cast<const float4*>(s_l + c0 + 4 * q);
          v[4 * q] = i4.x == 0.f ? 0.f : v[4 * q] * i4.x;
          v[4 * q + 1] = i4.y == 0.f ? 0.f : v[4 * q + 1] * i4.y;
          v[4 * q + 2] = i4.z == 0.f ? 0.f : v[4 * q + 2] * i4.z;
          v[4 * q + 3] = i4.w == 0.f ? 0.f : v[4 * q + 3] * i4.w;
        }
        const size_t at = out0 * D_V + t * 256 + static_cast<int>(rank) * 128 + quad * 32 + lane;
        if (s.whole && p.out_bf16) {
          __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c < rows) o[c * D_V] = __float2bfloat16_rn(v[c]);
        } else {
          float* o = (s.whole ? reinterpret_cast<float*>(p.out) : p.part_o) + at;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c < rows) o[c * D_V] = v[c];
        }
      }
      tc::fence_before_sync();   // the next segment's O^T overwrites these columns after MB_P
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0 && s_abort[0] != 0) st_peer(tc::peer_addr(smem_u32(s_tmem + 4), peer), 1);
  // Neither CTA leaves while the peer may still write into its shared
  // memory, signal its barriers or (even CTA) read its operands.
  tc::cluster_sync();
  tc::fence_after_sync();
  if (s_abort[0] != 0 || s_abort[1] != 0) {   // the same in both CTAs
    // Copies and stores under way land within microseconds: far longer than
    // that.  And every MMA issued is done before tensor memory is freed.
    settle(1LL << 22);
    if (warp == MMA_WARP) {
      if (rank == 0) tc::commit_pair(mbar(MB_DONE));
      wait_drain(mbar(MB_DONE), 0, p.err);
    }
    const SharedPos end{range.z, range.w};
    for (int tile = from.tile; next_segment(p, share, from, end, tile, s); tile = s.tile + 1)
      write_nan_segment(p, s, cluster, rank, tid);
    tc::cluster_sync();
    tc::fence_after_sync();
  }
  if (warp == MMA_WARP) tc::tmem_dealloc_pair<TMEM_COLS>(tmem);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

}  // namespace

cudaError_t make_shared_maps(SharedMaps* maps, void* k16, long long k_plane, void* q16, long long q_plane) {
  // (Looked up once per process: a look-up takes longer than the three maps.)
  struct Encoder {
    EncodeTiled fn;
    cudaError_t e;
  };
  static const Encoder encoder = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    const bool found = e == cudaSuccess && q == cudaDriverEntryPointSuccess && fn;
    return Encoder{reinterpret_cast<EncodeTiled>(fn), found ? cudaSuccess : e != cudaSuccess ? e : cudaErrorNotSupported};
  }();
  if (encoder.e != cudaSuccess) return encoder.e;
  const EncodeTiled encode = encoder.fn;
  // Nine planes of rows of 64 fp16 (128 bytes), swizzled on the way in.
  auto planes = [&](CUtensorMap* map, void* base, long long rows, cuuint32_t box_rows, cuuint32_t box_planes) {
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), 9};
    const cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(rows) * 128};
    const cuuint32_t box[3] = {64, box_rows, box_planes}, estrides[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, base, dims, strides, box, estrides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  if (planes(&maps->pair, k16, k_plane, BN, 2) != CUDA_SUCCESS || planes(&maps->chunk, k16, k_plane, BN, 1) != CUDA_SUCCESS ||
      planes(&maps->q, q16, q_plane, HROWS, Q_PLANES) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

cudaError_t partial_shared_prepare() {
  cudaError_t e = cudaFuncSetAttribute(partial_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(partial_shared_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

cudaError_t launch_partial_shared(const SharedParams& p, const SharedMaps& maps, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.clusters);
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = SMEM_TOTAL;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, partial_shared_kernel, p, maps.pair, maps.chunk, maps.q);
}

}  // namespace mlav
