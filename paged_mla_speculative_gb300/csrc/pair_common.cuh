// What the CTA-pair kernels (partial_pair.cu, partial_shared.cu, weigh_kv.cu)
// have in common: bounded waits, the shuffle reduction and the order of the
// ring units; and two instructions that tc_ptx.cuh does not have.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace mlav {
namespace tc {

// TMA tile load of a 2-D tensor for this CTA alone, signalled on a barrier of
// its own.  Warp-collective; the elected lane issues.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t mbar) {
  asm volatile(
      "{\n.reg .pred e;\n"
      "elect.sync _|e, 0xffffffff;\n"
      "@e cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}
// An 8x8 matrix of 16-bit values, a row's pairs in four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(w));
  return r;
}

}  // namespace tc

constexpr long long WAIT_LIMIT = 1LL << 31;     // cycles before a wait gives up

__device__ __forceinline__ void named_sync(int id, int count) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(count) : "memory");
}

// Bounded wait (acquire at cluster scope: some arrivals come from the peer
// CTA).  A timeout, or an earlier one in this CTA, returns false.
__device__ __forceinline__ bool wait_phase(uint32_t mbar, uint32_t parity, volatile int* abort, int* err) {
  if (tc::mbar_try_cluster(mbar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (tc::mbar_try_cluster(mbar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > WAIT_LIMIT) {
      *abort = 1;
      atomicOr(err, ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ void wait_warp(uint32_t mbar, uint32_t parity, volatile int* abort, int* err) {
  wait_phase(mbar, parity, abort, err);
  __syncwarp();
}
// Bounded wait that ignores the abort flag (own copies in flight at exit).
__device__ __forceinline__ void wait_drain(uint32_t mbar, uint32_t parity, int* err) {
  const long long t0 = clock64();
  while (!tc::mbar_try(mbar, parity)) {
    if (clock64() - t0 > WAIT_LIMIT) {
      atomicOr(err, ERR_TIMEOUT);
      return;
    }
  }
}

// Column maxima / sums of a warp's 32 x 32 tile (lane = key, v[c] = column
// c) in 31 shuffles: lane l ends with column l's result in v[0].
template <bool SUM>
__device__ __forceinline__ void transpose_reduce32(float (&v)[32], int lane) {
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) {
    const bool upper = (lane & w) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = upper ? v[i] : v[i + w];
      const float keep = upper ? v[i + w] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, w);
      v[i] = SUM ? keep + got : fmaxf(keep, got);
    }
  }
}

// Ring unit order shared by the copy warps and the MMA warp.  Phase f of 2n:
// S(0), S(1), O(0), S(2), O(1), .., S(n-1), O(n-2), O(n-1); S(i) = the CTA's
// own block's chunk pairs 0..3 (and its rope chunk, into the rope slot),
// O(i) = for t in 0,1 and key half h in 0,1: chunk pair 2t + rank of block
// 2i + h.  Unit n goes to slot n % 3.
__device__ __forceinline__ void phase_of(int f, int n, bool& is_s, int& i) {
  if (f == 0) { is_s = true; i = 0; }
  else if (f == 2 * n - 1) { is_s = false; i = n - 1; }
  else if (f & 1) { is_s = true; i = (f + 1) >> 1; }
  else { is_s = false; i = (f >> 1) - 1; }
}

// Spin about `cycles` (an abort path: lets copies and remote stores that
// are still in flight land before the pair leaves).
__device__ __forceinline__ void settle(long long cycles) {
  const long long t0 = clock64();
  while (clock64() - t0 < cycles) {
  }
}

}  // namespace mlav
