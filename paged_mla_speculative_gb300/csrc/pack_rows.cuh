// What the two kernels that lay out a call and pack its keys (shared_pack.cu,
// chunk_pack.cu) have in common: the block scan, the gather of rows into fp16
// planes, and the merge of a row's partials.
#pragma once

#include "shared.cuh"

#include <cuda_bf16.h>

namespace mlav {

constexpr int PACK_THREADS = 256;
constexpr int PACK_KEYS = 32;                                   // rows per CTA iteration
constexpr int PER_THREAD = PACK_KEYS * ROW_CHUNKS / PACK_THREADS;    // 9 granules
static_assert(PER_THREAD * PACK_THREADS == PACK_KEYS * ROW_CHUNKS, "even split");

// Inclusive block scan; `all` receives the block's total.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* s_warp, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < PACK_THREADS / 32; ++w) {
    if (w == warp) x += all;
    all += s_warp[w];
  }
  return x;
}

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
template <typename T>
__device__ __forceinline__ int last_not_above(const T* a, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct Rows {
  uint4 v[PER_THREAD];
};
// A granule that the call reads once.  (No read-only load: those are for
// memory that nothing writes while the kernel runs, and this one is launched
// while the kernel before it may still write its inputs.)
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
// Row r of 32 (each PACK_THREADS / 8 granules apart) at src + s_row[r] * 576, or
// zeros where s_row is negative.
__device__ __forceinline__ void load_rows(const uint16_t* src, const long long* s_row, Rows& x) {
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * PACK_THREADS;
    const int r = e / ROW_CHUNKS, c = e - r * ROW_CHUNKS;
    const long long row = s_row[r];
    x.v[u] = row >= 0 ? load_once(reinterpret_cast<const uint4*>(src + row * D_QK) + c) : make_uint4(0, 0, 0, 0);
  }
}
// Widened into the planes at plane rows row0 .. row0 + rows - 1.  A value
// outside fp16 is packed as zero and sets s_bad of its row; returns whether
// this thread met one.
__device__ __forceinline__ bool store_rows(const Rows& x, int* s_bad, uint16_t* dst, long long plane, long long row0, int rows) {
  bool any = false;
#pragma unroll
  for (int u = 0; u < PER_THREAD; ++u) {
    const int e = threadIdx.x + u * PACK_THREADS;
    const int r = e / ROW_CHUNKS, c = e - r * ROW_CHUNKS;
    bool bad = false;
    uint4 w = widen_bf16x8(x.v[u], bad);
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


// The LSE merge of a row's `nseg` parts, part s in partial row at(s): value
// dims 4 col .. 4 col + 3 and the row's log-sum-exp.  Up to JOIN_FLIGHT parts
// are loaded before any is used.
constexpr int JOIN_FLIGHT = 8;
constexpr int JOIN_MAX = SH_MAX_CLUSTERS / 32;   // parts per lane

template <typename At>
__device__ __forceinline__ void merge_parts(const SharedParams& p, int nseg, const At& at, int col, float4& acc, float& lse) {
  const int lane = threadIdx.x & 31;
  const float nan = __int_as_float(0x7fc00000);
  float L[JOIN_MAX], mx = -INFINITY;
  bool any_nan = false;
#pragma unroll
  for (int k = 0; k < JOIN_MAX; ++k) {
    L[k] = 32 * k + lane < nseg ? p.part_lse[at(32 * k + lane)] : -INFINITY;
    any_nan |= L[k] != L[k];
    mx = fmaxf(mx, L[k]);
  }
  any_nan = __any_sync(0xffffffffu, any_nan);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float top = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < JOIN_MAX; ++k) {
    L[k] = ex2((L[k] - top) * kLog2e);
    sum += L[k];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  // Every key masked (bad slots): weight 0 everywhere.
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < JOIN_MAX; ++k) {
    for (int s0 = 32 * k; s0 < min(nseg, 32 * k + 32); s0 += JOIN_FLIGHT) {
      float4 x[JOIN_FLIGHT];
#pragma unroll
      for (int f = 0; f < JOIN_FLIGHT; ++f)
        if (s0 + f < nseg) x[f] = __ldcs(reinterpret_cast<const float4*>(p.part_o + at(s0 + f) * D_V) + col);
#pragma unroll
      for (int f = 0; f < JOIN_FLIGHT; ++f) {
        const float w = __shfl_sync(0xffffffffu, L[k], (s0 + f) & 31) * inv;
        if (s0 + f >= nseg || w == 0.f) continue;   // (a part of weight 0 may hold anything)
        acc.x += w * x[f].x;
        acc.y += w * x[f].y;
        acc.z += w * x[f].z;
        acc.w += w * x[f].w;
      }
    }
  }
  lse = sum > 0.f ? top + logf(sum) : -INFINITY;
  if (any_nan) {
    acc = make_float4(nan, nan, nan, nan);
    lse = nan;
  }
}

__device__ __forceinline__ void store_merged(const SharedParams& p, int row, int col, float4 acc, float lse) {
  const size_t at = static_cast<size_t>(row) * (D_V / 4) + col;
  if (p.out_bf16) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
    reinterpret_cast<uint2*>(p.out)[at] = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  } else {
    reinterpret_cast<float4*>(p.out)[at] = acc;
  }
  if (col == 0) p.lse[row] = lse;
}

}  // namespace mlav
