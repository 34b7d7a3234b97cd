// New tokens' cache rows and queries: the norm of each token's latent, the
// position rotation of its shared rope dims and of every query head's, and
// the write into the paged cache, in one pass.
//
// Definition (token n with slot s and position p; (cos, sin)_i = row p of the
// table):
//   row[0:512]   = bf16(c * rsqrt(mean(c^2) + eps) * w),  c = kv[n, 0:512]
//   row[512:576] = rot(kv[n, 512:576], p)            -> cache[s]
//   q[n, h]      = q_nope[n, h] | rot(q_pe[n, h], p)
//   rot(x)_a = x_a cos_i - x_b sin_i,  rot(x)_b = x_b cos_i + x_a sin_i, with
//   (a, b) = (2i, 2i + 1), or (i, i + 32) when the two halves are rotated.
// A token with slot -1 is padding; one whose slot is outside the cache
// (ERR_SLOT) or whose position is outside the table (ERR_POS) is reported:
// nothing of either is written.  Sums and products are fp32, rounded to bf16
// once, when they are stored.
//
// HBM is the bound: a token reads and writes 1152 bytes, and 1152 (or 128,
// when the absorbed part is already in place) for every head.  A warp takes
// one item -- a token's cache row, or four of its heads -- and has the item's
// nine 16-byte loads per lane in flight before it uses any: with four heads
// the 4 x 64 copied granules and the 4 x 8 rotated ones divide evenly over
// the lanes.
#include "common.cuh"
#include "kernels.h"

#include <cuda_bf16.h>

namespace mlav {
namespace {

constexpr int THREADS = 256;
constexpr int HEADS = 4;                 // heads per item
constexpr int NOPE_GRANULES = D_V / 8;   // 64 sixteen-byte granules
constexpr int DR = D_QK - D_V;           // 64 rotated dims

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
// Granules read once by the whole call.  (No read-only load: those are for
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

// The table entries granule g (0..7) of the rotated dims needs: pairs 4g ..
// 4g+3 when neighbours are rotated, 8(g & 3) .. +7 when the halves are.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ Angles load_angles(const float* row, int g, bool halves) {
  Angles a;
  const float4* cs = reinterpret_cast<const float4*>(row);
  const int i = halves ? 2 * (g & 3) : g;
  const float4 c0 = cs[i], s0 = cs[8 + i];
  const float4 c1 = halves ? cs[i + 1] : c0, s1 = halves ? cs[8 + i + 1] : s0;
  a.c[0] = c0.x, a.c[1] = c0.y, a.c[2] = c0.z, a.c[3] = c0.w;
  a.c[4] = c1.x, a.c[5] = c1.y, a.c[6] = c1.z, a.c[7] = c1.w;
  a.s[0] = s0.x, a.s[1] = s0.y, a.s[2] = s0.z, a.s[3] = s0.w;
  a.s[4] = s1.x, a.s[5] = s1.y, a.s[6] = s1.z, a.s[7] = s1.w;
  return a;
}

// Granule g of the eight that hold one vector's rotated dims, lane g of an
// aligned group of eight lanes (all of them call).
__device__ __forceinline__ uint4 rotate(uint4 v, const Angles& a, int g, bool halves) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (!halves) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = unpack(w[k]);
      w[k] = pack(x.x * a.c[k] - x.y * a.s[k], x.y * a.c[k] + x.x * a.s[k]);
    }
  } else {
    // The partner half of the same eight pairs is four lanes away; the lower
    // half takes -sin.
    const float sign = g < 4 ? -1.f : 1.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = unpack(w[k]), y = unpack(__shfl_xor_sync(0xffffffffu, w[k], 4));
      w[k] = pack(x.x * a.c[2 * k] + sign * y.x * a.s[2 * k], x.y * a.c[2 * k + 1] + sign * y.y * a.s[2 * k + 1]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Squares of bf16 values leave fp32 on both sides: a row whose sum of squares
// is too large, or too small to be held well, is summed again in units of 2^70
// or 2^-80.  Whole warp; returns the reciprocal root for values times `unit`.
// (A call: inlined, it took 8192 tokens of 64 heads from 178 to 189 us.)
constexpr float MAX_SUM = 0x1p120f, MIN_MEAN = 0x1p-80f;
__device__ __noinline__ float rms_in_units(const uint4* row, float eps, float unit) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = threadIdx.x & 31; c < NOPE_GRANULES; c += 32) {
    const uint4 x = row[c];
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    for (int k = 0; k < 4; ++k) {
      const float2 v = unpack(xs[k]);
      sum += (v.x * unit) * (v.x * unit) + (v.y * unit) * (v.y * unit);
    }
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return rsqrtf(sum * (1.f / D_V) + eps * unit * unit);
}

__global__ void __launch_bounds__(THREADS) append_kv_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31, g = lane & 7;
  const int head_items = a.q_pe ? (a.heads + HEADS - 1) / HEADS : 0;
  const long long item = static_cast<long long>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
  const long long n = item / (head_items + 1);
  if (n >= a.num_tokens) return;
  const int part = static_cast<int>(item - n * (head_items + 1));   // 0: the cache row; k: heads 4(k-1) ..
  const long long slot = a.slots[n], pos = a.positions[n];
  if (slot == -1) return;
  const bool slot_ok = slot >= 0 && slot < a.num_slots, pos_ok = pos >= 0 && pos < a.max_pos;
  if (!slot_ok || !pos_ok) {
    if (part == 0 && lane == 0) atomicOr(a.err, (slot_ok ? 0 : ERR_SLOT) | (pos_ok ? 0 : ERR_POS));
    return;
  }
  const bool halves = a.halves != 0;

  if (part == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(a.kv + n * a.kv_stride);
    const uint4* wsrc = reinterpret_cast<const uint4*>(a.weight);
    uint4 x[2], w[2], r = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      x[u] = load_once(src + lane + 32 * u);
      w[u] = wsrc[lane + 32 * u];
    }
    if (lane < 8) r = load_once(src + NOPE_GRANULES + lane);
    const Angles ang = load_angles(a.cos_sin + pos * DR, g, halves);
    float sum = 0.f, unit = 1.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack(xs[k]);
        sum += v.x * v.x + v.y * v.y;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float rms = rsqrtf(sum * (1.f / D_V) + a.eps);
    if (sum > MAX_SUM || sum * (1.f / D_V) + a.eps < MIN_MEAN) {   // (the same in all lanes)
      unit = sum > MAX_SUM ? 0x1p-70f : 0x1p80f;
      rms = rms_in_units(src, a.eps, unit);
    }
    uint4* dst = reinterpret_cast<uint4*>(a.kv_cache + slot * D_QK);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack(xs[k]), f = unpack(ws[k]);
        y[k] = pack(v.x * unit * rms * f.x, v.y * unit * rms * f.y);
      }
      dst[lane + 32 * u] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    r = rotate(r, ang, g, halves);
    if (lane < 8) dst[NOPE_GRANULES + lane] = r;
    return;
  }

  const int h0 = HEADS * (part - 1);
  const int hp = h0 + (lane >> 3);                 // this lane's head for the rotated dims
  const bool pe = hp < a.heads;
  uint4 r = make_uint4(0, 0, 0, 0);
  // Plain loads: q_pe may be the rotated dims of q itself.
  if (pe) r = reinterpret_cast<const uint4*>(a.q_pe + n * a.pe_stride_n + hp * a.pe_stride_h)[g];
  uint16_t* q = a.q + (n * a.heads + h0) * D_QK;
  const Angles ang = load_angles(a.cos_sin + pos * DR, g, halves);
  if (a.q_nope) {
    uint4 v[2 * HEADS];
#pragma unroll
    for (int u = 0; u < 2 * HEADS; ++u)
      if (h0 + u / 2 < a.heads)
        v[u] = load_once(reinterpret_cast<const uint4*>(a.q_nope + n * a.nope_stride_n + (h0 + u / 2) * a.nope_stride_h) +
                         lane + 32 * (u & 1));
#pragma unroll
    for (int u = 0; u < 2 * HEADS; ++u)
      if (h0 + u / 2 < a.heads) reinterpret_cast<uint4*>(q + (u / 2) * D_QK)[lane + 32 * (u & 1)] = v[u];
  }
  r = rotate(r, ang, g, halves);
  if (pe) reinterpret_cast<uint4*>(q + (lane >> 3) * D_QK + D_V)[g] = r;
}

}  // namespace

cudaError_t launch_append_kv(const AppendArgs& a, cudaStream_t stream) {
  const long long items = a.num_tokens * (a.q_pe ? (a.heads + HEADS - 1) / HEADS + 1 : 1);
  const long long ctas = (items + THREADS / 32 - 1) / (THREADS / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_overlapping(append_kv_kernel, dim3(static_cast<unsigned>(ctas)), THREADS, 0, stream, 1, a);
}

}  // namespace mlav
