// packed_rows.cuh -- what the kernels over packed token rows share. The two int8
// linear kernels give a token the same bits whichever of them a call takes, so
// the arithmetic behind their sums stands here once.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace pqk {

// Request s with cu[s] <= t < cu[s + 1] (the last such s when requests are
// empty); always in 0..B-1, whatever cu holds.
__device__ __forceinline__ int request_of(const int32_t* cu, int B, int64_t t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(__ldg(cu + mid)) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The two bf16 numbers of a 32-bit word.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// silu(g) * u
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// Four neighbouring int32 sums of a token times its scale and theirs.
__device__ __forceinline__ void scaled4(int4 sum, float row_scale, float4 w, float (&y)[4]) {
  y[0] = __int2float_rn(sum.x) * row_scale * w.x;
  y[1] = __int2float_rn(sum.y) * row_scale * w.y;
  y[2] = __int2float_rn(sum.z) * row_scale * w.z;
  y[3] = __int2float_rn(sum.w) * row_scale * w.w;
}

// x + g * y for four neighbouring outputs, x as bf16
__device__ __forceinline__ void gated4(uint2 x, float4 g, float (&y)[4]) {
  y[0] = fmaf(g.x, y[0], bf16_lo(x.x));
  y[1] = fmaf(g.y, y[1], bf16_hi(x.x));
  y[2] = fmaf(g.z, y[2], bf16_lo(x.y));
  y[3] = fmaf(g.w, y[3], bf16_hi(x.y));
}

}  // namespace pqk
