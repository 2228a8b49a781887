// norm_quant_i8.cu -- gated residual, normalisation and adaLN modulation with
// an int8 output and one scale per token: what modulate_swiglu writes as bf16,
// in the form the int8 linear layers read, in one pass over the rows (the
// pages fuse "residual connections", normalisation and modulation into fewer
// launches: "FastH3 在八卡 B300 上实现完整 MP4 生成快于播放时长", section "融合 DiT
// 算子"; that the layer behind reads 8-bit integers is a reading, not theirs).
//
//   x' = x + gate_res[s] * branch          (either may be left out)
//   h  = norm(x') * weight * (1 + scale[s]) + shift[s]
//   step = max_c |h_c| / 127 (1 for a zero row)
//   code_c = 127 h_c / max_c |h_c| to the nearest integer, ties to even
//
// HBM-bound: x and branch are read once, x' and the codes written once (7
// bytes an element with everything on). kTpr threads own one row and hold all
// of it in registers as fp32 (as bf16 where x itself is coded), kCpt chunks of 8
// elements a thread, so the three
// dependent passes over a row (its moments, its largest |h|, its codes) cost
// no memory traffic and h is never rounded before it is coded. Rows of one
// warp need only shuffles; longer ones exchange one word per warp.
//
// Sums are fp32: at most 64 elements in a thread's chain, then a tree. The
// largest |h| is taken on the bits (for non-negative floats their order is
// the numbers', with NaN above infinity), so that a NaN cannot get lost in a
// maximum: a row that is not finite gets scale NaN and codes 0, which makes
// its dequantised values NaN, and no other row's.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "packed_rows.cuh"
#include "pqk_internal.h"

namespace pqk {
namespace {

struct NormQuantParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* branch;
  __nv_bfloat16* x_out;
  int8_t* h8;
  float* h_scale;
  int64_t x_stride, branch_stride, x_out_stride, h8_stride;
  const __nv_bfloat16* weight;
  const float* shift;
  const float* scale;
  const float* gate_res;
  const int32_t* cu;
  int B;
  int64_t T;
  int C;
  int norm_type;
  float eps;
  bool wide;  // shift, scale and gate_res start on 32-byte boundaries
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Bits of the largest of eight |bf16|, as an fp32 number.
__device__ __forceinline__ uint32_t max_abs_bf16x8(const uint4& v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                              __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m << 16, m & 0xffff0000u);
}

__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Eight entries of a request's vector, in one 32-byte load where the vectors
// start on 32-byte boundaries: two 16-byte loads with 32 bytes between lanes
// pass twice as many lines through L1 ([58,048, 5,120] with all vectors: 395 us
// with the latter, 366 with the former).
__device__ __forceinline__ void load8f(const float* p, bool wide, float (&f)[8]) {
  if (wide) {
    asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
        : "l"(p));
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// The larger of a and |b|; NaN where one of them is. One instruction, where the
// maximum of the bits takes two.
__device__ __forceinline__ float max_abs_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The kTpr threads of a row: combine one value of each and give every thread
// the result. `slot`: kTpr / 32 words of shared memory used by this row only,
// and by this exchange only until the row's next barrier.
template <int kTpr, typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, T* slot, Op op) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, off));
  if constexpr (kTpr > 32) {
    const int warp_in_row = (threadIdx.x % kTpr) >> 5;
    if ((threadIdx.x & 31) == 0) slot[warp_in_row] = v;
    __syncthreads();  // such a row is a block of its own
    v = slot[0];
#pragma unroll
    for (int i = 1; i < kTpr / 32; ++i) v = op(v, slot[i]);
  }
  return v;
}

struct AddOp {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// Threads per block: one row, or four of a warp each (blocks of two or four
// rows of 128 threads leave more of an SM idle between rows: 364 and 491 us
// where these take 348 for [58,048, 5,120]).
template <int kTpr>
constexpr int kBlock = kTpr < 128 ? 128 : kTpr;

// Blocks per SM that a layout's registers have to allow, where the compiler by
// itself takes a few more registers than fit one more block of rows in flight
// (four or more chunks a thread): at most 64 to 80 of them. Without and with the
// bound, us at one stage of the kernel, everything on / without the branch /
// LayerNorm without vectors:
//   128 x 4  20,000 x 4,096   112 / 75 / 104   111 / 72 / 100
//   128 x 5  58,048 x 5,120   389 / 259 / 363  377 / 245 / 353
//   128 x 6  20,000 x 6,144   173 / 117 / 158  165 / 105 / 147
//   128 x 7  20,000 x 7,168   222 / 130 / 188  222 / 125 / 175
//   256 x 5  20,000 x 10,240  307 / 189 / 258  302 / 176 / 247
//   256 x 6  12,345 x 12,288  274 / 173 / 217  257 / 137 / 189
//   256 x 7  12,345 x 14,336  334 / 194 / 259  315 / 166 / 230 (32 bytes spilled)
//   512 x 4  12,345 x 16,384  441 / 305 / 368  332 / 195 / 272
// and for codes of x alone 512 x 4, 12,345 x 16,384 118 -> 105, x 14,344 113 -> 98.
template <int kTpr, int kCpt, bool kPlain>
constexpr int kBlocksPerSm = kPlain      ? (kTpr == 512 ? 3 : 1)
                             : kCpt < 4  ? 1
                             : kTpr == 128 ? (kCpt == 4 ? 8 : kCpt == 7 ? 6 : 7)
                             : kTpr == 256 ? (kCpt < 6 ? 4 : 3)
                             : kTpr == 512 ? 2
                                           : 1;

// kPlain: codes of x alone (no branch, norm or vectors), in fewer registers.
template <int kTpr, int kCpt, bool kPlain>
__global__ void __launch_bounds__(kBlock<kTpr>, kBlocksPerSm<kTpr, kCpt, kPlain>)
    norm_quant_i8_kernel(const NormQuantParams p) {
  constexpr int kRows = kBlock<kTpr> / kTpr;
  // one set of words for each of a row's exchanges, so that no exchange can
  // overwrite words that a slow warp still reads
  __shared__ float s_sum[kRows][3][kTpr / 32];
  __shared__ uint32_t s_max[kRows][kTpr / 32];
  const int group = threadIdx.x / kTpr;
  const int lane = threadIdx.x % kTpr;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + group;
  if (t >= p.T) return;  // a whole row's threads leave together: barriers count one row's threads
  const int nchunks = p.C >> 3;
  const int64_t mod_row =
      !kPlain && p.cu != nullptr ? static_cast<int64_t>(request_of(p.cu, p.B, t)) * p.C : 0;

  uint4 xr[kCpt];
#pragma unroll
  for (int i = 0; i < kCpt; ++i) {
    const int c = lane + i * kTpr;
    xr[i] = c < nchunks ? ld16(p.x + t * p.x_stride + c * 8) : make_uint4(0, 0, 0, 0);
  }
  // the row in fp32; codes of x alone keep it as it came, in half the registers
  float v[kPlain ? 1 : kCpt][8];
  if constexpr (!kPlain) {
    uint4 br[kCpt];
    if (p.branch != nullptr) {
#pragma unroll
      for (int i = 0; i < kCpt; ++i) {
        const int c = lane + i * kTpr;
        br[i] = c < nchunks ? ld16(p.branch + t * p.branch_stride + c * 8) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kCpt; ++i) {
      const int c = lane + i * kTpr;
      unpack8(xr[i], v[i]);
      if (p.branch != nullptr && c < nchunks) {
        float b[8], g[8];
        unpack8(br[i], b);
        if (p.gate_res != nullptr) {
          load8f(p.gate_res + mod_row + c * 8, p.wide, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = fmaf(g[e], b[e], v[i][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += b[e];
        }
      }
    }
  }
  // x' of every element is formed by the thread that read the element: x_out
  // may be x (or branch) itself
  if constexpr (!kPlain) {
    if (p.x_out != nullptr) {
#pragma unroll
      for (int i = 0; i < kCpt; ++i) {
        const int c = lane + i * kTpr;
        if (c < nchunks) {
          uint4 o;
          o.x = pack_bf16x2(v[i][0], v[i][1]);
          o.y = pack_bf16x2(v[i][2], v[i][3]);
          o.z = pack_bf16x2(v[i][4], v[i][5]);
          o.w = pack_bf16x2(v[i][6], v[i][7]);
          *reinterpret_cast<uint4*>(p.x_out + t * p.x_out_stride + c * 8) = o;
        }
      }
    }

    const float inv_c = 1.0f / static_cast<float>(p.C);
    if (p.norm_type != 2) {
      float mu = 0.f;
      if (p.norm_type == 1) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kCpt; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) s += v[i][e];
        // a quotient, not a product with 1 / C: a constant row's sum is exact, and
        // its mean has to be that constant
        mu = row_reduce<kTpr>(s, s_sum[group][0], AddOp()) / static_cast<float>(p.C);
      }
      // centred second moment (mu = 0 for RMS); elements past C stay 0
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < kCpt; ++i) {
        if (lane + i * kTpr < nchunks) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[i][e] -= mu;
            s2 = fmaf(v[i][e], v[i][e], s2);
          }
        }
      }
      s2 = row_reduce<kTpr>(s2, s_sum[group][1], AddOp());
      float inv;
      if (s2 <= 3.402823466e38f) {
        inv = 1.0f / sqrtf(s2 * inv_c + p.eps);
      } else {
        // The sum passed fp32's range; the mean square need not have: sum the
        // squares of 2^-12 v (C is at most 2^14). A row whose mean square passes
        // it counts as not finite.
        float small = 0.f;
#pragma unroll
        for (int i = 0; i < kCpt; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = lane + i * kTpr < nchunks ? v[i][e] * 0x1p-12f : 0.f;
            small = fmaf(u, u, small);
          }
        }
        const float mean = row_reduce<kTpr>(small, s_sum[group][2], AddOp()) * inv_c * 0x1p24f;
        inv = mean <= 3.402823466e38f ? 1.0f / sqrtf(mean + p.eps) : __int_as_float(0x7fffffff);
      }
#pragma unroll
      for (int i = 0; i < kCpt; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= inv;
    }
  }
  uint32_t top = 0;  // bits of the largest |h|
  float top_f = 0.f;
#pragma unroll
  for (int i = 0; i < kCpt; ++i) {
    const int c = lane + i * kTpr;
    if (c < nchunks) {
      if constexpr (kPlain) {
        top = max(top, max_abs_bf16x8(xr[i]));
      } else {
        if (p.weight != nullptr) {
          float w[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight + c * 8)), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
        }
        if (p.shift != nullptr) {
          float sc[8], sh[8];
          load8f(p.scale + mod_row + c * 8, p.wide, sc);
          load8f(p.shift + mod_row + c * 8, p.wide, sh);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = fmaf(v[i][e], 1.0f + sc[e], sh[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top_f = max_abs_or_nan(top_f, v[i][e]);
      }
    }
  }
  if constexpr (!kPlain) top = __float_as_uint(top_f);
  top = row_reduce<kTpr>(top, s_max[group], MaxOp());

  const bool finite = top < 0x7f800000u;
  const float amax = __uint_as_float(top);
  // 127 / amax as hi + lo, whose sum is off by less than 2^-46 of it: the
  // quotient below is the real one rounded once (but for real ones within 2^-40
  // of the border between two floats), and a tie stays a tie. With hi alone an
  // element of half the row's maximum, 63.5 steps, was coded 63 for 66 of the 128
  // mantissas that a bf16 maximum can have. Rows whose hi or lo would overflow or
  // be subnormal are scaled by a power of two first.
  const float shift_by = amax < 7.888609052e-31f  ? 18446744073709551616.0f  // 2^-100, 2^64
                         : amax > 1.267650600e30f ? 5.421010862e-20f         // 2^100, 2^-64
                                                  : 1.0f;
  const float a = amax * shift_by;
  if constexpr (!kPlain) {
    if (shift_by != 1.0f) {
#pragma unroll
      for (int i = 0; i < kCpt; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= shift_by;
    }
  }
  const float hi = a > 0.f ? 127.0f / a : 0.f;
  const float lo = fmaf(-hi, a, 127.0f) * (hi * (1.0f / 127.0f));
  if (lane == 0) p.h_scale[t] = finite ? (amax > 0.f ? amax / 127.0f : 1.0f) : __int_as_float(0x7fffffff);
#pragma unroll
  for (int i = 0; i < kCpt; ++i) {
    const int c = lane + i * kTpr;
    if (c < nchunks) {
      float h[8];
      if constexpr (kPlain) {
        unpack8(xr[i], h);
        if (shift_by != 1.0f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) h[e] *= shift_by;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = v[i][e];
      }
      // the quotient + 1.5 * 2^23: the integer nearest to it (ties to even) is
      // the sum's low byte
      uint32_t q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(fmaf(h[e], hi, h[e] * lo) + 12582912.0f);
      uint2 o;
      o.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
      o.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
      if (!finite) o = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(p.h8 + t * p.h8_stride + c * 8) = o;
    }
  }
}

template <int kTpr, int kCpt>
int launch(const NormQuantParams& p, bool plain, cudaStream_t stream) {
  constexpr int kRows = kBlock<kTpr> / kTpr;
  const unsigned blocks = static_cast<unsigned>((p.T + kRows - 1) / kRows);
  if (plain)
    norm_quant_i8_kernel<kTpr, kCpt, true><<<blocks, kBlock<kTpr>, 0, stream>>>(p);
  else
    norm_quant_i8_kernel<kTpr, kCpt, false><<<blocks, kBlock<kTpr>, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_norm_quant_i8(const void* x, int64_t x_stride, const void* branch, int64_t branch_stride, void* x_out,
                         int64_t x_out_stride, void* h8, int64_t h8_stride, float* h_scale, const void* weight,
                         const float* shift, const float* scale, const float* gate_res, const int32_t* cu, int B,
                         int64_t T, int C, int norm_type, float eps, cudaStream_t stream, int num_sms) {
  NormQuantParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.branch = static_cast<const __nv_bfloat16*>(branch);
  p.x_out = static_cast<__nv_bfloat16*>(x_out);
  p.h8 = static_cast<int8_t*>(h8);
  p.h_scale = h_scale;
  p.x_stride = x_stride;
  p.branch_stride = branch_stride;
  p.x_out_stride = x_out_stride;
  p.h8_stride = h8_stride;
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.shift = shift;
  p.scale = scale;
  p.gate_res = gate_res;
  p.cu = cu;
  p.B = B;
  p.T = T;
  p.C = C;
  p.norm_type = norm_type;
  p.eps = eps;
  p.wide = (reinterpret_cast<uintptr_t>(shift) | reinterpret_cast<uintptr_t>(scale) |
            reinterpret_cast<uintptr_t>(gate_res)) % 32 == 0;
  // How a row is laid over threads: the layout with the fewest idle chunks of
  // 8, and of equals the one with fewer threads a row (shorter exchanges) unless
  // that takes 8 chunks a thread. Measured at one stage of the kernel, threads x
  // chunks: C = 5,120, 58,048 rows: 128 x 5 394 us, 256 x 3 422; C = 13,824,
  // 12,345 rows: 256 x 7 104, 512 x 4 118; C = 16,384, 3,000 rows: 512 x 4 94,
  // 256 x 8 104; C = 2,048, 4,096 rows: 128 x 2 18.5, 32 x 8 34. With fewer rows
  // than would fill the GPU a row's latency counts, and more threads shorten it
  // (200 rows of 5,120: 512 x 2 4.8 us, 128 x 5 6.3).
  const int n = C / 8;
  const bool plain = branch == nullptr && x_out == nullptr && norm_type == 2 && weight == nullptr && shift == nullptr;
  const bool few = T <= 2 * num_sms;
  int tpr = 0, cpt = 0, best = INT_MAX;
  for (int t : {32, 128, 256, 512}) {
    const int c = (n + t - 1) / t;
    if (c > (few ? 2 : (t < 128 ? 4 : 7)) && t < 512) continue;
    if (t * c < best) {
      best = t * c;
      tpr = t;
      cpt = c;
    }
  }
  switch (tpr * 8 + cpt) {
#define PQK_LAYOUT(t, c) \
  case t * 8 + c: return launch<t, c>(p, plain, stream)
    PQK_LAYOUT(32, 1);
    PQK_LAYOUT(32, 2);
    PQK_LAYOUT(32, 3);
    PQK_LAYOUT(32, 4);
    PQK_LAYOUT(128, 1);
    PQK_LAYOUT(128, 2);
    PQK_LAYOUT(128, 3);
    PQK_LAYOUT(128, 4);
    PQK_LAYOUT(128, 5);
    PQK_LAYOUT(128, 6);
    PQK_LAYOUT(128, 7);
    PQK_LAYOUT(256, 2);
    PQK_LAYOUT(256, 4);
    PQK_LAYOUT(256, 5);
    PQK_LAYOUT(256, 6);
    PQK_LAYOUT(256, 7);
    PQK_LAYOUT(512, 2);
    PQK_LAYOUT(512, 3);
    PQK_LAYOUT(512, 4);
#undef PQK_LAYOUT
    default: return -1;  // unreachable: n <= 2048
  }
}

}  // namespace pqk
