// linear_i8_few.cu -- the int8 linear layers for few tokens (a pooled vector,
// a prompt's states): out = epilogue(A W^T) where reading W is most of the
// work, or where the 256-token tiles of linear_epilogue.cu would leave most
// SMs without one.
//
// The operands change places: 128 rows of W are the MMA's M side and up to kNT
// tokens its N side, so a tile with one token wastes no tensor-core rows that
// W needs, and there are N / 128 tiles to spread W over instead of N / 256
// pairs. Where that is still fewer than the SMs, the K range of a tile is
// split over the CTAs of a cluster. The int32 partial sums are exact, so their
// sum does not depend on how K was split: a token's result is the same bits as
// from the pair kernel.
//
//   warp 0      TMA producer: 128 bytes of K of 128 W rows and kNT tokens a stage
//   warp 1      tensor-memory allocator and single-thread MMA issuer
//   warps 2-5   move the accumulator (lane = W row, column = token) to shared
//               memory, token by token
//   all warps   after a cluster barrier, each CTA of the cluster finishes its
//               share of the tokens: sums the CTAs' partials over distributed
//               shared memory, scales, applies the epilogue and stores, 4
//               neighbouring outputs a lane.
// SwiGLU: the 128 rows are 64 gate rows and the same 64 up rows.
//
// Every wait is bounded; a wait that runs out raises the CTA's abort flag and
// the device status word, the CTA drains its copies and MMAs, and no CTA of the
// cluster stores the tile.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "packed_rows.cuh"
#include "pqk_internal.h"

namespace pqk {
namespace {

constexpr int kRows = 128;      // W rows per tile = MMA M
constexpr int kRowBytes = 128;  // K per stage: one 128-byte swizzle row
constexpr int kThreads = 192;
constexpr int kMaxSplit = 8;    // CTAs per cluster
constexpr uint32_t kWBytes = kRows * kRowBytes;

template <int kNT>
struct Layout {
  static constexpr uint32_t kABytes = kNT * kRowBytes;
  static constexpr uint32_t kStageBytes = kWBytes + kABytes;
  // about 100 KB, so that two CTAs share an SM and one's copies run while the
  // other starts or finishes
  static constexpr int kStages = 100 * 1024 / kStageBytes;
  static constexpr int kBarOff = kStages * kStageBytes;
  // full[S], empty[S], acc_full, drain
  static constexpr int kNumBars = 2 * kStages + 2;
  static constexpr int kTmemSlotOff = kBarOff + kNumBars * 8;
  static constexpr int kAbortOff = kTmemSlotOff + 4;
  static constexpr int kAlloc = kAbortOff + 4 + 1024;  // room to align the base to 1024
  // the partial sums [kNT][kRows] take the ring's place
  static_assert(kNT * kRows * 4 <= kBarOff, "partial sums fit the ring");
  static_assert(kStages >= 3 && kAlloc <= 232448 / 2, "two CTAs per SM");
};

struct Params {
  __nv_bfloat16* out;
  int64_t out_stride;
  const __nv_bfloat16* x;
  int64_t x_stride;
  const float* gate_res;
  const int32_t* cu;
  const float* a_scale;
  const float* w_scale;
  int B;
  int64_t T;
  int N;
  int n_kb;
  int* status;
  long long timeout_ns;
};

template <int kNT, int kEpi>
__global__ void __launch_bounds__(kThreads)
    linear_few_kernel(const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
                      const __grid_constant__ CUtensorMap tm_a, const Params p) {
  using L = Layout<kNT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ctarank();
  const uint32_t split = cluster_size();
  const uint32_t bar0 = base + L::kBarOff;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (L::kStages + s); };
  const uint32_t acc_full = bar0 + 8u * (2 * L::kStages);
  const uint32_t drain = acc_full + 8;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kTmemSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbortOff);
  auto raise_abort = [&]() {
    *abort_flag = 1;
    atomicCAS(p.status, 0, kStatusTimeout);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L::kTmemSlotOff, kNT);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensor_map(&tm_w0);
    if (kEpi == kEpiSwiglu) prefetch_tensor_map(&tm_w1);
    prefetch_tensor_map(&tm_a);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int tile = static_cast<int>(blockIdx.x / split);
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kNT;
  // this CTA's K blocks (the host keeps split <= n_kb, so there is at least one)
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.n_kb) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.n_kb) * (rank + 1) / split);
  const int n = kb1 - kb0;
  uint32_t loads = 0;  // stages this CTA's producer loaded, for the drain

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int s = i % L::kStages;
        const uint32_t round = i / L::kStages;
        if (round > 0 && !(ok = mbar_wait(empty(s), (round - 1) & 1, abort_flag, p.timeout_ns))) break;
        mbar_arrive_expect_tx(full(s), L::kStageBytes);
        const uint32_t w = base + s * L::kStageBytes;
        const int k = (kb0 + i) * kRowBytes;
        if constexpr (kEpi == kEpiSwiglu) {
          tma_load_2d(w, &tm_w0, full(s), k, tile * (kRows / 2));
          tma_load_2d(w + kWBytes / 2, &tm_w1, full(s), k, tile * (kRows / 2));
        } else {
          tma_load_2d(w, &tm_w0, full(s), k, tile * kRows);
        }
        tma_load_2d(w + kWBytes, &tm_a, full(s), k, static_cast<int>(t0));
        ++loads;
      }
      if (!ok) raise_abort();
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_s8_s32(kRows, kNT);
      constexpr uint32_t kDescHi = smem_desc_hi_sw128(1024);
      const uint32_t w_lo = smem_desc_lo(base, 16);
      const uint32_t a_lo = smem_desc_lo(base + kWBytes, 16);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int s = i % L::kStages;
        if (!(ok = mbar_wait(full(s), (i / L::kStages) & 1, abort_flag, p.timeout_ns))) break;
        tc_fence_after_sync();
        const uint32_t off = s * (L::kStageBytes >> 4);
#pragma unroll
        for (int k = 0; k < kRowBytes / 32; ++k)
          mma_i8_ss_w(tmem, w_lo + off + 2 * k, a_lo + off + 2 * k, kDescHi, kIdesc, (i > 0 || k > 0) ? 1u : 0u);
        tc_commit(empty(s));
      }
      if (ok) tc_commit(acc_full);
      else raise_abort();
    }
  } else {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, abort_flag, p.timeout_ns));
    if (ok) {
      // every copy has been read by an MMA and every MMA is complete: the
      // ring's memory is free
      tc_fence_after_sync();
      const int row = (warp & 3) * 32 + lane;
      int* part = reinterpret_cast<int*>(smem);
#pragma unroll 1
      for (int c0 = 0; c0 < kNT; c0 += 32) {
        if (t0 + c0 >= p.T) break;
        uint32_t v[32];
        tmem_ld_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, v);
#pragma unroll
        for (int c = 0; c < 32; ++c) part[(c0 + c) * kRows + row] = static_cast<int>(v[c]);
      }
    } else {
      raise_abort();
    }
  }

  tc_fence_before_sync();
  __syncwarp();
  cluster_sync_all();  // every CTA's partial sums are in place, or its abort flag is up
  if (*abort_flag) {
    // this CTA's roles have stopped: wait for what may still be in flight.
    // Copy idx was issued only after copy idx - kStages had landed, so the
    // last kStages issued are the ones outstanding
    if (warp == 0 && lane == 0) {
      const uint32_t first = loads > static_cast<uint32_t>(L::kStages) ? loads - L::kStages : 0;
      for (uint32_t idx = first; idx < loads; ++idx)
        mbar_drain_wait(full(idx % L::kStages), (idx / L::kStages) & 1);
    } else if (warp == 1 && lane == 0) {
      tc_commit(drain);  // completes once every MMA has
      mbar_drain_wait(drain, 0);
    }
    __syncwarp();
  }
  bool aborted = false;
  for (uint32_t r = 0; r < split; ++r) aborted |= ld_cluster_u32(in_cta(base + L::kAbortOff, r)) != 0;
  if (!aborted) {
    // this CTA's share of the tile's tokens
    const int valid = static_cast<int>(p.T - t0 < kNT ? p.T - t0 : kNT);
    const int first = valid * static_cast<int>(rank) / static_cast<int>(split);
    const int last = valid * (static_cast<int>(rank) + 1) / static_cast<int>(split);
    constexpr int kLanes = kEpi == kEpiSwiglu ? 16 : 32;  // lanes per token, 4 outputs each
    constexpr int kTokensPerWarp = 32 / kLanes;
    const int quad = lane % kLanes;
    const int col = tile * kLanes * 4 + quad * 4;
    if (col < p.N) {
      for (int c = first + warp * kTokensPerWarp + lane / kLanes; c < last; c += (kThreads / 32) * kTokensPerWarp) {
        const int64_t t = t0 + c;
        const uint32_t at = base + static_cast<uint32_t>(c * kRows + quad * 4) * 4;
        int4 sum = make_int4(0, 0, 0, 0), up = make_int4(0, 0, 0, 0);
        for (uint32_t r = 0; r < split; ++r) {
          const int4 v = ld_cluster16(in_cta(at, r));
          sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
          if constexpr (kEpi == kEpiSwiglu) {
            const int4 u = ld_cluster16(in_cta(at + kRows / 2 * 4, r));
            up.x += u.x; up.y += u.y; up.z += u.z; up.w += u.w;
          }
        }
        const float row_scale = __ldg(p.a_scale + t);
        float y[4];
        scaled4(sum, row_scale, __ldg(reinterpret_cast<const float4*>(p.w_scale + col)), y);
        if constexpr (kEpi == kEpiSwiglu) {
          float u[4];
          scaled4(up, row_scale, __ldg(reinterpret_cast<const float4*>(p.w_scale + p.N + col)), u);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = silu_mul(y[e], u[e]);
        } else if constexpr (kEpi == kEpiGatedResidual) {
          const int64_t g0 = static_cast<int64_t>(request_of(p.cu, p.B, t)) * p.N + col;
          const float4 g = __ldg(reinterpret_cast<const float4*>(p.gate_res + g0));
          gated4(*reinterpret_cast<const uint2*>(p.x + t * p.x_stride + col), g, y);
        }
        *reinterpret_cast<uint2*>(p.out + t * p.out_stride + col) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      }
    }
  }
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while another reads its partial sums
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, kNT);
}

template <int kNT, int kEpi>
bool prepare() {
  return cudaFuncSetAttribute(linear_few_kernel<kNT, kEpi>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Layout<kNT>::kAlloc) == cudaSuccess;
}
template <int kNT>
bool prepare_epis() {
  return prepare<kNT, kEpiNone>() && prepare<kNT, kEpiGatedResidual>() && prepare<kNT, kEpiSwiglu>();
}

template <int kNT, int kEpi>
int launch(const CUtensorMap& tw0, const CUtensorMap& tw1, const CUtensorMap& ta, const Params& p, int split,
           cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  const int tile_cols = kEpi == kEpiSwiglu ? kRows / 2 : kRows;
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + tile_cols - 1) / tile_cols * split),
                     static_cast<unsigned>((p.T + kNT - 1) / kNT), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<kNT>::kAlloc;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, linear_few_kernel<kNT, kEpi>, tw0, tw1, ta, p) != cudaSuccess) return -1;
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int kNT>
int launch_epi(int epi, const CUtensorMap& tw0, const CUtensorMap& tw1, const CUtensorMap& ta, const Params& p,
               int split, cudaStream_t stream) {
  if (epi == kEpiGatedResidual) return launch<kNT, kEpiGatedResidual>(tw0, tw1, ta, p, split, stream);
  if (epi == kEpiSwiglu) return launch<kNT, kEpiSwiglu>(tw0, tw1, ta, p, split, stream);
  return launch<kNT, kEpiNone>(tw0, tw1, ta, p, split, stream);
}

}  // namespace

bool prepare_linear_i8_few() { return prepare_epis<32>() && prepare_epis<64>() && prepare_epis<128>(); }

int launch_linear_i8_few(int epi, const void* a8, int64_t a_stride, const float* a_scale, const void* w8,
                         int64_t w_stride, const float* w_scale, const void* x, int64_t x_stride,
                         const float* gate_res, const int32_t* cu, int B, void* out, int64_t out_stride, int64_t T,
                         int K, int N, int token_tile, int split, int* status, long long timeout_ns,
                         cudaStream_t stream) {
  CUtensorMap tw0, tw1, ta;
  const bool swiglu = epi == kEpiSwiglu;
  bool ok = make_i8_rows_map(&ta, a8, T, K, a_stride, token_tile) &&
            make_i8_rows_map(&tw0, w8, N, K, w_stride, swiglu ? kRows / 2 : kRows);
  tw1 = tw0;
  if (swiglu)
    ok = ok && make_i8_rows_map(&tw1, static_cast<const char*>(w8) + static_cast<int64_t>(N) * w_stride, N, K,
                                w_stride, kRows / 2);
  if (!ok) return -2;
  Params p;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_stride = out_stride;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.x_stride = x_stride;
  p.gate_res = gate_res;
  p.cu = cu;
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.B = B;
  p.T = T;
  p.N = N;
  p.n_kb = (K + kRowBytes - 1) / kRowBytes;
  p.status = status;
  p.timeout_ns = timeout_ns;
  if (split < 1 || split > kMaxSplit || split > p.n_kb) return -1;
  if (token_tile == 32) return launch_epi<32>(epi, tw0, tw1, ta, p, split, stream);
  if (token_tile == 64) return launch_epi<64>(epi, tw0, tw1, ta, p, split, stream);
  return token_tile == 128 ? launch_epi<128>(epi, tw0, tw1, ta, p, split, stream) : -1;
}

}  // namespace pqk
