// varlen_attn_fwd.cu -- packed variable-length bf16 self-attention on the
// fifth-generation tensor cores (tcgen05 + tensor memory + TMA).
//
// The operation: every request's tokens attend to all tokens of the same
// request and to nothing else; requests are packed back to back without
// padding and only valid tokens are processed ("FastH3 在八卡 B300 上实现完整
// MP4 生成快于播放时长", section "长序列注意力与通信优化"; "MiniMax H3 FastH3
// real-time serving with vLLM-Omni", bullet "Long-sequence attention &
// communication").
//
// Work unit ("work tile"): (request, head, block of 256 query rows) = two
// 128-row query tiles Q0, Q1 that share every K/V tile. A one-block
// schedule kernel turns cu_seqlens into a tile list (requests longest
// first, then head, then query block, so that the CTAs running at the same
// time read the same head's K/V from L2) and resets a claim counter; a
// persistent kernel with one CTA per SM claims tiles from that list in
// order with an atomic on the counter (each CTA's producer claims its next
// tile when it is ready to load it and hands the index to the block's other
// roles through shared memory), so a CTA that runs faster simply takes more
// tiles. Each tile has exactly one owner and writes only its own rows, so the
// result does not depend on which CTA computed what.
//
// CTA roles (320 threads):
//   warps 0-3  softmax for Q0; thread r owns query row r (tensor-memory lane r)
//   warps 4-7  softmax for Q1
//   warp  8    TMA producer: Q tiles, then K_j, V_j into a ring of stages
//   warp  9    tensor-memory allocator and single-thread MMA issuer
// Tensor memory (512 columns x 128 lanes x 32 bit):
//   [0,128) S0 = Q0 K^T (fp32), [128,256) S1; P_i (bf16 pairs) overwrites the
//   first 64 columns of S_i once the softmax has read S_i; [256,256+D) O0,
//   [256+D,256+2D) O1 (fp32 accumulators).
// MMA issue order per K/V tile j: O0 += P0 V_j, S0 = Q0 K_{j+1}^T,
// O1 += P1 V_j, S1 = Q1 K_{j+1}^T, so each softmax group works on its S
// while the tensor core runs the other group's two products. MMAs from one
// thread execute in issue order, which makes the S_i write after P_i's read
// safe; every other hand-off goes through an mbarrier:
//   kv_full/kv_empty (TMA <-> MMA, per stage), q_full/q_empty,
//   s_full[i] (MMA -> softmax i: S_i ready, and all earlier products of
//   this thread complete), p_full[i] (softmax i -> MMA: P_i in tensor
//   memory, O_i rescaled), o_done[i] (MMA -> softmax i: last product of
//   the work tile complete).
// Online softmax in the log2 domain with lazy rescaling: the running row
// maximum is only raised (and O, l rescaled) when the tile maximum exceeds
// it by more than 2^8, which keeps every probability <= 256 and makes
// rescales rare after the first tiles.
// Every wait is bounded (pqk::mbar_wait, the caller's timeout); a wait that
// runs out raises the block's abort flag and the device status word, and
// every role stops issuing work. Once all roles have stopped (a block
// barrier), the producer waits for every copy it issued that no one consumed
// and the MMA thread for every MMA it issued (a commit on a barrier used only
// for that), both bounded by kDrainTimeoutNs rather than the caller's
// timeout; only then is the tensor memory freed and the block exits.
//
// CTA pairs (kPair; bf16, head_dim 128, no block skipping): two CTAs of a
// cluster share one work tile of 512 query rows, 256 per CTA as above, and
// one thread of the first CTA (the leader) issues every MMA of the pair with
// tcgen05 cta_group::2, M = 256: S_i = Q_i K^T over both CTAs' 128-row Q_i
// with each CTA holding 64 of K_j's 128 keys, and O_i += P_i V_j with P_i in
// each CTA's tensor memory and each CTA holding 64 of V_j's columns. Each SM
// thus streams half of every K/V tile (16 KB stages, ten of them) and reads
// 96 instead of 128 bytes of operands from shared memory per cycle of a
// Q K^T product, whose one-CTA form is bound by that bandwidth. The leader
// claims the tiles, posts the bytes of both CTAs' copies on its own
// barriers before it hands each tile and stage to the second CTA's
// producer, and commits "S ready" and "O done" to both CTAs' barriers; the
// second CTA's softmax warps report "P ready" with one remote arrive per
// warp. On a timeout both CTAs' abort flags are raised; after a cluster
// barrier the leader drains the copies and MMAs of the pair and a second
// cluster barrier keeps the second CTA, whose copies signal the leader's
// barriers, resident until then.
//
// Cross-attention (kCross; bf16): the queries attend to another packed
// sequence. A work unit has its own key range and key head; what else differs:
//   - the query heads that share a key head share a unit: a query tile is
//     128 / p.pack tokens x p.pack heads, so that K and V are read once for
//     all of them (one box of the Q map; p.pack is 1 without shared heads);
//   - a unit without rows for the second query tile leaves it out, so that a
//     few queries cost one product a key tile instead of two;
//   - where there are fewer tiles than SMs, the keys of a tile are cut into
//     parts, each a unit of its own that leaves its normalised fp32 rows and
//     their log-sum-exp in the workspace for combine_parts_kernel; in a part
//     of a tile without second query tile the two softmax groups take turns
//     on the key tiles (each with its own S, O and running maximum) and leave
//     two such rows;
//   - V rows past a unit's last key are set to zero in shared memory before
//     their product: they belong to another request, or to nobody, and a NaN
//     or infinity there would survive the product with P = 0;
//   - the producer claims and decodes the next unit while the current one
//     runs and hands the decoded unit to the other roles;
//   - output rows go through shared memory, a warp's 32 rows x 128 bytes at a
//     time, so that a store instruction covers 4 whole 128-byte lines instead
//     of 16 bytes of 32 lines. With four key tiles a unit (512 text keys) the
//     scattered stores took 220 of 790 us (55,296 queries x 512 keys, 40
//     heads); with the 454 of a long self-attention they do not show.
//
// Compile-time variants of the same pipeline:
//   kSkip  block skipping ("Skip-Softmax", first page, bullet on TRTLLM_ATTN
//          SAGE and Skip-Softmax): a softmax warp whose 32 rows all have the
//          tile maximum more than skip_tau below their earlier maximum writes
//          P = 0 and skips its exponentials; the MMA thread leaves out
//          O_i += P_i V_j when all four warps of the group voted so;
//   kFp8   Q and K as e4m3 bytes (SAGE FP8): S_i = Q_i K^T from 16 KB tiles
//          with kind::f8f6f4 MMAs, the heads' dequantisation factors folded
//          into the softmax scale;
//   kFp8Pv V as e4m3 bytes too and P rounded to e4m3 in tensor memory, so
//          that O_i += P_i V_j runs on the FP8 tensor cores as well; it
//          combines with kSkip (SAGE FP8 with Skip-Softmax).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "pqk_internal.h"

namespace pqk {
namespace {

constexpr int kBM = 128;          // query rows per Q tile
constexpr int kBN = 128;          // keys per K/V tile
constexpr int kRowsPerWork = 2 * kBM;      // one CTA: two 128-row query tiles
constexpr int kRowsPerPairWork = 4 * kBM;  // a CTA pair: two tiles in each CTA
constexpr int kThreads = 320;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
// The running row maximum only moves when a tile's maximum exceeds it by
// more than this (log2 units), so probabilities stay <= 2^threshold.
#ifndef PQK_ATTN_RESCALE_LOG2
#define PQK_ATTN_RESCALE_LOG2 8.0f
#endif
constexpr float kRescaleThreshold = PQK_ATTN_RESCALE_LOG2;
// Softmax arithmetic on packed fp32 pairs (fma/add .f32x2) and three-input
// max, halving the non-SFU instructions per score.
#ifndef PQK_ATTN_PACKED
#define PQK_ATTN_PACKED 1
#endif
constexpr bool kPacked = PQK_ATTN_PACKED != 0;
constexpr int kSlabBytes = 128 * 128;      // 128 rows x 64 bf16 (one 128-byte swizzle width)
// Ring of claimed work-tile indices in shared memory. The producer claims
// tile wt + 1 only once the Q K^T products of tile wt are complete, and the
// MMA thread starts tile wt + 1 only after the softmax warps have handed over
// the last P of tile wt, so the producer is at most two tiles ahead of the
// softmax warps: at most three slots are live. Cross-attention may issue the
// next unit's first S0 before the last P1 of the current one, so there the
// producer can be three units ahead of the second softmax group: all four.
constexpr int kWorkSlots = 4;

template <int D, bool kPair = false, bool kCross = false>
struct Layout {
  static constexpr int kSlabs = D / 64;
  static constexpr int kTileBytes = kSlabs * kSlabBytes;  // a Q tile; a whole K or V tile
  // a K/V stage: a whole tile, or on a CTA pair this CTA's half (64 keys of
  // K; 64 of V's columns for all 128 keys)
  static constexpr int kStageBytes = kPair ? kTileBytes / 2 : kTileBytes;
  static constexpr int kStages = kCross ? (D == 128 ? 4 : 8) : ((kPair || D != 128) ? 10 : 5);
  static constexpr int kQOff = 0;
  static constexpr int kKVOff = 2 * kTileBytes;
  // cross-attention: 32 output rows x 128 bytes for each softmax warp
  static constexpr int kOutOff = kKVOff + kStages * kStageBytes;
  static constexpr int kBarOff = kOutOff + (kCross ? 8 * 32 * 128 : 0);
  // barriers: kv_full[S], kv_empty[S], q_full, q_empty, s_full[2], p_full[2], o_done[2], drain,
  // work_full[kWorkSlots], and for cross-attention q_full and q_empty of the second query tile
  static constexpr int kNumBars = 2 * kStages + 9 + kWorkSlots + (kCross ? 2 : 0);
  static constexpr int kTmemSlotOff = kBarOff + kNumBars * 8;
  static constexpr int kAbortOff = kTmemSlotOff + 4;
  // block-skip votes: one byte per softmax warp, [group][tile parity][warp]
  static constexpr int kVoteOff = kAbortOff + 4;
  // claimed work-tile indices, a ring of kWorkSlots (-1: no more work)
  static constexpr int kWorkOff = kVoteOff + 16;
  // (kCross: the decoded units instead, eight words each)
  static constexpr int kUnitOff = (kWorkOff + 15) / 16 * 16;
  // the producer's copy counts (K/V stages, Q pairs; kCross: K/V stages, first and second Q tiles), left for the
  // drain
  static constexpr int kLoadsOff = kCross ? kUnitOff + 32 * kWorkSlots : kWorkOff + 4 * kWorkSlots;
  static constexpr int kBytes = kLoadsOff + (kCross ? 12 : 8);
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base to 1024
  static constexpr uint32_t kTmemS0 = 0, kTmemS1 = 128, kTmemO0 = 256, kTmemO1 = 256 + D;
  static_assert(kAlloc <= 232448, "shared memory budget");
};

// Schedule in the workspace (int32): [0] number of work tiles, [1] number of
// requests B, [2] the claim counter (reset to 0 by the schedule kernel on
// every call), [3] query rows per work tile, then for the requests in schedule order r =
// 0..B-1: tile_start[B+1] (prefix of tiles), seg_start[B], seg_len[B].
constexpr int kSchedHeader = 4;
__host__ __device__ constexpr size_t sched_words(int B) {
  return kSchedHeader + (B + 1) + 2 * static_cast<size_t>(B);
}

struct AttnParams {
  __nv_bfloat16* o;
  float* lse;
  int64_t o_stride;
  int64_t T;
  int H;
  float scale_log2;
  const int32_t* sched;
  int* status;
  long long timeout_ns;
  float skip_tau;                        // block-skip threshold (log2 units), kSkip only
  const float* deq;                      // kFp8: [2H] dequantisation factors of Q's, then K's heads
  unsigned long long* skip_counts;       // nullable: [0] skipped warp blocks, [1] skipped O += P V products
  int pack;                              // kCross: query heads per unit
  uint32_t pack_mul;                     // kCross: floor(2^16 / pack) + 1
  int group;                             // kCross: query heads per key head
  float* part_o;                         // kCross: [slots][kRowsPerWork][D] rows of cut tiles, and their
  float* part_lse;                       // [slots][kRowsPerWork] log2-sum-exps
};

struct Work {
  int seg_start;
  int seg_len;
  int head;
  int q0;      // first query row of the work tile
  int n_kv;    // number of K/V tiles
};

__device__ __forceinline__ Work decode_work(const int32_t* sched, int H, int w) {
  const int B = sched[1];
  const int32_t* tile_start = sched + kSchedHeader;
  const int32_t* seg_start = tile_start + B + 1;
  const int32_t* seg_len = seg_start + B;
  int lo = 0, hi = B - 1;  // last r with tile_start[r] <= w
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= w) lo = mid; else hi = mid - 1;
  }
  Work wk;
  wk.seg_start = seg_start[lo];
  wk.seg_len = seg_len[lo];
  const int rows_per_work = sched[3];
  const int nqb = (wk.seg_len + rows_per_work - 1) / rows_per_work;
  const int local = w - tile_start[lo];
  wk.head = local / nqb;
  wk.q0 = wk.seg_start + (local % nqb) * rows_per_work;
  wk.n_kv = (wk.seg_len + kBN - 1) / kBN;
  (void)H;
  return wk;
}

// Cross-attention: a unit's queries and keys. slot < 0: the unit holds all keys of its tile and writes the
// outputs itself.
struct CrossWork {
  int head;     // first of its p.pack query heads; -1: no more work
  int q0;
  int q_end;    // one past the request's last query
  int k_start;  // first key of the unit
  int k_len;    // its keys (at least one)
  int n_kv;
  int slot;
};

// Schedule of a cross-attention call (int32): [0] units, [1] B, [2] the claim
// counter, [3] tiles (2 * (128 / pack) queries x pack heads, requests with
// keys), [4] the same of requests without keys, [5] key tiles per part (0: no tile is cut);
// then, requests in schedule order, prefixes [B+1] of units, tiles and keyless
// tiles, and q_start, q_len, k_start, k_len [B] each.
constexpr int kCrossHeader = 8;
__host__ __device__ constexpr size_t cross_sched_words(int B) {
  return kCrossHeader + 3 * (static_cast<size_t>(B) + 1) + 4 * static_cast<size_t>(B);
}
struct CrossSched {
  int32_t *unit_start, *tile_start, *empty_start, *q_start, *q_len, *k_start, *k_len;
  __device__ __forceinline__ CrossSched(const int32_t* sched, int B) {
    unit_start = const_cast<int32_t*>(sched) + kCrossHeader;
    tile_start = unit_start + B + 1;
    empty_start = tile_start + B + 1;
    q_start = empty_start + B + 1;
    q_len = q_start + B;
    k_start = q_len + B;
    k_len = k_start + B;
  }
};
__device__ __forceinline__ int cross_parts(int n_kv, int part_tiles) {
  return part_tiles == 0 ? 1 : (n_kv + part_tiles - 1) / part_tiles;
}
// The last r < B with start[r] <= i.
__device__ __forceinline__ int find_last(const int32_t* start, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// tile_tokens: queries of a whole tile (both query tiles).
__device__ __forceinline__ CrossWork decode_cross(const int32_t* sched, int pack, int tile_tokens, int w) {
  const int B = sched[1];
  const CrossSched cs(sched, B);
  const int r = find_last(cs.unit_start, B, w);
  const int local = w - cs.unit_start[r];
  const int q_len = cs.q_len[r], k_len = cs.k_len[r];
  const int all_kv = (k_len + kBN - 1) / kBN;
  const int parts = cross_parts(all_kv, sched[5]);
  const int part = local % parts;
  const int tile = local / parts;
  const int nqb = (q_len + tile_tokens - 1) / tile_tokens;
  CrossWork wk;
  wk.head = tile / nqb * pack;
  wk.q0 = cs.q_start[r] + (tile % nqb) * tile_tokens;
  wk.q_end = cs.q_start[r] + q_len;
  // parts of equal size to one key tile
  const int first = parts == 1 ? 0 : static_cast<int>(static_cast<int64_t>(all_kv) * part / parts);
  const int last = parts == 1 ? all_kv : static_cast<int>(static_cast<int64_t>(all_kv) * (part + 1) / parts);
  wk.k_start = cs.k_start[r] + first * kBN;
  wk.k_len = (last < all_kv ? last * kBN : k_len) - first * kBN;
  wk.n_kv = last - first;
  wk.slot = parts > 1 ? w : -1;
  return wk;
}

// What the pipeline's roles ask of a unit of either kind.
__device__ __forceinline__ int key_count(const Work& wk) { return wk.seg_len; }
__device__ __forceinline__ int key_count(const CrossWork& wk) { return wk.k_len; }
__device__ __forceinline__ int end_of_queries(const Work& wk) { return wk.seg_start + wk.seg_len; }
__device__ __forceinline__ int end_of_queries(const CrossWork& wk) { return wk.q_end; }

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, int* status) {
  *abort_flag = 1;
  atomicCAS(status, 0, kStatusTimeout);
}

// Drain of an aborting block (after its final barrier). Kept out of line:
// inlined, the rarely run drain loops change the register allocation of the
// softmax loop.
// Producer: K/V copy idx was issued only after copy idx - n_stages had
// landed, so the last n_stages copies (and the last Q pair) are the ones
// that can be outstanding; each is the newest phase of its stage barrier
// (stage s at bar_kv_full + 8 s).
__device__ __noinline__ void drain_copies(uint32_t bar_kv_full, uint32_t bar_q_full, uint32_t n_stages,
                                          uint32_t load_idx, uint32_t q_loads) {
  const uint32_t first = load_idx > n_stages ? load_idx - n_stages : 0;
  for (uint32_t idx = first; idx < load_idx; ++idx)
    mbar_drain_wait(bar_kv_full + 8u * (idx % n_stages), (idx / n_stages) & 1);
  if (q_loads > 0) mbar_drain_wait(bar_q_full, (q_loads - 1) & 1);
}

// MMA thread: a commit on the (otherwise unused) drain barrier completes
// once every MMA this thread issued has, and with them the arrivals of their
// own commits.
__device__ __noinline__ void drain_mmas(uint32_t bar_drain) {
  tc_commit(bar_drain);
  mbar_drain_wait(bar_drain, 0);
}
__device__ __noinline__ void drain_mmas_pair(uint32_t bar_drain) {
  tc_commit_pair(bar_drain);
  mbar_drain_wait(bar_drain, 0);
}

// ------------------------------------------------------------ schedule

constexpr int kSchedThreads = 1024;
constexpr int kSortLimit = 8192;  // requests ordered longest first up to this B
// dynamic shared memory of the schedule kernel: one 64-bit sort key per request
constexpr int kSchedSmem = kSortLimit * 8;

// Fills sort_keys[0, B) with the requests of cu, longest first, ties by index
// (the request in each key's low word): a bitonic sort of the keys
// (INT32_MAX - length) << 32 | index over the next power of two, padded with
// keys above every real one. By the whole block.
template <int kThreadsN>
__device__ __forceinline__ void sort_longest_first(const int32_t* cu, int B, uint64_t* sort_keys) {
  int n = 1;
  while (n < B) n <<= 1;
  for (int i = threadIdx.x; i < n; i += kThreadsN)
    sort_keys[i] = i < B ? (static_cast<uint64_t>(static_cast<uint32_t>(INT32_MAX - (cu[i + 1] - cu[i]))) << 32) |
                               static_cast<uint32_t>(i)
                         : ~0ull;
  __syncthreads();
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < n; i += kThreadsN) {
        const int partner = i ^ j;
        if (partner > i) {
          const uint64_t a = sort_keys[i], b = sort_keys[partner];
          if ((a > b) == ((i & k) == 0)) {
            sort_keys[i] = b;
            sort_keys[partner] = a;
          }
        }
      }
      __syncthreads();
    }
  }
}

// out[i] = count(0) + ... + count(i - 1) for i < B; returns the total to every
// thread. One chunk of kThreadsN requests at a time (warp scans, then a
// scan of warp sums). By the whole block.
template <int kThreadsN, typename Count>
__device__ __forceinline__ int32_t exclusive_prefix(int B, int32_t* out, Count count) {
  __shared__ int32_t warp_sums[kThreadsN / 32];
  int32_t carry = 0;
  for (int base = 0; base < B; base += kThreadsN) {
    const int i = base + threadIdx.x;
    const int32_t n = i < B ? count(i) : 0;
    int32_t incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, incl, off);
      if ((threadIdx.x & 31) >= off) incl += y;
    }
    __syncthreads();  // the previous chunk's (or call's) sums have been read
    if ((threadIdx.x & 31) == 31) warp_sums[threadIdx.x >> 5] = incl;
    __syncthreads();
    int32_t before = carry, all = carry;
    for (int w = 0; w < kThreadsN / 32; ++w) {
      if (w < static_cast<int>(threadIdx.x >> 5)) before += warp_sums[w];
      all += warp_sums[w];
    }
    if (i < B) out[i] = before + incl - n;
    carry = all;
  }
  return carry;
}

__global__ void __launch_bounds__(kSchedThreads) build_schedule_kernel(const int32_t* cu, int B, int64_t T, int H,
                                                                        int rows_per_work, int32_t* sched,
                                                                        int* status) {
  extern __shared__ uint64_t sort_keys[];
  __shared__ int bad;
  if (threadIdx.x == 0) bad = (cu[0] != 0 || static_cast<int64_t>(cu[B]) != T) ? 1 : 0;
  __syncthreads();
  for (int i = threadIdx.x; i < B; i += kSchedThreads)
    if (cu[i + 1] < cu[i]) bad = 1;
  __syncthreads();
  int32_t* tile_start = sched + kSchedHeader;
  int32_t* seg_start = tile_start + B + 1;
  int32_t* seg_len = seg_start + B;
  if (bad) {
    if (threadIdx.x == 0) {
      sched[0] = 0;
      sched[1] = B;
      sched[2] = 0;
      sched[3] = rows_per_work;
      atomicCAS(status, 0, kStatusBadSeqlens);
    }
    return;
  }
  if (B <= kSortLimit) {
    sort_longest_first<kSchedThreads>(cu, B, sort_keys);
    for (int r = threadIdx.x; r < B; r += kSchedThreads) {
      const int i = static_cast<int>(sort_keys[r] & 0xffffffffu);
      seg_start[r] = cu[i];
      seg_len[r] = cu[i + 1] - cu[i];
    }
  } else {
    // the given order
    for (int i = threadIdx.x; i < B; i += kSchedThreads) {
      seg_start[i] = cu[i];
      seg_len[i] = cu[i + 1] - cu[i];
    }
  }
  __syncthreads();
  const int32_t total = exclusive_prefix<kSchedThreads>(
      B, tile_start, [&](int i) { return ((seg_len[i] + rows_per_work - 1) / rows_per_work) * H; });
  if (threadIdx.x == 0) {
    tile_start[B] = total;
    sched[0] = total;
    sched[1] = B;
    sched[2] = 0;  // claim counter
    sched[3] = rows_per_work;
  }
}

// Tiles are cut along their keys when there are fewer of them than this (one
// B200's SMs; a constant, since the workspace's size is given by B and D alone
// and holds a slot for each part): into parts of at most as many key tiles as
// make the units no more than that, but kMinPartTiles at least (a part costs its
// rows' way through the workspace).
constexpr int kCutUnits = 148;
constexpr int kMinPartTiles = 4;

__global__ void __launch_bounds__(kSchedThreads)
    build_cross_schedule_kernel(const int32_t* cu_q, const int32_t* cu_k, int B, int64_t Tq, int64_t Tk,
                                int head_blocks, int tile_tokens, int32_t* sched, int* status) {
  launch_dependents();
  extern __shared__ uint64_t sort_keys[];
  __shared__ int bad;
  __shared__ unsigned long long key_tiles;  // of all tiles together
  __shared__ int most_tiles, count;
  if (threadIdx.x == 0) {
    bad = (cu_q[0] != 0 || cu_k[0] != 0 || static_cast<int64_t>(cu_q[B]) > Tq || static_cast<int64_t>(cu_k[B]) > Tk)
              ? 1 : 0;
    key_tiles = 0;
    most_tiles = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < B; i += kSchedThreads)
    if (cu_q[i + 1] < cu_q[i] || cu_k[i + 1] < cu_k[i]) bad = 1;
  __syncthreads();
  if (bad) {
    if (threadIdx.x < kCrossHeader) sched[threadIdx.x] = threadIdx.x == 1 ? B : 0;
    if (threadIdx.x == 0) atomicCAS(status, 0, kStatusBadSeqlens);
    return;
  }
  const CrossSched cs(sched, B);
  const bool sorted = B <= kSortLimit;
  if (sorted) sort_longest_first<kSchedThreads>(cu_k, B, sort_keys);
  for (int r = threadIdx.x; r < B; r += kSchedThreads) {
    const int i = sorted ? static_cast<int>(sort_keys[r] & 0xffffffffu) : r;
    cs.q_start[r] = cu_q[i];
    cs.q_len[r] = cu_q[i + 1] - cu_q[i];
    cs.k_start[r] = cu_k[i];
    cs.k_len[r] = cu_k[i + 1] - cu_k[i];
  }
  __syncthreads();
  auto tiles_of = [&](int r) { return (cs.q_len[r] + tile_tokens - 1) / tile_tokens * head_blocks; };
  auto key_tiles_of = [&](int r) { return (cs.k_len[r] + kBN - 1) / kBN; };
  const int32_t tiles = exclusive_prefix<kSchedThreads>(
      B, cs.tile_start, [&](int r) { return cs.k_len[r] > 0 ? tiles_of(r) : 0; });
  const int32_t empty = exclusive_prefix<kSchedThreads>(
      B, cs.empty_start, [&](int r) { return cs.k_len[r] > 0 ? 0 : tiles_of(r); });
  int part_tiles = 0;
  if (tiles < kCutUnits) {
    unsigned long long mine = 0;
    int most = 0;
    for (int r = threadIdx.x; r < B; r += kSchedThreads) {
      const int kt = cs.q_len[r] > 0 ? key_tiles_of(r) : 0;
      mine += static_cast<unsigned long long>(tiles_of(r)) * kt;
      most = max(most, kt);
    }
    if (mine != 0) atomicAdd(&key_tiles, mine);
    if (most != 0) atomicMax(&most_tiles, most);
    __syncthreads();
    // the least part size in [lo, hi] with at most kCutUnits units; hi cuts nothing
    int hi = max(most_tiles, kMinPartTiles);
    int lo = max(kMinPartTiles, static_cast<int>((key_tiles + kCutUnits - 1) / kCutUnits));
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      __syncthreads();
      if (threadIdx.x == 0) count = 0;
      __syncthreads();
      int n = 0;
      for (int r = threadIdx.x; r < B; r += kSchedThreads)
        if (cs.k_len[r] > 0) n += tiles_of(r) * cross_parts(key_tiles_of(r), mid);
      if (n != 0) atomicAdd(&count, n);
      __syncthreads();
      if (count <= kCutUnits) hi = mid; else lo = mid + 1;
    }
    part_tiles = hi;
  }
  const int32_t units = exclusive_prefix<kSchedThreads>(B, cs.unit_start, [&](int r) {
    return cs.k_len[r] > 0 ? tiles_of(r) * cross_parts(key_tiles_of(r), part_tiles) : 0;
  });
  if (threadIdx.x == 0) {
    cs.unit_start[B] = units;
    cs.tile_start[B] = tiles;
    cs.empty_start[B] = empty;
    sched[0] = units;
    sched[1] = B;
    sched[2] = 0;  // claim counter
    sched[3] = tiles;
    sched[4] = empty;
    sched[5] = part_tiles;
    sched[6] = sched[7] = 0;
  }
}

// The same for at most 32 requests by one warp, a request a lane, without
// barriers or a way through memory (3 requests: 3 us where the block above
// takes 14).
constexpr int kWarpRequests = 32;
__global__ void __launch_bounds__(32)
    build_cross_schedule_warp_kernel(const int32_t* cu_q, const int32_t* cu_k, int B, int64_t Tq, int64_t Tk,
                                     int head_blocks, int tile_tokens, int32_t* sched, int* status) {
  launch_dependents();
  constexpr unsigned kAll = 0xffffffffu;
  __shared__ int4 sorted[kWarpRequests];
  const int lane = threadIdx.x;
  const int at = min(lane, B);
  const int q0 = cu_q[at], k0 = cu_k[at], q1 = cu_q[min(lane + 1, B)], k1 = cu_k[min(lane + 1, B)];
  const bool bad = q1 < q0 || k1 < k0 || (lane == 0 && (q0 != 0 || k0 != 0)) ||
                   static_cast<int64_t>(q1) > Tq || static_cast<int64_t>(k1) > Tk;
  if (__any_sync(kAll, bad)) {
    if (lane < kCrossHeader) sched[lane] = lane == 1 ? B : 0;
    if (lane == 0) atomicCAS(status, 0, kStatusBadSeqlens);
    return;
  }
  // longest keys first, ties by index; lanes past B hold requests of nothing
  int rank = 0;
  for (int i = 0; i < kWarpRequests; ++i) {
    const int other = __shfl_sync(kAll, k1 - k0, i);
    rank += other > k1 - k0 || (other == k1 - k0 && i < lane);
  }
  sorted[rank] = make_int4(q0, q1 - q0, k0, k1 - k0);
  __syncwarp();
  const int4 mine = sorted[lane];
  const int all_tiles = (mine.y + tile_tokens - 1) / tile_tokens * head_blocks;
  const int my_tiles = mine.w > 0 ? all_tiles : 0;
  const int key_tiles = (mine.w + kBN - 1) / kBN;
  // inclusive prefix over the lanes
  auto scan = [&](int v) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kAll, v, off);
      if (lane >= off) v += y;
    }
    return v;
  };
  const int tiles_incl = scan(my_tiles), empty_incl = scan(all_tiles - my_tiles);
  const int tiles = __shfl_sync(kAll, tiles_incl, 31), empty = __shfl_sync(kAll, empty_incl, 31);
  int part_tiles = 0;
  if (tiles < kCutUnits) {
    unsigned long long total = static_cast<unsigned long long>(my_tiles) * key_tiles;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) total += __shfl_xor_sync(kAll, total, off);
    int hi = max(__reduce_max_sync(kAll, my_tiles > 0 ? key_tiles : 0), kMinPartTiles);
    int lo = max(kMinPartTiles, static_cast<int>((total + kCutUnits - 1) / kCutUnits));
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__reduce_add_sync(kAll, my_tiles * cross_parts(key_tiles, mid)) <= kCutUnits) hi = mid; else lo = mid + 1;
    }
    part_tiles = hi;
  }
  const int my_units = my_tiles * cross_parts(key_tiles, part_tiles);
  const int units_incl = scan(my_units);
  const CrossSched cs(sched, B);
  if (lane < B) {
    cs.unit_start[lane] = units_incl - my_units;
    cs.tile_start[lane] = tiles_incl - my_tiles;
    cs.empty_start[lane] = empty_incl - (all_tiles - my_tiles);
    cs.q_start[lane] = mine.x;
    cs.q_len[lane] = mine.y;
    cs.k_start[lane] = mine.z;
    cs.k_len[lane] = mine.w;
  }
  if (lane == 31) {
    cs.unit_start[B] = units_incl;
    cs.tile_start[B] = tiles;
    cs.empty_start[B] = empty;
    sched[0] = units_incl;
    sched[1] = B;
    sched[2] = 0;  // claim counter
    sched[3] = tiles;
    sched[4] = empty;
    sched[5] = part_tiles;
    sched[6] = sched[7] = 0;
  }
}

// The rows of cut tiles from their parts' rows o_i and log2-sum-exps u_i:
// O = sum_i 2^(u_i - u) o_i / sum_i 2^(u_i - u) with u the largest u_i, and
// lse = (u + log2 of that sum) ln 2. Block (x, y) takes tile x's rows from 8 y
// on, a warp a row, the parts in order.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
constexpr int kCombineThreads = 256;
template <int D>
__global__ void __launch_bounds__(kCombineThreads)
    combine_parts_kernel(const int32_t* sched, const float* part_o, const float* part_lse, __nv_bfloat16* o,
                         float* lse, int64_t o_stride, int64_t Tq, int pack) {
  const int B = sched[1], tiles = sched[3], part_tiles = sched[5];
  const int tile = blockIdx.x;
  if (part_tiles == 0 || tile >= tiles) return;
  const CrossSched cs(sched, B);
  const int r = find_last(cs.tile_start, B, tile);
  const int parts = cross_parts((cs.k_len[r] + kBN - 1) / kBN, part_tiles);
  if (parts == 1) return;
  const int tokens = kBM / pack;  // queries of one query tile
  const int q_len = cs.q_len[r];
  const int nqb = (q_len + 2 * tokens - 1) / (2 * tokens);
  const int local = tile - cs.tile_start[r];
  const int q_tile0 = (local % nqb) * 2 * tokens;
  const int in_tile = min(2 * tokens, q_len - q_tile0);  // the tile's queries
  // rows of one query tile only: both softmax groups left some, 128 rows apart
  const bool one = in_tile <= tokens;
  const int n = one ? 2 * parts : parts;
  const int64_t step = one ? kBM : kRowsPerWork;
  const int64_t slot_row = (cs.unit_start[r] + static_cast<int64_t>(local) * parts) * kRowsPerWork;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.y * (kCombineThreads / 32) + (threadIdx.x >> 5);
  if (i < in_tile * pack) {
    const int token = i / pack;
    const int64_t row0 = slot_row + (token < tokens ? i : kBM + i - tokens * pack);
    const float* u = part_lse + row0;
    const float* src = part_o + row0 * D + lane * (D / 32);
    float top = -INFINITY;
    for (int k = lane; k < n; k += 32) top = max_or_nan(top, u[k * step]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    float sum = 0.f, acc[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
      // one part's weight a lane, then the parts in order, 16 rows in flight
      const float mine = k0 + lane < n ? ex2_approx(u[(k0 + lane) * step] - top) : 0.f;
      const int m = min(32, n - k0);
#pragma unroll 16
      for (int k = 0; k < m; ++k) {
        const float weight = __shfl_sync(0xffffffffu, mine, k);
        sum += weight;
        const float2* v = reinterpret_cast<const float2*>(src + (k0 + k) * step * D);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          const float2 x = v[e];
          acc[2 * e] = fmaf(weight, x.x, acc[2 * e]);
          acc[2 * e + 1] = fmaf(weight, x.y, acc[2 * e + 1]);
        }
      }
    }
    const float inv = 1.0f / sum;
    const int64_t t = cs.q_start[r] + q_tile0 + token;
    const int head = local / nqb * pack + i - token * pack;
    uint32_t* dst = reinterpret_cast<uint32_t*>(o + t * o_stride + head * D + lane * (D / 32));
#pragma unroll
    for (int e = 0; e < D / 64; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lse != nullptr && lane == 0)
      lse[static_cast<int64_t>(head) * Tq + t] =
          top == -INFINITY ? top : (top + __log2f(sum)) * 0.69314718055994530942f;  // no part has a finite score
  }
}

// ------------------------------------------------------------ attention

// The 128 fp32 scores of this thread's row from tensor memory; columns at
// or past `valid` become -inf.
__device__ __forceinline__ void load_scores(uint32_t taddr, int valid, float (&s)[128]) {
  uint32_t r[128];
  tmem_ld_x128(taddr, r);
#pragma unroll
  for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(r[c]);
  if (valid < kBN) {
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (c >= valid) s[c] = -INFINITY;
  }
}

__device__ __forceinline__ float row_max(const float (&s)[128]) {
  if constexpr (kPacked) {
    // eight independent chains of three-input maxima (two new columns each),
    // then a three-level tree
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaxf(s[i], s[i + 8]);
#pragma unroll
    for (int c = 16; c < 128; c += 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = max3(m[i], s[c + i], s[c + 8 + i]);
    }
    return fmaxf(max3(m[0], m[1], m[2]), max3(m[3], m[4], fmaxf(m[5], fmaxf(m[6], m[7]))));
  } else {
    float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
    for (int c = 4; c < 128; c += 4) {
      m0 = fmaxf(m0, s[c]);
      m1 = fmaxf(m1, s[c + 1]);
      m2 = fmaxf(m2, s[c + 2]);
      m3 = fmaxf(m3, s[c + 3]);
    }
    return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
  }
}

// Exponentials of 4 consecutive columns starting at c (a multiple of 4).
__device__ __forceinline__ void exp4(const float (&s)[128], int c, float scale_log2, float neg_m, float (&e)[4]) {
  float x0, x1, x2, x3;
  if constexpr (kPacked) {
    fma2_bcast(s[c], s[c + 1], scale_log2, neg_m, x0, x1);
    fma2_bcast(s[c + 2], s[c + 3], scale_log2, neg_m, x2, x3);
  } else {
    x0 = fmaf(s[c], scale_log2, neg_m);
    x1 = fmaf(s[c + 1], scale_log2, neg_m);
    x2 = fmaf(s[c + 2], scale_log2, neg_m);
    x3 = fmaf(s[c + 3], scale_log2, neg_m);
  }
  e[0] = ex2_approx(x0);
  e[1] = ex2_approx(x1);
  e[2] = ex2_approx(x2);
  e[3] = ex2_approx(x3);
}

// p_c = 2^(s_c * scale_log2 - m) for the 128 columns, rounded to bf16 pairs
// and written over the first 64 columns of S at `t_p` (tensor memory), or,
// with kE4m3P, rounded to e4m3 (four per column) over the first 32; returns
// their unrounded fp32 sum. Waits for its tensor-memory stores before
// returning. bf16 is V's type, and kind::f16 takes both operands of P V in one
// type; tf32 would keep more of P at half the MMA rate and twice P's columns.
// A probability is off by at most half a step, 2^-8 of itself, so O moves by at
// most that share of sum p |v|; measured on cross-attention, the output's
// relative distance from the 64-bit definition is 0.0020-0.0023 instead of the
// 0.0017 of rounding O alone.
template <bool kE4m3P>
__device__ __forceinline__ float exp_tile_store(const float (&s)[128], float scale_log2, float neg_m, uint32_t t_p) {
  float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
  if constexpr (kE4m3P) {
    uint32_t pk[32];
#pragma unroll
    for (int c = 0; c < 128; c += 4) {
      float e[4];
      exp4(s, c, scale_log2, neg_m, e);
      add2_acc(l0, l1, e[0], e[1]);
      add2_acc(l2, l3, e[2], e[3]);
      pk[c / 4] = pack_e4m3x2(e[0], e[1]) | (pack_e4m3x2(e[2], e[3]) << 16);
    }
    tmem_st_x32(t_p, pk);
    return (l0 + l1) + (l2 + l3);
  }
  uint32_t pk[64];
#pragma unroll
  for (int c = 0; c < 128; c += 4) {
    float e[4];
    exp4(s, c, scale_log2, neg_m, e);
    if constexpr (kPacked) {
      add2_acc(l0, l1, e[0], e[1]);
      add2_acc(l2, l3, e[2], e[3]);
    } else {
      l0 += e[0];
      l1 += e[1];
      l2 += e[2];
      l3 += e[3];
    }
    pk[c / 2] = pack_bf16x2(e[0], e[1]);
    pk[c / 2 + 1] = pack_bf16x2(e[2], e[3]);
  }
  tmem_st_x64(t_p, pk);
  return (l0 + l1) + (l2 + l3);
}

template <int D, bool kSkip, bool kFp8, bool kFp8Pv, bool kPair = false, bool kCross = false>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const AttnParams p) {
  using L = Layout<D, kPair, kCross>;
  static_assert(!kFp8 || D == 128, "FP8 Q K^T: one 128-byte swizzle row per token");
  static_assert(!kFp8Pv || kFp8, "FP8 P V comes with FP8 Q K^T");
  static_assert(!kPair || (D == 128 && !kSkip && !kFp8), "CTA pairs: bf16, head_dim 128, no block skipping");
  static_assert(!kCross || (!kSkip && !kFp8 && !kPair), "cross-attention: bf16, one SM a unit, no block skipping");
  // FP8 Q K^T: the MMA thread waits for the next V stage (loaded long ago)
  // while it waits for P1 anyway, and probes the next K stage there without
  // blocking (its copy may still be in flight), instead of waiting for both
  // at the top of the next iteration, just before P0 (-3 % time with FP8;
  // +1 % with bf16 operands, where it is left out).
  constexpr bool kEarlyKv = kFp8;
  // bytes of one Q or K tile: bf16 slabs, or 128 rows x 128 e4m3 bytes
  constexpr uint32_t kQKBytes = kFp8 ? static_cast<uint32_t>(kBM) * 128u : static_cast<uint32_t>(L::kTileBytes);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // CTA pair: rank 0 (the leader) issues every MMA of the pair and owns the
  // barriers of the K/V and Q copies; each CTA keeps its own 256 query rows
  const uint32_t rank = kPair ? ctarank() : 0u;
  const bool leader = rank == 0;
  const uint32_t q_smem = base + L::kQOff;
  const uint32_t kv_smem = base + L::kKVOff;
  const uint32_t bar0 = base + L::kBarOff;
  auto kv_full = [&](int s) { return bar0 + 8u * s; };
  auto kv_empty = [&](int s) { return bar0 + 8u * (L::kStages + s); };
  const uint32_t q_full = bar0 + 8u * (2 * L::kStages);
  const uint32_t q_empty = q_full + 8;
  auto s_full = [&](int i) { return q_full + 16 + 8u * i; };
  auto p_full = [&](int i) { return q_full + 32 + 8u * i; };
  auto o_done = [&](int i) { return q_full + 48 + 8u * i; };
  const uint32_t drain = q_full + 64;
  auto work_full = [&](int i) { return q_full + 72 + 8u * i; };
  // kCross: the two query tiles come and go separately
  const uint32_t q1_full = q_full + 72 + 8u * kWorkSlots, q1_empty = q1_full + 8;
  volatile int* work_slot = reinterpret_cast<volatile int*>(smem + (kCross ? L::kUnitOff : L::kWorkOff));
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kTmemSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbortOff);
  volatile uint8_t* votes = smem + L::kVoteOff;
  // a wait that ran out stops this CTA's roles and, on a pair, the other CTA's
  auto abort_all = [&]() {
    raise_abort(abort_flag, p.status);
    if constexpr (kPair) st_remote_u32(in_cta(base + L::kAbortOff, rank ^ 1u), 1u);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    if constexpr (kCross) {
      mbar_init(q1_full, 1);
      mbar_init(q1_empty, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      // one arrival per softmax thread, or on a pair one per softmax warp of either CTA
      mbar_init(p_full(i), kPair ? 8 : kBM);
      mbar_init(o_done(i), 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kWorkSlots; ++i) mbar_init(work_full(i), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    if constexpr (kPair) {
      tmem_alloc_pair(base + L::kTmemSlotOff, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(base + L::kTmemSlotOff, 512);
      tmem_relinquish();
    }
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
  }
  tc_fence_before_sync();
  if constexpr (kPair) {
    __syncwarp();
    cluster_sync_all();  // both CTAs' barriers are initialised before any remote arrive
  } else {
    __syncthreads();
  }
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  if constexpr (kCross) wait_for_primary();  // the schedule
  const int n_work = p.sched[0];
  int* claim_counter = const_cast<int*>(p.sched + 2);
  // copies issued by the producer thread (K/V stages, Q tile pairs), kept in
  // shared memory for the drain so that no other thread holds them
  volatile uint32_t* loads_done = reinterpret_cast<volatile uint32_t*>(smem + L::kLoadsOff);
  // The index of this block's work tile wt, published by the producer in
  // slot wt % kWorkSlots (-1 once the list is exhausted); false when the
  // block aborts first.
  auto next_work = [&](int wt, int& w) {
    if (!mbar_wait(work_full(wt % kWorkSlots), (wt / kWorkSlots) & 1, abort_flag, p.timeout_ns)) return false;
    // on a pair's second CTA the slot was written by the leader's producer
    if (kPair && !leader) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    w = kCross ? work_slot[8 * (wt % kWorkSlots)] : work_slot[wt % kWorkSlots];
    return true;
  };
  // Work tile w in full; cross-attention takes the producer's decoded copy,
  // which stays in its slot until the unit kWorkSlots further on is handed over.
  auto decode = [&](int wt, int w) {
    if constexpr (kCross) {
      const volatile int* src = work_slot + 8 * (wt % kWorkSlots);
      CrossWork wk;
      wk.head = src[0];
      wk.q0 = src[1];
      wk.q_end = src[2];
      wk.k_start = src[3];
      wk.k_len = src[4];
      wk.n_kv = src[5];
      wk.slot = src[6];
      return wk;
    } else {
      return decode_work(p.sched, p.H, w);
    }
  };
  auto unit_word = [&](int wt, int i) -> int { return work_slot[8 * (wt % kWorkSlots) + i]; };
  // kCross: queries of one query tile; whether a unit has rows for the second
  const int tile_q = kCross ? kBM / p.pack : kBM;
  auto two_tiles = [&](const auto& wk) { return !kCross || wk.q0 + tile_q < end_of_queries(wk); };

  if (warp == kProducerWarp) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      if (kCross) loads_done[2] = 0;
      uint32_t load_idx = 0;
      uint32_t q_loads = 0;
      bool ok = true;
      if constexpr (kPair) {
        // The leader claims each work tile, posts the bytes of both CTAs'
        // copies on its own barriers and only then hands the tile, and each
        // K/V stage, to the second CTA's producer (so that no copy completes
        // before the count it belongs to). Both CTAs copy their own two Q
        // tiles, their 64 of each K tile's keys and their 64 of each V
        // tile's columns; every copy completes on the leader's barrier.
        const uint32_t q_bar = in_cta(q_full, 0);
        for (int wt = 0; ok; ++wt) {
          int w;
          if (leader) {
            if (wt > 0 && !(ok = mbar_wait(q_empty, (wt - 1) & 1, abort_flag, p.timeout_ns))) break;
            const int claimed = atomicAdd(claim_counter, 1);
            w = claimed < n_work ? claimed : -1;
            if (w >= 0) {
              mbar_arrive_expect_tx(q_full, 4 * kQKBytes);
              ++q_loads;
            }
            work_slot[wt % kWorkSlots] = w;
            mbar_arrive(work_full(wt % kWorkSlots));
            st_remote_u32(in_cta(base + L::kWorkOff + 4u * (wt % kWorkSlots), 1), static_cast<uint32_t>(w));
            arrive_remote_release(in_cta(work_full(wt % kWorkSlots), 1));
          } else if (!(ok = next_work(wt, w))) {
            break;
          }
          if (w < 0) break;
          const Work wk = decode_work(p.sched, p.H, w);
          const int qrow = wk.q0 + static_cast<int>(rank) * kRowsPerWork;
          for (int i = 0; i < 2; ++i)
            for (int sl = 0; sl < L::kSlabs; ++sl)
              tma_load_3d_pair(q_smem + i * L::kTileBytes + sl * kSlabBytes, &tm_q, q_bar, sl * 64, wk.head,
                               qrow + i * kBM);
          for (int j = 0; j < wk.n_kv && ok; ++j) {
            const int key0 = wk.seg_start + j * kBN;
            for (int kv = 0; kv < 2; ++kv) {
              const int s = load_idx % L::kStages;
              const uint32_t round = load_idx / L::kStages;
              if (leader) {
                if (round > 0 && !(ok = mbar_wait(kv_empty(s), (round - 1) & 1, abort_flag, p.timeout_ns))) break;
                mbar_arrive_expect_tx(kv_full(s), 2 * L::kStageBytes);
                arrive_remote(in_cta(kv_empty(s), 1));
              } else if (!(ok = mbar_wait(kv_empty(s), round & 1, abort_flag, p.timeout_ns))) {
                break;
              }
              const uint32_t dst = kv_smem + s * L::kStageBytes;
              const uint32_t bar = in_cta(kv_full(s), 0);
              if (kv == 0) {
                for (int sl = 0; sl < L::kSlabs; ++sl)
                  tma_load_3d_pair(dst + sl * (kSlabBytes / 2), &tm_k, bar, sl * 64, wk.head,
                                   key0 + static_cast<int>(rank) * (kBN / 2));
              } else {
                tma_load_3d_pair(dst, &tm_v, bar, static_cast<int>(rank) * 64, wk.head, key0);
              }
              ++load_idx;
            }
          }
        }
      } else if constexpr (kCross) {
        const uint32_t q_tile_bytes = static_cast<uint32_t>(L::kSlabs * 128 * tile_q * p.pack);
        auto claim = [&]() {
          const int w = atomicAdd(claim_counter, 1);
          CrossWork wk = {};
          wk.head = -1;
          return w < n_work ? decode_cross(p.sched, p.pack, 2 * tile_q, w) : wk;
        };
        auto load_q = [&](const CrossWork& wk, int i) {
          mbar_arrive_expect_tx(i == 0 ? q_full : q1_full, q_tile_bytes);
          for (int sl = 0; sl < L::kSlabs; ++sl)
            tma_load_3d(q_smem + i * L::kTileBytes + sl * kSlabBytes, &tm_q, i == 0 ? q_full : q1_full, sl * 64,
                        wk.head, wk.q0 + i * tile_q);
        };
        uint32_t q1_loads = 0;
        CrossWork wk = claim();
        for (int wt = 0;; ++wt) {
          // the first Q tile of the previous unit is no longer needed: hand over the next unit
          if (wt > 0 && !(ok = mbar_wait(q_empty, (wt - 1) & 1, abort_flag, p.timeout_ns))) break;
          volatile int* dst = work_slot + 8 * (wt % kWorkSlots);
          dst[0] = wk.head;
          dst[1] = wk.q0;
          dst[2] = wk.q_end;
          dst[3] = wk.k_start;
          dst[4] = wk.k_len;
          dst[5] = wk.n_kv;
          dst[6] = wk.slot;
          dst[7] = static_cast<int>(load_idx);  // index of the unit's first copy
          mbar_arrive(work_full(wt % kWorkSlots));
          if (wk.head < 0) break;
          load_q(wk, 0);
          ++q_loads;
          const int kv_head = wk.head / p.group;
          // Copy i of the unit is key tile i / 2's K (even i) or V. In a unit whose
          // groups take turns S runs two tiles ahead of P V, so the order there is
          // K_0, K_1, V_0, K_2, V_1, ..., V_{n-2}, V_{n-1}: that of their use (one
          // query x 55,296 keys x 40 heads: 264 us for K_0, V_0, K_1, ..., where
          // K_{j+2} could not be asked for before V_{j+1} had a stage; 183 us so,
          // 6.2 TB/s. Copying the tiles into L2 ahead as well is slower, 192).
          const bool turns = wk.slot >= 0 && !two_tiles(wk);
          auto key_tile_of = [&](int i, bool& is_v) {
            if (!turns) {
              is_v = (i & 1) != 0;
              return i >> 1;
            }
            const int t = (i - 2) >> 1;
            is_v = i >= 2 && ((i & 1) == 0 || t + 2 >= wk.n_kv);
            return i < 2 ? i : ((i & 1) == 0 ? t : (is_v ? t + 1 : t + 2));
          };
          for (int i = 0; i < 2 * wk.n_kv; ++i) {
            bool is_v;
            const int t = key_tile_of(i, is_v);
            const int s = load_idx % L::kStages;
            const uint32_t round = load_idx / L::kStages;
            if (round > 0 && !(ok = mbar_wait(kv_empty(s), (round - 1) & 1, abort_flag, p.timeout_ns))) break;
            mbar_arrive_expect_tx(kv_full(s), L::kTileBytes);
            for (int sl = 0; sl < L::kSlabs; ++sl)
              tma_load_3d(kv_smem + s * L::kStageBytes + sl * kSlabBytes, is_v ? &tm_v : &tm_k, kv_full(s), sl * 64,
                          kv_head, wk.k_start + t * kBN);
            ++load_idx;
            if (i == 0 && two_tiles(wk)) {
              // the second Q tile once the last unit that had one is through with it
              if (q1_loads > 0 && !(ok = mbar_wait(q1_empty, (q1_loads - 1) & 1, abort_flag, p.timeout_ns))) break;
              load_q(wk, 1);
              ++q1_loads;
            }
          }
          loads_done[2] = q1_loads;
          if (!ok) break;
          // while the unit's last key tiles are worked on: the next unit, and its queries into L2
          wk = claim();
          if (wk.head >= 0)
            for (int i = 0; i < (two_tiles(wk) ? 2 : 1); ++i)
              for (int sl = 0; sl < L::kSlabs; ++sl) tma_prefetch_3d(&tm_q, sl * 64, wk.head, wk.q0 + i * tile_q);
        }
      } else {
      for (int wt = 0; ok; ++wt) {
        // the Q tiles of the previous work tile are no longer needed: claim the next one
        if (wt > 0 && !(ok = mbar_wait(q_empty, (wt - 1) & 1, abort_flag, p.timeout_ns))) break;
        const int claimed = atomicAdd(claim_counter, 1);
        const int w = claimed < n_work ? claimed : -1;
        work_slot[wt % kWorkSlots] = w;
        mbar_arrive(work_full(wt % kWorkSlots));
        if (w < 0) break;
        const Work wk = decode_work(p.sched, p.H, w);
        mbar_arrive_expect_tx(q_full, 2 * kQKBytes);
        ++q_loads;
        for (int i = 0; i < 2; ++i) {
          if constexpr (kFp8) {
            tma_load_3d(q_smem + i * L::kTileBytes, &tm_q, q_full, 0, wk.head, wk.q0 + i * kBM);
          } else {
            for (int sl = 0; sl < L::kSlabs; ++sl)
              tma_load_3d(q_smem + i * L::kTileBytes + sl * kSlabBytes, &tm_q, q_full, sl * 64, wk.head,
                          wk.q0 + i * kBM);
          }
        }
        for (int j = 0; j < wk.n_kv && ok; ++j) {
          for (int kv = 0; kv < 2; ++kv) {
            const int s = load_idx % L::kStages;
            const uint32_t round = load_idx / L::kStages;
            if (round > 0 && !(ok = mbar_wait(kv_empty(s), (round - 1) & 1, abort_flag, p.timeout_ns))) break;
            if ((kFp8 && kv == 0) || (kFp8Pv && kv == 1)) {
              // one 128-byte e4m3 row per token: a single 16 KB box
              mbar_arrive_expect_tx(kv_full(s), kQKBytes);
              tma_load_3d(kv_smem + s * L::kStageBytes, kv == 0 ? &tm_k : &tm_v, kv_full(s), 0, wk.head,
                          wk.seg_start + j * kBN);
            } else {
              mbar_arrive_expect_tx(kv_full(s), L::kTileBytes);
              const CUtensorMap* tm = kv == 0 ? &tm_k : &tm_v;
              for (int sl = 0; sl < L::kSlabs; ++sl)
                tma_load_3d(kv_smem + s * L::kStageBytes + sl * kSlabBytes, tm, kv_full(s), sl * 64, wk.head,
                            wk.seg_start + j * kBN);
            }
            ++load_idx;
          }
        }
      }
      }
      if (!ok) abort_all();
      loads_done[0] = load_idx;
      loads_done[1] = q_loads;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issuer (the leader's, on a pair)
    if (lane == 0 && leader) {
      // a pair's products have M = 256: each CTA's 128 rows of Q_i, S_i, P_i, O_i
      constexpr int kM = kPair ? 2 * kBM : kBM;
      constexpr uint32_t kIdescQK = kFp8 ? idesc_e4m3_f32(kBM, kBN) : idesc_bf16_f32(kM, kBN, false);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kM, D, true);
      // completions: of this CTA's copies' consumers (stages, Q), or seen by
      // both CTAs' softmax warps (S ready, O done)
      auto commit_own = [&](uint32_t bar) {
        if constexpr (kPair) tc_commit_pair(bar); else tc_commit(bar);
      };
      auto commit_all = [&](uint32_t bar) {
        if constexpr (kPair) tc_commit_pair_both(bar); else tc_commit(bar);
      };
      constexpr uint32_t kIdescPV8 = idesc_e4m3_f32(kBM, D, true);
      uint32_t cons_idx = 0;
      uint32_t p_phase = 0;
      uint32_t p_phase1 = 0;  // kCross: the second query tile's, which units with one tile pass by
      unsigned long long pv_skips = 0;
      // every softmax warp of group i voted to skip K/V tile j
      auto group_skips = [&](int i, int j) {
        return *reinterpret_cast<volatile uint32_t*>(votes + (i * 2 + (j & 1)) * 4) == 0x01010101u;
      };
      // kCross: units with a second query tile so far (their second Q tiles' phase), and whether the unit's first
      // S0 = Q0 K_0^T is already issued
      uint32_t q1_phase = 0;
      bool s0_issued = false;
      int wt = 0;
      bool ok = true;
      // Descriptor low words of Q0 and of stage 0 (K: K-major, V: MN-major
      // with 64-wide column slabs kSlabBytes apart); one high word for all.
      constexpr uint32_t kDescHi = smem_desc_hi_sw128(1024);
      constexpr uint32_t kTileWords = L::kTileBytes >> 4;
      constexpr uint32_t kStageWords = L::kStageBytes >> 4;
      // a K stage's two 64-column slabs (on a pair 64 keys each)
      constexpr uint32_t kKSlabBytes = kPair ? kSlabBytes / 2 : kSlabBytes;
      const uint32_t q_lo = smem_desc_lo(q_smem, 16);
      const uint32_t k_lo = smem_desc_lo(kv_smem, 16);
      const uint32_t v_lo = smem_desc_lo(kv_smem, kSlabBytes);
      // S_i = Q_i K^T over D/16 K-steps of 16 (32 bytes inside the 128-byte row)
      auto issue_qk_of = [&](int i, int q_tile, int stage) {
        const uint32_t a0 = q_lo + q_tile * kTileWords;
        const uint32_t b0 = k_lo + stage * kStageWords;
        if constexpr (kFp8) {
          // e4m3: K = 32 per instruction, 32 bytes inside the one 128-byte row
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8_ss_w(tmem + (i == 0 ? L::kTmemS0 : L::kTmemS1), a0 + 2 * k, b0 + 2 * k, kDescHi, kIdescQK,
                        k > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off_a = ((k / 4) * kSlabBytes + (k % 4) * 32) >> 4;
            const uint32_t off_b = ((k / 4) * kKSlabBytes + (k % 4) * 32) >> 4;
            if constexpr (kPair)
              mma_bf16_ss_pair(tmem + (i == 0 ? L::kTmemS0 : L::kTmemS1), a0 + off_a, b0 + off_b, kDescHi, kIdescQK,
                               k > 0 ? 1u : 0u);
            else
              mma_bf16_ss_w(tmem + (i == 0 ? L::kTmemS0 : L::kTmemS1), a0 + off_a, b0 + off_b, kDescHi, kIdescQK,
                            k > 0 ? 1u : 0u);
          }
        }
      };
      auto issue_qk = [&](int i, int stage) { issue_qk_of(i, i, stage); };
      // O_i (+)= P_i V over kBN/16 K-steps; V is MN-major: 64-wide column
      // slabs kSlabBytes apart, 8-row groups 1024 bytes apart
      auto issue_pv = [&](int i, int stage, bool accumulate) {
        const uint32_t b0 = v_lo + stage * kStageWords;
        const uint32_t p_col = tmem + (i == 0 ? L::kTmemS0 : L::kTmemS1);
        if constexpr (kFp8Pv) {
          // e4m3 P (four keys per column, 8 columns per K = 32 step) and V as
          // 128-byte rows: MN-major, one swizzle atom wide, 32 keys = 4096 bytes
#pragma unroll
          for (int k = 0; k < kBN / 32; ++k)
            mma_f8_ts_w(tmem + (i == 0 ? L::kTmemO0 : L::kTmemO1), p_col + 8 * k, b0 + ((k * 4096) >> 4), kDescHi,
                        kIdescPV8, (accumulate || k > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int k = 0; k < kBN / 16; ++k) {
            if constexpr (kPair)
              mma_bf16_ts_pair(tmem + (i == 0 ? L::kTmemO0 : L::kTmemO1), p_col + 8 * k, b0 + ((k * 2048) >> 4),
                               kDescHi, kIdescPV, (accumulate || k > 0) ? 1u : 0u);
            else
              mma_bf16_ts_w(tmem + (i == 0 ? L::kTmemO0 : L::kTmemO1), p_col + 8 * k, b0 + ((k * 2048) >> 4),
                            kDescHi, kIdescPV, (accumulate || k > 0) ? 1u : 0u);
          }
        }
      };
      auto wait_stage = [&](uint32_t idx) {
        return mbar_wait(kv_full(idx % L::kStages), (idx / L::kStages) & 1, abort_flag, p.timeout_ns);
      };
      for (;; ++wt) {
        int w;
        if (!(ok = next_work(wt, w)) || w < 0) break;
        const auto wk = decode(wt, w);
        const bool q1_in_request = wk.q0 + kBM < end_of_queries(wk);
        const bool two = two_tiles(wk);
        if constexpr (kCross) {
          // A unit without a second query tile: that group's softmax warps
          // arrive once when they have seen it, so that they cannot fall
          // behind the ring of claimed units. Waited for before the unit's
          // first product, so before the producer may claim the next unit:
          // the group cannot arrive for that one before this wait is over.
          if (!two && wk.slot < 0) {
            if (!(ok = mbar_wait(p_full(1), p_phase1, abort_flag, p.timeout_ns))) break;
            p_phase1 ^= 1u;
          }
          // A part of a tile without second query tile: the groups take turns,
          // group j % 2 on key tile j (there are at least two). Copies come in
          // the order of their use, so a product waits for none but its own.
          if (!two && wk.slot >= 0) {
            if (!(ok = mbar_wait(q_full, wt & 1, abort_flag, p.timeout_ns))) break;
            for (int j = 0; j < 2 && ok; ++j) {
              const uint32_t k_idx = cons_idx + j;
              if (!(ok = wait_stage(k_idx))) break;
              tc_fence_after_sync();
              issue_qk_of(j, 0, k_idx % L::kStages);
              commit_all(s_full(j));
              commit_own(kv_empty(k_idx % L::kStages));
            }
            if (!ok) break;
            if (wk.n_kv == 2) commit_own(q_empty);
            for (int j = 0; j < wk.n_kv; ++j) {
              const int g = j & 1;
              const bool more = j + 2 < wk.n_kv;
              const uint32_t v_idx = cons_idx + (j + 1 < wk.n_kv ? 2 * j + 2 : 2 * j + 1);
              if (!(ok = wait_stage(v_idx))) break;
              if (!(ok = mbar_wait(p_full(g), g == 0 ? p_phase : p_phase1, abort_flag, p.timeout_ns))) break;
              if (g == 0) p_phase ^= 1u; else p_phase1 ^= 1u;
              tc_fence_after_sync();
              issue_pv(g, v_idx % L::kStages, j >= 2);
              commit_own(kv_empty(v_idx % L::kStages));
              if (more) {
                const uint32_t nk_idx = cons_idx + 2 * j + 3;
                if (!(ok = wait_stage(nk_idx))) break;
                tc_fence_after_sync();
                issue_qk_of(g, 0, nk_idx % L::kStages);
                commit_all(s_full(g));
                commit_own(kv_empty(nk_idx % L::kStages));
                if (j + 3 == wk.n_kv) commit_own(q_empty);
              } else {
                commit_all(o_done(g));
              }
            }
            if (!ok) break;
            cons_idx += 2 * wk.n_kv;
            continue;
          }
        }
        uint32_t k_stage_idx = cons_idx;
        if (!s0_issued) {
          if (!(ok = mbar_wait(q_full, wt & 1, abort_flag, p.timeout_ns))) break;
          if (!(ok = wait_stage(k_stage_idx))) break;
          tc_fence_after_sync();
          issue_qk(0, k_stage_idx % L::kStages);
          commit_all(s_full(0));
          if (kCross && wk.n_kv == 1) commit_own(q_empty);
        }
        s0_issued = false;
        if (two) {
          if constexpr (kCross) {
            if (!(ok = mbar_wait(q1_full, q1_phase, abort_flag, p.timeout_ns))) break;
            q1_phase ^= 1u;
            tc_fence_after_sync();
          }
          issue_qk(1, k_stage_idx % L::kStages);
          commit_all(s_full(1));
        }
        commit_own(kv_empty(k_stage_idx % L::kStages));
        if (wk.n_kv == 1 && two) commit_own(kCross ? q1_empty : q_empty);
        ++cons_idx;
        // stages of iteration j: V_j and K_{j+1}
        uint32_t v_idx = cons_idx++;
        uint32_t nk_idx = wk.n_kv > 1 ? cons_idx++ : 0;
        bool v_ready = false, k_ready = false;
        for (int j = 0; j < wk.n_kv; ++j) {
          const bool more = j + 1 < wk.n_kv;
          // V_j and K_{j+1} are complete before P0 is waited for, so no copy
          // wait sits between O0 += P0 V_j and S0 = Q0 K_{j+1}^T
          if (!v_ready && !(ok = wait_stage(v_idx))) break;
          if (more && !k_ready && !(ok = wait_stage(nk_idx))) break;
          if (!(ok = mbar_wait(p_full(0), p_phase, abort_flag, p.timeout_ns))) break;
          tc_fence_after_sync();
          if (kSkip && j > 0 && group_skips(0, j)) {
            ++pv_skips;
          } else {
            issue_pv(0, v_idx % L::kStages, j > 0);
          }
          if (!more) commit_all(o_done(0));
          if (more) {
            issue_qk(0, nk_idx % L::kStages);
            commit_all(s_full(0));
            if (kCross && j + 2 == wk.n_kv) commit_own(q_empty);
          }
          uint32_t next_v = 0, next_nk = 0;
          if (more) {
            next_v = cons_idx++;
            next_nk = j + 2 < wk.n_kv ? cons_idx++ : 0;
          }
          v_ready = k_ready = false;
          if (kEarlyKv && more) {
            if (!(ok = wait_stage(next_v))) break;
            v_ready = true;
            k_ready = j + 2 < wk.n_kv &&
                      mbar_test_wait(kv_full(next_nk % L::kStages), (next_nk / L::kStages) & 1);
          }
          if constexpr (kCross) {
            if (!two) {
              commit_own(kv_empty(v_idx % L::kStages));
              if (more) {
                commit_own(kv_empty(nk_idx % L::kStages));
              }
              p_phase ^= 1u;
              v_idx = next_v;
              nk_idx = next_nk;
              continue;
            }
          }
          if constexpr (kCross) {
            // After the unit's last O0 += P0 V: the next unit's first
            // S0 = Q0 K_0^T as soon as its copies have landed, if that is
            // before P1 is ready, so that the first softmax group need not
            // wait for the second's. (Units without second query tile wait
            // for the second group's arrival first, above.)
            if (!more) {
              const uint64_t t0 = global_timer_ns();
              for (uint32_t polls = 1; !mbar_test_wait(p_full(1), p_phase1); ++polls) {
                if (!s0_issued && mbar_test_wait(work_full((wt + 1) % kWorkSlots), ((wt + 1) / kWorkSlots) & 1) &&
                    mbar_test_wait(q_full, (wt + 1) & 1) &&
                    mbar_test_wait(kv_full(cons_idx % L::kStages), (cons_idx / L::kStages) & 1)) {
                  const auto next = decode(wt + 1, 0);
                  if (two_tiles(next)) {
                    tc_fence_after_sync();
                    issue_qk(0, cons_idx % L::kStages);
                    commit_all(s_full(0));
                    if (next.n_kv == 1) commit_own(q_empty);
                    s0_issued = true;
                  }
                }
                if (*abort_flag || polls >= kMaxPolls ||
                    static_cast<long long>(global_timer_ns() - t0) > p.timeout_ns) {
                  ok = false;
                  break;
                }
              }
              if (!ok) break;
            }
          }
          if (!(ok = mbar_wait(p_full(1), kCross ? p_phase1 : p_phase, abort_flag, p.timeout_ns))) break;
          tc_fence_after_sync();
          if (kSkip && j > 0 && group_skips(1, j)) {
            if (q1_in_request) ++pv_skips;
          } else {
            issue_pv(1, v_idx % L::kStages, j > 0);
          }
          if (!more) commit_all(o_done(1));
          commit_own(kv_empty(v_idx % L::kStages));
          if (more) {
            issue_qk(1, nk_idx % L::kStages);
            commit_all(s_full(1));
            commit_own(kv_empty(nk_idx % L::kStages));
            if (j + 2 == wk.n_kv) commit_own(kCross ? q1_empty : q_empty);
          }
          p_phase ^= 1u;
          p_phase1 ^= 1u;
          v_idx = next_v;
          nk_idx = next_nk;
        }
        if (!ok) break;  // no product of another unit after a wait that ran out
      }
      if (kSkip && p.skip_counts != nullptr && pv_skips != 0) atomicAdd(&p.skip_counts[1], pv_skips);
      if (!ok) abort_all();
    }
  } else {
    // ------------------------------------------------ softmax groups
    const int grp = warp >> 2;  // 0 -> Q0, 1 -> Q1
    const int r = threadIdx.x & 127;
    // kCross: a query tile's row -> its token, r / pack (exact for r < 128, pack <= 32: the factor is
    // floor(2^16 / pack) + 1)
    auto token_of = [&](int row_in_tile) { return static_cast<int>((row_in_tile * p.pack_mul) >> 16); };
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + (grp == 0 ? L::kTmemS0 : L::kTmemS1);
    const uint32_t t_o = tmem + lane_off + (grp == 0 ? L::kTmemO0 : L::kTmemO1);
    uint32_t s_phase = 0;
    uint32_t o_phase = 0;  // kCross: this group's count of units, as a parity
    int wt = 0;
    bool ok = true;
    unsigned long long warp_skips = 0;
    for (;; ++wt) {
      int w;
      ok = __all_sync(0xffffffffu, next_work(wt, w));
      if (!ok || w < 0) break;
      const auto wk = decode(wt, w);
      // the groups take turns on the key tiles of a cut tile without second query tile
      bool turns = false;
      if constexpr (kCross) {
        turns = wk.slot >= 0 && !two_tiles(wk);
        if (grp == 1 && !turns && !two_tiles(wk)) {
          mbar_arrive(p_full(1));
          continue;
        }
      }
      const int step_j = turns ? 2 : 1;
      const int n_kv = wk.n_kv;
      const int row = kCross ? 0 : wk.q0 + static_cast<int>(rank) * kRowsPerWork + grp * kBM + r;
      // log2-domain score factor; FP8 scores carry the two heads' dequantisation factors
      const float sl2 = kFp8 ? p.scale_log2 * p.deq[wk.head] * p.deq[p.H + wk.head] : p.scale_log2;
      float m = -INFINITY, l = 0.f;
      float m_seen = -INFINITY;  // block skipping: running maximum over all earlier tiles
      for (int j = turns ? grp : 0; j < n_kv; j += step_j) {
        ok = __all_sync(0xffffffffu, mbar_wait(s_full(grp), s_phase, abort_flag, p.timeout_ns));
        if (!ok) break;
        s_phase ^= 1u;
        tc_fence_after_sync();
        // keys at or past the request end (last tile only) are masked
        // (kCross: what the loop seldom needs is read from the unit's slot again, not held in a register)
        const int valid = j == n_kv - 1 ? (kCross ? unit_word(wt, 4) : key_count(wk)) - j * kBN : kBN;
        float s[128];
        load_scores(t_s, valid, s);
        const float mx = row_max(s) * sl2;
        if constexpr (kSkip) {
          // Skip-Softmax: this warp's 32 rows drop K/V tile j when every row
          // of the request has its tile maximum more than skip_tau below its
          // maximum over tiles 0..j-1. The vote goes to the MMA thread, which
          // leaves out O_i += P_i V_j when all four warps of the group drop it.
          const bool in_request = row < end_of_queries(wk);
          const bool skip = __all_sync(0xffffffffu, !in_request || (j > 0 && mx < m_seen - p.skip_tau));
          m_seen = fmaxf(m_seen, mx);
          if (lane == 0) votes[(grp * 2 + (j & 1)) * 4 + (warp & 3)] = skip ? 1 : 0;
          if (skip) {
            if (__any_sync(0xffffffffu, in_request) && lane == 0) ++warp_skips;
            // P = 0 for these rows (the product still runs if another warp
            // keeps the tile): 64 columns of bf16 pairs, or 32 of e4m3 quads
            if constexpr (kFp8Pv) {
              uint32_t zero[32];
#pragma unroll
              for (int c = 0; c < 32; ++c) zero[c] = 0u;
              tmem_st_x32(t_s, zero);
            } else {
              uint32_t zero[64];
#pragma unroll
              for (int c = 0; c < 64; ++c) zero[c] = 0u;
              tmem_st_x64(t_s, zero);
            }
            tc_fence_before_sync();
            mbar_arrive(p_full(grp));
            continue;
          }
        }
        const bool need_rescale = j >= step_j && mx > m + kRescaleThreshold;
        float alpha = 1.0f;
        if (j < step_j) {
          // kCross: a first key tile of scores -inf alone (keys with infinities)
          // leaves P = 0 and l = 0 behind, not exp(-inf + inf)
          m = kCross ? fmaxf(mx, -3.402823466e38f) : mx;
        } else if (need_rescale) {
          alpha = ex2_approx(m - mx);
          l *= alpha;
          m = mx;
        }
        // O_i holds the products of tiles 0..j-1, all complete (s_full for
        // tile j completed after them): rescale it before P_j V_j. Tensor-
        // memory loads and stores are warp-collective (.sync.aligned), so
        // the whole warp takes this path when any of its rows needs it, the
        // other rows with alpha = 1. Eight columns at a time in a rolled
        // loop: the 128 scores are live here, and wider chunks push the
        // kernel past its register budget (spills in every variant).
        if (__any_sync(0xffffffffu, need_rescale)) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 8) {
            uint32_t ov[8];
            tmem_ld_x8(t_o + c0, ov);
#pragma unroll
            for (int c = 0; c < 8; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
            tmem_st_x8(t_o + c0, ov);
          }
        }
        l += exp_tile_store<kFp8Pv>(s, sl2, -m, t_s);
        if constexpr (kCross) {
          // V rows past the last key become zero before any product reads
          // them (the first group's "P ready" precedes both groups' products;
          // when they take turns, the tile is this group's alone)
          if ((grp == 0 || turns) && valid < kBN) {
            const uint32_t idx = static_cast<uint32_t>(unit_word(wt, 7)) + 2 * j + 1;  // the unit's last copy
            const int st = idx % L::kStages;
            ok = __all_sync(0xffffffffu, mbar_wait(kv_full(st), (idx / L::kStages) & 1, abort_flag, p.timeout_ns));
            if (!ok) break;
            if (r >= valid) {
#pragma unroll
              for (int c = 0; c < L::kSlabs * 8; ++c)
                *reinterpret_cast<uint4*>(smem + L::kKVOff + st * L::kStageBytes + (c / 8) * kSlabBytes + r * 128 +
                                          (c % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
          }
        }
        tc_fence_before_sync();
        if constexpr (kPair) {
          // one arrival per warp at the leader's barrier. P and the rescaled
          // O are in this CTA's tensor memory, their stores complete
          // (tcgen05.wait::st) and fenced before this point, so a plain
          // remote arrive hands them over; a cluster-scope release here,
          // on every tile's critical path, cost 15 % of the kernel's time
          __syncwarp();
          if (lane == 0) {
            if (leader) mbar_arrive(p_full(grp));
            else arrive_remote(in_cta(p_full(grp), 0));
          }
        } else {
          mbar_arrive(p_full(grp));
        }
      }
      if (!ok) break;
      // epilogue: normalise O_i and write the valid rows
      ok = __all_sync(0xffffffffu, mbar_wait(o_done(grp), kCross ? o_phase : wt & 1, abort_flag, p.timeout_ns));
      if (!ok) break;
      o_phase ^= 1u;
      tc_fence_after_sync();
      // FP8 P V accumulates V's codes: its dequantisation factor comes in here
      const float inv_l = (kFp8Pv ? p.deq[2 * p.H + wk.head] : 1.0f) / l;
      const bool valid_row = row < end_of_queries(wk);
      if constexpr (kCross) {
        // the unit again from its slot: holding all of it through the loop
        // over the key tiles cost spills
        const auto un = decode(wt, w);
        // this thread's token and head, of the query tile's tile_q x pack rows
        const int r_token = token_of(r);
        const int q_row = un.q0 + (un.slot >= 0 && !two_tiles(un) ? 0 : grp * tile_q) + r_token;
        const bool valid_row = r_token < tile_q && q_row < un.q_end;
        if (un.slot >= 0) {
          const int64_t prow = static_cast<int64_t>(un.slot) * kRowsPerWork + grp * kBM + r;
          float4* part = reinterpret_cast<float4*>(p.part_o + prow * D);
          // a part whose scores are all -inf: rows of 0, to be joined with weight 0
          const float part_inv_l = l == 0.f ? 0.f : inv_l;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t ov[32];
            tmem_ld_x32(t_o + c0, ov);
            if (valid_row) {
#pragma unroll
              for (int c = 0; c < 32; c += 4)
                part[(c0 + c) / 4] =
                    make_float4(__uint_as_float(ov[c]) * part_inv_l, __uint_as_float(ov[c + 1]) * part_inv_l,
                                __uint_as_float(ov[c + 2]) * part_inv_l, __uint_as_float(ov[c + 3]) * part_inv_l);
            }
          }
          if (valid_row) p.part_lse[prow] = m + __log2f(l);
          tc_fence_before_sync();
          continue;
        }
        // 64 columns of the warp's 32 rows at a time: each lane puts its row's
        // eight 16-byte pieces where no two lanes meet in a bank (piece ^ row
        // in the row's 128 bytes), then eight lanes store one row
        const int head = un.head + r - r_token * p.pack;
        const uint64_t dst = reinterpret_cast<uint64_t>(
            valid_row ? p.o + static_cast<int64_t>(q_row) * p.o_stride + head * D : nullptr);
        uint8_t* stage = smem + L::kOutOff + warp * (32 * 128);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t ov[32];
            tmem_ld_x32(t_o + c0 + half * 32, ov);
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              uint4 v;
              v.x = pack_bf16x2(__uint_as_float(ov[c]) * inv_l, __uint_as_float(ov[c + 1]) * inv_l);
              v.y = pack_bf16x2(__uint_as_float(ov[c + 2]) * inv_l, __uint_as_float(ov[c + 3]) * inv_l);
              v.z = pack_bf16x2(__uint_as_float(ov[c + 4]) * inv_l, __uint_as_float(ov[c + 5]) * inv_l);
              v.w = pack_bf16x2(__uint_as_float(ov[c + 6]) * inv_l, __uint_as_float(ov[c + 7]) * inv_l);
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((half * 4 + c / 8) ^ (lane & 7)) * 16)) = v;
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int srow = i * 4 + (lane >> 3), piece = lane & 7;
            const uint64_t to = __shfl_sync(0xffffffffu, dst, srow);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + srow * 128 + ((piece ^ (srow & 7)) * 16));
            if (to != 0) reinterpret_cast<uint4*>(to)[c0 / 8 + piece] = v;
          }
          __syncwarp();
        }
        if (valid_row && p.lse != nullptr)
          p.lse[static_cast<int64_t>(head) * p.T + q_row] = (m + __log2f(l)) * 0.69314718055994530942f;
        tc_fence_before_sync();
        continue;
      }
      __nv_bfloat16* dst = p.o + static_cast<int64_t>(row) * p.o_stride + wk.head * D;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t ov[32];
        tmem_ld_x32(t_o + c0, ov);
        if (valid_row) {
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint4 v;
            v.x = pack_bf16x2(__uint_as_float(ov[c]) * inv_l, __uint_as_float(ov[c + 1]) * inv_l);
            v.y = pack_bf16x2(__uint_as_float(ov[c + 2]) * inv_l, __uint_as_float(ov[c + 3]) * inv_l);
            v.z = pack_bf16x2(__uint_as_float(ov[c + 4]) * inv_l, __uint_as_float(ov[c + 5]) * inv_l);
            v.w = pack_bf16x2(__uint_as_float(ov[c + 6]) * inv_l, __uint_as_float(ov[c + 7]) * inv_l);
            *reinterpret_cast<uint4*>(dst + c0 + c) = v;
          }
        }
      }
      if (valid_row && p.lse != nullptr)
        p.lse[static_cast<int64_t>(wk.head) * p.T + row] = (m + __log2f(l)) * 0.69314718055994530942f;
      tc_fence_before_sync();
    }
    if constexpr (kCross) {
      // queries without keys: O = 0, lse = -inf; tiles spread over the blocks
      const int B = p.sched[1], n_empty = p.sched[4];
      const CrossSched cs(p.sched, B);
      for (int i = blockIdx.x; i < n_empty; i += gridDim.x) {
        const int q = find_last(cs.empty_start, B, i);
        const int nqb = (cs.q_len[q] + 2 * tile_q - 1) / (2 * tile_q);
        const int local = i - cs.empty_start[q];
        const int r_token = token_of(r);
        const int head = local / nqb * p.pack + r - r_token * p.pack;
        const int in_request = (local % nqb) * 2 * tile_q + grp * tile_q + r_token;
        if (r_token < tile_q && in_request < cs.q_len[q]) {
          const int64_t t = cs.q_start[q] + in_request;
          uint4* dst = reinterpret_cast<uint4*>(p.o + t * p.o_stride + head * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
          if (p.lse != nullptr) p.lse[static_cast<int64_t>(head) * p.T + t] = -INFINITY;
        }
      }
    }
    if (kSkip && p.skip_counts != nullptr && lane == 0 && warp_skips != 0) atomicAdd(&p.skip_counts[0], warp_skips);
    if (!ok) abort_all();
  }

  tc_fence_before_sync();
  auto block_sync = [&]() {
    if constexpr (kPair) {
      __syncwarp();
      cluster_sync_all();
    } else {
      __syncthreads();
    }
  };
  block_sync();
  // Every role (of both CTAs, on a pair) has stopped, so the abort flag is
  // final. On an abort, copies and MMAs may still be in flight into the
  // block's shared and tensor memory: wait for all of them before the memory
  // is freed. On a pair every copy completes on a leader's barrier, which
  // completes only once both CTAs' halves have landed; the second CTA waits
  // at the cluster barrier meanwhile.
  if (*abort_flag) {
    if (leader && warp == kProducerWarp && lane == 0)
    {
      drain_copies(kv_full(0), q_full, L::kStages, loads_done[0], loads_done[1]);
      if (kCross && loads_done[2] > 0) mbar_drain_wait(q1_full, (loads_done[2] - 1) & 1);
    }
    else if (leader && warp == kMmaWarp && lane == 0)
      kPair ? drain_mmas_pair(drain) : drain_mmas(drain);
    block_sync();
  }
  tc_fence_after_sync();
  if (warp == kMmaWarp) {
    if constexpr (kPair) tmem_dealloc_pair(tmem, 512); else tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------ self-test

__global__ void wait_selftest_kernel(int* status, long long timeout_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  const uint32_t b = smem_addr(&bar);
  if (threadIdx.x == 0) {
    mbar_init(b, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    // nothing ever arrives on `bar`: the bounded wait must give up
    if (!mbar_wait(b, 0, &abort_flag, timeout_ns)) atomicCAS(status, 0, kStatusTimeout);
  }
}

// ------------------------------------------------------------ host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// [T, H, D] bf16 with `stride` elements between tokens, read as boxes of
// 64 columns x box_heads heads x box_rows tokens, 128-byte swizzled; rows past
// T read as 0.
bool make_qkv_map(CUtensorMap* map, const void* ptr, int64_t T, int H, int D, int64_t stride, int box_rows = kBM,
                  int box_heads = 1) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T, H, D] e4m3 bytes with `stride` elements (bytes) between tokens, read
// as boxes of 128 bytes x 1 head x 128 tokens, 128-byte swizzled.
bool make_e4m3_map(CUtensorMap* map, const void* ptr, int64_t T, int H, int D, int64_t stride) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr || D != 128) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[3] = {128, 1, static_cast<cuuint32_t>(kBM)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kCross>
bool set_schedule_smem_attr() {
  static int done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (!done[dev]) {
    const void* kernel = kCross ? reinterpret_cast<const void*>(build_cross_schedule_kernel)
                                : reinterpret_cast<const void*>(build_schedule_kernel);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSchedSmem) != cudaSuccess)
      return false;
    done[dev] = 1;
  }
  return true;
}

// Per device: the shared-memory attribute of the pair kernel is set and the
// number of CTA pairs that can be resident at once is queried on the first
// call (which must precede any stream capture), so that the persistent grid
// never leaves a pair waiting for a second wave.
int resident_attn_pairs(cudaLaunchConfig_t* cfg) {
  static int pairs[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  if (pairs[dev] == 0) {
    if (cudaFuncSetAttribute(attn_fwd_kernel<128, false, false, false, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<128, true>::kAlloc) != cudaSuccess)
      return -1;
    int n = 0;
    cfg->gridDim = dim3(2, 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, attn_fwd_kernel<128, false, false, false, true>, cfg) != cudaSuccess ||
        n < 1)
      return -1;
    pairs[dev] = n;
  }
  return pairs[dev];
}

int launch_attn_pair(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                     int64_t max_work, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<128, true>::kAlloc;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int max_pairs = resident_attn_pairs(&cfg);
  if (max_pairs < 1) return -1;
  cfg.gridDim = dim3(2 * static_cast<unsigned>(max_work < max_pairs ? max_work : max_pairs), 1, 1);
  if (cudaLaunchKernelEx(&cfg, attn_fwd_kernel<128, false, false, false, true>, tq, tk, tv, p) != cudaSuccess)
    return -1;
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int D, bool kSkip, bool kFp8, bool kFp8Pv, bool kCross = false>
bool set_smem_attr() {
  static int done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_fwd_kernel<D, kSkip, kFp8, kFp8Pv, false, kCross>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<D, false, kCross>::kAlloc) != cudaSuccess)
      return false;
    done[dev] = 1;
  }
  return true;
}

}  // namespace

size_t attn_schedule_bytes(int B) { return ((sched_words(B) * sizeof(int32_t)) + 255) & ~static_cast<size_t>(255); }

int launch_varlen_attn(const void* q, const void* k, const void* v, void* o, float* lse, int64_t q_stride,
                       int64_t k_stride, int64_t v_stride, int64_t o_stride, const int32_t* cu_seqlens, int B,
                       int64_t T, int H, int D, float softmax_scale, void* workspace, int* status,
                       long long timeout_ns, cudaStream_t stream, int num_sms, bool skip, float skip_tau,
                       unsigned long long* skip_counts, const float* deq, bool fp8_pv, bool cta_pairs) {
  CUtensorMap tq, tk, tv;
  const bool maps_ok = deq != nullptr
                           ? make_e4m3_map(&tq, q, T, H, D, q_stride) && make_e4m3_map(&tk, k, T, H, D, k_stride)
                           : make_qkv_map(&tq, q, T, H, D, q_stride) && make_qkv_map(&tk, k, T, H, D, k_stride);
  const bool v_ok = fp8_pv ? make_e4m3_map(&tv, v, T, H, D, v_stride) : make_qkv_map(&tv, v, T, H, D, v_stride);
  if (!maps_ok || !v_ok) return -2;
  // bf16, head_dim 128, no block skipping: on CTA pairs when asked, whose K
  // copies are 64-key halves
  const bool pair = cta_pairs && deq == nullptr && !skip && D == 128;
  if (pair && !make_qkv_map(&tk, k, T, H, D, k_stride, kBN / 2)) return -2;
  const int rows_per_work = pair ? kRowsPerPairWork : kRowsPerWork;
  int32_t* sched = static_cast<int32_t*>(workspace);
  int sort_n = 1;
  while (sort_n < B) sort_n <<= 1;
  const size_t sched_smem = B <= kSortLimit ? static_cast<size_t>(sort_n) * 8 : 0;
  if (sched_smem > 48 * 1024 && !set_schedule_smem_attr<false>()) return -1;
  build_schedule_kernel<<<1, kSchedThreads, sched_smem, stream>>>(cu_seqlens, B, T, H, rows_per_work, sched,
                                                                  status);
  if (cudaGetLastError() != cudaSuccess) return -1;
  AttnParams p;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.o_stride = o_stride;
  p.T = T;
  p.H = H;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.sched = sched;
  p.status = status;
  p.timeout_ns = timeout_ns;
  p.skip_tau = skip_tau;
  p.skip_counts = skip_counts;
  p.deq = deq;
  p.pack = p.group = 1;
  p.part_o = p.part_lse = nullptr;
  // upper bound of work tiles: every request adds at most one partial block
  const int64_t max_work = static_cast<int64_t>(H) * ((T + rows_per_work - 1) / rows_per_work + B);
  const int grid = static_cast<int>(max_work < num_sms ? max_work : num_sms);
  if (pair) return launch_attn_pair(tq, tk, tv, p, max_work, stream);
  if (fp8_pv && !skip) {
    if (D != 128 || deq == nullptr) return -1;
    if (!set_smem_attr<128, false, true, true>()) return -1;
    attn_fwd_kernel<128, false, true, true><<<grid, kThreads, Layout<128>::kAlloc, stream>>>(tq, tk, tv, p);
  } else if (fp8_pv) {
    if (D != 128 || deq == nullptr) return -1;
    if (!set_smem_attr<128, true, true, true>()) return -1;
    attn_fwd_kernel<128, true, true, true><<<grid, kThreads, Layout<128>::kAlloc, stream>>>(tq, tk, tv, p);
  } else if (deq != nullptr && !skip) {
    if (D != 128) return -1;
    if (!set_smem_attr<128, false, true, false>()) return -1;
    attn_fwd_kernel<128, false, true, false><<<grid, kThreads, Layout<128>::kAlloc, stream>>>(tq, tk, tv, p);
  } else if (deq != nullptr) {
    if (D != 128) return -1;
    if (!set_smem_attr<128, true, true, false>()) return -1;
    attn_fwd_kernel<128, true, true, false><<<grid, kThreads, Layout<128>::kAlloc, stream>>>(tq, tk, tv, p);
  } else if (D == 128 && !skip) {
    if (!set_smem_attr<128, false, false, false>()) return -1;
    attn_fwd_kernel<128, false, false, false><<<grid, kThreads, Layout<128>::kAlloc, stream>>>(tq, tk, tv, p);
  } else if (D == 128) {
    if (!set_smem_attr<128, true, false, false>()) return -1;
    attn_fwd_kernel<128, true, false, false><<<grid, kThreads, Layout<128>::kAlloc, stream>>>(tq, tk, tv, p);
  } else if (!skip) {
    if (!set_smem_attr<64, false, false, false>()) return -1;
    attn_fwd_kernel<64, false, false, false><<<grid, kThreads, Layout<64>::kAlloc, stream>>>(tq, tk, tv, p);
  } else {
    if (!set_smem_attr<64, true, false, false>()) return -1;
    attn_fwd_kernel<64, true, false, false><<<grid, kThreads, Layout<64>::kAlloc, stream>>>(tq, tk, tv, p);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

namespace {

size_t cross_sched_bytes(int B) { return (cross_sched_words(B) * sizeof(int32_t) + 255) & ~static_cast<size_t>(255); }

template <int D>
int launch_cross(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p, int B,
                 int grid, bool may_cut, cudaStream_t stream) {
  // The attention kernel sets itself up while the schedule is still being
  // built (programmatic dependent launch) and waits for it where it first
  // needs it.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<D, false, true>::kAlloc;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_fwd_kernel<D, false, false, false, false, true>, tq, tk, tv, p) != cudaSuccess)
    return -1;
  if (may_cut) {
    // as many blocks as there can be cut tiles (fewer than kCutUnits) and rows in one
    const int tokens = kBM / p.pack;
    const int64_t tiles = static_cast<int64_t>(p.H / p.pack) * ((p.T + 2 * tokens - 1) / (2 * tokens) + B);
    const int64_t rows = (p.T < 2 * tokens ? p.T : 2 * tokens) * p.pack;
    const dim3 blocks(static_cast<unsigned>(tiles < kCutUnits ? tiles : kCutUnits),
                      static_cast<unsigned>((rows + kCombineThreads / 32 - 1) / (kCombineThreads / 32)));
    combine_parts_kernel<D><<<blocks, kCombineThreads, 0, stream>>>(
        p.sched, p.part_o, p.part_lse, p.o, p.lse, p.o_stride, p.T, p.pack);
    if (cudaGetLastError() != cudaSuccess) return -1;
  }
  return 0;
}

}  // namespace

// The schedule, then the parts' rows and log2-sum-exps (at most kCutUnits
// parts of kRowsPerWork rows).
size_t cross_attn_workspace_bytes(int B, int D) {
  return cross_sched_bytes(B) + static_cast<size_t>(kCutUnits) * kRowsPerWork * (D + 1) * sizeof(float);
}

int launch_varlen_cross_attn(const void* q, const void* k, const void* v, void* o, float* lse, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, int64_t o_stride, const int32_t* cu_q,
                             const int32_t* cu_k, int B, int64_t Tq, int64_t Tk, int H, int Hkv, int D,
                             float softmax_scale, void* workspace, int* status, long long timeout_ns,
                             cudaStream_t stream, int num_sms) {
  CUtensorMap tq, tk, tv;
  // all settings on the first call on a device: a later one, of other sizes, may be under capture
  if (!set_smem_attr<64, false, false, false, true>() || !set_smem_attr<128, false, false, false, true>() ||
      !set_schedule_smem_attr<true>())
    return -1;
  const int group = H / Hkv;
  // heads of one key head in one unit. Past 32 of them a query tile's 128 rows
  // may be a quarter empty (128 mod pack), and K and V are read 32 times less
  // often than the queries' rows as it is.
  const int pack = group <= 32 ? group : 1;
  const int tile_q = kBM / pack;
  if (!make_qkv_map(&tq, q, Tq, H, D, q_stride, tile_q, pack)) return -2;
  if (Tk > 0 ? !make_qkv_map(&tk, k, Tk, Hkv, D, k_stride) || !make_qkv_map(&tv, v, Tk, Hkv, D, v_stride) : false)
    return -2;
  if (Tk == 0) tk = tv = tq;  // without any key there is nothing to map, and these are not read
  int32_t* sched = static_cast<int32_t*>(workspace);
  int sort_n = 1;
  while (sort_n < B) sort_n <<= 1;
  const size_t sched_smem = B <= kSortLimit ? static_cast<size_t>(sort_n) * 8 : 0;
  if (B <= kWarpRequests)
    build_cross_schedule_warp_kernel<<<1, 32, 0, stream>>>(cu_q, cu_k, B, Tq, Tk, H / pack, 2 * tile_q, sched, status);
  else
    build_cross_schedule_kernel<<<1, kSchedThreads, sched_smem, stream>>>(cu_q, cu_k, B, Tq, Tk, H / pack, 2 * tile_q,
                                                                          sched, status);
  if (cudaGetLastError() != cudaSuccess) return -1;
  AttnParams p = {};
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.o_stride = o_stride;
  p.T = Tq;
  p.H = H;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.sched = sched;
  p.status = status;
  p.timeout_ns = timeout_ns;
  p.pack = pack;
  p.pack_mul = 65536 / pack + 1;
  p.group = group;
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + cross_sched_bytes(B));
  p.part_lse = p.part_o + static_cast<size_t>(kCutUnits) * kRowsPerWork * D;
  // no request has more than kMinPartTiles key tiles: no tile can be cut
  const bool may_cut = Tk > static_cast<int64_t>(kMinPartTiles) * kBN;
  const int64_t tiles = static_cast<int64_t>(H / pack) * ((Tq + 2 * tile_q - 1) / (2 * tile_q) + B);
  const int64_t max_units = tiles + (may_cut ? kCutUnits : 0);
  const int grid = static_cast<int>(max_units < num_sms ? max_units : num_sms);
  return D == 128 ? launch_cross<128>(tq, tk, tv, p, B, grid, may_cut, stream)
                  : launch_cross<64>(tq, tk, tv, p, B, grid, may_cut, stream);
}

int launch_wait_selftest(int* status, long long timeout_ns, cudaStream_t stream) {
  wait_selftest_kernel<<<1, 32, 0, stream>>>(status, timeout_ns);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace pqk
