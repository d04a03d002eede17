// Gradient of packed cross attention (and, with equal offsets, of packed self attention) for
// sm_103a: TMA + tcgen05 + TMEM.
//
//   P = exp(scale q k^T - lse),  dP = do v^T,  delta = rowsum(do * o),  dS = P * (dP - delta)
//   dv = P^T do,   dk = scale dS^T q,   dq = scale dS k
//
// Two kernels, because a sum over queries (dk, dv) and one over keys (dq) cannot both stay in one
// CTA's accumulators: the dK/dV kernel keeps a 128-key tile and runs over the queries, the dQ kernel
// keeps a 128-row query tile and runs over the keys.  Each recomputes S and dP (7 products in all
// instead of 5); in exchange nothing is summed through memory in an order that depends on timing
// (no atomics), and no fp32 gradient goes through memory, but for the tiles of a last, partly filled
// wave of CTAs: their range is cut into chunks so that they fill it too (4,096 x 4,096 x 24 heads is
// 5.05 waves of tiles in each kernel), and a last kernel adds the chunks' fp32 sums in order.
//
// dK/dV works on transposed scores: S^T = K Q^T and dP^T = V dO^T have keys as TMEM lanes, so P^T and
// dS^T are written back to TMEM as the A operands of dV += P^T dO and dK += dS^T Q, and one copy of Q
// and dO in shared memory serves both products that read it.  Each thread owns a key row and half the
// 128 query columns.  dV_i and S_{i+1} run while dS_i is computed, dK_i and dP_{i+1} while P_{i+1} is.
// TMEM (512 columns): S^T/P^T, dP^T/dS^T, dK, dV.
// dQ: S = Q K^T (two buffers), dP = dO V^T, dQ += dS K with dS written over S.  It runs from one item
// into the next, since key lists may be a few tiles.  A fourth warpgroup computes delta an item ahead (a
// kernel of its own for it reads do once more: 59 us of a text case's 589).
// In dQ the products come from two warps (S and dP from one, dQ from the other): a warp's polls queue
// behind its own products, so one warp alone leaves the tensor core idle at each wait (4,096 x 4,096 x
// 24 x 128: 290 us with one, 236 with two, 207 now).  In dK/dV the four products of a step alternate between two chains
// and one warp keeps them in that order; two warps measured slower there (350 us against 295, now 262).
// What bounds both: the chain scores -> exponential -> dS -> product of one tile, which keeps the tensor
// core 66 % busy in dK/dV, 63 % in dQ, and 47 % in dQ when key lists are five tiles, where reading dQ out
// of TMEM between two items is not hidden (the fourth warpgroup cannot do it: it has delta to compute).
//
// P and dS are rounded to bf16 for the tensor core (half a step, 2^-8 relative at most); everything
// else is fp32 until the gradients are rounded once.  Rows and keys past a segment's end are zeroed
// in shared memory as far as a product reads them, and masked by select where they would meet an
// exponential.  Every wait is bounded; a wait that runs out records a timeout and unwinds the CTA.
#include <cuda_bf16.h>

#include <cstddef>

#include "cross_segments.cuh"
#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 384;
constexpr int kDqThreads = 512;  // registers moved with setmaxnreg
constexpr int kDqRegsCompute = 168, kDqRegsRows = 80, kDqRegsControl = 96;
static_assert(2 * kDqRegsCompute + kDqRegsRows + kDqRegsControl == 65536 / 128, "the registers at launch");
constexpr int kTmemCols = 512;
constexpr int kPlanThreads = 1024;

__host__ __device__ constexpr int tiles_of(int n) { return (n + kTile - 1) / kTile; }
__device__ __forceinline__ int steps16(int n) { return (n + 15) / 16; }

// A row's LSE in units of log 2 as the exponent's offset.  A row without weights (LSE -inf: no keys, or
// all scores -inf) gets +inf, so that its weights are exp2(S - inf) = 0 and it takes no part.
__device__ __forceinline__ float lse_log2(float lse) {
  return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
}

// ---- plan ------------------------------------------------------------------------------------------
// Tiles of each kernel are numbered over the segments (head-major within one).  Whole waves of tiles are
// an item each; the tiles behind them are cut into `chunks` items each.
struct Plan {
  uint32_t items_q, items_k;  // of dQ and of dK/dV
  uint32_t whole_q, whole_k;  // tiles that are an item
  uint32_t chunks_q, chunks_k;
  uint32_t tiles_q, tiles_k;
  uint32_t prefix[1];  // exclusive prefix of query tiles x heads [S + 1], then of key tiles x key heads
};
static_assert(offsetof(Plan, prefix) == kCrossBwdHeader * sizeof(uint32_t), "the header's words");
__device__ __forceinline__ const Plan& plan_of(const uint32_t* ws) { return *reinterpret_cast<const Plan*>(ws); }
__device__ __forceinline__ int kv_steps(const CrossSegment& r, int group) {  // (head, query tile) pairs
  return r.used > 0 ? group * tiles_of(r.rows) : 0;
}
// Item of a kernel -> tile and chunk.
struct Cut {
  uint32_t tile;
  int chunk, chunks;
};
__device__ __forceinline__ Cut cut_of(uint32_t item, uint32_t whole, uint32_t chunks) {
  if (item < whole) return Cut{item, 0, 1};
  return Cut{whole + (item - whole) / chunks, static_cast<int>((item - whole) % chunks), static_cast<int>(chunks)};
}
// A tile of n steps is cut into at most n chunks; chunk c's steps begin at n c / chunks.
__device__ __forceinline__ int step_at(int n, int c, int chunks) {
  return static_cast<int>(static_cast<int64_t>(n) * c / chunks);
}

// Tiles and steps of each kernel.  Tiles are counted in 64 bits: overlapping segments can hold more than 32
// bits count.  Of the steps (rows x keys x heads pass 32 bits first) only the mean is wanted.
struct PlanSums {
  uint64_t tiles_q, tiles_k;
  float steps_q, steps_k;
  __device__ __forceinline__ void add(const PlanSums& o) {
    tiles_q += o.tiles_q;
    tiles_k += o.tiles_k;
    steps_q += o.steps_q;
    steps_k += o.steps_k;
  }
  __device__ __forceinline__ PlanSums shfl(int from) const {
    return PlanSums{__shfl_sync(0xffffffffu, tiles_q, from), __shfl_sync(0xffffffffu, tiles_k, from),
                    __shfl_sync(0xffffffffu, steps_q, from), __shfl_sync(0xffffffffu, steps_k, from)};
  }
};
// Sum over the block's threads (whole warps) before this one (tiles only) and over all; the four sums' shuffles
// overlap.
__device__ __forceinline__ PlanSums exclusive_scan(const PlanSums& v, PlanSums* s_warp, PlanSums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  PlanSums x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const PlanSums y = x.shfl((lane - o) & 31);
    if (lane >= o) x.add(y);
  }
  total = x.shfl(31);
  x.tiles_q -= v.tiles_q;
  x.tiles_k -= v.tiles_k;
  if (warps == 1) return x;
  if (lane == 31) s_warp[warp] = total;
  __syncthreads();
  total = PlanSums{};
#pragma unroll 1
  for (int w = 0; w < warps; ++w) {
    if (w == warp) x.add(total);
    total.add(s_warp[w]);
  }
  return x;
}

// One block: a warp when the segments fit its lanes (one scan, no block barrier), else 1,024
// threads with several segments each.
__global__ void __launch_bounds__(kPlanThreads)
cross_bwd_plan_kernel(const __grid_constant__ CrossSegments seg, uint32_t* __restrict__ ws, int slots, uint32_t sms,
                      unsigned int* err) {
  __shared__ PlanSums s_warp[kPlanThreads / 32];
  grid_dependency_wait();
  launch_dependents();
  const int S = seg.num_segments, tid = threadIdx.x, group = seg.num_q_heads / seg.num_kv_heads;
  const int chunk = (S + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
  const int lo = min(S, tid * chunk), hi = min(S, lo + chunk);
  auto q_tiles = [&](const CrossSegment& r) { return static_cast<uint32_t>(tiles_of(r.rows)) * seg.num_q_heads; };
  auto k_tiles = [&](const CrossSegment& r) { return static_cast<uint32_t>(tiles_of(r.keys)) * seg.num_kv_heads; };
  CrossSegment mine{};  // this thread's only segment, when it has one
  if (chunk == 1 && lo < hi) mine = checked_cross_segment(seg, lo, err);
  auto segment = [&](int g) { return chunk == 1 ? mine : checked_cross_segment(seg, g, err); };
  PlanSums own{}, all;
  for (int g = lo; g < hi; ++g) {
    const CrossSegment r = segment(g);
    const uint32_t nq = q_tiles(r), nk = k_tiles(r);
    own.add(PlanSums{nq, nk, static_cast<float>(nq) * static_cast<float>(tiles_of(r.used)),
                     static_cast<float>(nk) * static_cast<float>(kv_steps(r, group))});
  }
  const PlanSums before = exclusive_scan(own, s_warp, all);
  uint32_t at_q = static_cast<uint32_t>(before.tiles_q), at_k = static_cast<uint32_t>(before.tiles_k);
  // Segments that overlap can hold more tiles than the capacities: then no item.
  const bool over = all.tiles_q > (static_cast<uint64_t>(seg.capacity_q) / kTile + S) * seg.num_q_heads ||
                    all.tiles_k > (static_cast<uint64_t>(seg.capacity_k) / kTile + S) * seg.num_kv_heads;
  if (over && tid == 0) record_error(err, kErrBadCuSeqlens);
  const uint32_t tiles_q = over ? 0u : static_cast<uint32_t>(all.tiles_q);
  const uint32_t tiles_k = over ? 0u : static_cast<uint32_t>(all.tiles_k);
  uint32_t *pq = ws + kCrossBwdHeader, *pk = pq + S + 1;
  for (int g = lo; g < hi; ++g) {
    const CrossSegment r = segment(g);
    pq[g] = at_q;
    pk[g] = at_k;
    at_q += q_tiles(r);
    at_k += k_tiles(r);
  }
  // Chunks of the tiles behind the whole waves: what makes their waves of items (of steps / c steps,
  // and about 3 steps' time of start and end each; 2 more for the sum of several chunks) shortest, as
  // far as the slots reach.  Measured with other terms: 0 for the 3: 2,048 x 2,048 x 24 207 us, not 171, four
  // segments of 64 to 320 rows and 40 to 256 keys 57, not 42; 6: 157 and 42.  0 for the 2: 171 and 44; 8: 158 and
  // 43.5.  Six other shapes are the same within 2 % but for 130 x 5,000 x 8 (50 us, not 48, at 0 for the 2).  Lanes 0-15 weigh 1 to 16 chunks for the query tiles, 16-31 for the key
  // tiles.
  if (tid < 32) {
    const bool keys = tid >= 16;
    const uint32_t c = (tid & 15) + 1, tiles = keys ? tiles_k : tiles_q, rest = tiles % sms;
    const float steps = tiles > 0 ? (keys ? all.steps_k : all.steps_q) / static_cast<float>(tiles) : 0.f;
    float cost = static_cast<float>((rest * c + sms - 1) / sms) * (steps / static_cast<float>(c) + 3.f) + (c > 1 ? 2.f : 0.f);
    if (c > kCrossBwdMaxChunks || (c > 1 && rest * c > static_cast<uint32_t>(slots))) cost = INFINITY;
    uint32_t best = c;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, cost, o);
      const uint32_t other_c = __shfl_xor_sync(0xffffffffu, best, o);
      if (other < cost || (other == cost && other_c < best)) {
        cost = other;
        best = other_c;
      }
    }
    const uint32_t best_q = __shfl_sync(0xffffffffu, best, 0), best_k = __shfl_sync(0xffffffffu, best, 16);
    if (tid == 0) {
      pq[S] = tiles_q;
      pk[S] = tiles_k;
      Plan& p = *reinterpret_cast<Plan*>(ws);
      p.tiles_q = tiles_q;
      p.tiles_k = tiles_k;
      p.whole_q = tiles_q - tiles_q % sms;
      p.whole_k = tiles_k - tiles_k % sms;
      p.chunks_q = best_q;
      p.chunks_k = best_k;
      p.items_q = p.whole_q + (tiles_q - p.whole_q) * best_q;
      p.items_k = p.whole_k + (tiles_k - p.whole_k) * best_k;
    }
  }
}

__device__ __forceinline__ int find_segment(const uint32_t* __restrict__ prefix, int S, uint32_t item) {
  int lo = 0, hi = S - 1;  // last g with prefix[g] <= item
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= item) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// ---- shared pieces of the two product kernels ----------------------------------------------------------
template <int D>
struct Tiles {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBytes = kTile * D * 2;
  static constexpr int kBoxBytes = kTile * 128;
};

// One 128-row tile of one head.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int head, int row, uint32_t bar) {
  mbar_arrive_expect_tx(bar, Tiles<D>::kBytes);
#pragma unroll
  for (int b = 0; b < Tiles<D>::kBoxes; ++b)
    tma_load_3d(smem_u32(dst + b * Tiles<D>::kBoxBytes), map, b * 64, head, row, bar);
}

// Zero rows [n, 16 * steps16(n)) of a tile (whole 128-byte rows: the swizzle permutes 16-byte pieces
// within a row).  One warp; before any product reads the tile.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int n) {
  const int lane = threadIdx.x & 31, rows = 16 * steps16(n) - n;
  for (int i = lane; i < rows * Tiles<D>::kBoxes * 8; i += 32) {
    const int r = n + i / (Tiles<D>::kBoxes * 8), rem = i % (Tiles<D>::kBoxes * 8);
    *reinterpret_cast<uint4*>(tile + (rem >> 3) * Tiles<D>::kBoxBytes + r * 128 + (rem & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// D[128 x 16 n16] = A B^T over D, both tiles K-major in shared memory (descriptor low halves).
template <int D>
__device__ __forceinline__ void product_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                           uint32_t b_hi, int n16) {
  const uint32_t idesc = idesc_bf16_f32(kTile, 16 * n16, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * Tiles<D>::kBoxBytes + (kk & 3) * 32) >> 4;
    mma_ss_split(d_tmem, a_lo + off, a_hi, b_lo + off, b_hi, idesc, kk > 0 ? 1u : 0u);
  }
}
// D[128 x D] (+)= A B over 16 n16 rows of B (row-major tile): A in TMEM as packed bf16, its first 64
// columns at a, the others at a + 64.
template <int D>
__device__ __forceinline__ void product_ts(uint32_t d_tmem, uint32_t a, uint32_t b_lo, uint32_t b_hi, int n16,
                                           bool first) {
  constexpr uint32_t idesc = idesc_bf16_f32(kTile, D, true);
  if (n16 == 8) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_ts_split(d_tmem, a + (kk >> 2) * 64 + (kk & 3) * 8, b_lo + kk * (2048 >> 4), b_hi, idesc,
                   (!first || kk > 0) ? 1u : 0u);
  } else {
#pragma unroll 1
    for (int kk = 0; kk < n16; ++kk)
      mma_ts_split(d_tmem, a + (kk >> 2) * 64 + (kk & 3) * 8, b_lo + kk * (2048 >> 4), b_hi, idesc,
                   (!first || kk > 0) ? 1u : 0u);
  }
}

// 32 fp32 columns of this thread's TMEM lane, times f, as bf16 to columns [c0, c0 + 32) of its row:
// lanes 2i and 2i + 1 trade halves, so that each instruction writes 32-byte sectors.  p0: the even
// lane's row (+ 16 columns for the odd lane), p1 the odd lane's; wide: both are 32-byte aligned.
__device__ __forceinline__ void store_columns(const uint32_t* r, float f, __nv_bfloat16* p0, __nv_bfloat16* p1,
                                              bool ok0, bool ok1, bool wide) {
  const bool odd = threadIdx.x & 1;
  uint32_t pk[16];
#pragma unroll
  for (int c = 0; c < 16; ++c)
    pk[c] = pack_bf16x2(__uint_as_float(r[2 * c]) * f, __uint_as_float(r[2 * c + 1]) * f);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? pk[c] : pk[8 + c], 1);
    pk[c] = odd ? got : pk[c];
    pk[8 + c] = odd ? pk[8 + c] : got;
  }
  if (ok0) st_global_32(p0, pk, wide);
  if (ok1) st_global_32(p1, pk + 8, wide);
}

// ---- dK, dV ---------------------------------------------------------------------------------------------
struct KvWork {
  int more;                  // 0: no more work
  int steps, first;          // (head, query tile) steps of the item: first, first + 1, ...
  int head0, qtiles;         // step s: head head0 + s / qtiles, query tile s % qtiles
  int q0, q_end;
  int kv_head, k_row;        // the key tile
  int rows, used;            // its rows inside the segment, and how many of them are used
  int slot;                  // partial sums go to this slot; -1: straight to dk, dv
};

__device__ __forceinline__ KvWork decode_kv(uint32_t item, const uint32_t* __restrict__ ws, const CrossSegments& seg) {
  const int S = seg.num_segments, group = seg.num_q_heads / seg.num_kv_heads;
  const Plan& plan = plan_of(ws);
  const uint32_t* prefix = plan.prefix + S + 1;
  const Cut cut = cut_of(item, plan.whole_k, plan.chunks_k);
  const int g = find_segment(prefix, S, cut.tile);
  const CrossSegment r = cross_segment(seg, g);
  const int tiles = tiles_of(r.keys), local = static_cast<int>(cut.tile - prefix[g]);
  KvWork d;
  d.more = 1;
  d.kv_head = local / tiles;
  const int kt = local % tiles;
  d.k_row = r.k0 + kt * kTile;
  d.rows = min(kTile, r.keys - kt * kTile);
  d.used = max(0, min(kTile, r.used - kt * kTile));
  const int steps = d.used > 0 ? kv_steps(r, group) : 0;  // none: zeros, from the first chunk
  const int chunks = max(1, min(cut.chunks, steps));
  if (cut.chunk >= chunks) {
    d.steps = d.first = d.rows = 0;
  } else {
    d.first = step_at(steps, cut.chunk, chunks);
    d.steps = step_at(steps, cut.chunk + 1, chunks) - d.first;
  }
  d.slot = chunks > 1 && cut.chunk < chunks ? static_cast<int>(item - plan.whole_k) : -1;
  d.head0 = d.kv_head * group;
  d.qtiles = max(1, tiles_of(r.rows));
  d.q0 = r.q0;
  d.q_end = r.q0 + r.rows;
  return d;
}

template <int D>
struct KvCfg {
  // Q is held longest (S to dK), so its ring is a tile deeper than dO's (dP to dV): 7 tiles with K and
  // V, all that fits at D = 128.
  static constexpr int kStagesQ = 3, kStagesO = 2;
  // kv_full, kv_empty, s_full, dp_full, p_full, ds_full, acc_full, acc_empty, w_full[2], w_empty[2],
  // drain, then q_full, q_empty, st_full, st_empty, do_full, do_empty
  static constexpr int kNumBars = 13 + 2 * kStagesQ + 4 * kStagesO;
  static constexpr int kSmemBytes = Tiles<D>::kBytes * (2 + kStagesQ + kStagesO) + kStagesO * 2 * kTile * 4 +
                                    kNumBars * 8 + 16 + 2 * sizeof(KvWork);
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr int kColS = 0, kColP = 128, kColK = 256, kColV = 384;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_dkv_kernel(const __grid_constant__ CrossBwdArgs a) {
  using C = KvCfg<D>;
  using T = Tiles<D>;
  constexpr int SQ = C::kStagesQ, SO = C::kStagesO;
  extern __shared__ __align__(1024) uint8_t smem[];  // no room to align it by hand
  uint8_t* sK = smem;
  uint8_t* sV = sK + T::kBytes;
  uint8_t* sQ = sV + T::kBytes;
  uint8_t* sO = sQ + SQ * T::kBytes;
  float* s_lse = reinterpret_cast<float*>(sO + SO * T::kBytes);  // [SO][128], in units of log 2
  float* s_delta = s_lse + SO * kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_delta + SO * kTile);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  KvWork* work = reinterpret_cast<KvWork*>(tmem_slot + 4);
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * static_cast<uint32_t>(i); };
  const uint32_t kv_full = bar(0), kv_empty = bar(1), s_full = bar(2), dp_full = bar(3), p_full = bar(4),
                 ds_full = bar(5), acc_full = bar(6), acc_empty = bar(7), drain = bar(12);
  auto w_full = [&](int i) { return bar(8 + i); };
  auto w_empty = [&](int i) { return bar(10 + i); };
  auto q_full = [&](int s) { return bar(13 + s); };
  auto q_empty = [&](int s) { return bar(13 + SQ + s); };
  auto st_full = [&](int s) { return bar(13 + 2 * SQ + s); };
  auto st_empty = [&](int s) { return bar(13 + 2 * SQ + SO + s); };
  auto do_full = [&](int s) { return bar(13 + 2 * SQ + 2 * SO + s); };
  auto do_empty = [&](int s) { return bar(13 + 2 * SQ + 3 * SO + s); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, a.wait_limit_ns)) != 0;
  };
  auto wait2 = [&](uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1) {  // the polls overlap
    bool r0 = mbar_try_wait(b0, p0), r1 = mbar_try_wait(b1, p1);
    if (!r0) r0 = mbar_wait(b0, p0, a.wait_limit_ns);
    if (!r1) r1 = mbar_wait(b1, p1, a.wait_limit_ns);
    return __all_sync(0xffffffffu, r0 && r1) != 0;
  };
  auto wait_long = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_long(b, parity, a.wait_limit_ns)) != 0;
  };
  auto arrive_warp = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };
  auto take = [&](int k, KvWork& d) {
    if (!wait_long(w_full(k & 1), (k >> 1) & 1)) return false;
    d = work[k & 1];
    arrive_warp(w_empty(k & 1));
    return true;
  };

  grid_dependency_wait();
  launch_dependents();
  if (__syncthreads_or(a.err != nullptr && *reinterpret_cast<volatile unsigned int*>(a.err) == kErrTimeout)) return;
  const uint32_t total = plan_of(a.plan).items_k;
  if (blockIdx.x >= total) return;
  if ((smem_u32(smem) & 1023u) != 0) {  // the tiles' swizzle needs it; not met on any known driver
    if (threadIdx.x == 0) record_error(a.err, kErrSmemLayout);
    return;
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&a.tmap_q);
    tma_prefetch_desc(&a.tmap_k);
    tma_prefetch_desc(&a.tmap_v);
    tma_prefetch_desc(&a.tmap_do);
    const uint32_t one[] = {kv_full, kv_empty, s_full, dp_full, acc_full, drain};
    for (uint32_t b : one) mbar_init(b, 1);
    const uint32_t warps8[] = {p_full, ds_full, acc_empty};
    for (uint32_t b : warps8) mbar_init(b, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(w_full(i), 1);
      mbar_init(w_empty(i), 11);  // compute warps, loads, products, statistics
    }
    for (int s = 0; s < SQ; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
    }
    for (int s = 0; s < SO; ++s) {
      mbar_init(st_full(s), 1);
      mbar_init(st_empty(s), 8);
      mbar_init(do_full(s), 1);
      mbar_init(do_empty(s), 1);
    }
    fence_mbarrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ================= loads =================
    bool ok = true, stalled = false;
    uint32_t items = 0, n = 0, nd = 0;  // key tiles, Q tiles, dO tiles loaded so far
    KvWork d;
    for (int k = 0; ok && !stalled; ++k) {
      ok = take(k, d);
      if (!ok || !d.more) break;
      if (d.steps == 0) continue;
      ok = wait(kv_empty, (items & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(kv_full, 2 * T::kBytes);
        for (int b = 0; b < T::kBoxes; ++b) {
          tma_load_3d(smem_u32(sK + b * T::kBoxBytes), &a.tmap_k, b * 64, d.kv_head, d.k_row, kv_full);
          tma_load_3d(smem_u32(sV + b * T::kBoxBytes), &a.tmap_v, b * 64, d.kv_head, d.k_row, kv_full);
        }
      }
      ++items;
      for (int i = 0; i < d.steps; ++i) {
        if (n >= a.stall_after_tiles) {  // testing hook: as if the loads had stalled
          stalled = true;
          break;
        }
        const int s = static_cast<int>(n % SQ), o = static_cast<int>(nd % SO), step = d.first + i;
        const int head = d.head0 + step / d.qtiles, row = d.q0 + step % d.qtiles * kTile;
        ok = wait_long(q_empty(s), ((n / SQ) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) load_tile<D>(sQ + s * T::kBytes, &a.tmap_q, head, row, q_full(s));
        ++n;
        ok = wait_long(do_empty(o), ((nd / SO) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) load_tile<D>(sO + o * T::kBytes, &a.tmap_do, head, row, do_full(o));
        ++nd;
      }
    }
    if (!ok && lane == 0) record_error(a.err, kErrTimeout);
    // never leave while a copy may still land
    if (items > 0) mbar_wait(kv_full, (items - 1) & 1);
    for (uint32_t i = 0; i < SQ && i < n; ++i) mbar_wait(q_full((n - 1 - i) % SQ), ((n - 1 - i) / SQ) & 1);
    for (uint32_t i = 0; i < SO && i < nd; ++i) mbar_wait(do_full((nd - 1 - i) % SO), ((nd - 1 - i) / SO) & 1);
  } else if (warp == 9) {
    // ================= products =================
    const bool leader = elect_one();
    constexpr uint32_t kTile16 = T::kBytes >> 4;
    const SmemDesc dk = sw128_desc_split(smem_u32(sK), 16, 1024), dv = sw128_desc_split(smem_u32(sV), 16, 1024);
    const SmemDesc dq = sw128_desc_split(smem_u32(sQ), 16, 1024), dd = sw128_desc_split(smem_u32(sO), 16, 1024);
    // the same tiles as row-major B operands
    const SmemDesc rq = sw128_desc_split(smem_u32(sQ), T::kBoxBytes, 1024);
    const SmemDesc rd = sw128_desc_split(smem_u32(sO), T::kBoxBytes, 1024);
    bool ok = true, issued = false;
    uint32_t items = 0, n = 0;  // key tiles; steps whose dK has been issued
    KvWork d;
    for (int k = 0; ok; ++k) {
      ok = take(k, d);
      if (!ok || !d.more) break;
      if (d.steps == 0) continue;
      int tile = d.first % d.qtiles;  // query tile of the step whose scores are next
      auto next_rows = [&] {
        const int rows = min(kTile, d.q_end - d.q0 - tile * kTile);
        tile = tile + 1 == d.qtiles ? 0 : tile + 1;
        return rows;
      };
      auto scores = [&](uint32_t m, int rows) {  // S^T = K Q^T of step m (counted over all items)
        const int s = static_cast<int>(m % SQ);
        if (rows % 16 != 0) zero_rows<D>(sQ + s * T::kBytes, rows);
        tc_fence_after();
        if (leader) {
          product_ss<D>(tmem + C::kColS, dk.lo, dk.hi, dq.lo + s * kTile16, dq.hi, steps16(rows));
          mma_commit(s_full);
        }
        __syncwarp();
      };
      auto grads = [&](uint32_t m, int rows) {  // dP^T = V dO^T
        const int s = static_cast<int>(m % SO);
        if (rows % 16 != 0) zero_rows<D>(sO + s * T::kBytes, rows);
        tc_fence_after();
        if (leader) {
          product_ss<D>(tmem + C::kColP, dv.lo, dv.hi, dd.lo + s * kTile16, dd.hi, steps16(rows));
          mma_commit(dp_full);
        }
        __syncwarp();
      };
      int rows = next_rows(), rows_next = kTile;
      ok = wait(kv_full, items & 1) && wait2(q_full(n % SQ), (n / SQ) & 1, do_full(n % SO), (n / SO) & 1);
      if (!ok) break;
      scores(n, rows);
      grads(n, rows);
      issued = true;
      for (int i = 0; i < d.steps; ++i, ++n) {
        const int s = static_cast<int>(n % SQ), o = static_cast<int>(n % SO), n16 = steps16(rows);
        const uint32_t m = n + 1;
        const bool more = i + 1 < d.steps;
        // one wait before each product: it passes while the last ones of the product before it run
        ok = wait(p_full, n & 1);
        if (ok && i == 0) ok = wait(acc_empty, (items & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        if (leader) {  // dV += P^T dO
          product_ts<D>(tmem + C::kColV, tmem + C::kColS, rd.lo + o * kTile16, rd.hi, n16, i == 0);
          mma_commit(do_empty(o));
        }
        __syncwarp();
        if (more) {
          rows_next = next_rows();
          ok = wait(q_full(m % SQ), (m / SQ) & 1);
          if (!ok) break;
          scores(m, rows_next);
        }
        ok = wait(ds_full, n & 1);
        if (!ok) break;
        tc_fence_after();
        if (leader) {  // dK += dS^T Q
          product_ts<D>(tmem + C::kColK, tmem + C::kColP, rq.lo + s * kTile16, rq.hi, n16, i == 0);
          mma_commit(q_empty(s));
        }
        __syncwarp();
        if (more) {
          ok = wait(do_full(m % SO), (m / SO) & 1);
          if (!ok) break;
          grads(m, rows_next);
        }
        rows = rows_next;
      }
      if (!ok) break;
      if (leader) {
        mma_commit(acc_full);
        mma_commit(kv_empty);
      }
      __syncwarp();
      ++items;
    }
    if (!ok && leader) record_error(a.err, kErrTimeout);
    if (issued && leader) {  // every product issued has completed before TMEM is released
      mma_commit(drain);
      mbar_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ================= scheduler =================
    for (int k = 0;; ++k) {
      const uint32_t item = blockIdx.x + static_cast<uint32_t>(k) * gridDim.x;
      KvWork d{};
      if (item < total) d = decode_kv(item, a.plan, a.seg);
      if (!wait_long(w_empty(k & 1), ((k >> 1) & 1) ^ 1)) {
        if (lane == 0) record_error(a.err, kErrTimeout);
        break;
      }
      if (lane == 0) {
        work[k & 1] = d;
        mbar_arrive(w_full(k & 1));
      }
      __syncwarp();
      if (!d.more) break;
    }
  } else if (warp == 11) {
    // ================= row statistics of the query tiles =================
    bool ok = true;
    uint32_t n = 0;
    KvWork d;
    for (int k = 0; ok; ++k) {
      ok = take(k, d);
      if (!ok || !d.more) break;
      for (int i = 0; i < d.steps; ++i, ++n) {
        const int s = static_cast<int>(n % SO), step = d.first + i;
        const size_t at = static_cast<size_t>(d.head0 + step / d.qtiles) * a.seg.capacity_q;
        const int row = d.q0 + step % d.qtiles * kTile;
        float l[4], e[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // rows past the end: weight exp2(0 - inf) = 0
          const int r = row + lane + 32 * x;
          l[x] = r < d.q_end ? lse_log2(a.lse[at + r]) : INFINITY;
          e[x] = r < d.q_end ? a.delta[at + r] : 0.f;
        }
        ok = wait_long(st_empty(s), ((n / SO) & 1) ^ 1);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s_lse[s * kTile + lane + 32 * x] = l[x];
          s_delta[s * kTile + lane + 32 * x] = e[x];
        }
        arrive_warp(st_full(s));
      }
    }
    if (!ok && lane == 0) record_error(a.err, kErrTimeout);
  } else {
    // ================= P, dS and the epilogue: key row = TMEM lane, query columns by warpgroup =====
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + C::kColS + 64 * half;
    const uint32_t p_addr = tmem + lane_base + C::kColP + 64 * half;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    bool ok = true;
    uint32_t n = 0, items = 0;
    KvWork d;
    for (int k = 0; ok; ++k) {
      ok = take(k, d);
      if (!ok || !d.more) break;
      // key rows that take no part (their K and V may be anything): masked by select
      const bool dead = row >= d.used, any_dead = d.used < kTile;
      for (int i = 0; i < d.steps; ++i, ++n) {
        const int s = static_cast<int>(n % SO);
        const float4* lse4 = reinterpret_cast<const float4*>(s_lse + s * kTile + 64 * half);
        const float4* del4 = reinterpret_cast<const float4*>(s_delta + s * kTile + 64 * half);
        ok = wait(st_full(s), (n / SO) & 1) && wait(s_full, n & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[64];
        tmem_ld32(s_addr, x);
        tmem_ld32(s_addr + 32, x + 32);
        tmem_ld_wait();
        tmem_reg_fence<64>(x);
        float p[64];
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 v = lse4[c];
          p[4 * c] = ex2_approx(fmaf(__uint_as_float(x[4 * c]), scale_log2, -v.x));
          p[4 * c + 1] = ex2_approx(fmaf(__uint_as_float(x[4 * c + 1]), scale_log2, -v.y));
          p[4 * c + 2] = ex2_approx(fmaf(__uint_as_float(x[4 * c + 2]), scale_log2, -v.z));
          p[4 * c + 3] = ex2_approx(fmaf(__uint_as_float(x[4 * c + 3]), scale_log2, -v.w));
        }
        if (any_dead) {
#pragma unroll
          for (int c = 0; c < 64; ++c) p[c] = dead ? 0.f : p[c];
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
        tmem_st32(s_addr, w);
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(p_full);
        ok = wait(dp_full, n & 1);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(p_addr, x);
        tmem_ld32(p_addr + 32, x + 32);
        tmem_ld_wait();
        tmem_reg_fence<64>(x);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 v = del4[c];
          p[4 * c] *= __uint_as_float(x[4 * c]) - v.x;
          p[4 * c + 1] *= __uint_as_float(x[4 * c + 1]) - v.y;
          p[4 * c + 2] *= __uint_as_float(x[4 * c + 2]) - v.z;
          p[4 * c + 3] *= __uint_as_float(x[4 * c + 3]) - v.w;
        }
        arrive_warp(st_empty(s));
        if (any_dead) {
#pragma unroll
          for (int c = 0; c < 64; ++c) p[c] = dead ? 0.f : p[c];
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
        tmem_st32(p_addr, w);
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(ds_full);
      }
      if (!ok) break;
      // epilogue: warpgroup 0 takes dV, warpgroup 1 dK
      if (d.steps > 0) {
        ok = wait(acc_full, items & 1);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t acc = tmem + lane_base + (half == 0 ? C::kColV : C::kColK);
      const float f = half == 0 ? 1.f : a.scale;
      const int odd = lane & 1, r0 = row - odd;
      const int64_t stride = half == 0 ? a.dv_stride : a.dk_stride;
      __nv_bfloat16* p0 = (half == 0 ? a.dv : a.dk) + (static_cast<int64_t>(d.k_row) + r0) * stride +
                          d.kv_head * D + 16 * odd;
      float* part = a.partials + ((static_cast<size_t>(max(d.slot, 0)) * 2 + half) * kTile + row) * D;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t x[32];
        if (d.steps > 0) {
          tmem_ld32(acc + c0, x);
          tmem_ld_wait();
          tmem_reg_fence<32>(x);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0u;
        }
        if (d.slot >= 0) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4*>(part + c0 + 4 * c) =
                make_float4(__uint_as_float(x[4 * c]) * f, __uint_as_float(x[4 * c + 1]) * f,
                            __uint_as_float(x[4 * c + 2]) * f, __uint_as_float(x[4 * c + 3]) * f);
        } else {
          store_columns(x, f, p0 + c0, p0 + stride + c0, r0 < d.rows, r0 + 1 < d.rows, a.wide);
        }
      }
      if (d.steps > 0) {
        tc_fence_before();
        arrive_warp(acc_empty);
        ++items;
      }
    }
    if (!ok && lane == 0) record_error(a.err, kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Sums the chunks of every cut tile, in chunk order: 16 rows of one tile's dV, dK or dQ to a unit.
template <int D>
__global__ void __launch_bounds__(256)
cross_bwd_sum_kernel(const __grid_constant__ CrossBwdArgs a) {
  // Nothing is read before the wait, the plan and the offsets included (they say where this kernel writes):
  // only the wait makes another kernel's writes visible here.
  grid_dependency_wait();
  launch_dependents();
  const unsigned int code = a.err != nullptr ? *reinterpret_cast<const volatile unsigned int*>(a.err) : 0u;
  const Plan& plan = plan_of(a.plan);
  const int S = a.seg.num_segments, group = a.seg.num_q_heads / a.seg.num_kv_heads;
  constexpr uint32_t kParts = 8;
  constexpr int kRows = kTile / kParts;
  const uint32_t units_k = plan.chunks_k > 1 ? (plan.tiles_k - plan.whole_k) * 2 * kParts : 0;
  const uint32_t units_q = plan.chunks_q > 1 ? (plan.tiles_q - plan.whole_q) * kParts : 0;
  struct Unit {
    int chunks, r0, rows;
    size_t step;  // floats between chunks
    const float* part;
    int64_t stride;
    __nv_bfloat16* out;
  };
  auto locate = [&](uint32_t u) {
    const bool keys = u < units_k;
    const uint32_t v = keys ? u : u - units_k, per_tile = keys ? 2 * kParts : kParts;
    const uint32_t index = v / per_tile;  // of the tile behind the whole waves
    const int which = keys ? static_cast<int>(v / kParts % 2) : 0;
    const uint32_t* prefix = keys ? plan.prefix + S + 1 : plan.prefix;
    const uint32_t tile = (keys ? plan.whole_k : plan.whole_q) + index;
    const int most = static_cast<int>(keys ? plan.chunks_k : plan.chunks_q);
    const int g = find_segment(prefix, S, tile);
    const CrossSegment r = cross_segment(a.seg, g);
    const int tiles = tiles_of(keys ? r.keys : r.rows), local = static_cast<int>(tile - prefix[g]);
    const int head = local / tiles, row_tile = local % tiles * kTile;
    const int steps = keys ? (row_tile < r.used ? kv_steps(r, group) : 0) : tiles_of(r.used);
    const size_t slot = static_cast<size_t>(index) * most;
    Unit x;
    x.chunks = max(1, min(most, steps));
    x.r0 = static_cast<int>(v % kParts) * kRows;
    x.rows = min(kTile, (keys ? r.keys : r.rows) - row_tile);
    x.step = keys ? 2 * kTile * D : kTile * D;
    x.part = keys ? a.partials + slot * x.step + static_cast<size_t>(which) * kTile * D : a.partials_q + slot * x.step;
    x.stride = keys ? (which == 0 ? a.dv_stride : a.dk_stride) : a.dq_stride;
    x.out = (keys ? (which == 0 ? a.dv : a.dk) : a.dq) +
            (static_cast<int64_t>(keys ? r.k0 : r.q0) + row_tile) * x.stride + head * D;
    return x;
  };
  for (uint32_t u = blockIdx.x; u < units_k + units_q; u += gridDim.x) {
    const Unit x = locate(u);
    if (code == kErrTimeout || code == kErrSmemLayout) return;  // the sums are incomplete
    if (x.chunks == 1) continue;  // written already
    for (int i = threadIdx.x; i < kRows * (D / 8); i += 256) {
      const int row = x.r0 + i / (D / 8), col = i % (D / 8) * 8;
      if (row >= x.rows) continue;
      float f[8] = {};
#pragma unroll 8
      for (int c = 0; c < x.chunks; ++c) {
        const float4* src = reinterpret_cast<const float4*>(x.part + c * x.step + row * D + col);
        const float4 y = src[0], z = src[1];
        f[0] += y.x; f[1] += y.y; f[2] += y.z; f[3] += y.w;
        f[4] += z.x; f[5] += z.y; f[6] += z.z; f[7] += z.w;
      }
      *reinterpret_cast<uint4*>(x.out + row * x.stride + col) =
          make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
  }
}

// ---- dQ -------------------------------------------------------------------------------------------------
struct QWork {
  int more;
  int head, kv_head;
  int q_row, q_end;
  int k_row, nkv, last_keys;  // nkv 0: no keys (such items are not handed on)
  int slot;                   // the chunk's sum goes to this slot; -1: straight to dq
};

__device__ __forceinline__ QWork decode_q(uint32_t item, const uint32_t* __restrict__ ws, const CrossSegments& seg) {
  const int S = seg.num_segments, group = seg.num_q_heads / seg.num_kv_heads;
  const Plan& plan = plan_of(ws);
  const Cut cut = cut_of(item, plan.whole_q, plan.chunks_q);
  const int g = find_segment(plan.prefix, S, cut.tile);
  const CrossSegment r = cross_segment(seg, g);
  const int tiles = tiles_of(r.rows), local = static_cast<int>(cut.tile - plan.prefix[g]);
  const int steps = tiles_of(r.used), chunks = max(1, min(cut.chunks, steps));
  QWork d;
  d.more = 1;
  d.head = local / tiles;
  d.kv_head = d.head / group;
  d.q_row = r.q0 + local % tiles * kTile;
  d.q_end = cut.chunk < chunks ? r.q0 + r.rows : d.q_row;  // a chunk past the last has no rows
  const int first = step_at(steps, min(cut.chunk, chunks), chunks);
  const int end = step_at(steps, min(cut.chunk + 1, chunks), chunks);
  d.k_row = r.k0 + first * kTile;
  d.nkv = end - first;
  d.last_keys = min(kTile, r.used - (end - 1) * kTile);
  d.slot = chunks > 1 ? static_cast<int>(item - plan.whole_q) : -1;
  return d;
}

template <int D>
struct QCfg {
  static constexpr int kStagesK = 3, kStagesV = 2;
  static constexpr int kWork = 4;  // items decoded ahead
  // q_full, q_empty, do_full, do_empty, s_full[2], s_empty[2], ds_full[2], dp_full, dp_read, acc_full,
  // acc_empty, drain[2], d_full[2], d_empty[2], w_full[kWork], w_empty[kWork], then k_full, k_empty, v_full, v_empty
  static constexpr int kNumBars = 20 + 2 * kWork + 2 * kStagesK + 2 * kStagesV;
  static constexpr int kSmemBytes = Tiles<D>::kBytes * (2 + kStagesK + kStagesV) + kNumBars * 8 + 16 +
                                    kWork * sizeof(QWork) + 2 * kTile * sizeof(float2);
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr int kColS = 0, kColP = 256, kColQ = 384;
};

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1)
cross_dq_kernel(const __grid_constant__ CrossBwdArgs a) {
  using C = QCfg<D>;
  using T = Tiles<D>;
  constexpr int SK = C::kStagesK, SV = C::kStagesV;
  extern __shared__ __align__(1024) uint8_t smem[];  // no room to align it by hand
  uint8_t* sQ = smem;
  uint8_t* sO = sQ + T::kBytes;
  uint8_t* sK = sO + T::kBytes;
  uint8_t* sV = sK + SK * T::kBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + SV * T::kBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  QWork* work = reinterpret_cast<QWork*>(tmem_slot + 4);
  // [2][128]: an item's (lse in units of log 2, delta)
  float2* s_rows = reinterpret_cast<float2*>(work + C::kWork);
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * static_cast<uint32_t>(i); };
  const uint32_t q_full = bar(0), q_empty = bar(1), do_full = bar(2), do_empty = bar(3), dp_full = bar(10),
                 dp_read = bar(11), acc_full = bar(12), acc_empty = bar(13);
  auto s_full = [&](uint32_t i) { return bar(4 + static_cast<int>(i)); };
  auto s_empty = [&](uint32_t i) { return bar(6 + static_cast<int>(i)); };
  // two of them: a warp may finish its next dS while another still works on this one
  auto ds_full = [&](uint32_t i) { return bar(8 + static_cast<int>(i)); };
  auto drain = [&](int i) { return bar(14 + i); };
  auto d_full = [&](int i) { return bar(16 + (i & 1)); };
  auto d_empty = [&](int i) { return bar(18 + (i & 1)); };
  auto w_full = [&](int k) { return bar(20 + k % C::kWork); };
  auto w_empty = [&](int k) { return bar(20 + C::kWork + k % C::kWork); };
  constexpr int kRing = 20 + 2 * C::kWork;
  auto k_full = [&](int s) { return bar(kRing + s); };
  auto k_empty = [&](int s) { return bar(kRing + SK + s); };
  auto v_full = [&](int s) { return bar(kRing + 2 * SK + s); };
  auto v_empty = [&](int s) { return bar(kRing + 2 * SK + SV + s); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, a.wait_limit_ns)) != 0;
  };
  auto wait2 = [&](uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1) {  // the polls overlap
    bool r0 = mbar_try_wait(b0, p0), r1 = mbar_try_wait(b1, p1);
    if (!r0) r0 = mbar_wait(b0, p0, a.wait_limit_ns);
    if (!r1) r1 = mbar_wait(b1, p1, a.wait_limit_ns);
    return __all_sync(0xffffffffu, r0 && r1) != 0;
  };
  auto wait_long = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_long(b, parity, a.wait_limit_ns)) != 0;
  };
  auto arrive_warp = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };
  auto take = [&](int k, QWork& d) {
    if (!wait(w_full(k), k / C::kWork & 1)) return false;
    d = work[k % C::kWork];
    arrive_warp(w_empty(k));
    return true;
  };

  grid_dependency_wait();
  launch_dependents();
  if (__syncthreads_or(a.err != nullptr && *reinterpret_cast<volatile unsigned int*>(a.err) == kErrTimeout)) return;
  const uint32_t total = plan_of(a.plan).items_q;
  if (blockIdx.x >= total) return;
  if ((smem_u32(smem) & 1023u) != 0) {  // the tiles' swizzle needs it; not met on any known driver
    if (threadIdx.x == 0) record_error(a.err, kErrSmemLayout);
    return;
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&a.tmap_q);
    tma_prefetch_desc(&a.tmap_k);
    tma_prefetch_desc(&a.tmap_v);
    tma_prefetch_desc(&a.tmap_do);
    const uint32_t one[] = {q_full, q_empty, do_full, do_empty, s_full(0), s_full(1), s_empty(0), s_empty(1),
                            dp_full, acc_full, drain(0), drain(1)};
    for (uint32_t b : one) mbar_init(b, 1);
    const uint32_t warps8[] = {ds_full(0), ds_full(1), dp_read, acc_empty};
    for (uint32_t b : warps8) mbar_init(b, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(d_full(i), 4);
      mbar_init(d_empty(i), 8);
    }
    for (int i = 0; i < C::kWork; ++i) {
      mbar_init(w_full(i), 1);
      mbar_init(w_empty(i), 15);  // compute warps, key/value loads, two product warps, row warps
    }
    for (int s = 0; s < SK; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    fence_mbarrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 12) {
    // ================= the rows' lse and delta = rowsum(do * o), an item or two ahead ===========
    setmaxnreg_dec<kDqRegsRows>();
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kUnroll = 4;
    const int row = threadIdx.x & 127;
    // an item's rows of o and do into L2 an item before they are read: their latency is a large part
    // of a short item's time
    auto prefetch_rows = [&](const QWork& d) {
      if (d.q_row + row >= d.q_end) return;
      const size_t at = (static_cast<size_t>(d.q_row + row) * a.seg.num_q_heads + d.head) * D;
#pragma unroll
      for (int c = 0; c < D; c += 64) {
        prefetch_l2(static_cast<const __nv_bfloat16*>(a.o) + at + c);
        prefetch_l2(static_cast<const __nv_bfloat16*>(a.dout) + at + c);
      }
    };
    auto delta_rows = [&](int k, const QWork& d) {
      if (!wait_long(d_empty(k), ((k >> 1) & 1) ^ 1)) return false;
      const int64_t step = static_cast<int64_t>(a.seg.num_q_heads) * kLanes;  // 16-byte pieces between rows
      const int64_t at = d.q_row * step + d.head * kLanes + lane % kLanes;
      const int rows = min(kTile, d.q_end - d.q_row);
      const size_t stats = static_cast<size_t>(d.head) * a.seg.capacity_q + d.q_row;
      s_rows[(k & 1) * kTile + row].x = row < rows ? lse_log2(a.lse[stats + row]) : 0.f;
#pragma unroll 1
      for (int r0 = (warp & 3) * 32; r0 < (warp & 3) * 32 + 32; r0 += kRows * kUnroll) {
        uint4 x[kUnroll], y[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int r = r0 + u * kRows + lane / kLanes;
          x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) {
            x[u] = __ldg(static_cast<const uint4*>(a.o) + at + r * step);
            y[u] = __ldg(static_cast<const uint4*>(a.dout) + at + r * step);
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int r = r0 + u * kRows + lane / kLanes;
          const uint32_t p[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, q[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
          float f = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f = fmaf(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16), f);
            f = fmaf(__uint_as_float(p[i] & 0xffff0000u), __uint_as_float(q[i] & 0xffff0000u), f);
          }
#pragma unroll
          for (int m = kLanes / 2; m > 0; m >>= 1) f += __shfl_xor_sync(0xffffffffu, f, m);
          if (lane % kLanes == 0) {
            s_rows[(k & 1) * kTile + r].y = f;
            if (r < rows) a.delta[stats + r] = f;  // for dK
          }
        }
      }
      arrive_warp(d_full(k));
      return true;
    };
    QWork d, nxt{};
    bool ok = take(0, d);
    for (int k = 0; ok && d.more; ++k) {
      ok = take(k + 1, nxt);
      if (ok && nxt.more) prefetch_rows(nxt);
      if (ok) ok = delta_rows(k, d);
      d = nxt;
    }
    if (!ok && lane == 0) record_error(a.err, kErrTimeout);
  } else if (warp >= 8) {
    setmaxnreg_dec<kDqRegsControl>();
    if (warp == 8) {
      // ================= key/value loads =================
      bool ok = true, stalled = false;
      uint32_t kt = 0, vt = 0;
      QWork d;
      for (int k = 0; ok && !stalled; ++k) {
        ok = take(k, d);
        if (!ok || !d.more) break;
        for (int j = 0; j < d.nkv; ++j) {
          if (kt >= a.stall_after_tiles) {
            stalled = true;
            break;
          }
          const int s = static_cast<int>(kt % SK), v = static_cast<int>(vt % SV);
          ok = wait_long(k_empty(s), ((kt / SK) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) load_tile<D>(sK + s * T::kBytes, &a.tmap_k, d.kv_head, d.k_row + j * kTile, k_full(s));
          ++kt;
          ok = wait_long(v_empty(v), ((vt / SV) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) load_tile<D>(sV + v * T::kBytes, &a.tmap_v, d.kv_head, d.k_row + j * kTile, v_full(v));
          ++vt;
        }
      }
      if (!ok && lane == 0) record_error(a.err, kErrTimeout);
      for (uint32_t i = 0; i < SK && i < kt; ++i) mbar_wait(k_full((kt - 1 - i) % SK), ((kt - 1 - i) / SK) & 1);
      for (uint32_t i = 0; i < SV && i < vt; ++i) mbar_wait(v_full((vt - 1 - i) % SV), ((vt - 1 - i) / SV) & 1);
    } else if (warp == 10) {
      // ================= scheduler, query and output-gradient loads =================
      // Items are handed out kWork - 1 ahead of their queries: the others prepare while the query
      // tiles' buffers are still taken.
      bool ok = true, ended = false;
      uint32_t item = blockIdx.x, n = 0;
      auto post = [&](int k) {
        QWork d{};
        for (; item < total; item += gridDim.x) {
          d = decode_q(item, a.plan, a.seg);
          if (d.nkv > 0) break;
          // no keys: zero the tile's rows here
          const int rows = min(kTile, d.q_end - d.q_row);
          for (int i = lane; i < rows * (D / 8); i += 32)
            *reinterpret_cast<uint4*>(a.dq + (static_cast<int64_t>(d.q_row) + i / (D / 8)) * a.dq_stride + d.head * D +
                                      i % (D / 8) * 8) = make_uint4(0u, 0u, 0u, 0u);
          d.more = 0;
        }
        item += gridDim.x;
        if (!wait_long(w_empty(k), (k / C::kWork & 1) ^ 1)) return false;
        if (lane == 0) {
          work[k % C::kWork] = d;
          mbar_arrive(w_full(k));
        }
        __syncwarp();
        ended = !d.more;
        return true;
      };
      int posted = 0;
      for (int k = 0; ok; ++k) {
        while (ok && !ended && posted < k + C::kWork - 1) ok = post(posted++);
        if (!ok) break;
        const QWork d = work[k % C::kWork];  // not overwritten before it is done with here
        if (!d.more) break;
        ok = wait_long(q_empty, (n & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) load_tile<D>(sQ, &a.tmap_q, d.head, d.q_row, q_full);
        ok = wait_long(do_empty, (n & 1) ^ 1);
        if (!ok) {
          mbar_wait(q_full, n & 1);
          break;
        }
        if (lane == 0) load_tile<D>(sO, &a.tmap_do, d.head, d.q_row, do_full);
        ++n;
      }
      if (!ok && lane == 0) record_error(a.err, kErrTimeout);
      if (n > 0) mbar_wait(q_full, (n - 1) & 1);
      if (n > 0) mbar_wait(do_full, (n - 1) & 1);
    } else if (warp == 9) {
      // ================= S and dP =================
      const bool leader = elect_one();
      constexpr uint32_t kTile16 = T::kBytes >> 4;
      const SmemDesc dq = sw128_desc_split(smem_u32(sQ), 16, 1024), dd = sw128_desc_split(smem_u32(sO), 16, 1024);
      const SmemDesc dk = sw128_desc_split(smem_u32(sK), 16, 1024), dv = sw128_desc_split(smem_u32(sV), 16, 1024);
      bool ok = true, issued = false;
      uint32_t n = 0, items = 0;
      QWork d;
      for (int k = 0; ok; ++k, ++items) {
        ok = take(k, d);
        if (!ok || !d.more) break;
        for (int j = 0; j < d.nkv; ++j, ++n) {
          const int s = static_cast<int>(n % SK), v = static_cast<int>(n % SV);
          const bool last = j == d.nkv - 1;
          const int keys = last ? d.last_keys : kTile;
          ok = wait2(s_empty(n & 1), ((n >> 1) & 1) ^ 1, k_full(s), (n / SK) & 1);
          if (ok && j == 0) ok = wait(q_full, items & 1);
          if (!ok) break;
          if (keys % 16 != 0) zero_rows<D>(sK + s * T::kBytes, keys);
          tc_fence_after();
          if (leader) {  // S = Q K^T
            product_ss<D>(tmem + C::kColS + 128 * (n & 1), dq.lo, dq.hi, dk.lo + s * kTile16, dk.hi, steps16(keys));
            mma_commit(s_full(n & 1));
            if (last) mma_commit(q_empty);
          }
          __syncwarp();
          issued = true;
          ok = wait(v_full(v), (n / SV) & 1);
          if (ok && j == 0) ok = wait(do_full, items & 1);
          if (ok && n > 0) ok = wait(dp_read, (n - 1) & 1);
          if (!ok) break;
          if (keys % 16 != 0) zero_rows<D>(sV + v * T::kBytes, keys);
          tc_fence_after();
          if (leader) {  // dP = dO V^T
            product_ss<D>(tmem + C::kColP, dd.lo, dd.hi, dv.lo + v * kTile16, dv.hi, steps16(keys));
            mma_commit(dp_full);
            mma_commit(v_empty(v));
            if (last) mma_commit(do_empty);
          }
          __syncwarp();
        }
      }
      if (!ok && leader) record_error(a.err, kErrTimeout);
      if (issued && leader) {
        mma_commit(drain(0));
        mbar_wait(drain(0), 0);
      }
      __syncwarp();
    } else if (warp == 11) {
      // ================= dQ += dS K =================
      const bool leader = elect_one();
      constexpr uint32_t kTile16 = T::kBytes >> 4;
      const SmemDesc rk = sw128_desc_split(smem_u32(sK), T::kBoxBytes, 1024);
      bool ok = true, issued = false;
      uint32_t n = 0, items = 0;
      QWork d;
      for (int k = 0; ok; ++k, ++items) {
        ok = take(k, d);
        if (!ok || !d.more) break;
        for (int j = 0; j < d.nkv; ++j, ++n) {
          const int s = static_cast<int>(n % SK);
          const bool last = j == d.nkv - 1;
          ok = wait(ds_full(n & 1), (n >> 1) & 1);
          if (ok && j == 0) ok = wait(acc_empty, (items & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            product_ts<D>(tmem + C::kColQ, tmem + C::kColS + 128 * (n & 1), rk.lo + s * kTile16, rk.hi,
                          steps16(last ? d.last_keys : kTile), j == 0);
            mma_commit(k_empty(s));
            mma_commit(s_empty(n & 1));
            if (last) mma_commit(acc_full);
          }
          __syncwarp();
          issued = true;
        }
      }
      if (!ok && leader) record_error(a.err, kErrTimeout);
      if (issued && leader) {
        mma_commit(drain(1));
        mbar_wait(drain(1), 0);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kDqRegsCompute>();
    // ================= dS and the epilogue: query row = TMEM lane, keys by warpgroup ==============
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t p_addr = tmem + lane_base + C::kColP + 64 * half;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    bool ok = true;
    uint32_t n = 0;
    QWork d, nxt;
    float2 mine = make_float2(0.f, 0.f);  // this row's lse and delta
    auto begin = [&](int k, QWork& item) {
      if (!take(k, item)) return false;
      if (!item.more) return true;
      if (!wait(d_full(k), (k >> 1) & 1)) return false;
      return true;
    };
    ok = begin(0, d);
    for (int k = 0; ok && d.more; ++k) {
      mine = s_rows[(k & 1) * kTile + row];
      arrive_warp(d_empty(k));
      for (int j = 0; j < d.nkv; ++j, ++n) {
        const uint32_t s_addr = tmem + lane_base + C::kColS + 128 * (n & 1) + 64 * half;
        const bool last = j == d.nkv - 1;
        // the next item's values, while the products of the last step run
        if (last) ok = begin(k + 1, nxt);
        if (ok) ok = wait(s_full(n & 1), (n >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (last && d.last_keys <= 64 * half) {  // no keys in this warpgroup's columns
          ok = wait(dp_full, n & 1);
          if (!ok) break;
          tc_fence_after();
          tc_fence_before();
          arrive_warp(dp_read);
          arrive_warp(ds_full(n & 1));
          continue;
        }
        uint32_t x[64];
        tmem_ld32(s_addr, x);
        tmem_ld32(s_addr + 32, x + 32);
        tmem_ld_wait();
        tmem_reg_fence<64>(x);
        float p[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) p[c] = ex2_approx(fmaf(__uint_as_float(x[c]), scale_log2, -mine.x));
        if (last && d.last_keys < kTile) {
          // Columns past the keys: their K and V rows are zeros (or not multiplied at all), so any
          // finite weight adds nothing; a row's own weights are at most 1.
#pragma unroll
          for (int c = 0; c < 64; ++c) p[c] = fminf(p[c], 2.f);
        }
        ok = wait(dp_full, n & 1);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(p_addr, x);
        tmem_ld32(p_addr + 32, x + 32);
        tmem_ld_wait();
        tmem_reg_fence<64>(x);
        tc_fence_before();
        arrive_warp(dp_read);
#pragma unroll
        for (int c = 0; c < 64; ++c) p[c] *= __uint_as_float(x[c]) - mine.y;
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
        tmem_st32(s_addr, w);
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(ds_full(n & 1));
      }
      if (ok) ok = wait(acc_full, k & 1);
      if (!ok) break;
      tc_fence_after();
      // epilogue: each warpgroup stores half the columns
      float* part = a.partials_q + (static_cast<size_t>(max(d.slot, 0)) * kTile + row) * D;
      const int odd = lane & 1, r0 = d.q_row + row - odd;
      __nv_bfloat16* p0 = a.dq + static_cast<int64_t>(r0) * a.dq_stride + d.head * D + 16 * odd;
#pragma unroll 1
      for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
        uint32_t x[32];
        tmem_ld32(tmem + lane_base + C::kColQ + c0, x);
        tmem_ld_wait();
        tmem_reg_fence<32>(x);
        if (c0 + 32 == (half + 1) * (D / 2)) {
          tc_fence_before();
          arrive_warp(acc_empty);
        }
        if (d.slot >= 0) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4*>(part + c0 + 4 * c) =
                make_float4(__uint_as_float(x[4 * c]) * a.scale, __uint_as_float(x[4 * c + 1]) * a.scale,
                            __uint_as_float(x[4 * c + 2]) * a.scale, __uint_as_float(x[4 * c + 3]) * a.scale);
        } else {
          store_columns(x, a.scale, p0 + c0, p0 + a.dq_stride + c0, r0 < d.q_end, r0 + 1 < d.q_end, a.wide);
        }
      }
      d = nxt;
    }
    if (!ok && lane == 0) record_error(a.err, kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const CrossBwdArgs& a, cudaStream_t stream) {
  cudaError_t e = allow_shared_memory<KvCfg<D>::kSmemBytes>(cross_dkv_kernel<D>);
  if (e != cudaSuccess) return e;
  e = allow_shared_memory<QCfg<D>::kSmemBytes>(cross_dq_kernel<D>);
  if (e != cudaSuccess) return e;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  e = launch_programmatic(cross_bwd_plan_kernel, dim3(1), dim3(a.seg.num_segments <= 32 ? 32 : kPlanThreads), 0, stream,
                          a.seg, a.plan, a.slots, static_cast<uint32_t>(sms), a.err);
  if (e != cudaSuccess) return e;
  if (a.seg.capacity_q > 0) {
    e = launch_programmatic(cross_dq_kernel<D>, dim3(sms), dim3(kDqThreads), QCfg<D>::kSmemBytes, stream, a);
    if (e != cudaSuccess) return e;
  }
  if (a.seg.capacity_k > 0) {
    e = launch_programmatic(cross_dkv_kernel<D>, dim3(sms), dim3(kThreads), KvCfg<D>::kSmemBytes, stream, a);
    if (e != cudaSuccess) return e;
  }
  // as many CTAs as fit at once: a unit is a chain of dependent loads (2 CTAs an SM: 39.5 us, not 36.2,
  // for four segments of 64 to 320 rows and 40 to 256 keys x 24 heads x 64)
  if (a.slots > 0)
    e = launch_programmatic(cross_bwd_sum_kernel<D>, dim3(8 * sms), dim3(256), 0, stream, a);
  return e;
}

}  // namespace

cudaError_t launch_cross_bwd(const CrossBwdArgs& a, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace h3
