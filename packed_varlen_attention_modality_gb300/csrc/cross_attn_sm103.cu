// Packed cross attention forward for sm_103a (TMA + tcgen05 + TMEM): query segments attend to key
// segments of other lengths (an encoder's states), query heads share key heads.
//
//   S = scale q k^T over the segment's keys,  P = softmax(S),  o = P v,  lse = log sum exp(S)
//
// Work item: two 128-row query tiles that share a (segment, key head): consecutive tiles of the
// key head's query heads, so with shared heads a segment of few rows still fills both tiles.  Both
// stream the same key/value tiles.  One CTA per SM takes items c, c + G, ... of a list ordered by
// key count; what a last, partly filled wave leaves idle is used by cutting its items' key ranges
// into chunks, which a merge kernel joins in chunk order.
//
// An encoder's key lists are short (a few 128-key tiles), so an item is over after a few thousand
// cycles and what happens between items costs as much as the items do.  Hence:
//   - the MMA warps run straight on from one item into the next (order PV0_last, S0_first of the
//     next item, PV1_last, S1_first: the boundary looks like any other step);
//   - they are two, one for each query tile, and take turns: a warp's polls wait behind the products that
//     it has issued, so with one warp the tensor core runs dry at each poll (4,096 x 4,096 x 24 x 128:
//     148 us, 162 with one);
//   - O is read out, normalised and stored by a warpgroup of its own, which hands the accumulator
//     back before it stores, while the softmax warpgroups are in the next item;
//   - items are decoded one ahead, and queries and keys have a producer each, so neither waits on
//     the other's ring;
//   - a last key tile is multiplied only as far as it holds keys (in steps of 16).
// 58,758 rows x 558 keys x 40 heads x 128 take 558 to 565 us so (1,190 to 1,200 TFLOP/s; 530 at best); with
// all of it in the softmax warpgroups and one producer (the packed self-attention kernel's structure) they
// took 787 us.  What bounds it: a step takes some 2,700 cycles (2,048 of tensor work: the chain scores ->
// softmax -> product of each tile sets the pace), the step between two items, here every fifth, 3,700; the
// tensor pipe is 51 % busy (62 % with 32 key tiles an item).  The GPU is at its power cap then, at 1.91 to
// 1.95 GHz, as it is in the packed self-attention kernel at 1,640 TFLOP/s, so the cap is not the bound.  Tried and slower: both tiles' softmax by
// all eight warps, half a row each (581 us); a third query tile's buffer for a key/value tile's (556 us); one
// copy of the issuing code for both kinds of step (615 us); two issuing warps without turns (the tiles fall
// in phase).
//
// Warp roles (512 threads; registers moved with setmaxnreg):
//   warps 0-3 / 4-7   softmax of query tile 0 / 1: thread r owns row r = TMEM lane r
//   warps 8-11        epilogue of both tiles
//   warps 12-15       key/value producer, MMA issuers of tile 0 and 1, scheduler + query producer
// TMEM (512 columns): O0 [0,128), O1 [128,256), S0/P0 [256,384), S1/P1 [384,512).
// Shared memory at D = 128: 2 Q tiles and a ring of 5 K and V tiles in turn, 32 KB each.
//
// Keys past the segment's end are masked to -inf by select and the value rows PV reads past it are
// zeroed in shared memory (by the producer), so NaN/Inf there cannot leak.  A segment without keys takes one tile
// whose keys are all masked: its rows come out as 0 with an LSE of -inf.
// P is rounded to bf16 for the tensor core (half a step, 2^-8 relative at most); scores,
// running max and sum, and O stay fp32, and the result is rounded to bf16 once.
// Every wait is bounded; a wait that runs out records a timeout and unwinds the CTA.
#include <cuda_bf16.h>

#include "cross_segments.cuh"
#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kBlockM = 128, kBlockN = 128;
constexpr int kThreads = 512;
constexpr int kRegsSoftmax = 176, kRegsEpilogue = 80, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + kRegsEpilogue + kRegsOther == 65536 / 128, "the split of the registers at launch");
constexpr int kTmemCols = 512, kColO = 0, kColS = 256;
constexpr float kRescaleLog2 = 8.0f;  // rescale O only when the running max grows by > 2^8
constexpr int kPlanThreads = 1024;   // at most: kSortMax when the segments are that few
// Segments are ordered by keys, and the last wave cut, up to this count (the ordering compares all pairs).
// Segments of 200 rows and 64, 200 or 4,000 keys x 8 heads: 256 of them 348 us (106 ns a key tile), 257 478 us (145).
constexpr int kSortMax = 256;
constexpr int kHeader = kAttnWsHeaderWords;
// The last, partly filled wave, in steps of a key tile (one query tile alone takes nearly as long as two:
// the chain of each sets the pace).  An item's start and end take about two, joining chunks (partial
// results through memory, a kernel with something to do) about eight: 2,048 x 2,048 x 24 heads, 16 steps
// whole or 11 in shares, take 64 us whole, 55 us cut; 3 x 300 x 2,500 x 40 heads, 20 or 16 with the items of
// the last wave short, 81 us either way.
constexpr uint32_t kCostItem = 2, kCostJoin = 8;
// Items of at least 8 key tiles are cut, into chunks of at least 3.  Items of 4 or of 16 at least: the same times
// within 1 % at ten shapes of 1,000 to 30,000 keys.  Chunks of 6 at least: 2,048 x 2,048 x 24 61 us, not 53; of one
// tile: 4,096 x 4,096 x 24 146 us, not 148, 8 x 128 x 1,500 x 24 50, not 53, 100 x 30,000 x 8 50.2, not 49.4.
constexpr int kSplitMinTiles = 8;
constexpr int kSplitMinChunk = 3;
constexpr int kSplitMaxChunks = 64;

__host__ __device__ constexpr int key_tiles(int keys) {
  return keys > 0 ? (keys + kBlockN - 1) / kBlockN : 1;
}

// A chunk of the last wave (or a whole item of it): key tiles [kv0, kv1) of a segment's item.
struct CrossEntry {
  int segment, kv_head, pair, kv0, kv1;
  int first;          // the item's first entry
  int chunk, chunks;  // chunks == 1: whole
};
static_assert(sizeof(CrossEntry) == 8 * sizeof(int32_t), "entries are 8 words");
// first entries of the cut items (fewer than a wave), then the first entry of each CTA and their number
__host__ __device__ constexpr size_t split_items_offset() {
  return static_cast<size_t>(kSplitMaxEntries) * sizeof(CrossEntry);
}
__host__ __device__ constexpr size_t split_partials_offset() {
  return split_items_offset() + static_cast<size_t>(kSplitMaxEntries) * sizeof(uint32_t);
}
template <int D>
constexpr size_t kPartial = static_cast<size_t>(kBlockM) * (D + 1);  // floats of a tile's partial

// Items of a segment per key head: pairs of its group * ceil(rows / 128) tiles.
__device__ __forceinline__ int pairs_of(int rows, int group) {
  return ((rows + kBlockM - 1) / kBlockM * group + 1) / 2;
}

template <typename T>
__device__ __forceinline__ T block_exclusive_scan(T v, T* s_warp, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll 1
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  total = all;
  return before + x - v;
}

// Plan: segment order and item prefix, and the entries of the last wave.  Words of ws: [0] cut
// items, [1] unused, [2] whole items before the last wave, [3] its entries, then the order [S] and the
// exclusive prefix [S + 1].
// The last wave's work is laid end to end and dealt to the CTAs in equal shares, so an item is cut where
// a share ends (four requests of 213 to 292 rows x 12,369 to 13,961 keys x 24 heads, 120 items of about 100
// key tiles on 152 CTAs: 163 us when an item per CTA took 183 us; the same without the heads apart 188 us,
// as each row of K and V then comes from memory in pieces at different times).
__global__ void __launch_bounds__(kPlanThreads)
cross_plan_kernel(const __grid_constant__ CrossSegments seg, uint32_t* __restrict__ ws,
                  uint8_t* __restrict__ split_area, int wave, unsigned int* err) {
  __shared__ int s_rows[kSortMax], s_keys[kSortMax], s_order[kSortMax];
  __shared__ uint32_t s_prefix[kSortMax + 1];
  __shared__ uint32_t s_warp[kPlanThreads / 32];
  __shared__ uint64_t s_warp64[kPlanThreads / 32];
  __shared__ uint32_t s_cut, s_most;
  __shared__ uint2 s_item[kSplitMaxEntries / 2];  // of the last wave: where it starts, its key tiles
  __shared__ uint4 s_at[kSplitMaxEntries / 2];    // of each CTA: where its share starts, cuts before it
  grid_dependency_wait();
  launch_dependents();
  const int S = seg.num_segments, tid = threadIdx.x;
  uint32_t* order = ws + kHeader;
  uint32_t* prefix = ws + kHeader + S;
  const bool sorted = S <= kSortMax;
  const int group = seg.num_q_heads / seg.num_kv_heads;
  if (sorted) {
    if (tid < S) {
      const CrossSegment r = checked_cross_segment(seg, tid, err);
      s_rows[tid] = r.rows;
      s_keys[tid] = r.used;
    }
    __syncthreads();
    if (tid < S) {  // most keys first, ties by position
      int rank = 0;
      for (int h = 0; h < S; ++h)
        rank += s_keys[h] > s_keys[tid] || (s_keys[h] == s_keys[tid] && h < tid);
      s_order[rank] = tid;
    }
    __syncthreads();
  }
  auto items_at = [&](int i) -> uint32_t {  // of the segment in place i
    const int rows = sorted ? s_rows[s_order[i]] : checked_cross_segment(seg, i, err).rows;
    return static_cast<uint32_t>(pairs_of(rows, group)) * seg.num_kv_heads;
  };
  const int chunk = (S + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
  const int lo = min(S, tid * chunk), hi = min(S, lo + chunk);
  uint64_t local = 0, items;
  for (int i = lo; i < hi; ++i) local += items_at(i);
  uint32_t run = static_cast<uint32_t>(block_exclusive_scan(local, s_warp64, items));
  // Segments that overlap can hold more tiles than the capacity (and more than 32 bits count): then no item.
  if (items > (static_cast<uint64_t>(seg.capacity_q) / kBlockM + S) * seg.num_q_heads) {
    if (tid == 0) {
      record_error(err, kErrBadCuSeqlens);
      ws[0] = ws[2] = ws[3] = 0;
    }
    return;
  }
  const uint32_t total = static_cast<uint32_t>(items);
  for (int i = lo; i < hi; ++i) {
    order[i] = static_cast<uint32_t>(sorted ? s_order[i] : i);
    prefix[i] = run;
    if (sorted) s_prefix[i] = run;
    run += items_at(i);
  }
  if (tid == 0) {
    prefix[S] = total;
    if (sorted) s_prefix[S] = total;
  }
  const uint32_t tail = total / wave * wave, R = total - tail;
  if (split_area == nullptr || !sorted || R == 0 || 2 * wave + 1 > kSplitMaxEntries) {
    if (tid == 0) {
      ws[0] = 0;
      ws[2] = total;
      ws[3] = 0;
    }
    return;
  }
  const bool mine = tid < static_cast<int>(R);  // fewer than a wave
  if (tid == 0) s_cut = s_most = 0u;
  __syncthreads();  // also: the prefix is complete
  CrossEntry e{};
  int nkv = 0;
  uint32_t cost = 0;
  // Key heads apart, a group of CTAs each, where no whole wave comes before: then the heads of a segment
  // are cut alike and read the same key rows at the same time (175 us where one space of all heads takes 181 for
  // 213 to 292 rows x 12,369 to 13,961 keys x 24, 49.4 and 50.8 for 100 x 30,000 x 8; eight shorter shapes within 1 %).
  const int heads = seg.num_kv_heads;
  const bool apart = tail == 0 && heads <= wave;
  const int groups = apart ? heads : 1, members = wave / groups;  // of CTAs; CTAs in a group
  const uint32_t per = R / groups;                                // items of a group
  if (mine) {
    const uint32_t item = apart ? tid % per * heads : tail + tid;  // (prefixes count all heads)
    int l = 0, h = S - 1;
    while (l < h) {
      const int mid = (l + h + 1) >> 1;
      if (s_prefix[mid] <= item) l = mid; else h = mid - 1;
    }
    e.segment = s_order[l];
    const int rows = s_rows[e.segment], pairs = pairs_of(rows, group);
    const int loc = static_cast<int>(item - s_prefix[l]);
    e.kv_head = apart ? tid / static_cast<int>(per) : loc / pairs;
    e.pair = apart ? loc / heads : loc % pairs;
    nkv = key_tiles(s_keys[e.segment]);
    cost = static_cast<uint32_t>(nkv) + kCostItem;  // a wave's sum fits 32 bits
    atomicMax(&s_most, cost);
  }
  uint32_t all;
  const uint32_t start = block_exclusive_scan(cost, s_warp, all);  // (its barriers also order s_most)
  if (mine) s_item[tid] = make_uint2(start, static_cast<uint32_t>(nkv));
  __syncthreads();
  // a CTA's share; no cut where whole items end as soon as the shares and their joining would
  const uint32_t whole = all / groups;  // a group's
  uint32_t share = max((whole + members - 1) / members, s_most / (kSplitMaxChunks - 4) + 1);
  share = max(share, 2u * kSplitMinChunk);
  const bool cut = s_most > share + kCostJoin;
  // CTA k starts in item at.x, at its key tile at.y (0: at its start)
  uint2 at = make_uint2(R, 0u);
  const uint32_t from = tid / members * whole, into = share * (tid % members);
  if (tid < groups * members && cut) {
    const uint32_t x = from + min(into, whole);
    int l = 0, h = static_cast<int>(R) - 1;
    while (l < h) {
      const int mid = (l + h + 1) >> 1;
      if (s_item[mid].x <= x) l = mid; else h = mid - 1;
    }
    const uint32_t n = s_item[l].y, j = min(n, x - s_item[l].x);
    const bool inside = n >= static_cast<uint32_t>(kSplitMinTiles) && j >= static_cast<uint32_t>(kSplitMinChunk) &&
                        j + kSplitMinChunk <= n;
    at = inside ? make_uint2(l, j) : make_uint2(2 * j < n ? l : l + 1, 0u);
  } else if (!cut) {
    at.x = min(static_cast<uint32_t>(tid), R);
  }
  uint32_t cuts;
  const uint32_t before = block_exclusive_scan(tid < wave && at.y > 0 ? 1u : 0u, s_warp, cuts);
  uint32_t* listed = reinterpret_cast<uint32_t*>(split_area + split_items_offset());
  if (tid < wave) {
    s_at[tid] = make_uint4(at.x, at.y, before, 0u);
    listed[wave + tid] = at.x + before + (at.y > 0 ? 1u : 0u);
  }
  if (tid == 0) listed[2 * wave] = R + cuts;
  __syncthreads();
  if (mine) {
    // the cuts inside this item, in order: CTAs whose share starts inside it
    uint32_t k = cut ? start / whole * members + start % whole / share : static_cast<uint32_t>(wave);
    while (k < static_cast<uint32_t>(wave) && s_at[k].x < static_cast<uint32_t>(tid)) ++k;
    const uint32_t earlier = k < static_cast<uint32_t>(wave) ? s_at[k].z : (cut ? cuts : 0u);
    uint32_t last = k;
    int c = 1;
    for (; last < static_cast<uint32_t>(wave) && s_at[last].x == static_cast<uint32_t>(tid); ++last)
      c += s_at[last].y > 0;
    const uint32_t first = tid + earlier;
    if (c > 1) listed[atomicAdd(&s_cut, 1u)] = first;  // listed for the merge; the list's order is immaterial
    e.first = static_cast<int>(first);
    e.chunks = c;
    e.kv0 = 0;
    for (e.chunk = 0; e.chunk < c; ++e.chunk, ++k) {
      while (k < last && s_at[k].y == 0) ++k;
      e.kv1 = k < last ? static_cast<int>(s_at[k].y) : nkv;
      reinterpret_cast<CrossEntry*>(split_area)[first + e.chunk] = e;
      e.kv0 = e.kv1;
    }
  }
  __syncthreads();
  if (tid == 0) {
    ws[0] = s_cut;
    ws[2] = tail;
    ws[3] = R + cuts;
  }
}

struct CrossWork {
  int ntiles;           // 0: no more work
  int q0[2], head[2];   // first row and query head of each tile
  int seg_end;
  int kv_row, kv_head;  // first key row of the item's first key tile
  int nkv, last_keys;   // key tiles, and keys in the last of them (0: a segment without keys)
  int partial;          // entry whose partial results the item writes, -1 for o itself
};

__device__ __forceinline__ CrossWork decode(uint32_t item, const uint32_t* __restrict__ ws,
                                            const CrossSegments& seg,
                                            const uint8_t* __restrict__ split_area) {
  const int S = seg.num_segments, group = seg.num_q_heads / seg.num_kv_heads;
  const uint32_t tail = ws[2];
  CrossWork d;
  int g, pair, kv0 = 0, kv1 = -1;
  d.partial = -1;
  if (item >= tail) {
    const CrossEntry e = reinterpret_cast<const CrossEntry*>(split_area)[item - tail];
    g = e.segment;
    pair = e.pair;
    d.kv_head = e.kv_head;
    kv0 = e.kv0;
    kv1 = e.kv1;
    if (e.chunks > 1) d.partial = e.first + e.chunk;
  } else {
    const uint32_t* prefix = ws + kHeader + S;
    int lo = 0, hi = S - 1;  // last i with prefix[i] <= item
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= item) lo = mid; else hi = mid - 1;
    }
    g = static_cast<int>((ws + kHeader)[lo]);
    const int pairs = pairs_of(seg.cu_q[g + 1] - seg.cu_q[g], group);
    const int loc = static_cast<int>(item - prefix[lo]);
    d.kv_head = loc / pairs;
    pair = loc % pairs;
  }
  const int a = seg.cu_q[g];
  d.seg_end = seg.cu_q[g + 1];
  const int per_head = (d.seg_end - a + kBlockM - 1) / kBlockM;
  d.ntiles = min(2, per_head * group - 2 * pair);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int tile = 2 * pair + t;
    d.head[t] = d.kv_head * group + tile / per_head;
    d.q0[t] = a + tile % per_head * kBlockM;
  }
  const int ka = seg.cu_k[g];
  const int keys = seg.seqused_k != nullptr ? seg.seqused_k[g] : seg.cu_k[g + 1] - ka;
  const int all = key_tiles(keys);
  if (kv1 < 0) kv1 = all;
  d.nkv = kv1 - kv0;
  d.last_keys = kv1 == all ? keys - (all - 1) * kBlockN : kBlockN;
  d.kv_row = ka + kv0 * kBlockN;
  return d;
}

template <int D>
struct Cfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBlockM * D * 2;
  static constexpr int kBoxBytes = kBlockM * 128;
  static constexpr int kStages = D == 128 ? 5 : 8;  // key and value tiles in turn
  // q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_final[2], o_empty[2], l_full[2],
  // w_full[2], w_empty[2], drain[2], turn[2], then kv_full, kv_empty, v_tail
  static constexpr int kNumBars = 24 + 3 * kStages;
  static constexpr int kSmemBytes = 1024 + kTileBytes * (2 + kStages) + kNumBars * 8 + 24 +
                                    2 * sizeof(CrossWork) + 2 * kBlockM * sizeof(float);
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(kBlockM, kBlockN, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(kBlockM, D, true);
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, __nv_bfloat16* __restrict__ out, int wide,
                  float* __restrict__ lse, const __grid_constant__ CrossSegments seg, float scale,
                  float scale_log2, const uint32_t* __restrict__ ws, uint8_t* __restrict__ split_area,
                  unsigned int* err, unsigned long long wait_ns, unsigned int stall_after) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + 2 * C::kTileBytes;
  float* s_norm = reinterpret_cast<float*>(sKV + kStages * C::kTileBytes);  // [2][128]: 1 / row sum
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_norm + 2 * kBlockM);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  CrossWork* work = reinterpret_cast<CrossWork*>(tmem_slot + 2);  // 2-slot ring
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * static_cast<uint32_t>(i); };
  auto bar_qfull = [&](int t) { return bar(t); };
  auto bar_qempty = [&](int t) { return bar(2 + t); };
  auto bar_sfull = [&](int t) { return bar(4 + t); };
  auto bar_phalf = [&](int t) { return bar(6 + t); };
  auto bar_pfull = [&](int t) { return bar(8 + t); };
  auto bar_ofinal = [&](int t) { return bar(10 + t); };
  auto bar_oempty = [&](int t) { return bar(12 + t); };
  auto bar_lfull = [&](int t) { return bar(14 + t); };
  auto bar_wfull = [&](int i) { return bar(16 + i); };
  auto bar_wempty = [&](int i) { return bar(18 + i); };
  auto bar_drain = [&](int t) { return bar(20 + t); };
  auto bar_turn = [&](int t) { return bar(22 + t); };
  auto bar_full = [&](int s) { return bar(24 + s); };
  auto bar_empty = [&](int s) { return bar(24 + kStages + s); };
  auto bar_vtail = [&](int s) { return bar(24 + 2 * kStages + s); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto pwait = [&](uint32_t b, uint32_t parity) { return mbar_wait(b, parity, wait_ns); };
  // The whole warp polls: a branch for one lane would leave the warp diverged behind it.
  auto wait_all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, pwait(b, parity)) != 0; };
  auto wait_long = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_long(b, parity, wait_ns)) != 0;
  };
  // One arrival for the warp, after what all its lanes did.
  auto arrive_warp = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };

  grid_dependency_wait();
  launch_dependents();
  // a timeout recorded earlier and not read yet: leave at once, all threads together
  if (__syncthreads_or(err != nullptr && *reinterpret_cast<volatile unsigned int*>(err) == kErrTimeout))
    return;
  // this CTA's items: every gridDim.x-th of the whole ones, then its entries of the last wave
  const uint32_t whole = ws[2];
  uint32_t entry = 0, entry_end = 0;
  if (ws[3] > 0) {
    const uint32_t* firsts = reinterpret_cast<const uint32_t*>(split_area + split_items_offset()) + gridDim.x;
    entry = firsts[blockIdx.x];
    entry_end = firsts[blockIdx.x + 1];
  }
  if (blockIdx.x >= whole && entry == entry_end) return;

  if (warp == 12 && lane == 0) {
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_qfull(t), 1);
      mbar_init(bar_qempty(t), 1);
      mbar_init(bar_sfull(t), 1);
      mbar_init(bar_phalf(t), 4);  // warps
      mbar_init(bar_pfull(t), 4);  // warps
      mbar_init(bar_ofinal(t), 1);
      mbar_init(bar_oempty(t), 4);  // warps
      mbar_init(bar_lfull(t), 4);  // warps
      mbar_init(bar_wfull(t), 1);
      mbar_init(bar_drain(t), 1);
      mbar_init(bar_turn(t), 1);
      mbar_init(bar_wempty(t), 15);  // softmax and epilogue warps, key/value producer, MMA warps
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 2);  // MMA warps
      mbar_init(bar_vtail(s), 1);
    }
    fence_mbarrier_init();
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Item k from the ring, for one warp (every lane calls).  False when the wait ran out.
  auto take = [&](int k, CrossWork& d) {
    if (!wait_long(bar_wfull(k & 1), (k >> 1) & 1)) return false;
    d = work[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_wempty(k & 1));
    return true;
  };

  // An item's last key tile is multiplied as far as it holds keys, in steps of 16 and at least one; value
  // rows past the keys that PV reads all the same are zeroed.
  auto steps16 = [](int keys) { return max(1, (keys + 15) / 16); };
  auto has_tail = [&](int keys) { return keys < 16 * steps16(keys); };

  if (warp >= 12) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == 12) {
      // ================= key/value producer =================
      const uint64_t pol_keep = l2_policy_evict_last();  // shared by the CTAs of a key head
      uint32_t loaded = 0, v_last = 0;  // tiles; the last value tile of an item
      int tail_keys = 0;
      bool ok = true, stalled = false, tail = false;
      CrossWork d;
      // The tail of an item's last value tile, once it has landed: while the next key tile is on its way,
      // before the next value tile.  (Whole 128-byte rows: the swizzle permutes 16-byte pieces within a row.)
      auto zero_tail = [&] {
        if (!tail) return true;
        tail = false;
        const uint32_t s = v_last % kStages;
        if (!wait_long(bar_full(s), (v_last / kStages) & 1)) return false;
        uint8_t* vb = sKV + s * C::kTileBytes;
        for (int i = lane; i < (16 * steps16(tail_keys) - tail_keys) * C::kBoxes * 8; i += 32) {
          const int r = tail_keys + i / (C::kBoxes * 8), rem = i % (C::kBoxes * 8);
          *reinterpret_cast<uint4*>(vb + (rem >> 3) * C::kBoxBytes + r * 128 + (rem & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        arrive_warp(bar_vtail(s));
        return true;
      };
      for (int k = 0; ok && !stalled; ++k) {
        ok = take(k, d);
        if (!ok || d.ntiles == 0) break;
        auto load = [&](uint8_t* dst, const CUtensorMap* map, int row, uint32_t b) {
          if (lane != 0) return;
          mbar_arrive_expect_tx(b, C::kTileBytes);
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_3d_hint(smem_u32(dst + x * C::kBoxBytes), map, x * 64, d.kv_head, row, b, pol_keep);
        };
        for (int j = 0; j < d.nkv; ++j) {
          if (loaded / 2 >= stall_after) {  // testing hook: as if the loads had stalled
            stalled = true;
            break;
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int s = static_cast<int>(loaded % kStages);
            ok = (v == 0 || zero_tail()) && wait_long(bar_empty(s), ((loaded / kStages) & 1) ^ 1);
            if (!ok) break;
            load(sKV + s * C::kTileBytes, v == 0 ? &tmap_k : &tmap_v, d.kv_row + j * kBlockN, bar_full(s));
            ++loaded;
          }
          if (!ok) break;
        }
        tail = ok && !stalled && has_tail(d.last_keys);
        tail_keys = d.last_keys;
        v_last = loaded - 1;
      }
      if (ok && !stalled) ok = zero_tail();
      if (!ok && lane == 0) record_error(err, kErrTimeout);
      // never leave while a copy may still land: the last loads sit on distinct stages
      for (uint32_t i = 0; i < kStages && i < loaded; ++i)
        mbar_wait(bar_full((loaded - 1 - i) % kStages), ((loaded - 1 - i) / kStages) & 1);
    } else if (warp == 15) {
      // ================= scheduler and query producer =================
      const uint64_t pol_stream = l2_policy_evict_first();
      uint32_t qn[2] = {0u, 0u};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const uint32_t item = blockIdx.x + static_cast<uint32_t>(k) * gridDim.x;
        CrossWork d{};
        if (item < whole) d = decode(item, ws, seg, split_area);
        else if (entry < entry_end) d = decode(whole + entry++, ws, seg, split_area);
        ok = wait_long(bar_wempty(k & 1), ((k >> 1) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          work[k & 1] = d;
          mbar_arrive(bar_wfull(k & 1));
        }
        __syncwarp();
        if (d.ntiles == 0) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= d.ntiles) break;
          ok = wait_long(bar_qempty(t), (qn[t] & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar_qfull(t), C::kTileBytes);
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d_hint(smem_u32(sQ + t * C::kTileBytes + x * C::kBoxBytes), &tmap_q, x * 64,
                               d.head[t], d.q0[t], bar_qfull(t), pol_stream);
          }
          ++qn[t];
        }
      }
      if (!ok && lane == 0) record_error(err, kErrTimeout);
      for (int t = 0; t < 2; ++t)
        if (qn[t] > 0) mbar_wait(bar_qfull(t), (qn[t] - 1) & 1);
    } else {
      // ================= MMA issuers: warp 13 for tile 0, 14 for tile 1 =================
      // A warp's polls wait for the products that it has issued before, so the tensor core would run dry at
      // each poll of a single issuer.  Two take turns: what one polls for, it does while the other's products
      // run.  Their order is kept (a turn barrier each), or the tiles would fall in phase.
      const int t = warp - 13;
      constexpr uint32_t kTile16 = C::kTileBytes >> 4;
      const SmemDesc dq = sw128_desc_split(smem_u32(sQ) + t * C::kTileBytes, 16, 1024);
      const SmemDesc dk = sw128_desc_split(smem_u32(sKV), 16, 1024);
      const SmemDesc dv = sw128_desc_split(smem_u32(sKV), C::kBoxBytes, 1024);
      const uint32_t s_tmem = tmem + kColS + 128 * t, o_tmem = tmem + kColO + 128 * t;
      auto issue_qk = [&](int s, uint32_t idesc) {  // S_t = Q_t K_s^T
        const uint32_t klo = dk.lo + s * kTile16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_split(s_tmem, dq.lo + off, dq.hi, klo + off, dk.hi, idesc, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar_sfull(t));
      };
      auto issue_pv = [&](int s, bool first, int from) {  // O_t += P_t V_s over four steps of 16 keys
        const uint32_t vlo = dv.lo + s * kTile16;
#pragma unroll
        for (int kk = from; kk < from + 4; ++kk)
          mma_ts_split(o_tmem, s_tmem + kk * 8, vlo + kk * (2048 >> 4), dv.hi, C::kIdescPV,
                       (!first || kk > 0) ? 1u : 0u);
      };
      const bool leader = elect_one();
      struct Item {  // what is needed of an item here
        int ntiles, nkv, last_keys;
      } cur{0, 0, 0}, nxt{0, 0, 0};
      auto take_item = [&](int k, Item& i) {
        if (!wait_all(bar_wfull(k & 1), (k >> 1) & 1)) return false;
        i = Item{work[k & 1].ntiles, work[k & 1].nkv, work[k & 1].last_keys};
        __syncwarp();
        if (leader) mbar_arrive(bar_wempty(k & 1));
        return true;
      };
      auto idesc_last = [&](const Item& i) {
        return i.last_keys < kBlockN ? idesc_bf16_f32(kBlockM, 16 * steps16(i.last_keys), false) : C::kIdescQK;
      };
      int sk = 0, sv = 1;
      uint32_t pk = 0, pv = 0;  // phases of the stages of the next key and value tile
      uint32_t qp = 0u, pp = 0u, op = 1u, turn = t == 0 ? 1u : 0u;  // phases of Q, P, O and the turns
      uint32_t tails = 0;  // phases of the value tails, a bit per stage
      auto next_k = [&] {
        if ((sk += 2) >= kStages) {
          sk -= kStages;
          pk ^= 1;
        }
      };
      auto next_v = [&] {
        if ((sv += 2) >= kStages) {
          sv -= kStages;
          pv ^= 1;
        }
      };
      // Waits for this warp's turn and whatever else is asked for; the polls overlap.
      auto wait_turn = [&](bool v, bool k, bool q, bool p, uint32_t p_bar, bool o, bool z) {
        bool r[7];
        r[0] = !p || mbar_try_wait(p_bar, pp);
        r[1] = mbar_try_wait(bar_turn(t), turn);
        r[2] = !v || mbar_try_wait(bar_full(sv), pv);
        r[3] = !k || mbar_try_wait(bar_full(sk), pk);
        r[4] = !q || mbar_try_wait(bar_qfull(t), qp);
        r[5] = !o || mbar_try_wait(bar_oempty(t), op);
        r[6] = !z || mbar_try_wait(bar_vtail(sv), tails >> sv & 1u);
        bool all = true;
        if (!r[0]) all = pwait(p_bar, pp);
        if (!r[1]) all = pwait(bar_turn(t), turn) && all;
        if (!r[2]) all = pwait(bar_full(sv), pv) && all;
        if (!r[3]) all = pwait(bar_full(sk), pk) && all;
        if (!r[4]) all = pwait(bar_qfull(t), qp) && all;
        if (!r[5]) all = pwait(bar_oempty(t), op) && all;
        if (!r[6]) all = pwait(bar_vtail(sv), tails >> sv & 1u) && all;
        turn ^= 1;
        if (z) tails ^= 1u << sv;
        if (q) qp ^= 1;
        if (o) op ^= 1;
        return __all_sync(0xffffffffu, all) != 0;
      };
      bool ok = take_item(0, cur), issued = false;
      if (ok && cur.ntiles > 0) {  // the first item's first scores
        ok = wait_all(bar_full(0), 0);
        if (ok && t < cur.ntiles) {
          ok = wait_all(bar_qfull(t), 0);
          qp = 1;
          tc_fence_after();
          if (ok && leader) {
            issue_qk(0, cur.nkv == 1 ? idesc_last(cur) : C::kIdescQK);
            if (cur.nkv == 1) mma_commit(bar_qempty(t));
            mma_commit(bar_empty(0));
          }
          issued = ok;
          __syncwarp();
        } else if (ok && leader) {
          mbar_arrive(bar_empty(0));
        }
        next_k();
      }
      // One step within an item: PV of its key tile, and the scores of the next one.
      auto step = [&](bool first, uint32_t idesc, bool q_done) {
        if (t < cur.ntiles) {
          if (!wait_turn(true, true, false, true, bar_phalf(t), first, false)) return false;
          tc_fence_after();
          if (leader) issue_pv(sv, first, 0);
          __syncwarp();
          if (!wait_all(bar_pfull(t), pp)) return false;
          pp ^= 1;
          tc_fence_after();
          if (leader) issue_pv(sv, false, 4);
          if (leader) {
            mma_commit(bar_empty(sv));
            issue_qk(sk, idesc);
            if (q_done) mma_commit(bar_qempty(t));
            mma_commit(bar_empty(sk));
            mbar_arrive(bar_turn(t ^ 1));
          }
          __syncwarp();
        } else {
          if (!wait_turn(true, true, false, false, 0, false, false)) return false;
          if (leader) {
            mbar_arrive(bar_empty(sv));
            mbar_arrive(bar_empty(sk));
            mbar_arrive(bar_turn(t ^ 1));
          }
          __syncwarp();
        }
        next_v();
        next_k();
        return true;
      };
      // The step between two items: PV of the last key tile, as far as it holds keys, and the next item's
      // first scores.
      auto boundary = [&](bool first) {
        const bool has_pv = t < cur.ntiles, has_qk = t < nxt.ntiles, more = nxt.ntiles > 0;
        const int end = steps16(cur.last_keys);
        const uint32_t idesc = nxt.nkv == 1 ? idesc_last(nxt) : C::kIdescQK;
        if (!wait_turn(true, more, has_qk, has_pv, bar_pfull(t), has_pv && first,
                       has_tail(cur.last_keys))) return false;
        if (has_pv) pp ^= 1;
        tc_fence_after();
        if (has_pv) {
          if (end == kBlockN / 16) {
            if (leader) {
              issue_pv(sv, first, 0);
              issue_pv(sv, false, 4);
            }
          } else if (leader) {
#pragma unroll 1
            for (int kk = 0; kk < end; ++kk)
              mma_ts_split(o_tmem, s_tmem + kk * 8, dv.lo + sv * kTile16 + kk * (2048 >> 4), dv.hi, C::kIdescPV,
                           (!first || kk > 0) ? 1u : 0u);
          }
          if (leader) {
            mma_commit(bar_ofinal(t));
            mma_commit(bar_empty(sv));
          }
        } else if (leader) {
          mbar_arrive(bar_empty(sv));
        }
        __syncwarp();
        if (has_qk) {
          if (leader) {
            issue_qk(sk, idesc);
            if (nxt.nkv == 1) mma_commit(bar_qempty(t));
            mma_commit(bar_empty(sk));
          }
          issued = true;
        } else if (more && leader) {
          mbar_arrive(bar_empty(sk));
        }
        __syncwarp();
        if (leader) mbar_arrive(bar_turn(t ^ 1));
        __syncwarp();
        next_v();
        if (more) next_k();
        return true;
      };
      for (int k = 0; ok && cur.ntiles > 0; ++k) {
        const uint32_t idesc_end = idesc_last(cur);
        for (int j = 0; j + 1 < cur.nkv && ok; ++j) {
          const bool q_done = j + 2 == cur.nkv;
          ok = step(j == 0, q_done ? idesc_end : C::kIdescQK, q_done);
        }
        if (ok) ok = take_item(k + 1, nxt);
        if (ok) ok = boundary(cur.nkv == 1);
        cur = nxt;
      }
      if (!ok && leader) record_error(err, kErrTimeout);
      if (issued && leader) {  // every MMA issued has completed before TMEM is released
        mma_commit(bar_drain(t));
        mbar_wait(bar_drain(t), 0);
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<kRegsEpilogue>();
    // ================= epilogue: O / l -> bf16 rows (or fp32 partials) =================
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t fn[2] = {0u, 0u};
    bool ok = true;
    CrossWork d;
    for (int k = 0; ok; ++k) {
      ok = take(k, d);
      if (!ok || d.ntiles == 0) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t >= d.ntiles) break;
        ok = wait_long(bar_lfull(t), fn[t] & 1);
        if (ok) ok = wait_long(bar_ofinal(t), fn[t] & 1);
        ++fn[t];
        if (!ok) break;
        tc_fence_after();
        const float inv_l = s_norm[t * kBlockM + row];
        const uint32_t o_addr = tmem + lane_base + kColO + 128 * t;
        if (d.partial >= 0) {
          float* mine = reinterpret_cast<float*>(split_area + split_partials_offset()) +
                        (static_cast<size_t>(d.partial) * 2 + t) * kPartial<D> + static_cast<size_t>(row) * D;
          const bool sectors = (reinterpret_cast<uintptr_t>(mine) & 31u) == 0;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(o_addr + c0, r);
            tmem_ld_wait();
            tmem_reg_fence<32>(r);
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * inv_l);
#pragma unroll
            for (int c = 0; c < 32; c += 8) st_global_32(mine + c0 + c, r + c, sectors);
          }
          tc_fence_before();
          arrive_warp(bar_oempty(t));
          continue;
        }
        // Lanes 2i and 2i + 1 trade halves of each 64 bytes, so that an instruction writes whole
        // 32-byte sectors, two neighbours of a row at a time.
        const int odd = lane & 1;
        const int r0 = d.q0[t] + row - odd;  // the even lane's row
        __nv_bfloat16* p0 = out + (static_cast<size_t>(r0) * seg.num_q_heads + d.head[t]) * D + 16 * odd;
        __nv_bfloat16* p1 = p0 + static_cast<size_t>(seg.num_q_heads) * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t r[32], pk[16];
          tmem_ld32(o_addr + c0, r);
          tmem_ld_wait();
          tmem_reg_fence<32>(r);
          if (c0 == D - 32) {
            tc_fence_before();
            arrive_warp(bar_oempty(t));
          }
#pragma unroll
          for (int c = 0; c < 16; ++c)
            pk[c] = pack_bf16x2(__uint_as_float(r[2 * c]) * inv_l, __uint_as_float(r[2 * c + 1]) * inv_l);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? pk[c] : pk[8 + c], 1);
            pk[c] = odd ? got : pk[c];
            pk[8 + c] = odd ? pk[8 + c] : got;
          }
          if (r0 < d.seg_end) st_global_32(p0 + c0, pk, wide);
          if (r0 + 1 < d.seg_end) st_global_32(p1 + c0, pk + 8, wide);
        }
      }
    }
    if (!ok && lane == 0) record_error(err, kErrTimeout);
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ================= softmax (warps 0-3: tile 0, 4-7: tile 1) =================
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kColS + 128 * t;
    const uint32_t o_addr = tmem + lane_base + kColO + 128 * t;
    const float2 c2 = make_float2(scale_log2, scale_log2);
    uint32_t sn = 0, un = 0;  // score tiles and items of this query tile seen
    bool ok = true;
    CrossWork d;
    for (int k = 0; ok; ++k) {
      ok = take(k, d);
      if (!ok || d.ntiles == 0) break;
      if (t >= d.ntiles) continue;
      float m_used = -INFINITY, l = 0.f;
      // New row max: the reference max moves (and l and O_t are rescaled) only when it grows by more
      // than 2^kRescaleLog2.  O_t is stable here: PV_t,{j-1} was issued before the scores whose
      // completion this thread has seen.
      auto update_max = [&](float mx, int j) {
        float alpha = 1.f;
        bool rescale = false;
        if (mx > m_used && (m_used == -INFINITY || (mx - m_used) * scale_log2 > kRescaleLog2)) {
          alpha = ex2_approx((m_used - mx) * scale_log2);
          rescale = j > 0;
          l *= alpha;
          m_used = mx;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(o_addr + c0, r);
            tmem_ld_wait();
            tmem_reg_fence<32>(r);
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * alpha);
            tmem_st32(o_addr + c0, r);
          }
        }
        // a row without keys has no max: its weights are exp2(-inf) = 0
        const float mb = m_used == -INFINITY ? 0.f : m_used * scale_log2;
        return make_float2(-mb, -mb);
      };
      // weights of 64 scores as 32 packed bf16 pairs; acc: four running sums
      auto weights = [&](const uint32_t* s, float2 nm2, float2 (&acc)[4], uint32_t* p) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 x = ffma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), c2, nm2);
          const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          acc[c & 3] = fadd2(acc[c & 3], e);
          p[c] = pack_bf16x2(e.x, e.y);
        }
      };
      for (int j = 0; j < d.nkv; ++j) {
        ok = wait_all(bar_sfull(t), sn++ & 1);
        if (!ok) break;
        tc_fence_after();
        const int keys = j == d.nkv - 1 ? d.last_keys : kBlockN;
        float2 acc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        // row max of columns: four chains of 3-input steps
        auto max_of = [&](const uint32_t* s, int n) {
#pragma unroll
          for (int c = 0; c < n; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              m4[u] = fmax3(m4[u], __uint_as_float(s[c + u]), __uint_as_float(s[c + 4 + u]));
          return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        };
        uint32_t s[128], p[32];
        tmem_ld32(s_addr, s);
        tmem_ld32(s_addr + 32, s + 32);
        if (keys <= 64) {  // a short last tile: half the columns
          tmem_ld_wait();
          tmem_reg_fence<64>(s);
#pragma unroll
          for (int c = 0; c < 64; ++c) s[c] = c < keys ? s[c] : 0xff800000u;
          weights(s, update_max(max_of(s, 64), j), acc, p);
          tmem_st32(s_addr, p);
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(bar_phalf(t));
        } else {
          tmem_ld32(s_addr + 64, s + 64);
          tmem_ld32(s_addr + 96, s + 96);
          tmem_ld_wait();
          tmem_reg_fence<128>(s);
          if (keys < kBlockN) {  // keys past the end: by select, so NaN/Inf there is discarded
#pragma unroll
            for (int c = 64; c < 128; ++c) s[c] = c < keys ? s[c] : 0xff800000u;
          }
          const float2 nm2 = update_max(max_of(s, 128), j);
          weights(s, nm2, acc, p);
          tmem_st32(s_addr, p);
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(bar_phalf(t));
          weights(s + 64, nm2, acc, p);
          tmem_st32(s_addr + 32, p);
          tmem_st_wait();
          tc_fence_before();
        }
        arrive_warp(bar_pfull(t));
        const float2 a01 = fadd2(acc[0], acc[1]), a23 = fadd2(acc[2], acc[3]);
        l += (a01.x + a01.y) + (a23.x + a23.y);
      }
      if (!ok) break;
      // hand the row's norm to the epilogue, once it has read the previous item's
      if (un > 0) ok = wait_all(bar_oempty(t), (un - 1) & 1);
      if (!ok) break;
      ++un;
      s_norm[t * kBlockM + row] = l == 0.f ? 0.f : 1.f / l;
      arrive_warp(bar_lfull(t));
      const float lse_row = m_used * scale + logf(l);  // -inf without keys
      const int q_row = d.q0[t] + row;
      if (d.partial >= 0)
        (reinterpret_cast<float*>(split_area + split_partials_offset()) +
         (static_cast<size_t>(d.partial) * 2 + t) * kPartial<D>)[static_cast<size_t>(kBlockM) * D + row] = lse_row;
      else if (lse != nullptr && q_row < d.seg_end)
        lse[static_cast<size_t>(d.head[t]) * seg.capacity_q + q_row] = lse_row;
    }
    if (!ok && lane == 0) record_error(err, kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of cut items, in chunk order: lse = log sum_c exp(lse_c), o = sum_c exp(lse_c - lse) o_c.
// A unit is 16 rows of one tile; memory-bound and short (the partials are in L2).
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 16;
static_assert(kMergeThreads == 16 * kMergeRows, "16 lanes to a row");
constexpr int kMergeUnits = 2 * (kBlockM / kMergeRows);
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
cross_merge_kernel(const uint32_t* __restrict__ ws, const uint8_t* __restrict__ split_area,
                   __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                   const __grid_constant__ CrossSegments seg, const unsigned int* err) {
  __shared__ float s_w[kMergeRows][kSplitMaxChunks];
  grid_dependency_wait();
  launch_dependents();
  // after a timeout the partials are incomplete: leave the output as it is
  if (err != nullptr && *reinterpret_cast<const volatile unsigned int*>(err) == kErrTimeout) return;
  const int n_units = static_cast<int>(ws[0]) * kMergeUnits;
  const uint32_t* items = reinterpret_cast<const uint32_t*>(split_area + split_items_offset());
  const float* parts = reinterpret_cast<const float*>(split_area + split_partials_offset());
  const int group = seg.num_q_heads / seg.num_kv_heads;
  for (int unit = blockIdx.x; unit < n_units; unit += gridDim.x) {
    const int e = static_cast<int>(items[unit / kMergeUnits]);
    const int t = unit % kMergeUnits / (kBlockM / kMergeRows);
    const int r0 = unit % (kBlockM / kMergeRows) * kMergeRows;
    const CrossEntry en = reinterpret_cast<const CrossEntry*>(split_area)[e];
    const int a = seg.cu_q[en.segment], seg_end = seg.cu_q[en.segment + 1];
    const int per_head = (seg_end - a + kBlockM - 1) / kBlockM, tile = 2 * en.pair + t;
    const int head = en.kv_head * group + tile / per_head;
    const int row0 = a + tile % per_head * kBlockM + r0;
    if (tile >= per_head * group || row0 >= seg_end) continue;  // the whole CTA
    auto part = [&](int ch) { return parts + (static_cast<size_t>(e + ch) * 2 + t) * kPartial<D>; };
    __syncthreads();  // the previous unit's weights have been used
    {  // 16 lanes to a row
      const int r = threadIdx.x / 16, lane16 = threadIdx.x % 16;
      float mx = -INFINITY, den = 0.f;
      for (int ch = lane16; ch < en.chunks; ch += 16) {
        const float v = part(ch)[static_cast<size_t>(kBlockM) * D + r0 + r];
        s_w[r][ch] = v;
        mx = fmaxf(mx, v);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float base = mx == -INFINITY ? 0.f : mx;  // no chunk has weights: o is 0, the LSE -inf
      for (int ch = lane16; ch < en.chunks; ch += 16) den += __expf(s_w[r][ch] - base);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      const float all = base + logf(den);
      for (int ch = lane16; ch < en.chunks; ch += 16) s_w[r][ch] = den == 0.f ? 0.f : __expf(s_w[r][ch] - all);
      if (lane16 == 0 && lse != nullptr && row0 + r < seg_end)
        lse[static_cast<size_t>(head) * seg.capacity_q + row0 + r] = all;
    }
    __syncthreads();
    for (int u = threadIdx.x; u < kMergeRows * (D / 8); u += kMergeThreads) {
      const int r = u / (D / 8), c = u % (D / 8) * 8;
      if (row0 + r >= seg_end) continue;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int ch = 0; ch < en.chunks; ++ch) {
        const float4* src = reinterpret_cast<const float4*>(part(ch) + static_cast<size_t>(r0 + r) * D + c);
        const float4 x = src[0], y = src[1];
        const float w = s_w[r][ch];
        acc[0] = fmaf(w, x.x, acc[0]);
        acc[1] = fmaf(w, x.y, acc[1]);
        acc[2] = fmaf(w, x.z, acc[2]);
        acc[3] = fmaf(w, x.w, acc[3]);
        acc[4] = fmaf(w, y.x, acc[4]);
        acc[5] = fmaf(w, y.y, acc[5]);
        acc[6] = fmaf(w, y.z, acc[6]);
        acc[7] = fmaf(w, y.w, acc[7]);
      }
      *reinterpret_cast<uint4*>(out + (static_cast<size_t>(row0 + r) * seg.num_q_heads + head) * D + c) =
          make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                     pack_bf16x2(acc[6], acc[7]));
    }
  }
}

template <int D>
cudaError_t launch(const CrossArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  cudaError_t e = allow_shared_memory<C::kSmemBytes>(cross_attn_kernel<D>);
  if (e != cudaSuccess) return e;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  uint32_t* ws = static_cast<uint32_t*>(a.workspace);
  uint8_t* split = static_cast<uint8_t*>(a.split_area);
  e = launch_programmatic(cross_plan_kernel, dim3(1), dim3(a.seg.num_segments <= kSortMax ? kSortMax : kPlanThreads), 0,
                          stream, a.seg, ws, split, sms, a.err);
  if (e != cudaSuccess) return e;
  e = launch_programmatic(cross_attn_kernel<D>, dim3(sms), dim3(kThreads), C::kSmemBytes, stream, a.tmap_q,
                          a.tmap_k, a.tmap_v, static_cast<__nv_bfloat16*>(a.o), a.wide, a.lse, a.seg, a.scale,
                          a.scale * 1.4426950408889634f, static_cast<const uint32_t*>(ws), split, a.err,
                          static_cast<unsigned long long>(a.wait_limit_ns), a.stall_after_tiles);
  if (e != cudaSuccess) return e;
  if (split != nullptr)
    e = launch_programmatic(cross_merge_kernel<D>, dim3(8 * sms), dim3(kMergeThreads), 0, stream,
                            static_cast<const uint32_t*>(ws), static_cast<const uint8_t*>(split),
                            static_cast<__nv_bfloat16*>(a.o), a.lse, a.seg,
                            static_cast<const unsigned int*>(a.err));
  return e;
}

}  // namespace

cudaError_t launch_cross_attn(const CrossArgs& a, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace h3
