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

#include "attn_tile.cuh"
#include "cross_segments.cuh"
#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kPlanThreads = 1024;   // at most: kSortMax when the segments are that few
// Segments are ordered by keys, and the last wave cut, up to this count (the ordering compares all pairs).
// Segments of 200 rows and 64, 200 or 4,000 keys x 8 heads: 256 of them 348 us (106 ns a key tile), 257 478 us (145).
constexpr int kSortMax = 256;
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

// A chunk of the last wave (or a whole item of it): key tiles [kv0, kv1) of a segment's item.
struct TileEntry {
  int segment, kv_head, pair, kv0, kv1;
  int first;          // the item's first entry
  int chunk, chunks;  // chunks == 1: whole
};
static_assert(sizeof(TileEntry) == 8 * sizeof(int32_t), "entries are 8 words");

// Items of a segment per key head: pairs of its group * ceil(rows / 128) tiles.
__device__ __forceinline__ int pairs_of(int rows, int group) {
  return ((rows + kBlockM - 1) / kBlockM * group + 1) / 2;
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
  TileEntry e{};
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
  uint32_t* listed = reinterpret_cast<uint32_t*>(split_area + split_items_offset<TileEntry>());
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
      reinterpret_cast<TileEntry*>(split_area)[first + e.chunk] = e;
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

template <int kD>
struct CrossSource {
  static constexpr int kDim = kD, kChunks = kSplitMaxChunks;
  static constexpr bool kConvert = false, kRowLimits = false;
  using Entry = TileEntry;
  CUtensorMap tmap_q, tmap_k, tmap_v;
  CrossSegments seg;

  struct Work {
    int ntiles;           // 0: no more work
    int q0[2], head[2];   // first row and query head of each tile
    int seg_end;
    int kv_row, kv_head;  // first key row of the item's first key tile
    int nkv, last_keys;   // key tiles, and keys in the last of them (0: a segment without keys)
    int partial;          // entry whose partial results the item writes, -1 for o itself
    __device__ __forceinline__ int q_head(int t) const { return head[t]; }
  };

  __device__ __forceinline__ uint32_t q_bytes() const { return kBlockM * kD * 2; }
  __device__ static __forceinline__ uint32_t whole_item(uint32_t k) { return blockIdx.x + k * gridDim.x; }
  __device__ static __forceinline__ TileRow row(int r) { return TileRow{r, 0}; }
  __device__ static __forceinline__ int row_keys(const Work&, int, TileRow) { return 0; }  // all of them

  __device__ __forceinline__ Work decode(uint32_t item, const uint32_t* __restrict__ ws,
                                         const uint8_t* __restrict__ split_area) const {
    const int S = seg.num_segments, group = seg.num_q_heads / seg.num_kv_heads;
    const uint32_t tail = ws[2];
    Work d;
    int g, pair, kv0 = 0, kv1 = -1;
    d.partial = -1;
    if (item >= tail) {
      const TileEntry e = reinterpret_cast<const TileEntry*>(split_area)[item - tail];
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
  __device__ __forceinline__ TilePlace place(const TileEntry& en, int t) const {
    const int group = seg.num_q_heads / seg.num_kv_heads;
    const int a = seg.cu_q[en.segment], end = seg.cu_q[en.segment + 1];
    const int per_head = (end - a + kBlockM - 1) / kBlockM, tile = 2 * en.pair + t;
    return TilePlace{tile < per_head * group, a + tile % per_head * kBlockM, en.kv_head * group + tile / per_head, end};
  }

  struct Fetch {
    __device__ __forceinline__ Fetch(const CrossSource&, const Work&) {}
    // Key (value) tile j of an item into a stage.
    __device__ __forceinline__ void tile(const CrossSource& s, const Work& d, int j, int v, uint8_t* dst, uint8_t*,
                                         uint32_t bar, uint64_t policy, unsigned int*) {
      if ((threadIdx.x & 31) != 0) return;
      mbar_arrive_expect_tx(bar, kBlockN * kD * 2);
      for (int x = 0; x < kD / 64; ++x)
        tma_load_3d_hint(smem_u32(dst + x * kBlockN * 128), v == 0 ? &s.tmap_k : &s.tmap_v, x * 64, d.kv_head,
                         d.kv_row + j * kBlockN, bar, policy);
    }
  };
};

template <int D>
cudaError_t launch(const CrossArgs& a, cudaStream_t stream) {
  using Source = CrossSource<D>;
  using C = TileCfg<Source>;
  cudaError_t e = allow_shared_memory<C::kSmemBytes>(attn_tile_kernel<Source>);
  if (e != cudaSuccess) return e;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  uint32_t* ws = static_cast<uint32_t*>(a.workspace);
  uint8_t* split = static_cast<uint8_t*>(a.split_area);
  e = launch_programmatic(cross_plan_kernel, dim3(1), dim3(a.seg.num_segments <= kSortMax ? kSortMax : kPlanThreads), 0,
                          stream, a.seg, ws, split, sms, a.err);
  if (e != cudaSuccess) return e;
  const Source src{a.tmap_q, a.tmap_k, a.tmap_v, a.seg};
  e = launch_programmatic(attn_tile_kernel<Source>, dim3(sms), dim3(kTileThreads), C::kSmemBytes, stream, src,
                          static_cast<__nv_bfloat16*>(a.o), a.wide, a.lse, a.scale, a.scale * 1.4426950408889634f,
                          static_cast<const uint32_t*>(ws), split, a.err,
                          static_cast<unsigned long long>(a.wait_limit_ns), a.stall_after_tiles);
  if (e != cudaSuccess) return e;
  if (split != nullptr)
    e = launch_programmatic(attn_tile_merge_kernel<Source>, dim3(8 * sms), dim3(kMergeThreads), 0, stream,
                            static_cast<const uint32_t*>(ws), static_cast<const uint8_t*>(split),
                            static_cast<__nv_bfloat16*>(a.o), a.lse, src, static_cast<const unsigned int*>(a.err));
  return e;
}

}  // namespace

cudaError_t launch_cross_attn(const CrossArgs& a, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace h3
