// Attention of chunks of new tokens over a paged cache, on the tile kernel of attn_tile.cuh (TMA + tcgen05 + TMEM).
//
//   S = scale q k^T over the keys that a row sees,  P = softmax(S),  o = P v,  lse = log sum exp(S)
//
// A 128-row query tile holds 128 / group tokens with all the query heads that share a key head, so a chunk of a few
// tokens fills a tile and every key is read once for the whole group.  An item is two consecutive tiles of a
// (segment, key head); both stream the same 128-key tiles, which a key/value producer gathers from pages: each of its
// lanes looks up one page of the tile, a tile ahead, and issues that page's copy.  An e4m3 tile arrives as bytes
// with its rows' scales, and the epilogue's warps, idle between items, turn it into bf16 in shared memory (exactly);
// the products and the softmax then are those of a bf16 cache.
//
// P is rounded to bf16 for the tensor core (half a step, 2^-8 of itself at most); scores, running max and sum, and O
// stay fp32, and the result is rounded to bf16 once.
//
// What it measured: 2,000 rows over 58,758 bf16 tokens, causal by frame, 24 heads x 128, 873 us on a cool GPU (1,650
// TFLOP/s) and up to 1,020 at the power cap on a warm one, as the packed kernel; first chunks of 900 to 4,096 tokens, 24 heads on 8 x 64, 78 us, of which
// the plan is 6 and the join 8.  Two chunks of 1,000 to 1,500 rows over 14,000 to 24,000 e4m3 tokens, 40 heads x 128,
// took 1,025 us converted as they are read: shared memory's bandwidth bounds that, for a step of 2,700 cycles moves the
// operands of the products (1,536 cycles of 128 bytes), the arriving bytes (256) and the conversion's reads and writes
// (768); without the conversion it took 667 us, without its arithmetic 828, with a second converting warpgroup 1,338.
// Where an item's keys are converted more than twice the host has them unpacked first (842 us; some 200 are the
// unpacking, at the rate of a plain copy), and this file sees a bf16 cache.
//
// Causal by blocks of tokens: an item's key tiles end at its last row's limit, a tile in which some row sees less is
// masked row by row, others are not.  Items come with the longest first and waves alternate in direction, so the
// CTAs' sums stay near one another; what a last, partly filled wave and unlike items leave idle is evened out by
// cutting that wave's items where each CTA's share of the whole ends.
#include <cuda_bf16.h>

#include "attn_tile.cuh"
#include "h3_internal.h"
#include "launch.h"
#include "paged_segments.cuh"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kSegments = 256;   // whose lengths the plan keeps in shared memory
constexpr int kSorted = 1024;    // pairs of tiles that are ordered by length (the ordering compares all of them)
constexpr int kWave = kSplitMaxEntries / 2;  // CTAs, at most
// In steps of a key tile, as measured for cross attention: an item's start and end, joining chunks; items cut at
// all, least chunk.
constexpr uint32_t kCostItem = 2, kCostJoin = 8;
constexpr int kSplitMinTiles = 8, kSplitMinChunk = 3;
constexpr int kMaxChunks = 160;  // of an item: one for each CTA

__device__ __forceinline__ int tiles_of(int rows, int tokens) { return (rows + tokens - 1) / tokens; }
__device__ __forceinline__ int pairs_of(int rows, int tokens) { return (tiles_of(rows, tokens) + 1) / 2; }

// Whole item k of CTA c of `ctas`: the waves alternate in direction.
__device__ __forceinline__ uint32_t item_of(uint32_t k, uint32_t c, uint32_t ctas) {
  return k * ctas + (k & 1 ? ctas - 1 - c : c);
}

// A pair of query tiles of a segment, and the keys that its last row sees.  Item i is head i % heads of pair
// i / heads of the plan's list.
static_assert(sizeof(PagedPair) == 8 * sizeof(int32_t), "whole vectors");
__device__ __forceinline__ PagedPair pair_of(const PagedSegment& s, int segment, int pair, int tokens, int block) {
  const int64_t end = static_cast<int64_t>(2 * pair + 2) * tokens;
  const int keys = row_limit(s, (end < s.rows ? static_cast<int>(end) : s.rows) - 1, block);
  return PagedPair{segment, s.q0 + 2 * pair * tokens, s.q0 + s.rows, s.used, keys,
                   min(2, tiles_of(s.rows, tokens) - 2 * pair), 0, 0};
}
struct PagedEntry {
  PagedPair pair;
  int kv_head, kv0, kv1;
  int first;          // the item's first entry
  int chunk, chunks;  // chunks == 1: whole
  int unused[2];
};
static_assert(sizeof(PagedEntry) <= kPagedEntryBytes, "the host makes room for them");

// Exclusive prefix of v over the block's threads, and the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  const T mine = lane < warps ? s_warp[lane] : 0;
  T w = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  return __shfl_sync(0xffffffffu, w - mine, warp) + x - v;
}

// Plan: the list of pairs, the longest first (up to kSorted of them; else segment by segment), and the entries of the
// last wave.  Words of ws: [0] cut items, [1] unused, [2] whole items before the last wave, [3] its entries; the list
// lies behind them.
__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(const __grid_constant__ PagedSegments seg, int tokens, uint32_t* __restrict__ ws,
                  PagedPair* __restrict__ list, uint8_t* __restrict__ split_area, int wave, unsigned int* err) {
  __shared__ PagedSegment s_seg[kSegments];
  __shared__ int s_first[kSegments];  // pairs before a segment's
  __shared__ __align__(16) uint32_t s_tiles[kSorted];  // key tiles of a pair, by its place in the segments
  __shared__ uint32_t s_sorted[kSorted];               // the same in the list's order
  __shared__ uint64_t s_warp64[32];
  __shared__ uint32_t s_warp[32];
  __shared__ uint32_t s_cut, s_most, s_uncut, s_top;
  __shared__ uint2 s_item[kWave];     // of the last wave: where it starts, its key tiles
  __shared__ uint32_t s_load[kWave];  // of each CTA before the last wave
  __shared__ uint2 s_at[kWave];       // of each CTA: the item in which its share starts, cuts before it
  __shared__ uint32_t s_tile[kWave];  // the cuts: key tile
  if (threadIdx.x == 0) s_cut = s_most = s_uncut = s_top = 0u;
  grid_dependency_wait();
  launch_dependents();
  const int S = seg.num_segments, tid = threadIdx.x, threads = blockDim.x;
  const uint32_t heads = seg.num_kv_heads;
  // ---- the pairs of each segment
  const int chunk = (S + threads - 1) / threads;  // segments of a thread: one each up to kSegments
  const int lo = min(S, tid * chunk), hi = min(S, lo + chunk);
  uint64_t local = 0, all;
  for (int g = lo; g < hi; ++g) {
    const PagedSegment s = checked_paged_segment(seg, g, err);
    local += pairs_of(s.rows, tokens);
    if (S <= kSegments) s_seg[g] = s;
  }
  const uint64_t before = block_scan(local, s_warp64, &all);
  // Segments that overlap can hold more tiles than the capacity (and more than 32 bits count): then no item.
  if (all > static_cast<uint64_t>(paged_max_pairs(seg.capacity_q, S, tokens))) {
    if (tid == 0) {
      record_error(err, kErrBadCuSeqlens);
      ws[0] = ws[2] = ws[3] = 0;
    }
    return;
  }
  const uint32_t n = static_cast<uint32_t>(all), total = n * heads;
  const bool sorted = n <= kSorted && S <= kSegments;
  if (S <= kSegments) {
    if (tid < S) s_first[tid] = static_cast<int>(before);
    __syncthreads();
    for (uint32_t i = tid; i < n; i += threads) {
      int l = 0, h = S - 1;  // the last segment that starts at i or before
      while (l < h) {
        const int mid = (l + h + 1) >> 1;
        if (static_cast<uint32_t>(s_first[mid]) <= i) l = mid; else h = mid - 1;
      }
      const int pair = pairs_of(s_seg[l].rows, tokens) - 1 - static_cast<int>(i - s_first[l]);  // the last one first
      const PagedPair p = pair_of(s_seg[l], l, pair, tokens, seg.causal_block);
      if (sorted) s_tiles[i] = key_tiles(p.keys);
      else list[i] = p;
    }
  } else {
    uint32_t i = static_cast<uint32_t>(before);
    for (int g = lo; g < hi; ++g) {
      const PagedSegment s = checked_paged_segment(seg, g, nullptr);
      for (int pair = pairs_of(s.rows, tokens) - 1; pair >= 0; --pair)
        list[i++] = pair_of(s, g, pair, tokens, seg.causal_block);
    }
  }
  if (sorted) {  // a pair's place: those that are longer, and those as long that come before
    for (uint32_t i = n + tid; i < (n + 3) / 4 * 4; i += threads) s_tiles[i] = 0u;
    __syncthreads();
    for (uint32_t i = tid; i < n; i += threads) {
      const uint32_t mine = s_tiles[i];
      uint32_t rank = 0;
      for (uint32_t j = 0; j < n; j += 4) {
        const uint4 t = *reinterpret_cast<const uint4*>(s_tiles + j);
        rank += (t.x > mine || (t.x == mine && j < i)) + (t.y > mine || (t.y == mine && j + 1 < i)) +
                (t.z > mine || (t.z == mine && j + 2 < i)) + (t.w > mine || (t.w == mine && j + 3 < i));
      }
      int l = 0, h = S - 1;
      while (l < h) {
        const int mid = (l + h + 1) >> 1;
        if (static_cast<uint32_t>(s_first[mid]) <= i) l = mid; else h = mid - 1;
      }
      const int pair = pairs_of(s_seg[l].rows, tokens) - 1 - static_cast<int>(i - s_first[l]);
      list[rank] = pair_of(s_seg[l], l, pair, tokens, seg.causal_block);
      s_sorted[rank] = mine;
    }
  }
  const uint32_t waves = total / wave, tail = waves * wave, R = total - tail;
  if (split_area == nullptr || R == 0 || 2 * wave + 1 > kSplitMaxEntries) {
    if (tid == 0) {
      ws[0] = 0;
      ws[2] = total;
      ws[3] = 0;
    }
    return;
  }
  __syncthreads();  // the list is complete (written by this CTA: the barrier makes it visible here)
  auto tiles_at = [&](uint32_t item) -> uint32_t {
    return sorted ? s_sorted[item / heads] : key_tiles(list[item / heads].keys);
  };
  uint32_t load = 0;
  if (tid < wave) {
    for (uint32_t w = 0; w < waves; ++w) load += tiles_at(item_of(w, tid, wave)) + kCostItem;
    s_load[tid] = load;
    atomicMax(&s_top, load);
  }
  // Behind an odd number of waves the CTAs' loads fall with their number reversed, so the items come reversed too.
  const bool reversed = waves & 1;
  const bool mine = tid < static_cast<int>(R);  // fewer than a wave
  const uint32_t item = tail + (reversed ? R - 1 - tid : tid);
  uint32_t nkv = 0, cost = 0;
  if (mine) {
    nkv = tiles_at(item);
    cost = nkv + kCostItem;  // a wave's sum fits 32 bits
    atomicMax(&s_most, cost);
  }
  // (two sums in one: the costs, and above them the loads; its barriers also order s_most, s_top and s_load)
  uint64_t sums;
  const uint32_t start =
      static_cast<uint32_t>(block_scan(static_cast<uint64_t>(tid < wave ? load : 0u) << 32 | cost, s_warp64, &sums));
  const uint32_t rest = static_cast<uint32_t>(sums), before_all = static_cast<uint32_t>(sums >> 32);
  if (mine) {
    s_item[tid] = make_uint2(start, nkv);
    atomicMax(&s_uncut, cost + s_load[reversed ? wave - static_cast<int>(R) + tid : tid]);
  }
  __syncthreads();
  // a CTA's share fills it up to the mean; no cut where whole items end as soon as the shares and their joining would
  const uint32_t target = (rest + before_all + wave - 1) / wave;
  const bool cut = s_uncut > max(target, s_top) + kCostJoin;
  uint32_t share = 0;
  if (tid < wave && load < target)
    share = max(max(target - load, 2u * kSplitMinChunk), s_most / (kMaxChunks - 4) + 1);
  uint32_t shares;
  const uint32_t from = block_scan(share, s_warp, &shares);
  // CTA k starts in item at.x, at its key tile at.y (0: at its start)
  uint2 at = make_uint2(R, 0u);
  if (tid < wave && cut) {
    if (from < rest) {
      int l = 0, h = static_cast<int>(R) - 1;
      while (l < h) {
        const int mid = (l + h + 1) >> 1;
        if (s_item[mid].x <= from) l = mid; else h = mid - 1;
      }
      const uint32_t m = s_item[l].y, j = min(m, from - s_item[l].x);
      const bool inside = m >= static_cast<uint32_t>(kSplitMinTiles) && j >= static_cast<uint32_t>(kSplitMinChunk) &&
                          j + kSplitMinChunk <= m;
      at = inside ? make_uint2(l, j) : make_uint2(2 * j < m ? l : l + 1, 0u);
    }
    if (tid == 0) at = make_uint2(0u, 0u);
  } else if (!cut) {
    const int first = reversed ? max(0, tid - (wave - static_cast<int>(R))) : tid;
    at.x = min(static_cast<uint32_t>(first), R);
  }
  // CTAs without a share start where the next one does: one of them stands for the cut there
  const bool counts = tid < wave && at.y > 0 && share > 0;
  uint32_t cuts;
  const uint32_t earlier_cuts = block_scan(counts ? 1u : 0u, s_warp, &cuts);
  uint32_t* listed = reinterpret_cast<uint32_t*>(split_area + split_items_offset<PagedEntry>());
  if (tid < wave) {
    s_at[tid] = make_uint2(at.x, earlier_cuts);
    if (counts) s_tile[earlier_cuts] = at.y;
    listed[wave + tid] = at.x + earlier_cuts + (at.y > 0 ? 1u : 0u);  // (the cut where it starts, whoever stands for it)
  }
  if (tid == 0) listed[2 * wave] = R + cuts;
  __syncthreads();
  // Cuts in the items before item i: those before the first CTA that starts in it or behind.
  auto cuts_before = [&](uint32_t i) {
    int l = 0, h = wave;
    while (l < h) {
      const int mid = (l + h) >> 1;
      if (s_at[mid].x < i) l = mid + 1; else h = mid;
    }
    return l < wave ? s_at[l].y : cuts;
  };
  // An entry: chunk `chunk` of item i of the last wave, whose cuts are [c0, c1).
  auto write_entry = [&](uint32_t i, uint32_t c0, uint32_t c1, uint32_t chunk, uint32_t tiles) {
    const uint32_t of = tail + (reversed ? R - 1 - i : i);
    PagedEntry e{};
    e.pair = list[of / heads];
    e.kv_head = static_cast<int>(of % heads);
    e.first = static_cast<int>(i + c0);
    e.chunk = static_cast<int>(chunk);
    e.chunks = static_cast<int>(1 + c1 - c0);
    e.kv0 = chunk == 0 ? 0 : static_cast<int>(s_tile[c0 + chunk - 1]);
    e.kv1 = c0 + chunk < c1 ? static_cast<int>(s_tile[c0 + chunk]) : static_cast<int>(tiles);
    reinterpret_cast<PagedEntry*>(split_area)[i + c0 + chunk] = e;
  };
  if (mine) {
    const uint32_t c0 = cuts_before(tid), c1 = cuts_before(tid + 1);
    if (c1 > c0) listed[atomicAdd(&s_cut, 1u)] = tid + c0;  // for the merge; the list's order is immaterial
    write_entry(tid, c0, c1, 0, nkv);
  }
  if (counts) {
    const uint32_t c0 = cuts_before(at.x);
    write_entry(at.x, c0, cuts_before(at.x + 1), earlier_cuts - c0 + 1, s_item[at.x].y);
  }
  __syncthreads();
  if (tid == 0) {
    ws[0] = s_cut;
    ws[2] = tail;
    ws[3] = R + cuts;
  }
}

template <int kD, bool kE4m3>
struct PagedSource {
  static constexpr int kDim = kD, kChunks = kMaxChunks;
  static constexpr bool kConvert = kE4m3, kRowLimits = true;
  using Entry = PagedEntry;
  CUtensorMap tmap_q, tmap_k, tmap_v;
  PagedSegments seg;
  const PagedPair* list;
  const uint8_t *k_scale, *v_scale;
  int group, tokens;  // query heads of a key head, tokens of a tile

  struct Work {
    int ntiles;          // 0: no more work
    int q0[2];           // first row of each tile
    int seg_end, head;   // the segment's last row + 1, the key head's first query head
    int segment, kv_head;
    int kv0;             // the item's first key tile
    int nkv, last_keys;  // key tiles, and keys in the last of them (0: rows that see no key)
    int used;            // tokens of the segment
    int partial;         // entry whose partial results the item writes, -1 for o itself
    __device__ __forceinline__ int q_head(int) const { return head; }
  };

  __device__ __forceinline__ uint32_t q_bytes() const { return tokens * group * kD * 2; }
  __device__ static __forceinline__ uint32_t whole_item(uint32_t k) { return item_of(k, blockIdx.x, gridDim.x); }
  __device__ __forceinline__ TileRow row(int r) const {
    return TileRow{r < tokens * group ? r / group : 1 << 29, r % group};
  }
  __device__ __forceinline__ int row_keys(const Work& d, int t, TileRow r) const {
    const int rows = d.seg_end - (d.q0[t] + r.token);  // from this one to the segment's last
    return row_limit(PagedSegment{0, rows, d.used}, 0, seg.causal_block) - d.kv0 * kBlockN;
  }

  __device__ __forceinline__ Work decode(uint32_t item, const uint32_t* __restrict__ ws,
                                         const uint8_t* __restrict__ split_area) const {
    const uint32_t tail = ws[2], heads = seg.num_kv_heads;
    Work d;
    PagedPair p;
    int kv1 = -1;
    d.kv0 = 0;
    d.partial = -1;
    if (item >= tail) {
      const PagedEntry e = reinterpret_cast<const PagedEntry*>(split_area)[item - tail];
      p = e.pair;
      d.kv_head = e.kv_head;
      d.kv0 = e.kv0;
      kv1 = e.kv1;
      if (e.chunks > 1) d.partial = e.first + e.chunk;
    } else {
      p = list[item / heads];
      d.kv_head = static_cast<int>(item % heads);
    }
    d.segment = p.segment;
    d.seg_end = p.seg_end;
    d.used = p.used;
    d.head = d.kv_head * group;
    d.ntiles = p.ntiles;
    d.q0[0] = p.q0;
    d.q0[1] = p.q0 + tokens;
    const int all = key_tiles(p.keys);
    if (kv1 < 0) kv1 = all;
    d.nkv = kv1 - d.kv0;
    d.last_keys = kv1 == all ? p.keys - (all - 1) * kBlockN : kBlockN;
    return d;
  }

  __device__ __forceinline__ TilePlace place(const PagedEntry& e, int t) const {
    return TilePlace{t < e.pair.ntiles, e.pair.q0 + t * tokens, e.kv_head * group, e.pair.seg_end};
  }

  // The key/value producer: lane i has page i of a key tile, looked up a tile ahead.
  struct Fetch {
    int shift, rows;  // log2 of a page, its rows in a tile
    int id, next;     // this lane's page of the current tile and the next one
    __device__ __forceinline__ int pages(const Work& d, int j) const {
      const int keys = j == d.nkv - 1 ? d.last_keys : kBlockN;
      return (keys + rows - 1) / rows;
    }
    __device__ __forceinline__ int look(const PagedSource& s, const Work& d, int j) const {
      const int lane = threadIdx.x & 31;
      if (j >= d.nkv || lane >= pages(d, j)) return 0;
      return page_id(s.seg.table, d.segment, ((d.kv0 + j) * kBlockN >> shift) + lane);
    }
    __device__ __forceinline__ Fetch(const PagedSource& s, const Work& d)
        : shift(s.seg.table.page_shift), rows(min(1 << shift, kBlockN)), id(0), next(look(s, d, 0)) {}
    // Key (value) tile j of an item into a stage: v = 0, then v = 1.
    __device__ __forceinline__ void tile(const PagedSource& s, const Work& d, int j, int v, uint8_t* dst, uint8_t* scales,
                                         uint32_t bar, uint64_t policy, unsigned int* err) {
      const int lane = threadIdx.x & 31, n = pages(d, j);
      if (v == 0) {
        id = next;
        next = look(s, d, j + 1);
        if (lane < n && !page_ok(s.seg.table, id)) {
          record_error(err, kErrBadPage);
          id = 0;
        }
      }
      const uint32_t row_bytes = kE4m3 ? kD + 1 : 2 * kD;
      if (lane == 0) mbar_arrive_expect_tx(bar, n * rows * row_bytes);
      __syncwarp();
      if (lane < n) {
        const CUtensorMap* map = v == 0 ? &s.tmap_k : &s.tmap_v;
        const int first = (d.kv0 + j) * kBlockN & ((1 << shift) - 1);  // of the page's rows (pages over 128 tokens)
        const int plane = id * s.seg.num_kv_heads + d.kv_head;
        if constexpr (kE4m3) {
          tma_load_3d_hint(smem_u32(dst + lane * rows * kD), map, 0, first, plane, bar, policy);
          const uint8_t* scale = (v == 0 ? s.k_scale : s.v_scale) + (static_cast<size_t>(plane) << shift) + first;
          bulk_load(smem_u32(scales + lane * rows), scale, rows, bar);
        } else {
          for (int x = 0; x < kD / 64; ++x)
            tma_load_3d_hint(smem_u32(dst + x * kBlockN * 128 + lane * rows * 128), map, x * 64, first, plane, bar,
                             policy);
        }
      }
      __syncwarp();
    }
  };

  // Row `row` of a tile of bytes (swizzled as it came) into a bf16 tile (128-byte swizzle, 64 columns apart).
  __device__ static __forceinline__ void convert_row(const uint8_t* raw, uint32_t biased, uint8_t* tile, int row, bool key,
                                                     bool zero) {
    auto at = [&](int piece) {  // 16 bytes of the bf16 row
      return reinterpret_cast<uint4*>(tile + (piece >> 3) * kBlockN * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
    };
    if (key) {
      // value = bits * 2^120 * 2^e, in one product where 2^(120 + e) is a bf16
      const bool two = biased > 127 + 7;
      const uint32_t first = (two ? 247u : biased + 120u) << 7, f2 = first | first << 16;
#pragma unroll
      for (int p = 0; p < kD / 16; ++p) {
        const int swizzled = kD == 128 ? p ^ (row & 7) : p ^ ((row >> 1) & 3);
        const uint4 w4 = *reinterpret_cast<const uint4*>(raw + row * kD + (swizzled << 4));
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b[2 * i] = bf16x2_mul(e4m3_pair_bits<0>(w[i]), f2);
          b[2 * i + 1] = bf16x2_mul(e4m3_pair_bits<2>(w[i]), f2);
        }
        *at(2 * p) = make_uint4(b[0], b[1], b[2], b[3]);
        *at(2 * p + 1) = make_uint4(b[4], b[5], b[6], b[7]);
      }
      if (two) {  // rows of values past 57,344, or with a NaN: a second product (apart, to keep the loop above straight)
        const uint32_t second = biased == kScaleNan ? 0x7fffu : biased << 7, s2 = second | second << 16;
#pragma unroll 1
        for (int p = 0; p < kD / 8; ++p) {
          const uint4 v = *at(p);
          *at(p) = make_uint4(bf16x2_mul(v.x, s2), bf16x2_mul(v.y, s2), bf16x2_mul(v.z, s2), bf16x2_mul(v.w, s2));
        }
      }
    } else if (zero) {
#pragma unroll
      for (int p = 0; p < kD / 8; ++p) *at(p) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

template <int D, bool kE4m3>
cudaError_t launch(const PagedTileArgs& a, cudaStream_t stream) {
  using Source = PagedSource<D, kE4m3>;
  using C = TileCfg<Source>;
  cudaError_t e = allow_shared_memory<C::kSmemBytes>(attn_tile_kernel<Source>);
  if (e != cudaSuccess) return e;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  uint32_t* ws = static_cast<uint32_t*>(a.workspace);
  PagedPair* list = reinterpret_cast<PagedPair*>(ws + 2 * kHeader);
  uint8_t* split = static_cast<uint8_t*>(a.split_area);
  const int group = a.seg.num_q_heads / a.seg.num_kv_heads, tokens = kBlockM / group;
  e = launch_programmatic(paged_plan_kernel, dim3(1), dim3(a.seg.num_segments <= kSegments ? kSegments : kPlanThreads), 0,
                          stream, a.seg, tokens, ws, list, split, sms, a.err);
  if (e != cudaSuccess) return e;
  const Source src{a.tmap_q, a.tmap_k, a.tmap_v, a.seg, list, a.k_scale, a.v_scale, group, tokens};
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

cudaError_t launch_paged_attn(const PagedTileArgs& a, int head_dim, cudaStream_t stream) {
  if (a.k_scale != nullptr) return head_dim == 128 ? launch<128, true>(a, stream) : launch<64, true>(a, stream);
  return head_dim == 128 ? launch<128, false>(a, stream) : launch<64, false>(a, stream);
}

}  // namespace h3
