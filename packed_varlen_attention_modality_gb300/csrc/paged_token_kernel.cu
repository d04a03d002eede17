// Attention over a paged cache for a few rows per segment (the single tokens of running streams): every key
// row is read once and meets at most 16 query rows, so the call is bound by reading K and V.
//
// Work is laid out in units of 64 keys (e4m3: 128, or 256 of 64 values) of a (segment, key head) and dealt to two
// CTAs an SM in equal shares, so streams of unlike lengths keep the GPU even; every CTA finds its share by a scan of
// the lengths.  A pair that a
// share's end cuts leaves fp32 partial results (O normalised by its own sum, and the LSE), which a second kernel
// joins in order.  The 16 rows of the tensor-core tile are the segment's rows times the query heads that share
// the key head, so shared heads cost no second read.  Each of a CTA's four warps streams blocks of 16 (32, 64) keys of K
// and V through its own ring in shared memory (16-byte asynchronous copies, the next piece's blocks included), computes
// S = Q K^T and O += P V with 16 x 8 x 16 matrix instructions, and keeps a running max and sum; the warps are
// added in order at the end of a piece.  16 keys lie in one page, whose id is looked up a block ahead.
//
// An e4m3 block becomes f16 in registers, one instruction for two values, and exactly: the rows' scales go to the
// scores and the weights, which are fp32.  Q's rows are brought to f16 by a power of two each (their largest value to
// 2^14: what that rounds is 2^-39 of it at most).  The weights of V's rows are 2^(score + V's exponent) over a
// reference of their own, which puts their largest between 2^7 and 2^15: f16 rounds each by 2^-11 of itself (bf16 by
// 2^-8) or, below 2^-21 of the largest, by 2^-32 of the largest.  So a row that outweighs the others by its score or its
// scale leaves them their digits up to a ratio of 2^21.  The order of the dims in S's product and in O's columns is
// chosen so that a lane's bytes lie together.
// Scores, max, sum and O are fp32; P is rounded to bf16 (2^-8 of itself at most; e4m3: f16, as above) for the product
// with V, o once at the end.
//
// With at most eight rows (a head group's single token) the products take keys as rows and query rows as columns:
// half the matrix instructions, exponentials and registers, for a transposition of the weights (64 streams of 20,000
// tokens x 8 heads x 64: 215 us, 280 the other way).  A bf16 cache is bound by HBM either way.
//
// 32 streams of 512 to 4,096 tokens, 64 heads on 8 x 128, bf16: 62 us (floor 48; some 9 us are the launch, the scan
// and the join; 128 streams of 4,096 tokens read at the rate of a plain copy).  Two streams of 90,000 to 100,000
// tokens, 40 heads on 8 x 128, e4m3: 79 us (floor 57; 124 with a conversion to bf16).  Eight warps in one CTA an SM: 93.
#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "paged_segments.cuh"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16;    // query rows of a CTA
constexpr int kCtasPerSm = 2;
constexpr int kMinShare = 2;   // units
constexpr int kMaxPieces = 16;  // looked up at once
constexpr float kTopWeight = 7.f;  // e4m3: log2 of the largest weight when the reference is set (f16 ends at 2^16)
static_assert(kRows == kPagedTokenRows, "host and device agree");

template <int D, bool kE4m3>
struct Cfg {
  // Keys of a block: steps of 16.  An e4m3 block is bound by its instructions, and look-ups, maxima and exchanges
  // cost the same for each (64 streams of 20,000 tokens x 8 heads x 64: 280 us at 4 steps, 319 at 2, with 16 rows; 2
  // streams of 95,000 x 8 x 128: 85 us at 2, 96 at 1; with eight rows 82 at 2, 90 at 4).  Three stages do for all: bf16 reads at the rate of a plain copy.
  static constexpr int kSteps = kE4m3 ? 256 / D : 1, kBlock = 16 * kSteps;
  static constexpr int kUnit = kBlock * kWarps;
  static constexpr int kRowBytes = kE4m3 ? D : 2 * D;
  static constexpr int kHalf = kBlock * kRowBytes;                          // K's part of a stage
  static constexpr int kStageBytes = 2 * kHalf + (kE4m3 ? 2 * kBlock : 0);  // K, V, their scales
  static constexpr int kStages = 3;
  static constexpr int kOut = D + 8;  // floats of a row while the warps are added (the pad keeps banks apart)
  static constexpr int kSmemBytes = kWarps * kStages * kStageBytes + kRows * kOut * 4;
  // where a 16-byte piece of a row lies: as the reads below meet no bank twice
  __device__ static __forceinline__ int piece_at(int row, int piece) {
    return row * kRowBytes + ((kRowBytes == 64 ? piece ^ ((row >> 1) & 3) : piece ^ (row & 7)) << 4);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// An 8 x 8 tile of 16-bit values with rows and columns exchanged: lane l's pair of row l / 4 becomes that of column l / 4.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The part of a (segment, key head) pair that a CTA takes: keys [first, end).
struct Piece {
  PagedSegment s;
  int g, head, first, end;
  int slot;  // -1: the whole pair
};

// Units of a pair.
template <int kUnit>
__device__ __forceinline__ int units_of(const PagedSegment& s, int block) {
  const int keys = s.rows == 0 ? 0 : row_limit(s, s.rows - 1, block);
  return s.rows == 0 ? 0 : keys <= kUnit ? 1 : (keys + kUnit - 1) / kUnit;
}

// What the scan of the segments leaves: those of a tile of kThreads, and the units before each.
struct Scan {
  PagedSegment seg[kThreads];
  uint64_t before[kThreads + 1];  // units of all key heads
  uint64_t warp[kWarps];
};

__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* s_warp, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *total = all;
  return before + x - v;
}

template <int D>
__device__ __forceinline__ float* partial_of(const PagedTokenArgs& a, int cta, int slot) {
  return a.partials + (static_cast<size_t>(cta) * 2 + slot) * paged_token_partial(a.max_rows, D);
}

// kNarrow (e4m3, at most eight rows): keys are the products' rows and query rows their columns.
template <int D, bool kE4m3, bool kNarrow>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
paged_token_kernel(const __grid_constant__ PagedTokenArgs a) {
  static_assert(kE4m3 || !kNarrow);
  using C = Cfg<D, kE4m3>;
  constexpr int kStages = C::kStages, kSteps = C::kSteps, kBlock = C::kBlock, kUnit = C::kUnit;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Scan scan;
  __shared__ Piece pieces[kMaxPieces];
  __shared__ int s_pieces, s_more;
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_w[kWarps][kRows];
  grid_dependency_wait();
  launch_dependents();
  const int S = a.seg.num_segments, heads = a.seg.num_kv_heads, block = a.seg.causal_block;
  const int group = a.seg.num_q_heads / heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, quad = lane & 3, c2 = quad * 2;  // this lane's rows gr, gr + 8 and columns c2, c2 + 1
  // of a tile of scores, of which it has kValues of each of two query rows
  constexpr int kScores = kNarrow ? kSteps : 2 * kSteps, kValues = 2 * kScores;
  auto row_of = [&](int h) { return kNarrow ? c2 + h : gr + 8 * h; };
  auto key_of = [&](int v) { return kNarrow ? (v >> 1) * 16 + gr + 8 * (v & 1) : (v >> 1) * 8 + c2 + (v & 1); };
  auto value = [](float (&x)[kScores][4], int h, int v) -> float& {
    return kNarrow ? x[v >> 1][2 * (v & 1) + h] : x[v >> 1][2 * h + (v & 1)];
  };
  auto over_row = [](float x, auto op) {  // over the lanes that share a query row
#pragma unroll
    for (int o = kNarrow ? 4 : 1; o < (kNarrow ? 32 : 4); o *= 2) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  };
  unsigned int* scan_err = blockIdx.x == 0 ? a.err : nullptr;  // one CTA records what is wrong with the offsets

  // ---- this CTA's share of the units
  auto scan_tile = [&](int g0, uint64_t base, unsigned int* err) {  // returns the units up to the tile's end
    PagedSegment s{0, 0, 0};
    if (g0 + tid < S) s = checked_paged_segment(a.seg, g0 + tid, err);
    const uint64_t n = static_cast<uint64_t>(units_of<kUnit>(s, block)) * heads;
    uint64_t total;
    const uint64_t at = block_scan(n, scan.warp, &total);
    scan.seg[tid] = s;
    scan.before[tid] = base + at;
    if (tid == 0) scan.before[kThreads] = base + total;
    __syncthreads();
    return base + total;
  };
  uint64_t all = 0;
  for (int g0 = 0; g0 < S; g0 += kThreads) all = scan_tile(g0, all, scan_err);
  uint64_t share = (all + gridDim.x - 1) / gridDim.x;
  if (share < kMinShare) share = kMinShare;
  const uint64_t begin = share * blockIdx.x;
  const uint64_t stop = begin + share < all ? begin + share : all;
  if (tid == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (begin >= stop) return;

  uint8_t* ring = smem + warp * kStages * C::kStageBytes;
  const uint32_t ring32 = smem_u32(ring);
  float* s_o = reinterpret_cast<float*>(smem + kWarps * kStages * C::kStageBytes);
  const float scale_log2 = a.scale * 1.4426950408889634f;

  int tile = 0;
  uint64_t at = begin;
  if (S > kThreads) {  // the tile with the first unit (with one tile it is there already)
    for (uint64_t base = 0;; tile += kThreads) {
      base = scan_tile(tile, base, nullptr);
      if (at < base) break;
      __syncthreads();
    }
  }
  for (;;) {
    // ---- the next pieces, by one thread
    if (tid == 0) {
      int n = 0;
      while (n < kMaxPieces && at < stop && at < scan.before[kThreads]) {
        int lo = 0, hi = kThreads - 1;  // the last segment with before <= at
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (scan.before[mid] <= at) lo = mid; else hi = mid - 1;
        }
        Piece p;
        p.s = scan.seg[lo];
        p.g = tile + lo;
        const int units = units_of<kUnit>(p.s, block);
        const uint64_t in = at - scan.before[lo];
        p.head = static_cast<int>(in / units);
        const int u0 = static_cast<int>(in % units);
        const int u1 = static_cast<int>(u0 + (stop - at) < static_cast<uint64_t>(units) ? u0 + (stop - at) : units);
        const int keys = row_limit(p.s, p.s.rows - 1, block);
        p.first = u0 * kUnit;
        p.end = u1 == units ? keys : u1 * kUnit;
        // the piece at the start of the share has slot 0, one at its end slot 1
        p.slot = u0 == 0 && u1 == units ? -1 : at == begin ? 0 : 1;
        if (u0 == 0 && u1 < units) {  // the first of a cut pair: all but the first of the others are whole shares
          const uint64_t rest = units - u1;
          a.joins[blockIdx.x] = make_int4(p.g, p.head, p.slot, 1 + static_cast<int>((rest + share - 1) / share));
        }
        pieces[n++] = p;
        at += u1 - u0;
      }
      s_pieces = n;
      s_more = at < stop;
    }
    __syncthreads();
    const int num_pieces = s_pieces;

    // ---- loads: a cursor that runs ahead of the computation, over the pieces' blocks
    struct Cursor {
      int piece, b, blocks;  // this warp's block b of the piece's
    };
    auto blocks_of = [&](int p) { return (pieces[p].end - pieces[p].first + kBlock - 1) / kBlock; };
    auto settle = [&](Cursor& c) {  // onto the next block there is
      while (c.piece < num_pieces && c.b >= c.blocks) {
        ++c.piece;
        c.b = warp;
        c.blocks = c.piece < num_pieces ? blocks_of(c.piece) : 0;
      }
    };
    const int shift = a.seg.table.page_shift;
    struct Ids {
      int id[kSteps];  // pages of a block's steps
    };
    auto lookup = [&](const Cursor& c) {
      Ids r{};
      if (c.piece >= num_pieces) return r;
      const Piece& p = pieces[c.piece];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int key = p.first + c.b * kBlock + 16 * i;
        if (key < p.end) r.id[i] = page_id(a.seg.table, p.g, key >> shift);
      }
      return r;
    };
    auto load = [&](const Cursor& c, const Ids& ids, int stage) {
      if (c.piece >= num_pieces) return;
      const Piece& p = pieces[c.piece];
      const uint32_t dst = ring32 + stage * C::kStageBytes;
#pragma unroll
      for (int step = 0; step < kSteps; ++step) {
        int id = ids.id[step];
        if (!page_ok(a.seg.table, id)) {
          if (lane == 0) record_error(a.err, kErrBadPage);
          id = 0;
        }
        const int key = p.first + c.b * kBlock + 16 * step, left = p.end - key;
        const size_t row = ((static_cast<size_t>(id) * heads + p.head) << shift) + (key & ((1 << shift) - 1));
        constexpr int kPieces = C::kRowBytes / 16;
        const uint8_t* kp = static_cast<const uint8_t*>(a.k) + row * C::kRowBytes;
        const uint8_t* vp = static_cast<const uint8_t*>(a.v) + row * C::kRowBytes;
#pragma unroll
        for (int i = lane; i < 16 * kPieces; i += 32) {  // a step's rows lie back to back; zeros past the end
          const int r = i / kPieces;
          const uint32_t bytes = r < left ? 16u : 0u, off = C::piece_at(16 * step + r, i % kPieces);
          cp_async16(dst + off, kp + i * 16, bytes);
          cp_async16(dst + C::kHalf + off, vp + i * 16, bytes);
        }
        if (kE4m3 && lane < 2 && left > 0)
          cp_async16(dst + 2 * C::kHalf + lane * kBlock + 16 * step, (lane == 0 ? a.k_scale : a.v_scale) + row, 16);
      }
    };
    Cursor ahead{0, warp, blocks_of(0)};
    settle(ahead);
    int stage = 0;
    Ids id = lookup(ahead);
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
      load(ahead, id, i);
      cp_async_commit();
      ahead.b += kWarps;
      settle(ahead);
      id = lookup(ahead);
    }

#pragma unroll 1
    for (int pi = 0; pi < num_pieces; ++pi) {
      const Piece& p = pieces[pi];
      const int rows = p.s.rows * group;
      // Q fragments: row r = (segment row r / group, head r % group of the key head's)
      uint32_t q[D / 16][4];
      int limit[2], low = p.end;  // keys that this lane's rows see; the least of all rows
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = gr + 8 * h;
        const __nv_bfloat16* row = a.q + static_cast<size_t>(p.s.q0 + r / group) * a.q_stride +
                                   (p.head * group + r % group) * D;
        if (kNarrow && h == 1) {
          // (its only row is gr)
        } else if (kE4m3) {  // step kk: dims 4 kk + {0, 1} and {2, 3} of the lane's D / 4
          const uint2* src = reinterpret_cast<const uint2*>(row + quad * (D / 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint2 x = r < rows ? src[kk] : make_uint2(0u, 0u);
            q[kk][h] = x.x;
            q[kk][2 + h] = x.y;
          }
        } else {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(row + c2);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            q[kk][h] = r < rows ? src[kk * 8] : 0u;
            q[kk][2 + h] = r < rows ? src[kk * 8 + 4] : 0u;
          }
        }
        const int scored = row_of(h);
        limit[h] = scored < rows ? row_limit(p.s, scored / group, block) : p.end;
      }
      float q_scale[2] = {1.f, 1.f};  // e4m3: what the f16 rows are to be multiplied with
      if (kE4m3) {
#pragma unroll
        for (int h = 0; h < (kNarrow ? 1 : 2); ++h) {
          uint32_t most = 0u;  // the largest magnitude's bits (of both halves: the upper decides)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = q[kk][h + 2 * i];
              most = max(most, max(x << 16 & 0x7fffffffu, x & 0x7fff0000u));
            }
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          // 2^(e - 14) for the exponent e of the largest; both powers are fp32
          const int e = min(max(static_cast<int>(most >> 23), 16), 254);
          q_scale[h] = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
          const float inv = __uint_as_float(static_cast<uint32_t>(254 - (e - 14)) << 23);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t& x = q[kk][h + 2 * i];
              x = pack_f16x2(__uint_as_float(x << 16) * inv, __uint_as_float(x & 0xffff0000u) * inv);
            }
        }
        if (kNarrow) {  // of the rows whose scores the lane has
          const float own = q_scale[0];
#pragma unroll
          for (int h = 0; h < 2; ++h) q_scale[h] = __shfl_sync(0xffffffffu, own, 4 * (c2 + h));
        }
      }
      low = min(low, row_limit(p.s, 0, block));

      // wide: column tile n of the rows; narrow: dims gr * D / 8 + 2 n and the next, of rows c2 and c2 + 1
      constexpr int kTiles = kNarrow ? D / 16 : D / 8;
      float o[kTiles][4] = {};
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      float top_w[2] = {-INFINITY, -INFINITY};  // e4m3: log2 of the weights' reference
      const int nblocks = (p.end - p.first + kBlock - 1) / kBlock;
#pragma unroll 1
      for (int b = warp; b < nblocks; b += kWarps) {
        load(ahead, id, stage == 0 ? kStages - 1 : stage - 1);
        cp_async_commit();
        ahead.b += kWarps;
        settle(ahead);
        id = lookup(ahead);
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint32_t kb = ring32 + stage * C::kStageBytes, vb = kb + C::kHalf;
        const uint8_t* base = ring + stage * C::kStageBytes;
        const int key = p.first + b * kBlock;
        const int mat = lane >> 3, mr = lane & 7;
        float sc[kScores][4] = {};
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
          if (!kE4m3) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              uint32_t f[4];  // keys 0-7: dims 0-7, 8-15 of the step; keys 8-15 the same
              ldmatrix4(f, kb + C::piece_at(16 * step + (mat >> 1) * 8 + mr, 2 * kk + (mat & 1)));
              mma_16816(sc[2 * step], q[kk], f[0], f[1]);
              mma_16816(sc[2 * step + 1], q[kk], f[2], f[3]);
            }
            continue;
          }
          if constexpr (kNarrow) {
            const int row = 16 * step + gr;
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              const uint4 k0 = *reinterpret_cast<const uint4*>(base + C::piece_at(row, quad * (D / 64) + x));
              const uint4 k1 = *reinterpret_cast<const uint4*>(base + C::piece_at(row + 8, quad * (D / 64) + x));
              const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t f[4] = {e4m3_pair_f16<0>(w0[i]), e4m3_pair_f16<0>(w1[i]), e4m3_pair_f16<1>(w0[i]),
                                       e4m3_pair_f16<1>(w1[i])};
                mma_16816_f16(sc[step], f, q[4 * x + i][0], q[4 * x + i][2]);
              }
            }
#pragma unroll
            for (int v = 2 * step; v < 2 * step + 2; ++v) {
              const float scale = scale_of(base[2 * C::kHalf + key_of(v)]);
#pragma unroll
              for (int h = 0; h < 2; ++h) value(sc, h, v) *= scale * q_scale[h];
            }
            continue;
          }
#pragma unroll
          for (int n = 2 * step; n < (kNarrow ? 0 : 2 * step + 2); ++n) {
            const int row = n * 8 + gr;
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              const uint4 w4 = *reinterpret_cast<const uint4*>(base + C::piece_at(row, quad * (D / 64) + x));
              const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_16816_f16(sc[n], q[4 * x + i], e4m3_pair_f16<0>(w[i]), e4m3_pair_f16<1>(w[i]));
            }
            const uint32_t ks = *reinterpret_cast<const uint16_t*>(base + 2 * C::kHalf + n * 8 + c2);
            const float s0 = scale_of(ks & 0xffu), s1 = scale_of(ks >> 8);
            sc[n][0] *= s0 * q_scale[0];
            sc[n][1] *= s1 * q_scale[0];
            sc[n][2] *= s0 * q_scale[1];
            sc[n][3] *= s1 * q_scale[1];
          }
        }
        if (key + kBlock > low) {  // by select, so NaN/Inf there is discarded
#pragma unroll
          for (int v = 0; v < kValues; ++v)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (key + key_of(v) >= min(limit[h], p.end)) value(sc, h, v) = -INFINITY;
        }
        // e4m3: the log2 of V's rows' weights, score and V's exponent together (a masked key's stays -inf: past the end
        // lie rows whose scale may be anything)
        float u[kScores][4];
        if (kE4m3) {
#pragma unroll
          for (int v = 0; v < kValues; v += 2) {
            const uint8_t* vs = base + 2 * C::kHalf + kBlock;
            uint32_t pair;
            if (kNarrow) pair = vs[key_of(v)] | vs[key_of(v + 1)] << 8;
            else pair = *reinterpret_cast<const uint16_t*>(vs + key_of(v));
            const float v0 = scale_log2_of(pair & 0xffu), v1 = scale_log2_of(pair >> 8);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float s0 = value(sc, h, v), s1 = value(sc, h, v + 1);
              value(u, h, v) = s0 == -INFINITY ? -INFINITY : fmaf(s0, scale_log2, v0);
              value(u, h, v + 1) = s1 == -INFINITY ? -INFINITY : fmaf(s1, scale_log2, v1);
            }
          }
        }
        // row maxima; a reference moves only when it grows by more than 2^8
        auto row_max = [&](float (&x)[kScores][4], int h) {
          float y = fmaxf(value(x, h, 0), value(x, h, 1));
#pragma unroll
          for (int v = 2; v < kValues; v += 2) y = fmax3(y, value(x, h, v), value(x, h, v + 1));
          return over_row(y, [](float p, float q) { return fmaxf(p, q); });
        };
        float alpha[2] = {1.f, 1.f};  // of O
        bool moved = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = row_max(sc, h);
          if (x > m[h] && (m[h] == -INFINITY || (x - m[h]) * scale_log2 > 8.f)) {
            const float f = ex2_approx((m[h] - x) * scale_log2);
            m[h] = x;
            l[h] *= f;
            if (!kE4m3) {
              alpha[h] = f;
              moved = true;
            }
          }
          if (kE4m3) {
            const float w = row_max(u, h) - kTopWeight;
            if (w > top_w[h] && (top_w[h] == -INFINITY || w - top_w[h] > 8.f)) {
              alpha[h] = ex2_approx(top_w[h] - w);
              top_w[h] = w;
              moved = true;
            }
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] *= alpha[kNarrow ? i & 1 : i >> 1];
        }
        uint32_t pw[kSteps][4];
        float weight[2][kNarrow ? 2 : 1];  // of two keys, of both rows
#pragma unroll
        for (int v = 0; v < kValues; v += 2)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mb = m[h] == -INFINITY ? 0.f : m[h] * scale_log2;
            const float e0 = ex2_approx(fmaf(value(sc, h, v), scale_log2, -mb));
            const float e1 = ex2_approx(fmaf(value(sc, h, v + 1), scale_log2, -mb));
            l[h] += e0 + e1;
            const int n = v / 2;
            if (kE4m3) {
              const float wb = top_w[h] == -INFINITY ? 0.f : top_w[h];
              const float w0 = ex2_approx(value(u, h, v) - wb), w1 = ex2_approx(value(u, h, v + 1) - wb);
              if constexpr (kNarrow) {
                weight[0][h] = w0;
                weight[1][h] = w1;
                if (h == 1) {
#pragma unroll
                  for (int k = 0; k < 2; ++k) pw[n][k] = transpose8x8(pack_f16x2(weight[k][0], weight[k][1]));
                }
              } else {
                pw[n / 2][2 * (n & 1) + h] = pack_f16x2(w0, w1);
              }
            } else {
              pw[n / 2][2 * (n & 1) + h] = pack_bf16x2(e0, e1);
            }
          }
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
          if (!kE4m3) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t f[4];  // dims 0-7 of the step: keys 0-7, 8-15; dims 8-15 the same
              ldmatrix4_trans(f, vb + C::piece_at(16 * step + (mat & 1) * 8 + mr, 2 * n + (mat >> 1)));
              mma_16816(o[2 * n], pw[step], f[0], f[1]);
              mma_16816(o[2 * n + 1], pw[step], f[2], f[3]);
            }
            continue;
          }
          // column gr of tile j is dim gr * D / 8 + j: the lane's dims of a key are D / 8 bytes in a row
          const uint8_t* vbase = base + C::kHalf;
          uint32_t w[4][D / 32];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 16 * step + c2 + (k & 1) + 8 * (k >> 1);
            if (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(vbase + C::piece_at(row, gr));
              w[k][0] = x.x;
              w[k][1] = x.y;
              w[k][D / 32 - 2] = x.z;
              w[k][D / 32 - 1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(vbase + C::piece_at(row, gr >> 1) + (gr & 1) * 8);
              w[k][0] = x.x;
              w[k][1] = x.y;
            }
          }
#pragma unroll
          for (int j = 0; j < D / 8; j += 2) {  // bytes j and j + 1 of two keys each, in one word
            const uint32_t pick = j % 4 == 0 ? 0x5140 : 0x7362;
            const uint32_t lo = __byte_perm(w[0][j / 4], w[1][j / 4], pick), hi = __byte_perm(w[2][j / 4], w[3][j / 4], pick);
            const uint32_t f[4] = {e4m3_pair_f16<0>(lo), e4m3_pair_f16<1>(lo), e4m3_pair_f16<0>(hi), e4m3_pair_f16<1>(hi)};
            if constexpr (kNarrow) {
              mma_16816_f16(o[j / 2], f, pw[step][0], pw[step][1]);
            } else {
              mma_16816_f16(o[j], pw[step], f[0], f[2]);
              mma_16816_f16(o[j + 1], pw[step], f[1], f[3]);
            }
          }
        }
        __syncwarp();  // the stage is read: it may be loaded again
        stage = stage == kStages - 1 ? 0 : stage + 1;
      }

      // ---- the warps, added in order
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] = over_row(l[h], [](float p, float q) { return p + q; });
        if (kNarrow ? gr == 0 : quad == 0) {
          s_m[warp][row_of(h)] = m[h];
          s_l[warp][row_of(h)] = l[h];
          s_w[warp][row_of(h)] = kE4m3 ? top_w[h] : m[h] * scale_log2;  // O's reference
        }
      }
      __syncthreads();
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_w[w][row_of(h)]);
        f[h] = top == -INFINITY ? 0.f : ex2_approx(s_w[warp][row_of(h)] - top);  // 0 for a warp without keys
      }
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        if (warp == w) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int col = kNarrow ? gr * (D / 8) + 2 * n + e : kE4m3 ? (c2 + e) * (D / 8) + n : n * 8 + c2 + e;
                float* dst = s_o + row_of(h) * C::kOut + col;
                const float x = f[h] * o[n][kNarrow ? 2 * e + h : 2 * h + e];
                *dst = w == 0 ? x : *dst + x;
              }
        }
        __syncthreads();
      }
      for (int i = tid; i < rows * (D / 8); i += kThreads) {
        const int r = i / (D / 8), col = i % (D / 8) * 8;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
        const float mb = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum = fmaf(ex2_approx((s_m[w][r] - mb) * scale_log2), s_l[w][r], sum);
        // no keys: 0, and an LSE of -inf.  O's reference is not the sum's for e4m3.
        float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (kE4m3) {
          float o_top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) o_top = fmaxf(o_top, s_w[w][r]);
          inv = o_top == -INFINITY ? 0.f : inv * exp2f(o_top - mb * scale_log2);
        }
        const float lse = top * a.scale + logf(sum);
        const float* x = s_o + r * C::kOut + col;
        if (p.slot >= 0) {
          float* part = partial_of<D>(a, blockIdx.x, p.slot);
          float4* dst = reinterpret_cast<float4*>(part + r * D + col);
          dst[0] = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
          dst[1] = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
          if (col == 0) part[a.max_rows * D + r] = lse;
        } else {
          const int row = p.s.q0 + r / group, head = p.head * group + r % group;
          *reinterpret_cast<uint4*>(a.o + (static_cast<size_t>(row) * a.seg.num_q_heads + head) * D + col) =
              make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                         pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
          if (col == 0 && a.lse != nullptr) a.lse[static_cast<size_t>(head) * a.seg.capacity_q + row] = lse;
        }
      }
      __syncthreads();  // s_o, s_m and s_l are read
    }
    cp_async_wait<0>();
    const bool more = s_more != 0;
    __syncthreads();  // the pieces and s_more are read
    if (!more) return;
    // the tile's segments are used up, or the list of pieces was full
    uint64_t next;
    if (tid == 0) scan.warp[0] = at;
    __syncthreads();
    next = scan.warp[0];
    const uint64_t tile_end = scan.before[kThreads];
    __syncthreads();
    if (next >= tile_end) {
      tile += kThreads;
      scan_tile(tile, tile_end, nullptr);
    }
  }
}

// Joins the pieces of a cut pair, in order, kBatch loaded at once.  CTA c joins the pair whose first piece CTA c of
// the kernel before took; nothing is read before the wait.
template <int D>
__global__ void __launch_bounds__(kThreads)
paged_token_join_kernel(const __grid_constant__ PagedTokenArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const int4 join = a.joins[blockIdx.x];
  const int n = join.w;
  if (n <= 1) return;
  const int g = join.x, kv_head = join.y;
  const PagedSegment s = checked_paged_segment(a.seg, g, nullptr);
  const int group = a.seg.num_q_heads / a.seg.num_kv_heads;
  auto piece = [&](int c) { return partial_of<D>(a, blockIdx.x + c, c == 0 ? join.z : 0); };
  for (int i = threadIdx.x; i < s.rows * group * (D / 8); i += kThreads) {
    const int r = i / (D / 8), col = i % (D / 8) * 8;
    float top = -INFINITY, sum = 0.f, x[8] = {};
    constexpr int kBatch = 16;  // pieces loaded at once (19 of them: 2.5 us less than 4 at once)
    for (int c0 = 0; c0 < n; c0 += kBatch) {
      float w[kBatch];
      float4 u[kBatch], v[kBatch];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        w[c] = -INFINITY;
        u[c] = v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + c >= n) continue;
        const float* p = piece(c0 + c);
        w[c] = p[a.max_rows * D + r];
        u[c] = reinterpret_cast<const float4*>(p + r * D + col)[0];
        v[c] = reinterpret_cast<const float4*>(p + r * D + col)[1];
      }
      float mx = top;
#pragma unroll
      for (int c = 0; c < kBatch; ++c) mx = fmaxf(mx, w[c]);
      const float base = mx == -INFINITY ? 0.f : mx;
      const float old = __expf(top - base);
      top = mx;
      sum *= old;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= old;
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const float f = __expf(w[c] - base);
        const float y[8] = {u[c].x, u[c].y, u[c].z, u[c].w, v[c].x, v[c].y, v[c].z, v[c].w};
        sum += f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = c0 + c < n ? fmaf(f, y[e], x[e]) : x[e];
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int row = s.q0 + r / group, head = kv_head * group + r % group;
    *reinterpret_cast<uint4*>(a.o + (static_cast<size_t>(row) * a.seg.num_q_heads + head) * D + col) =
        make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                   pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
    if (col == 0 && a.lse != nullptr) a.lse[static_cast<size_t>(head) * a.seg.capacity_q + row] = top + logf(sum);
  }
}

template <int D, bool kE4m3, bool kNarrow>
cudaError_t launch(const PagedTokenArgs& a, cudaStream_t stream) {
  using C = Cfg<D, kE4m3>;
  cudaError_t e = allow_shared_memory<C::kSmemBytes>(paged_token_kernel<D, kE4m3, kNarrow>);
  if (e != cudaSuccess) return e;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int ctas = sms * kCtasPerSm < kPagedTokenCtas ? sms * kCtasPerSm : kPagedTokenCtas;
  e = launch_programmatic(paged_token_kernel<D, kE4m3, kNarrow>, dim3(ctas), dim3(kThreads), C::kSmemBytes, stream, a);
  if (e != cudaSuccess) return e;
  return launch_programmatic(paged_token_join_kernel<D>, dim3(ctas), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_paged_token(const PagedTokenArgs& a, int head_dim, cudaStream_t stream) {
  if (a.k_scale == nullptr) return head_dim == 128 ? launch<128, false, false>(a, stream) : launch<64, false, false>(a, stream);
  if (a.max_rows <= 8) return head_dim == 128 ? launch<128, true, true>(a, stream) : launch<64, true, true>(a, stream);
  return head_dim == 128 ? launch<128, true, false>(a, stream) : launch<64, true, false>(a, stream);
}

}  // namespace h3
