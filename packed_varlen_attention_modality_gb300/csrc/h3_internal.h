// Host-side launchers shared between the C-ABI translation unit and the kernel translation units.
// Arguments arrive already validated by h3attn_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace h3 {

// ---- RoPE ---------------------------------------------------------------------------------
constexpr int kMaxPairs = 64;  // head_dim <= 128

// Per-pair fp32 inverse frequencies (computed on the host in fp64, rounded once) and, for video
// rows, which coordinate drives each pair (0 = t, 1 = h, 2 = w).
struct RopeTables {
  float inv_text[kMaxPairs];
  float inv_audio[kMaxPairs];
  float inv_video[kMaxPairs];
  uint8_t video_axis[kMaxPairs];
  float audio_hz;
  float video_fps;
};

cudaError_t launch_rope(const void* q_in, void* q_out, const void* k_in, void* k_out,
                        int num_tokens, int num_heads, int head_dim, const float* pos,
                        const uint8_t* tag, const int32_t* cu_requests, int num_requests,
                        const float* start_frames, const RopeTables& tables, cudaStream_t stream);

// ---- norm of Q and K rows with the rotation ------------------------------------------------
// Frequencies in turns per position unit (inverse frequency / 2 pi) as hi + lo float pairs, from
// fp64 on the host; video_axis as in RopeTables.
struct NormRopeTables {
  float2 text[kMaxPairs];
  float2 audio[kMaxPairs];
  float2 video[kMaxPairs];
  uint8_t video_axis[kMaxPairs];
  float audio_hz;
  float video_fps;
};
// One of Q and K; strides in elements between tokens, heads and dims contiguous.  Forward: out =
// the normed and rotated rows; backward: out = dx.
struct NormRopeTensor {
  int heads;  // 0: absent
  const __nv_bfloat16* x;
  const __nv_bfloat16* dy;
  __nv_bfloat16* out;
  int64_t x_stride, dy_stride, out_stride;
  const void* weight;  // [D], bf16 or fp32
  float* dw;           // backward: [D]
};
struct NormRopeArgs {
  NormRopeTensor t[2];
  int num_tokens;
  int weight_bf16;
  float eps;
  const float* pos;  // null: no rotation
  const uint8_t* tag;
  const int32_t* cu_requests;
  int num_requests;
  const float* start_frames;
  float* partials;  // backward: norm_bwd_workspace_bytes()
  NormRopeTables tab;
};
constexpr int kNormBwdMaxCtas = 608;  // 4 x 152 SMs
constexpr size_t norm_bwd_workspace_bytes(int head_dim) {
  return static_cast<size_t>(kNormBwdMaxCtas) * 2 * head_dim * sizeof(float);
}
cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, bool backward, cudaStream_t stream);

// ---- gated residual and modulated norm of the stream ----------------------------------------
constexpr int kNormNone = 0, kNormRms = 1, kNormLayer = 2;
// Strides in elements between the rows of a tensor; vectors of a request `*_stride` elements apart.
struct ResidualNormArgs {
  int num_tokens, dim, num_requests, norm, branch_norm;
  int x_fp32, weight_bf16, mod_bf16;
  float eps, residual_scale;
  const void* x;  // forward: the stream before the branch; backward: after it
  const __nv_bfloat16* y;
  const void *weight, *branch_weight, *scale, *shift, *gate;
  int64_t x_stride, y_stride, scale_stride, shift_stride, gate_stride;
  const int32_t* cu_requests;
  // forward
  void* x_out;
  __nv_bfloat16* h;
  int64_t x_out_stride, h_stride;
  // backward
  const void* dx_out;
  const __nv_bfloat16* dh;
  void* dx;
  __nv_bfloat16* dy;
  int64_t dx_out_stride, dh_stride, dx_stride, dy_stride;
  float *dweight, *dbranch_weight, *dscale, *dshift, *dgate;  // null: not wanted
  float* partials;  // residual_norm_bwd_bytes()
  unsigned int* err;
};
constexpr int kResidualNormMaxDim = 8192;
constexpr int kResidualNormMaxBwdCtas = 8 * 152;
inline int residual_norm_ctas(int num_tokens, int resident) {
  return num_tokens < resident ? num_tokens : resident;
}
// three column sums for each pair of a CTA and a request with rows in it
inline size_t residual_norm_bwd_bytes(int num_tokens, int num_requests, int dim) {
  const size_t pairs = static_cast<size_t>(residual_norm_ctas(num_tokens, kResidualNormMaxBwdCtas)) + num_requests;
  return pairs * 3 * dim * sizeof(float);
}
cudaError_t launch_residual_norm(const ResidualNormArgs& a, bool backward, cudaStream_t stream);

// ---- paged key/value cache --------------------------------------------------------------------
// Cache [pages, heads, page, D]; e4m3 with one biased exponent per row, [pages, heads, page].
constexpr int kScaleMin = -110, kScaleMax = 120;
constexpr uint32_t kScaleNan = 255;
struct PagedTable {
  const int32_t* pages;  // [segments, per_segment]
  int per_segment, num_pages, page_shift;
};
struct KvCacheArgs {
  __nv_bfloat16 *k, *v;  // packed rows (only read when the cache is written)
  int64_t k_stride, v_stride;
  void *k_cache, *v_cache;
  uint8_t *k_scale, *v_scale;  // null: a bf16 cache
  PagedTable table;
  const int32_t *cu, *start;
  int num_segments, capacity, heads;
  unsigned int* err;
};
cudaError_t launch_kv_cache(const KvCacheArgs& a, int head_dim, bool write, cudaStream_t stream);

// ---- window partition ---------------------------------------------------------------------
struct WindowGeom {
  int L[3];      // grid extent per axis (T, H, W)
  int w[3];      // window size per axis
  int s[3];      // shift per axis
  int nwin[3];   // axis window counts
};

constexpr int kMaxPackTensors = 8;
struct PackPtrs {
  const void* src[kMaxPackTensors];
  void* dst[kMaxPackTensors];
};

cudaError_t launch_window_pack(const WindowGeom& g, int32_t* perm, int32_t* cu_seqlens,
                               const PackPtrs& ptrs, int num_tensors, int row_bytes,
                               cudaStream_t stream);
cudaError_t launch_window_unpack(const int32_t* perm, int num_tokens, const void* src, void* dst,
                                 int row_bytes, unsigned int* err, cudaStream_t stream);

// ---- attention ------------------------------------------------------------------------------
// Attention kernel variants: packed varlen segments; 3D windows read in place on the grid;
// block-sparse video attention over selected 64-token blocks read in place on the grid.
constexpr int kAttnModePacked = 0;
constexpr int kAttnModeWindow = 1;
constexpr int kAttnModeVsa = 2;

// Attention straight on the (T, H, W) grid.
// Windows: windows of w[] cut with shift s[] (edge windows cropped), nwin[] windows per axis,
// frames_per_tile = 128 / (w[1] * w[2]) frames of a window per 128-row tile.
// VSA: blocks of w[] (w[0] * w[1] * w[2] = 64) cut without shift (s = 0), nwin[] blocks per axis,
// topk selected key blocks per query block.
struct WindowAttnGeom {
  int L[3];
  int w[3];
  int s[3];
  int nwin[3];
  int frames_per_tile;
  int half_h;  // windows: half-height maps exist (window H even) for edge windows
  int topk;
};

struct AttnArgs {
  // packed: 3-D views {D, H, capacity} of Q, K, V; window: 5-D views {D, H, W, Hgrid, T}
  CUtensorMap tmap_q, tmap_k, tmap_v;
  // window: the same views with half-height boxes (edge windows); otherwise copies of the above
  CUtensorMap tmap_q2, tmap_k2, tmap_v2;
  int mode;            // kAttnModePacked / kAttnModeWindow / kAttnModeVsa
  WindowAttnGeom wg;
  // VSA: the key/value steps of every (head, pair of query blocks), from launch_vsa_schedule
  const uint2* vsa_steps;
  const int2* vsa_counts;
  void* o;
  float* lse;
  const int32_t* cu_seqlens;
  int num_segments;
  int max_seqlen;
  int capacity;
  int num_heads;
  int head_dim;
  float scale;
  void* workspace;  // attn_plan_bytes(num_segments) bytes: the work plan
  void* split_area;  // packed: attn_split_bytes(head_dim) bytes after the plan, or null (no split)
  unsigned int* err;
  uint64_t wait_limit_ns;  // limit of the kernel's pipeline waits (wait_limit_ns() below)
  uint32_t stall_after_tiles;  // testing hook: producers stop after this many K/V tiles
};

// Limit of the attention kernels' pipeline waits for launches from now on: 2 s unless
// h3_set_wait_limit_ns changed it.
constexpr uint64_t kDefaultWaitLimitNs = 2000000000ull;
uint64_t wait_limit_ns();
// Key/value tiles a producer of an attention CTA issues before it stops (all, unless
// h3_debug_stall_loads changed it).
uint32_t stall_after_tiles();

// Workspace of the packed variant.  The plan (uint32 words): [0] split items, [1] work items, [2] whole items
// before the split last wave, [3] entries of that wave, [kAttnWsHeaderWords, +S) segment order,
// [kAttnWsHeaderWords + S, +S+1) exclusive prefix of whole items in that order; rounded up to
// 256 bytes.  Then, optionally, the split area of the last wave (entries, arrival counters and
// partial results of up to kSplitMaxEntries chunks): with it the call may cut the long items of
// its last wave into chunks of their key range; without it every item stays whole.
constexpr int kAttnWsHeaderWords = 4;
constexpr int kSplitMaxEntries = 320;  // chunks of the last wave (>= 2 x 152 SMs)
constexpr int kSplitMinSeqlen = 1024;  // the area is only asked for when a segment can be this long
constexpr size_t attn_plan_bytes(int num_segments) {
  return ((kAttnWsHeaderWords + 2 * static_cast<size_t>(num_segments) + 1) * sizeof(uint32_t) + 255) /
         256 * 256;
}
// entries (8 words each), a list of split items (one word each), then per entry and query tile
// 128 rows of head_dim fp32 values followed by their 128 fp32 LSEs
constexpr size_t attn_split_bytes(int head_dim) {
  return static_cast<size_t>(kSplitMaxEntries) * (8 + 1) * sizeof(uint32_t) +
         static_cast<size_t>(kSplitMaxEntries) * 2 * 128 * (head_dim + 1) * sizeof(float);
}
constexpr size_t attn_workspace_bytes(int num_segments, int max_seqlen, int head_dim) {
  return attn_plan_bytes(num_segments) + (max_seqlen >= kSplitMinSeqlen ? attn_split_bytes(head_dim) : 0);
}
cudaError_t launch_attn_fwd(const AttnArgs& a, cudaStream_t stream);

// ---- cross attention ------------------------------------------------------------------------
struct CrossSegments {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* seqused_k;  // keys used of each segment, or null: all
  int num_segments, max_seqlen_q, max_seqlen_k, capacity_q, capacity_k, num_q_heads, num_kv_heads;
};
struct CrossArgs {
  CUtensorMap tmap_q, tmap_k, tmap_v;  // 3-D views {D, H, rows}
  CrossSegments seg;
  void* o;
  int wide;  // o may be stored in 32-byte pieces
  float* lse;
  float scale;
  void* workspace;   // attn_plan_bytes(num_segments): the work plan
  void* split_area;  // attn_split_bytes(head_dim) after it, or null (no item is cut)
  unsigned int* err;
  uint64_t wait_limit_ns;
  uint32_t stall_after_tiles;
};
cudaError_t launch_cross_attn(const CrossArgs& a, int head_dim, cudaStream_t stream);

// Gradient.  Work plan: header words, then the prefixes of query and key tiles.  A tile of the last,
// partly filled wave may be cut into up to kCrossBwdMaxChunks chunks, whose partial sums take a slot
// each: two tiles of 128 x head_dim fp32 for a key tile, one for a query tile.
constexpr int kCrossBwdHeader = 8;
constexpr int kCrossBwdMaxSlots = 608;  // 4 x 152
constexpr int kCrossBwdMaxChunks = 16;
struct CrossBwdArgs {
  CUtensorMap tmap_q, tmap_k, tmap_v, tmap_do;
  CrossSegments seg;
  const void *o, *dout;
  const float* lse;
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t dq_stride, dk_stride, dv_stride;
  int wide;  // gradients may be stored in 32-byte pieces
  float scale;
  uint32_t* plan;
  float* delta;     // [num_q_heads, capacity_q]
  float* partials;    // slots x 2 x 128 x head_dim: dV, dK
  float* partials_q;  // slots x 128 x head_dim: dQ
  int slots;
  unsigned int* err;
  uint64_t wait_limit_ns;
  uint32_t stall_after_tiles;
};
struct CrossBwdWorkspace {
  size_t delta, partials, partials_q, bytes;  // offsets (the plan is at 0) and the whole
  int slots;
};
inline CrossBwdWorkspace cross_bwd_workspace(const CrossSegments& s, int head_dim) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  CrossBwdWorkspace w;
  w.delta = up((kCrossBwdHeader + 2 * (static_cast<size_t>(s.num_segments) + 1)) * sizeof(uint32_t));
  w.partials = w.delta + up(static_cast<size_t>(s.num_q_heads) * s.capacity_q * sizeof(float));
  // no more slots than chunks of all tiles that the capacities allow
  const int64_t k_tiles = (static_cast<int64_t>(s.capacity_k) / 128 + s.num_segments) * s.num_kv_heads;
  const int64_t q_tiles = (static_cast<int64_t>(s.capacity_q) / 128 + s.num_segments) * s.num_q_heads;
  const int64_t k_steps = static_cast<int64_t>(s.num_q_heads / s.num_kv_heads) * ((s.max_seqlen_q + 127) / 128);
  const int64_t q_steps = (s.capacity_k + 127) / 128;
  auto slots = [](int64_t tiles, int64_t steps) {
    const int64_t chunks = steps < kCrossBwdMaxChunks ? steps : kCrossBwdMaxChunks;
    return chunks > 1 ? tiles * chunks : 0;  // one chunk goes straight to the gradients
  };
  const int64_t a = slots(k_tiles, k_steps), b = slots(q_tiles, q_steps), all = a > b ? a : b;
  w.slots = static_cast<int>(all < kCrossBwdMaxSlots ? all : kCrossBwdMaxSlots);
  const size_t slot = static_cast<size_t>(w.slots) * 128 * head_dim * sizeof(float);
  w.partials_q = w.partials + 2 * slot;
  w.bytes = w.partials_q + slot;
  return w;
}
cudaError_t launch_cross_bwd(const CrossBwdArgs& a, int head_dim, cudaStream_t stream);

// Few rows per segment: at most kCrossTokenRows of (rows x query heads per key head).
constexpr int kCrossTokenRows = 16;
constexpr int kCrossTokenCtas = 608;  // CTAs aimed at: two waves of 2 x 152 (8 waves: 64 us, not 58)
struct CrossTokenArgs {
  CrossSegments seg;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  __nv_bfloat16* o;
  float* lse;
  float scale;
  int max_rows;            // max_seqlen_q x query heads per key head
  int chunk_keys, chunks;  // cross_token_split
  float* partials;         // cross_token_bytes()
  unsigned int* err;
};
void cross_token_split(const CrossSegments& s, int* chunk_keys, int* chunks);
// floats of a chunk's partial results: rows of head_dim values, then the rows' LSEs (16-byte units)
constexpr size_t cross_token_partial(int rows, int head_dim) {
  return static_cast<size_t>(rows) * head_dim + (rows + 3) / 4 * 4;
}
inline size_t cross_token_bytes(const CrossSegments& s, int head_dim) {
  int keys = 0, chunks = 0;
  cross_token_split(s, &keys, &chunks);
  const int rows = s.max_seqlen_q * (s.num_q_heads / s.num_kv_heads);
  const size_t all = static_cast<size_t>(s.num_segments) * s.num_kv_heads * chunks *
                     cross_token_partial(rows, head_dim) * sizeof(float);
  return chunks == 1 || all < 256 ? 256 : all;  // never none: the call always takes a workspace
}
cudaError_t launch_cross_token(const CrossTokenArgs& a, int head_dim, cudaStream_t stream);

// ---- attention over a paged cache ---------------------------------------------------------------
constexpr int kPagedMaxTokens = 1 << 30;  // of a segment: key counts then fit 32 bits with room for a tile
struct PagedSegments {
  const int32_t* cu_q;
  const int32_t* used;  // tokens of each segment, the new ones included
  PagedTable table;
  int num_segments, max_seqlen_q, max_seqlen_k, capacity_q, num_q_heads, num_kv_heads;
  int causal_block;  // tokens of a causal block; 0: every row sees every key
};

// Few rows per segment: at most kPagedTokenRows of (rows x query heads per key head).
constexpr int kPagedTokenRows = 16;
constexpr int kPagedTokenCtas = 304;  // 2 x 152
struct PagedTokenArgs {
  PagedSegments seg;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const void *k, *v;  // [pages, heads, page, D]
  const uint8_t *k_scale, *v_scale;
  __nv_bfloat16* o;
  float* lse;
  float scale;
  int max_rows;  // max_seqlen_q x query heads per key head
  int4* joins;   // [kPagedTokenCtas]: segment, key head, slot of the first piece, pieces
  float* partials;
  unsigned int* err;
};
// floats of a piece's partial results: rows of head_dim values, then the rows' LSEs (16-byte units)
constexpr size_t paged_token_partial(int rows, int head_dim) {
  return static_cast<size_t>(rows) * head_dim + (rows + 3) / 4 * 4;
}
constexpr size_t paged_token_joins_bytes() { return kPagedTokenCtas * sizeof(int4); }
constexpr size_t paged_token_bytes(int rows, int head_dim) {
  return paged_token_joins_bytes() + 2 * kPagedTokenCtas * paged_token_partial(rows, head_dim) * sizeof(float);
}
cudaError_t launch_paged_token(const PagedTokenArgs& a, int head_dim, cudaStream_t stream);

// A pair of 128-row query tiles of a segment (an item is a key head of one).
struct alignas(16) PagedPair {
  int segment;
  int q0, seg_end;  // its first row, the segment's last + 1
  int used, keys;   // tokens of the segment, and those that the pair's last row sees
  int ntiles;
  int unused[2];
};
__host__ __device__ constexpr int64_t paged_max_pairs(int capacity_q, int num_segments, int tokens) {
  return static_cast<int64_t>(capacity_q) / (2 * tokens) + num_segments;
}
// Workspace: 8 header words, the list of pairs; then, where a segment can be kSplitMinSeqlen tokens, the split area
// (entries, their lists, partial results as in attn_split_bytes).
constexpr size_t kPagedEntryBytes = 64;
constexpr size_t paged_plan_bytes(int capacity_q, int num_segments, int tokens) {
  return (8 * sizeof(uint32_t) + static_cast<size_t>(paged_max_pairs(capacity_q, num_segments, tokens)) * sizeof(PagedPair) +
          255) / 256 * 256;
}
constexpr size_t paged_split_bytes(int head_dim) {
  return static_cast<size_t>(kSplitMaxEntries) * (kPagedEntryBytes + sizeof(uint32_t)) +
         static_cast<size_t>(kSplitMaxEntries) * 2 * 128 * (head_dim + 1) * sizeof(float);
}
// An e4m3 cache's pages as bf16 (a page a slot, [slots, heads, page, D] of K, then of V) behind a table of the slots:
// segment g's page p is slot g * per_segment + p.
struct PagedUnpackArgs {
  PagedSegments seg;  // of the cache
  const uint8_t *k, *v, *k_scale, *v_scale;
  int per_segment;
  int32_t* table;
  __nv_bfloat16 *k_out, *v_out;
  unsigned int* err;
};
constexpr size_t paged_unpack_table_bytes(int64_t slots) { return (static_cast<size_t>(slots) * 4 + 255) / 256 * 256; }
constexpr size_t paged_unpack_cache_elements(int64_t slots, int heads, int page_size, int head_dim) {
  return static_cast<size_t>(slots) * heads * page_size * head_dim;
}
cudaError_t launch_paged_unpack(const PagedUnpackArgs& a, int head_dim, cudaStream_t stream);

struct PagedTileArgs {
  CUtensorMap tmap_q;          // {D, H, rows}, a box of a key head's query heads x 128 / their number
  CUtensorMap tmap_k, tmap_v;  // {D, page, pages x heads}, a box of a page (128 rows of it at most)
  PagedSegments seg;
  const uint8_t *k_scale, *v_scale;
  void* o;
  int wide;  // o may be stored in 32-byte pieces
  float* lse;
  float scale;
  void* workspace;   // paged_plan_bytes()
  void* split_area;  // paged_split_bytes(head_dim) after it, or null (no item is cut)
  unsigned int* err;
  uint64_t wait_limit_ns;
  uint32_t stall_after_tiles;
};
cudaError_t launch_paged_attn(const PagedTileArgs& a, int head_dim, cudaStream_t stream);

// ---- VSA block gate + top-k ----------------------------------------------------------------
struct VsaGeom {
  int L[3];   // grid (T, H, W)
  int b[3];   // block size per axis
  int nb[3];  // blocks per axis = ceil(L / b)
};
// Workspace: block means of Q and K, fp32 [2][heads][nblk][head_dim].
size_t vsa_pool_bytes(int nblk, int heads, int head_dim);
// scores: fp32 [heads, nblk, nblk] out; sel: int32 [heads, nblk, topk] out (ascending ids).
cudaError_t launch_vsa_select(const void* q, const void* k, const VsaGeom& g, int heads,
                              int head_dim, int topk, float scale, float* scores, int32_t* sel,
                              void* workspace, cudaStream_t stream);

// VSA key/value schedule.  Query blocks 2p and 2p + 1 (the two halves of one 128-row tile; the
// second is block 2p again past the last block) form pair p.  Step j of pair p loads two key
// blocks into the two 64-row halves of a key tile: steps[(h * npairs + p) * topk + j] holds
// {block of half 0 | use0 << kVsaUseShift, block of half 1 | use1 << kVsaUseShift}, where bit q
// of use_s says whether query block 2p + q attends to that half's keys.  counts[h * npairs + p]
// = {steps used (<= topk), s = blocks both query blocks selected}.  The steps follow a fixed
// layout: s / 2 steps of two shared blocks (both halves used by both), one step with the odd
// shared block in half 0 when s is odd, then steps whose half q is query block 2p + q's own.
constexpr int kVsaUseShift = 28;
constexpr uint32_t kVsaBlockMask = (1u << kVsaUseShift) - 1u;
inline int vsa_pairs(int nblk) { return (nblk + 1) / 2; }
size_t vsa_schedule_bytes(int nblk, int heads, int topk);
// sel: int32 [heads, nblk, topk]; workspace: vsa_schedule_bytes() bytes, 16-byte aligned.
cudaError_t launch_vsa_schedule(const int32_t* sel, int nblk, int heads, int topk, void* workspace,
                                unsigned int* err, cudaStream_t stream);

// ---- continuation window ---------------------------------------------------------------------
struct ContinuationGeom {
  int offset[5];  // first packed row of each group (offset[0] = 0)
  int num_rows;
  int frame_h, frame_w;  // latent grid of a video frame
};
// src[k]: device base of group k's source rows; first_row[k]: its first source row.
cudaError_t launch_continuation_pack(const ContinuationGeom& g, const void* const src[5],
                                     const int64_t first_row[5], int row_bytes, void* rows,
                                     float* pos, uint8_t* tag, uint8_t* target, cudaStream_t stream);
// Two contiguous device copies (bytes multiples of 16, 16-byte aligned) in one launch.
cudaError_t launch_copy_ranges(const void* const src[2], void* const dst[2], const int64_t bytes[2],
                               cudaStream_t stream);
cudaError_t launch_masked_row_update(void* dst, const void* src, const uint8_t* mask, int num_rows,
                                     int row_bytes, cudaStream_t stream);

}  // namespace h3
