// Cross attention for a few rows per segment (single tokens of a running sequence): every key row
// is read once and meets at most 16 query rows, so the call is bound by reading K and V.
//
// A CTA takes a (segment, key head) and a chunk of its keys; the 16 rows of the tensor-core tile are
// the segment's rows times the query heads that share the key head, so shared heads cost no second
// read.  Each of its four warps streams 16-key blocks of K and V through its own ring in shared
// memory (16-byte asynchronous copies, no barrier between warps), computes S = Q K^T and O += P V
// with 16 x 8 x 16 matrix instructions, and keeps a running max and sum; the warps are merged in
// order at the end.  Rows this few leave tcgen05's 128-row tiles all but empty: 32 segments of one
// row x 8 key heads x 64 query heads with 512 to 4,096 keys take 242 us there, 58 us here (323 MB read:
// 5.6 TB/s, 82 % of a plain copy's rate; the merge's launch is 4 us of it).
// Behind the tile's 16 rows is a step: with one or two rows a segment these take 54 to 58 us, with three (24 rows
// a key head) 224 us in the tile kernel, which gives each query head 128 rows of its own; 24 heads of their own keys
// 144 us at 16 rows, 181 at 17.  The rule goes by max_seqlen_q, so a loose bound takes the slower kernel too.
// Chunks write partial results (O normalised by its own sum, fp32, and the LSE), which a merge
// kernel joins in chunk order; with one chunk the CTA writes o itself.
// Scores, max, sum and O are fp32; P is rounded to bf16 for the product with V, o once at the end.
#include <cuda_bf16.h>

#include "cross_segments.cuh"
#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16;    // query rows of a CTA
constexpr int kBlock = 16;   // keys of a block
constexpr int kStages = 3;   // blocks of a warp's ring
constexpr int kCtasPerSm = 2;
static_assert(kRows == kCrossTokenRows, "host and device agree");

template <int D>
struct Cfg {
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kStageBytes = 2 * kBlock * kRowBytes;  // K then V
  static constexpr int kSmemBytes = kWarps * kStages * kStageBytes;
  static_assert(kSmemBytes >= kWarps * kRows * (D + 2) * 4, "the merge of the warps reuses the rings");
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

struct TokenSegment {
  int row0, rows;  // first query row; rows times shared heads (0: nothing to do)
  int key0, keys;
};
__device__ __forceinline__ TokenSegment token_segment(const CrossSegments& s, int g, unsigned int* err) {
  const CrossSegment r = checked_cross_segment(s, g, err);
  return TokenSegment{r.q0, r.rows * (s.num_q_heads / s.num_kv_heads), r.k0, r.used};
}

// Partial results of chunk c of (segment, key head) pair p: max_rows rows of D values, their LSEs.
template <int D>
__device__ __forceinline__ float* partial_of(float* partials, const CrossTokenArgs& a, size_t pair, int c) {
  return partials + (pair * a.chunks + c) * cross_token_partial(a.max_rows, D);
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
cross_token_kernel(const __grid_constant__ CrossTokenArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_wait();
  launch_dependents();
  const int g = blockIdx.z, kv_head = blockIdx.y, chunk = blockIdx.x;
  const TokenSegment s = token_segment(a.seg, g, chunk == 0 && kv_head == 0 ? a.err : nullptr);
  const int first = chunk * a.chunk_keys;
  if (s.rows == 0 || (first >= s.keys && (chunk > 0 || a.chunks > 1))) return;
  // the last chunk takes whatever is left, also keys past the host's bound
  const int end = chunk == a.chunks - 1 ? s.keys : min(s.keys, first + a.chunk_keys);
  const int group = a.seg.num_q_heads / a.seg.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, c2 = (lane & 3) * 2;  // this lane's rows gr, gr + 8 and column pair
  uint8_t* ring = smem + warp * kStages * C::kStageBytes;
  const uint32_t ring32 = smem_u32(ring);

  // 16 keys of K and V: 16-byte pieces, swizzled by the row so that ldmatrix meets no bank twice;
  // keys past the end are filled with zeros
  const __nv_bfloat16* k_base = a.k + static_cast<size_t>(s.key0) * a.k_stride + kv_head * D;
  const __nv_bfloat16* v_base = a.v + static_cast<size_t>(s.key0) * a.v_stride + kv_head * D;
  const int nblocks = (end - first + kBlock - 1) / kBlock;
  auto load = [&](int b, int stage) {  // block b of the chunk
    const uint32_t dst = ring32 + stage * C::kStageBytes;
    constexpr int kPieces = D / 8;
#pragma unroll
    for (int i = lane; i < kBlock * kPieces; i += 32) {
      const int r = i / kPieces, p = i % kPieces;
      const int key = first + b * kBlock + r;
      const uint32_t bytes = key < end ? 16u : 0u;
      const size_t at = key < end ? key : 0;
      const uint32_t off = r * C::kRowBytes + ((p ^ (r & 7)) << 4);
      cp_async16(dst + off, k_base + at * a.k_stride + p * 8, bytes);
      cp_async16(dst + kBlock * C::kRowBytes + off, v_base + at * a.v_stride + p * 8, bytes);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (warp + i * kWarps < nblocks) load(warp + i * kWarps, i);
    cp_async_commit();
  }

  // Q fragments: row r = (segment row r / group, head r % group of the key head's)
  uint32_t q[D / 16][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = gr + 8 * h;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(
        a.q + static_cast<size_t>(s.row0 + r / group) * a.q_stride + (kv_head * group + r % group) * D + c2);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      q[kk][h] = r < s.rows ? p[kk * 8] : 0u;
      q[kk][2 + h] = r < s.rows ? p[kk * 8 + 4] : 0u;
    }
  }

  float o[D / 8][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float scale_log2 = a.scale * 1.4426950408889634f;
  int stage = 0;
  for (int b = warp; b < nblocks; b += kWarps) {
    {
      const int ahead = b + (kStages - 1) * kWarps;
      if (ahead < nblocks) load(ahead, stage == 0 ? kStages - 1 : stage - 1);
      cp_async_commit();
    }
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t kb = ring32 + stage * C::kStageBytes, vb = kb + kBlock * C::kRowBytes;
    const int mat = lane >> 3, mr = lane & 7;
    float sc[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t f[4];  // keys 0-7: dims 0-7, 8-15 of the step; keys 8-15 the same
      const int row = (mat >> 1) * 8 + mr, piece = 2 * kk + (mat & 1);
      ldmatrix4(f, kb + row * C::kRowBytes + ((piece ^ (row & 7)) << 4));
      mma_16816(sc[0], q[kk], f[0], f[1]);
      mma_16816(sc[1], q[kk], f[2], f[3]);
    }
    const int left = end - first - b * kBlock;  // keys of this block
    if (left < kBlock) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n * 8 + c2 + (i & 1) >= left) sc[n][i] = -INFINITY;
    }
    // row maxima over the quad; the reference max moves only when it grows by more than 2^8
    float alpha[2] = {1.f, 1.f};
    bool moved = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      if (x > m[h] && (m[h] == -INFINITY || (x - m[h]) * scale_log2 > 8.f)) {
        alpha[h] = ex2_approx((m[h] - x) * scale_log2);
        m[h] = x;
        l[h] *= alpha[h];
        moved = true;
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] *= alpha[i >> 1];
    }
    uint32_t p[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float mb = m[h] == -INFINITY ? 0.f : m[h] * scale_log2;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float e0 = ex2_approx(fmaf(sc[n][2 * h], scale_log2, -mb));
        const float e1 = ex2_approx(fmaf(sc[n][2 * h + 1], scale_log2, -mb));
        l[h] += e0 + e1;
        p[2 * n + h] = pack_bf16x2(e0, e1);
      }
    }
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t f[4];  // dims 0-7 of the step: keys 0-7, 8-15; dims 8-15 the same
      const int row = (mat & 1) * 8 + mr, piece = 2 * n + (mat >> 1);
      ldmatrix4_trans(f, vb + row * C::kRowBytes + ((piece ^ (row & 7)) << 4));
      mma_16816(o[2 * n], p, f[0], f[1]);
      mma_16816(o[2 * n + 1], p, f[2], f[3]);
    }
    __syncwarp();  // the stage is read: it may be loaded again
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }

  // merge of the warps, in order
  cp_async_wait<0>();
  __syncthreads();
  float* s_o = reinterpret_cast<float*>(smem);  // [warp][row][D], then [warp][row] max, sum
  float* s_m = s_o + kWarps * kRows * D;
  float* s_l = s_m + kWarps * kRows;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    const int at = warp * kRows + gr + 8 * h;
    if ((lane & 3) == 0) {
      s_m[at] = m[h];
      s_l[at] = l[h];
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(s_o + at * D + n * 8 + c2) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < s.rows * (D / 8); i += kThreads) {
    const int r = i / (D / 8), col = i % (D / 8) * 8;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * kRows + r]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, x[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2_approx((s_m[w * kRows + r] - base) * scale_log2);  // 0 for a warp without keys
      sum = fmaf(f, s_l[w * kRows + r], sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(f, s_o[(w * kRows + r) * D + col + e], x[e]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no keys: 0, and an LSE of -inf
    const float lse = top * a.scale + logf(sum);
    if (a.chunks > 1) {
      float* part = partial_of<D>(a.partials, a, static_cast<size_t>(g) * a.seg.num_kv_heads + kv_head, chunk);
      float4* dst = reinterpret_cast<float4*>(part + r * D + col);
      dst[0] = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      dst[1] = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
      if (col == 0) part[a.max_rows * D + r] = lse;
    } else {
      const int row = s.row0 + r / group, head = kv_head * group + r % group;
      *reinterpret_cast<uint4*>(a.o + (static_cast<size_t>(row) * a.seg.num_q_heads + head) * D + col) =
          make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                     pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
      if (col == 0 && a.lse != nullptr) a.lse[static_cast<size_t>(head) * a.seg.capacity_q + row] = lse;
    }
  }
}

// Joins the chunks of each (segment, key head), in chunk order, four chunks loaded at once.  Nothing is read
// before the wait, the offsets included: only the wait makes another kernel's writes visible here.
template <int D>
__global__ void __launch_bounds__(kThreads)
cross_token_merge_kernel(const __grid_constant__ CrossTokenArgs a) {
  grid_dependency_wait();
  launch_dependents();
  const int kv_head = blockIdx.x, g = blockIdx.y;
  const TokenSegment s = token_segment(a.seg, g, nullptr);
  const int group = a.seg.num_q_heads / a.seg.num_kv_heads;
  const int n = min(a.chunks, (s.keys + a.chunk_keys - 1) / a.chunk_keys);
  const float* part = partial_of<D>(a.partials, a, static_cast<size_t>(g) * a.seg.num_kv_heads + kv_head, 0);
  const size_t step = cross_token_partial(a.max_rows, D);
  for (int i = threadIdx.x; i < s.rows * (D / 8); i += kThreads) {
    const int r = i / (D / 8), col = i % (D / 8) * 8;
    float top = -INFINITY, sum = 0.f, x[8] = {};
    constexpr int kBatch = 4;  // chunks loaded at once
    for (int c0 = 0; c0 < n; c0 += kBatch) {
      float w[kBatch];
      float4 u[kBatch], v[kBatch];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const float* p = part + min(c0 + c, n - 1) * step;
        w[c] = c0 + c < n ? p[a.max_rows * D + r] : -INFINITY;
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
    const int row = s.row0 + r / group, head = kv_head * group + r % group;
    *reinterpret_cast<uint4*>(a.o + (static_cast<size_t>(row) * a.seg.num_q_heads + head) * D + col) =
        make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                   pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
    if (col == 0 && a.lse != nullptr) a.lse[static_cast<size_t>(head) * a.seg.capacity_q + row] = top + logf(sum);
  }
}

template <int D>
cudaError_t launch(const CrossTokenArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  cudaError_t e = allow_shared_memory<C::kSmemBytes>(cross_token_kernel<D>);
  if (e != cudaSuccess) return e;
  const CrossSegments& s = a.seg;
  e = launch_programmatic(cross_token_kernel<D>, dim3(a.chunks, s.num_kv_heads, s.num_segments), dim3(kThreads),
                          C::kSmemBytes, stream, a);
  if (e != cudaSuccess || a.chunks == 1) return e;
  return launch_programmatic(cross_token_merge_kernel<D>, dim3(s.num_kv_heads, s.num_segments), dim3(kThreads), 0,
                             stream, a);
}

}  // namespace

// Chunks of keys: enough CTAs for several waves (kCtasPerSm on each of 152 SMs), so that segments of
// unlike lengths even out, but chunks of at least 128 keys and no more partial results than that
// takes.
void cross_token_split(const CrossSegments& s, int* chunk_keys, int* chunks) {
  const int64_t pairs = static_cast<int64_t>(s.num_segments) * s.num_kv_heads;
  const int64_t want = (kCrossTokenCtas + pairs - 1) / pairs;
  const int64_t keys = s.max_seqlen_k > 0 ? s.max_seqlen_k : 1;
  int64_t per = (keys + want - 1) / want;
  per = per < 128 ? 128 : (per + 63) / 64 * 64;
  *chunks = static_cast<int>((keys + per - 1) / per);
  *chunk_keys = static_cast<int>(per);
}

cudaError_t launch_cross_token(const CrossTokenArgs& a, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace h3
