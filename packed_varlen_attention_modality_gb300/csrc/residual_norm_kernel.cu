// The step between two branches of a block: the branch's output y joins the residual stream x through a
// norm, a gate and a residual scale, and the stream is normed and modulated for the next branch.  And the
// gradient of both.
//
// Per row (a token; dim values), with r the token's request:
//   u = norm_b(y) w_b,  x' = alpha x + gate_r u,  h = norm(x') w (1 + scale_r) + shift_r
//   norm(x) = c / sqrt(mean(c^2) + eps),  c = x (RMS) or x - mean(x) (layer)
// backward, with xh = norm(x'), yh = norm_b(y), rs and ry their factors:
//   g = dh w (1 + scale),  t = dx' + rs (g - [mean g] - xh mean(g xh)),  dx = alpha t
//   gy = t gate w_b,       dy = ry (gy - [mean gy] - yh mean(gy yh))          ([..]: layer norm only)
//   U_r = sum of dh xh, V_r = sum of t yh over the request's rows:  dshift = sum of dh,
//   dscale = w U, dgate = w_b V,  dw = sum_r (1 + scale_r) U_r,  dw_b = sum_r gate_r V_r
//
// Memory-bound: the forward reads x, y and writes x', h once; the backward reads dx', dh, x', y and writes
// dx, dy once.  A CTA takes a contiguous range of rows, so the request's vectors (w (1 + scale), shift,
// w_b gate) stay in registers from row to row, eight columns a thread, and so do the backward's column
// sums.  Rows come through a ring in shared memory by bulk copies that run several rows ahead: the row sums
// of a row (a shuffle tree and one barrier each) wait on no load.  All arithmetic is fp32; the mean of a layer
// norm is subtracted before the squares are summed, so a large mean costs no digits.
#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kMaxStages = 8;

struct Vec8 {
  float v[8];
};
__device__ __forceinline__ Vec8 unpack(const uint4& p) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ Vec8 load8(const __nv_bfloat16* p) { return unpack(*reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ Vec8 load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Vec8& r) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]),
                                                 pack_bf16x2(r.v[4], r.v[5]), pack_bf16x2(r.v[6], r.v[7])));
}
__device__ __forceinline__ void store8(float* p, const Vec8& r) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(r.v[0], r.v[1], r.v[2], r.v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(r.v[4], r.v[5], r.v[6], r.v[7]));
}
// Eight values of a weight or modulation vector; `none` where there is no vector.
__device__ __forceinline__ Vec8 load_vector(const void* base, int64_t at, int bf16, float none) {
  if (base == nullptr) return Vec8{{none, none, none, none, none, none, none, none}};
  return bf16 ? load8(static_cast<const __nv_bfloat16*>(base) + at) : load8(static_cast<const float*>(base) + at);
}

// Rows [first, first + rows) of CTA c of `ctas`.
__host__ __device__ __forceinline__ int range_start(int n, int ctas, int c) {
  return static_cast<int>(static_cast<int64_t>(n) * c / ctas);
}

// The request of row n and the row at which the next one begins.  Offsets that are not what they should be
// give some request in range.
__device__ __forceinline__ int request_of(const ResidualNormArgs& a, int n, int* end) {
  int lo = 0;
  if (a.cu_requests != nullptr) {
    int hi = a.num_requests - 1;  // largest r with cu_requests[r] <= n
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu_requests[mid] <= n) lo = mid; else hi = mid - 1;
    }
  }
  *end = a.cu_requests == nullptr || lo == a.num_requests - 1 ? a.num_tokens : a.cu_requests[lo + 1];
  return lo;
}

// Sums of two values over the CTA, in a fixed order.  One barrier: the slots alternate, and a slot is
// written again only behind the next sum's barrier, which all threads reach after reading this one's.
struct BlockSum {
  float2 (*slots)[32];
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane == 0) slots[turn][warp] = make_float2(a, b);
    __syncthreads();
    float2 t = lane < warps ? slots[turn][lane] : make_float2(0.f, 0.f);
    turn ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
      t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    }
    return t;
  }
};

// A CTA's rows through a ring of stages in shared memory.  kTensors rows a stage, those of the stream's type
// first; an absent tensor's place is not loaded.
struct RowSource {
  const uint8_t* base;
  int64_t stride;  // bytes
  uint32_t bytes;
};
template <int kTensors>
struct RowRing {
  uint8_t* smem;
  uint64_t* bars;
  RowSource src[kTensors];
  uint32_t at[kTensors], stage_bytes, load_bytes;
  int stages, first, rows;

  __device__ __forceinline__ void issue(int i) {  // one thread; row first + i
    const int s = i % stages;
    const uint32_t bar = smem_u32(bars + s);
    mbar_arrive_expect_tx(bar, load_bytes);
#pragma unroll
    for (int t = 0; t < kTensors; ++t)
      if (src[t].base != nullptr)
        bulk_load(smem_u32(smem + s * stage_bytes + at[t]), src[t].base + (first + i) * src[t].stride, src[t].bytes, bar);
  }
  __device__ __forceinline__ void start() {
    if (threadIdx.x == 0) {
      for (int s = 0; s < stages; ++s) mbar_init(smem_u32(bars + s), 1);
      fence_mbarrier_init();
      for (int i = 0; i < min(stages, rows); ++i) issue(i);
    }
    __syncthreads();
  }
  __device__ __forceinline__ bool wait(int i) const {
    return mbar_wait(smem_u32(bars + i % stages), (i / stages) & 1);
  }
  __device__ __forceinline__ const uint8_t* row(int i, int t) const { return smem + i % stages * stage_bytes + at[t]; }
  // behind a barrier that follows the last read of row i
  __device__ __forceinline__ void refill(int i) {
    if (threadIdx.x == 0 && i + stages < rows) issue(i + stages);
  }
  // a wait ran out: nothing is left in flight
  __device__ __forceinline__ void drain(int i, unsigned int* err) {
    if (threadIdx.x != 0) return;
    record_error(err, kErrTimeout);
    for (int j = i; j < min(i + stages, rows); ++j) wait(j);
  }
};

__host__ __device__ constexpr uint32_t row_place(uint32_t bytes) { return (bytes + 127) / 128 * 128; }

// 1 / sqrt(mean(c^2) + eps) of the row, which is centred in place for a layer norm; 1 without a norm.
template <int kVecs>
__device__ __forceinline__ float row_factor(Vec8 (&x)[kVecs], const bool (&own)[kVecs], int kind, float inv_dim, float eps,
                                            BlockSum& sum) {
  if (kind == kNormNone) return 1.f;
  if (kind == kNormLayer) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[k].v[e];
    const float mean = sum(s, 0.f).x * inv_dim;
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k].v[e] = own[k] ? x[k].v[e] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[k].v[e], x[k].v[e], s);
  return rsqrtf(sum(s, 0.f).x * inv_dim + eps);
}

template <typename X, int kVecs, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas)
residual_norm_kernel(const __grid_constant__ ResidualNormArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kMaxStages];
  __shared__ float2 slots[2][32];
  grid_dependency_wait();
  launch_dependents();
  const int dim = a.dim, ctas = static_cast<int>(gridDim.x);
  RowRing<2> ring;
  ring.smem = smem;
  ring.bars = bars;
  ring.stages = stages;
  ring.first = range_start(a.num_tokens, ctas, blockIdx.x);
  ring.rows = range_start(a.num_tokens, ctas, blockIdx.x + 1) - ring.first;
  const uint32_t xb = dim * sizeof(X), yb = a.y != nullptr ? dim * 2 : 0;
  ring.src[0] = RowSource{static_cast<const uint8_t*>(a.x), a.x_stride * static_cast<int64_t>(sizeof(X)), xb};
  ring.src[1] = RowSource{reinterpret_cast<const uint8_t*>(a.y), a.y_stride * 2, yb};
  ring.at[0] = 0;
  ring.at[1] = row_place(xb);
  ring.stage_bytes = row_place(xb) + row_place(yb);
  ring.load_bytes = xb + yb;
  ring.start();

  BlockSum sum{slots};
  const float inv_dim = 1.f / dim;
  int col[kVecs];
  bool own[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    col[k] = (k * blockDim.x + threadIdx.x) * 8;
    own[k] = col[k] < dim;
  }
  Vec8 gain[kVecs], shift[kVecs], gate[kVecs];
  int request_end = ring.first;
  for (int i = 0; i < ring.rows; ++i) {
    const int n = ring.first + i;
    if (n >= request_end) {
      const int r = request_of(a, n, &request_end);
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!own[k]) continue;
        const Vec8 w = load_vector(a.weight, col[k], a.weight_bf16, 1.f);
        const Vec8 sc = load_vector(a.scale, r * a.scale_stride + col[k], a.mod_bf16, 0.f);
        const Vec8 wb = load_vector(a.branch_weight, col[k], a.weight_bf16, 1.f);
        const Vec8 g = load_vector(a.gate, r * a.gate_stride + col[k], a.mod_bf16, 1.f);
        shift[k] = load_vector(a.shift, r * a.shift_stride + col[k], a.mod_bf16, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          gain[k].v[e] = w.v[e] * (1.f + sc.v[e]);
          gate[k].v[e] = wb.v[e] * g.v[e];
        }
      }
    }
    const bool ok = ring.wait(i);
    Vec8 x[kVecs], y[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      x[k] = y[k] = Vec8{};
      if (!own[k]) continue;
      x[k] = load8(reinterpret_cast<const X*>(ring.row(i, 0)) + col[k]);
      if (yb > 0) y[k] = load8(reinterpret_cast<const __nv_bfloat16*>(ring.row(i, 1)) + col[k]);
    }
    if (__syncthreads_or(!ok)) {  // the whole CTA leaves together
      ring.drain(i, a.err);
      return;
    }
    ring.refill(i);
    if (yb > 0) {
      const float ry = row_factor(y, own, a.branch_norm, inv_dim, a.eps, sum);
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!own[k]) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k].v[e] = fmaf(y[k].v[e] * ry, gate[k].v[e], a.residual_scale * x[k].v[e]);
        store8(static_cast<X*>(a.x_out) + n * a.x_out_stride + col[k], x[k]);
      }
    }
    if (a.norm == kNormNone) continue;
    const float rs = row_factor(x, own, a.norm, inv_dim, a.eps, sum);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!own[k]) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k].v[e] = fmaf(x[k].v[e] * rs, gain[k].v[e], shift[k].v[e]);
      store8(a.h + n * a.h_stride + col[k], x[k]);
    }
  }
}

// Backward.  Column sums of a CTA's rows of request r (dh, dh xh, t yh) go to slot c + r: along the rows c and
// r only grow, one at least at each new pair, so no two pairs share a slot.
constexpr int kSums = 3;

template <typename X, int kVecs, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas)
residual_norm_bwd_kernel(const __grid_constant__ ResidualNormArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kMaxStages];
  __shared__ float2 slots[2][32];
  grid_dependency_wait();
  launch_dependents();
  const int dim = a.dim, ctas = static_cast<int>(gridDim.x);
  RowRing<4> ring;
  ring.smem = smem;
  ring.bars = bars;
  ring.stages = stages;
  ring.first = range_start(a.num_tokens, ctas, blockIdx.x);
  ring.rows = range_start(a.num_tokens, ctas, blockIdx.x + 1) - ring.first;
  const uint32_t xb = dim * sizeof(X), yb = dim * 2;
  const bool has_dx = a.dx_out != nullptr, has_h = a.norm != kNormNone, has_y = a.y != nullptr;
  ring.src[0] = RowSource{static_cast<const uint8_t*>(a.x), a.x_stride * static_cast<int64_t>(sizeof(X)), xb};
  ring.src[1] = RowSource{static_cast<const uint8_t*>(a.dx_out), a.dx_out_stride * static_cast<int64_t>(sizeof(X)), xb};
  ring.src[2] = RowSource{reinterpret_cast<const uint8_t*>(a.dh), a.dh_stride * 2, yb};
  ring.src[3] = RowSource{reinterpret_cast<const uint8_t*>(a.y), a.y_stride * 2, yb};
  if (!has_h) ring.src[0].base = ring.src[2].base = nullptr;
  uint32_t place = 0;
  ring.load_bytes = 0;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    ring.at[t] = place;
    if (ring.src[t].base == nullptr) continue;
    place += row_place(ring.src[t].bytes);
    ring.load_bytes += ring.src[t].bytes;
  }
  ring.stage_bytes = place;
  ring.start();

  BlockSum sum{slots};
  const float inv_dim = 1.f / dim;
  int col[kVecs];
  bool own[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    col[k] = (k * blockDim.x + threadIdx.x) * 8;
    own[k] = col[k] < dim;
  }
  Vec8 gain[kVecs], gate[kVecs];
  Vec8 sums[kSums][kVecs] = {};
  int request = -1, request_end = ring.first;
  auto flush = [&] {
    if (request < 0) return;
    float* slot = a.partials + static_cast<size_t>(blockIdx.x + request) * kSums * dim;
#pragma unroll
    for (int j = 0; j < kSums; ++j)
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (own[k]) {
          float4* p = reinterpret_cast<float4*>(slot + static_cast<size_t>(j) * dim + col[k]);
          const Vec8& s = sums[j][k];
          p[0] = make_float4(s.v[0], s.v[1], s.v[2], s.v[3]);
          p[1] = make_float4(s.v[4], s.v[5], s.v[6], s.v[7]);
        }
        sums[j][k] = Vec8{};
      }
  };
  for (int i = 0; i < ring.rows; ++i) {
    const int n = ring.first + i;
    if (n >= request_end) {
      flush();
      request = request_of(a, n, &request_end);
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!own[k]) continue;
        const Vec8 w = load_vector(a.weight, col[k], a.weight_bf16, 1.f);
        const Vec8 sc = load_vector(a.scale, request * a.scale_stride + col[k], a.mod_bf16, 0.f);
        const Vec8 wb = load_vector(a.branch_weight, col[k], a.weight_bf16, 1.f);
        const Vec8 g = load_vector(a.gate, request * a.gate_stride + col[k], a.mod_bf16, 1.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          gain[k].v[e] = w.v[e] * (1.f + sc.v[e]);
          gate[k].v[e] = wb.v[e] * g.v[e];
        }
      }
    }
    const bool ok = ring.wait(i);
    Vec8 x[kVecs], t[kVecs], g[kVecs], y[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      x[k] = t[k] = g[k] = y[k] = Vec8{};
      if (!own[k]) continue;
      if (has_h) {
        x[k] = load8(reinterpret_cast<const X*>(ring.row(i, 0)) + col[k]);
        g[k] = load8(reinterpret_cast<const __nv_bfloat16*>(ring.row(i, 2)) + col[k]);
      }
      if (has_dx) t[k] = load8(reinterpret_cast<const X*>(ring.row(i, 1)) + col[k]);
      if (has_y) y[k] = load8(reinterpret_cast<const __nv_bfloat16*>(ring.row(i, 3)) + col[k]);
    }
    if (__syncthreads_or(!ok)) {
      ring.drain(i, a.err);
      return;
    }
    ring.refill(i);
    if (has_h) {
      const float rs = row_factor(x, own, a.norm, inv_dim, a.eps, sum);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[k].v[e] *= rs;
          sums[0][k].v[e] += g[k].v[e];
          sums[1][k].v[e] = fmaf(g[k].v[e], x[k].v[e], sums[1][k].v[e]);
          g[k].v[e] = own[k] ? g[k].v[e] * gain[k].v[e] : 0.f;
          s0 += g[k].v[e];
          s1 = fmaf(g[k].v[e], x[k].v[e], s1);
        }
      const float2 m = sum(s0, s1);
      const float mean = a.norm == kNormLayer ? m.x * inv_dim : 0.f, dot = m.y * inv_dim;
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          t[k].v[e] = fmaf(rs, g[k].v[e] - mean - x[k].v[e] * dot, t[k].v[e]);
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!own[k]) continue;
      Vec8 d;
#pragma unroll
      for (int e = 0; e < 8; ++e) d.v[e] = a.residual_scale * t[k].v[e];
      store8(static_cast<X*>(a.dx) + n * a.dx_stride + col[k], d);
    }
    if (!has_y) continue;
    const float ry = row_factor(y, own, a.branch_norm, inv_dim, a.eps, sum);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[k].v[e] *= ry;
        sums[2][k].v[e] = fmaf(t[k].v[e], y[k].v[e], sums[2][k].v[e]);
        t[k].v[e] = own[k] ? t[k].v[e] * gate[k].v[e] : 0.f;
        s0 += t[k].v[e];
        s1 = fmaf(t[k].v[e], y[k].v[e], s1);
      }
    float mean = 0.f, dot = 0.f;
    if (a.branch_norm != kNormNone) {
      const float2 m = sum(s0, s1);
      mean = a.branch_norm == kNormLayer ? m.x * inv_dim : 0.f;
      dot = m.y * inv_dim;
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!own[k]) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[k].v[e] = ry * (t[k].v[e] - mean - y[k].v[e] * dot);
      store8(a.dy + n * a.dy_stride + col[k], t[k]);
    }
  }
  flush();
}

// The requests' column sums: their CTAs' slots, in CTA order within each strand, then over the strands.
// A request's terms of the weights' gradients replace its first slot (its own columns of this block alone),
// where weight_sum_kernel adds them over the requests; a single request's are the gradients themselves.
constexpr int kSumColumns = 32, kSumStrands = 8;
__global__ void __launch_bounds__(kSumColumns* kSumStrands)
request_sum_kernel(const __grid_constant__ ResidualNormArgs a, int ctas) {
  __shared__ float part[kSums][kSumStrands][kSumColumns];
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x % kSumColumns, strand = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + lane;
  const bool own = c < a.dim;
  const bool single = a.num_requests == 1;
  for (int r = blockIdx.y; r < a.num_requests; r += gridDim.y) {
    const int n = a.num_tokens;
    const int first = r == 0 || a.cu_requests == nullptr ? 0 : min(max(a.cu_requests[r], 0), n);
    const int end = r == a.num_requests - 1 || a.cu_requests == nullptr ? n : min(max(a.cu_requests[r + 1], 0), n);
    int lo = 0, hi = -1;  // CTAs with rows of this request
    if (first < end) {
      // the CTA of row i: the largest c with start(c) <= i
      lo = static_cast<int>(((static_cast<int64_t>(first) + 1) * ctas - 1) / n);
      hi = static_cast<int>((static_cast<int64_t>(end) * ctas - 1) / n);
    }
    float s[kSums] = {};
    if (own) {
      for (int k = lo + strand; k <= hi; k += kSumStrands) {
        const float* p = a.partials + static_cast<size_t>(k + r) * kSums * a.dim + c;
#pragma unroll
        for (int j = 0; j < kSums; ++j) s[j] += p[static_cast<size_t>(j) * a.dim];
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSums; ++j) part[j][strand][lane] = s[j];
    __syncthreads();
    if (strand != 0 || !own) continue;
#pragma unroll
    for (int j = 0; j < kSums; ++j) {
      s[j] = 0.f;
#pragma unroll
      for (int k = 0; k < kSumStrands; ++k) s[j] += part[j][k][lane];
    }
    auto value = [&](const void* base, int64_t at, int bf16, float none) {
      if (base == nullptr) return none;
      return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]) : static_cast<const float*>(base)[at];
    };
    const size_t at = static_cast<size_t>(r) * a.dim + c;
    if (a.dshift != nullptr) a.dshift[at] = s[0];
    if (a.dscale != nullptr) a.dscale[at] = s[1] * value(a.weight, c, a.weight_bf16, 1.f);
    if (a.dgate != nullptr) a.dgate[at] = s[2] * value(a.branch_weight, c, a.weight_bf16, 1.f);
    const float w = s[1] * (1.f + value(a.scale, r * a.scale_stride + c, a.mod_bf16, 0.f));
    const float b = s[2] * value(a.gate, r * a.gate_stride + c, a.mod_bf16, 1.f);
    if (single) {
      if (a.dweight != nullptr) a.dweight[c] = w;
      if (a.dbranch_weight != nullptr) a.dbranch_weight[c] = b;
    } else if (lo <= hi) {
      float* p = a.partials + static_cast<size_t>(lo + r) * kSums * a.dim + c;
      p[0] = w;
      p[a.dim] = b;
    }
  }
}

__global__ void __launch_bounds__(kSumColumns* kSumStrands)
weight_sum_kernel(const __grid_constant__ ResidualNormArgs a, int ctas) {
  __shared__ float part[2][kSumStrands][kSumColumns];
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x % kSumColumns, strand = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + lane;
  float w = 0.f, b = 0.f;
  for (int r = strand; r < a.num_requests && c < a.dim; r += kSumStrands) {
    const int n = a.num_tokens;
    const int first = r == 0 ? 0 : min(max(a.cu_requests[r], 0), n);
    const int end = r == a.num_requests - 1 ? n : min(max(a.cu_requests[r + 1], 0), n);
    if (first >= end) continue;
    const int lo = static_cast<int>(((static_cast<int64_t>(first) + 1) * ctas - 1) / n);
    const float* p = a.partials + static_cast<size_t>(lo + r) * kSums * a.dim + c;
    w += p[0];
    b += p[a.dim];
  }
  part[0][strand][lane] = w;
  part[1][strand][lane] = b;
  __syncthreads();
  if (strand != 0 || c >= a.dim) return;
  w = b = 0.f;
#pragma unroll
  for (int k = 0; k < kSumStrands; ++k) {
    w += part[0][k][lane];
    b += part[1][k][lane];
  }
  if (a.dweight != nullptr) a.dweight[c] = w;
  if (a.dbranch_weight != nullptr) a.dbranch_weight[c] = b;
}

// Threads of a row: eight columns each (sixteen above 5,120), whole warps.
int row_threads(int dim, int vecs) { return (dim + 256 * vecs - 1) / (256 * vecs) * 32; }

template <typename X, int kVecs, int kThreads, int kCtas>
cudaError_t launch_rows(const ResidualNormArgs& a, bool backward, int sms, cudaStream_t stream) {
  constexpr int kSmem = 224 * 1024 / kCtas - 2048;
  auto fwd = residual_norm_kernel<X, kVecs, kThreads, kCtas>;
  auto bwd = residual_norm_bwd_kernel<X, kVecs, kThreads, kCtas>;
  const uint32_t xb = row_place(a.dim * sizeof(X)), yb = row_place(a.dim * 2);
  const bool has_h = a.norm != kNormNone, has_y = a.y != nullptr;
  const uint32_t stage = backward ? (has_h ? xb + yb : 0) + (a.dx_out != nullptr ? xb : 0) + (has_y ? yb : 0)
                                  : xb + (has_y ? yb : 0);
  int stages = static_cast<int>(kSmem / stage);
  stages = stages < 1 ? 1 : stages > kMaxStages ? kMaxStages : stages;
  const cudaError_t e = allow_shared_memory<kSmem>(backward ? bwd : fwd);
  if (e != cudaSuccess) return e;
  const int ctas = residual_norm_ctas(a.num_tokens, sms * kCtas);
  return launch_programmatic(backward ? bwd : fwd, dim3(ctas), dim3(row_threads(a.dim, kVecs)), stages * stage, stream, a,
                             stages);
}

template <typename X>
cudaError_t launch_type(const ResidualNormArgs& a, bool backward, int sms, int* ctas, cudaStream_t stream) {
  *ctas = residual_norm_ctas(a.num_tokens, sms * (a.dim <= 2560 ? 2 : 1));
  if (a.dim <= 2560) return launch_rows<X, 1, 320, 2>(a, backward, sms, stream);
  if (a.dim <= 5120) return launch_rows<X, 1, 640, 1>(a, backward, sms, stream);
  return launch_rows<X, 2, 512, 1>(a, backward, sms, stream);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs& a, bool backward, cudaStream_t stream) {
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  int ctas = 0;
  if (a.num_tokens > 0) {
    const cudaError_t e = a.x_fp32 ? launch_type<float>(a, backward, sms, &ctas, stream)
                                   : launch_type<__nv_bfloat16>(a, backward, sms, &ctas, stream);
    if (e != cudaSuccess) return e;
  }
  const bool weights = a.dweight != nullptr || a.dbranch_weight != nullptr;
  if (!backward || (!weights && a.dshift == nullptr && a.dscale == nullptr && a.dgate == nullptr)) return cudaSuccess;
  const int columns = (a.dim + kSumColumns - 1) / kSumColumns;
  const cudaError_t e = launch_programmatic(request_sum_kernel, dim3(columns, a.num_requests < 1024 ? a.num_requests : 1024),
                                            dim3(kSumColumns * kSumStrands), 0, stream, a, ctas);
  if (e != cudaSuccess || !weights || a.num_requests == 1) return e;
  return launch_programmatic(weight_sum_kernel, dim3(columns), dim3(kSumColumns * kSumStrands), 0, stream, a, ctas);
}

}  // namespace h3
