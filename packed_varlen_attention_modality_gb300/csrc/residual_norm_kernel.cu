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
// Memory-bound: the forward reads x, y and writes x', h once; the backward reads dx', dh, x', y and writes dx, dy
// once.  Measured with a bf16 stream of 5,120 values a row: forward, 58,758 rows of four requests, a layer norm and a
// gate, 378 us (floor 355 at the rate of a copy, 94 %); backward, 29,001 rows of three requests, both norms RMS, 357 us
// (floor 263, 74 %).
//
// A CTA takes a contiguous range of rows, so the request's vectors (w (1 + scale), shift, w_b gate) stay in registers
// from row to row, 16 columns a thread, and so do the backward's column sums.  (8 columns, with the registers of twice
// the threads: backward 436 us against 390.)  Rows come through a ring in shared memory by bulk copies that run
// several rows ahead, so a row waits on no load but on its sums alone.  The copies name their lines as the first to
// leave L2, since nothing reads them again: forward 386 us against 411 at that step.  The warps exchange a row's sums
// once for each norm forward.  Backward all that the inputs give goes round once, the branch's dot product among it;
// only with a layer norm a second exchange follows (for all norms: 390 us against 375).  All arithmetic is fp32, two
// values an instruction (one at a time: forward 395 us, backward 441).
#include <algorithm>

#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kMaxStages = 8;
constexpr int kVecs = 2;  // groups of eight columns a thread

// Eight values as packed pairs: an instruction takes two of them.
struct Vec8 {
  float2 p[4];
};
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ Vec8 all8(float v) { return Vec8{{both(v), both(v), both(v), both(v)}}; }
// Eight values as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ Vec8 values() const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    Vec8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    return r;
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ Vec8 values() const {
    return Vec8{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
  }
};
template <typename T>
__device__ __forceinline__ Vec8 load8(const T* p) {
  Raw8<T> r;
  r.load(p);
  return r.values();
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Vec8& r) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(r.p[0].x, r.p[0].y), pack_bf16x2(r.p[1].x, r.p[1].y),
                                                 pack_bf16x2(r.p[2].x, r.p[2].y), pack_bf16x2(r.p[3].x, r.p[3].y)));
}
__device__ __forceinline__ void store8(float* p, const Vec8& r) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(r.p[0].x, r.p[0].y, r.p[1].x, r.p[1].y));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(r.p[2].x, r.p[2].y, r.p[3].x, r.p[3].y));
}
// Eight values of a weight or modulation vector; `none` where there is no vector.
__device__ __forceinline__ Vec8 load_vector(const void* base, int64_t at, int bf16, float none) {
  if (base == nullptr) return all8(none);
  return bf16 ? load8(static_cast<const __nv_bfloat16*>(base) + at) : load8(static_cast<const float*>(base) + at);
}

// Rows [first, first + rows) of CTA c of `ctas`.
__host__ __device__ __forceinline__ int range_start(int n, int ctas, int c) {
  return static_cast<int>(static_cast<int64_t>(n) * c / ctas);
}

// The request of row n and the row at which the next one begins.  Offsets that are not what they should be
// (check_offsets records them) give some request in range.
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

// The grid looks over the offsets: they start at 0, do not fall, end at num_tokens.
__device__ __forceinline__ void check_offsets(const ResidualNormArgs& a) {
  if (a.cu_requests == nullptr) return;
  const int first = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x);
  bool bad = first == 0 && (a.cu_requests[0] != 0 || a.cu_requests[a.num_requests] != a.num_tokens);
  for (int64_t r = first; r < a.num_requests; r += gridDim.x * blockDim.x) bad |= a.cu_requests[r + 1] < a.cu_requests[r];
  if (bad) record_error(a.err, kErrBadCuSeqlens);
}

// The sums of N values over the lanes, on every lane.  Of three values and more a lane gives half to a partner and
// takes the partner's share of the others while more than one is left, so they cost little more than one: lane l ends
// with the value whose number its first bits spell, and hands it round.
template <int N>
__device__ __forceinline__ void lane_sums(float (&v)[N]) {
  if constexpr (N <= 2) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  } else {
    constexpr int P = N <= 4 ? 4 : 8;  // values, filled up to a power of two
    const int lane = threadIdx.x & 31;
    float w[P];
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = i < N ? v[i] : 0.f;
    int o = 16;
#pragma unroll
    for (int n = P / 2; n > 0; n /= 2, o /= 2) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = upper ? w[i] : w[n + i], keep = upper ? w[n + i] : w[i];
        w[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
#pragma unroll
    for (; o > 0; o /= 2) w[0] += __shfl_xor_sync(0xffffffffu, w[0], o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, w[0], i * (32 / P));
  }
}

// What the warps tell one another about a row, one barrier each time: the slots alternate, and one is written again
// only behind the next exchange's barrier, which all threads reach after reading this one's.
constexpr int kMaxTold = 6;
template <int kWarps>
struct Told {
  float v[2][kWarps][kMaxTold];
};
template <int kWarps>
struct Exchange {
  Told<kWarps>& told;
  int turn = 0;
  // Publishes the warp's v; then each lane holds the values of warp `lane` (0 past the last), `first` those of warp
  // 0.  False if any thread says so.
  template <int N>
  __device__ __forceinline__ bool operator()(float (&v)[N], float (&first)[N], bool ok) {
    static_assert(N <= kMaxTold);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) told.v[turn][warp][i] = v[i];
    }
    const bool failed = __syncthreads_or(!ok);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = lane < static_cast<int>(blockDim.x >> 5) ? told.v[turn][lane][i] : 0.f;
      first[i] = told.v[turn][0][i];
    }
    turn ^= 1;
    return !failed;
  }
};

// The same in two halves, so that a warp can do something else while it waits for the others: say() publishes,
// hear() waits.  Calls alternate; slots are written again two calls later, behind a hear() for which every warp has
// left its own call before.
template <int kWarps>
struct Parley {
  float v[2][kWarps][kMaxTold];
  uint64_t bar;
  int failed[2];
};
template <int kWarps, int N>
struct Talk {
  Parley<kWarps>& p;
  int turn = 0, heard = 0;
  __device__ __forceinline__ void say(const float (&v)[N], bool ok) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!ok) p.failed[turn & 1] = 1;
    __syncwarp();
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) p.v[turn & 1][warp][i] = v[i];
      mbar_arrive(smem_u32(&p.bar));
    }
    ++turn;
  }
  // Each lane's v: the values of warp `lane` (0 past the last); `first`: those of warp 0.  False if any thread said
  // so, or a wait runs out.
  __device__ __forceinline__ bool hear(float (&v)[N], float (&first)[N]) {
    const int lane = threadIdx.x & 31;
    const bool there = mbar_wait(smem_u32(&p.bar), heard & 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = lane < static_cast<int>(blockDim.x >> 5) ? p.v[heard & 1][lane][i] : 0.f;
      first[i] = p.v[heard & 1][0][i];
    }
    const bool fine = *const_cast<volatile int*>(&p.failed[heard & 1]) == 0;
    ++heard;
    return __all_sync(0xffffffffu, there && fine);
  }
};

// Columns of warp w's.
template <int kVecs>
__device__ __forceinline__ float columns_of(int w, int dim) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) n += min(max(dim - (k * static_cast<int>(blockDim.x) + w * 32) * 8, 0), 256);
  return static_cast<float>(w < static_cast<int>(blockDim.x >> 5) ? n : 0);
}

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

  int stage, parity;   // of the row that is read
  int freed, freed_at;  // rows whose stages have been given back, the stage of the next one

  __device__ __forceinline__ void issue(int i, int s) {  // one thread; the CTA's row i into stage s
    const uint64_t policy = l2_policy_evict_first();  // every row is read once
    const uint32_t bar = smem_u32(bars + s);
    mbar_arrive_expect_tx(bar, load_bytes);
#pragma unroll
    for (int t = 0; t < kTensors; ++t)
      if (src[t].base != nullptr)
        bulk_load_hint(smem_u32(smem + s * stage_bytes + at[t]), src[t].base + (first + i) * src[t].stride,
                       src[t].bytes, bar, policy);
  }
  __device__ __forceinline__ void start() {
    stage = parity = freed = freed_at = 0;
    if (threadIdx.x == 0) {
      for (int s = 0; s < stages; ++s) mbar_init(smem_u32(bars + s), 1);
      fence_mbarrier_init();
      for (int i = 0; i < min(stages, rows); ++i) issue(i, i);
    }
    __syncthreads();
  }
  __device__ __forceinline__ bool wait() const { return mbar_wait(smem_u32(bars + stage), parity); }
  __device__ __forceinline__ const uint8_t* row(int t) const { return smem + stage * stage_bytes + at[t]; }
  __device__ __forceinline__ void advance() {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
  // Gives the stages of all rows before row i back, behind a barrier that follows their last read.
  __device__ __forceinline__ void release(int i) {
    for (; freed < i; ++freed) {
      if (threadIdx.x == 0 && freed + stages < rows) issue(freed + stages, freed_at);
      if (++freed_at == stages) freed_at = 0;
    }
  }
  // A wait ran out (the current row's, or another warp's): nothing is left in flight.
  __device__ __forceinline__ void drain(unsigned int* err) {
    if (threadIdx.x != 0) return;
    record_error(err, kErrTimeout);
    for (int j = freed; j < min(freed + stages, rows); ++j)
      mbar_wait(smem_u32(bars + j % stages), (j / stages) & 1);
  }
};

__host__ __device__ constexpr uint32_t row_place(size_t bytes) { return static_cast<uint32_t>((bytes + 127) / 128 * 128); }

// The sums of a row that a norm needs, in two steps around an exchange.  A layer norm's squares are summed about the
// warp's own mean, and the warps' sums are joined about the mean of all (from the first warp's, exactly in the
// sense that no large numbers cancel), so a large mean costs no digits and one exchange does.
template <int kVecs>
__device__ __forceinline__ float warp_mean(const Vec8 (&x)[kVecs], float inv_columns) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fadd2(s, x[k].p[e]);
  float t[1] = {s.x + s.y};
  lane_sums(t);
  return t[0] * inv_columns;
}
template <bool kLayer, int kVecs>
__device__ __forceinline__ float lane_squares(const Vec8 (&x)[kVecs], const bool (&own)[kVecs], float mean) {
  float2 s = make_float2(0.f, 0.f);
  const float2 m = both(-mean);
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    if (!own[k]) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 c = kLayer ? fadd2(x[k].p[e], m) : x[k].p[e];
      s = ffma2(c, c, s);
    }
  }
  return s.x + s.y;
}
struct Stats {
  float mean, factor;  // 0 and 1 / sqrt(mean(x^2) + eps) for an RMS norm
};
// One norm's statistics, by an exchange of their own.  (kLayer: a norm of the call is a layer norm.)
template <int kVecs, bool kLayer, typename Tell>
__device__ __forceinline__ bool row_stats(const Vec8 (&x)[kVecs], const bool (&own)[kVecs], int kind, float inv_mine,
                                          float theirs, float inv_dim, float eps, Tell& tell, bool ok, Stats* r) {
  if constexpr (kLayer) {
    const bool layer = kind == kNormLayer;
    float first[2], v[2];
    v[0] = layer ? warp_mean(x, inv_mine) : 0.f;
    float q[1] = {lane_squares<true>(x, own, v[0])};
    lane_sums(q);
    v[1] = q[0];
    ok = tell(v, first, ok);
    const float d = v[0] - first[0];  // of this lane's warp's mean from the first's
    float t[2] = {theirs * d, fmaf(theirs * d, d, v[1])};
    lane_sums(t);
    const float shift = t[0] * inv_dim;
    r->mean = first[0] + shift;
    r->factor = rsqrtf((t[1] - t[0] * shift) * inv_dim + eps);
  } else {
    float q[1] = {lane_squares<false>(x, own, 0.f)}, first[1];
    lane_sums(q);
    ok = tell(q, first, ok);
    lane_sums(q);
    r->mean = 0.f;
    r->factor = rsqrtf(q[0] * inv_dim + eps);
  }
  return ok;
}

template <typename X, int kVecs, int kThreads, int kCtas, bool kLayer>
__global__ void __launch_bounds__(kThreads, kCtas)
residual_norm_kernel(const __grid_constant__ ResidualNormArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kMaxStages];
  __shared__ Told<kThreads / 32> told;
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
  check_offsets(a);

  Exchange<kThreads / 32> tell{told};
  const float inv_dim = 1.f / dim;
  const float mine = columns_of<kVecs>(threadIdx.x >> 5, dim), theirs = columns_of<kVecs>(threadIdx.x & 31, dim);
  const float inv_mine = mine > 0.f ? 1.f / mine : 0.f;
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
        for (int e = 0; e < 4; ++e) {
          gain[k].p[e] = fmul2(w.p[e], fadd2(both(1.f), sc.p[e]));
          gate[k].p[e] = fmul2(wb.p[e], g.p[e]);
        }
      }
    }
    const bool ok = ring.wait();
    Vec8 x[kVecs], y[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      x[k] = y[k] = Vec8{};
      if (!own[k]) continue;
      x[k] = load8(reinterpret_cast<const X*>(ring.row(0)) + col[k]);
      if (yb > 0) y[k] = load8(reinterpret_cast<const __nv_bfloat16*>(ring.row(1)) + col[k]);
    }
    // the first exchange of the row is also where a wait that ran out is heard of, and the last read of its stage
    const bool branch = yb > 0 && a.branch_norm != kNormNone, norm = a.norm != kNormNone;
    Stats st{0.f, 1.f};
    bool fine = true;
    if (branch) {
      fine = row_stats<kVecs, kLayer>(y, own, a.branch_norm, inv_mine, theirs, inv_dim, a.eps, tell, ok, &st);
    }
    if (yb > 0) {
      const float2 m = both(-st.mean), f = both(st.factor), alpha = both(a.residual_scale);
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!own[k]) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c = kLayer ? fadd2(y[k].p[e], m) : y[k].p[e];
          x[k].p[e] = ffma2(fmul2(c, f), gate[k].p[e], fmul2(alpha, x[k].p[e]));
        }
      }
    }
    if (norm) fine = row_stats<kVecs, kLayer>(x, own, a.norm, inv_mine, theirs, inv_dim, a.eps, tell, ok && fine, &st);
    else if (!branch) fine = !__syncthreads_or(!ok);
    if (!fine) {  // the whole CTA leaves together
      ring.drain(a.err);
      return;
    }
    ring.advance();
    ring.release(i + 1);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!own[k]) continue;
      if (yb > 0) store8(static_cast<X*>(a.x_out) + n * a.x_out_stride + col[k], x[k]);
      if (!norm) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 c = kLayer ? fadd2(x[k].p[e], both(-st.mean)) : x[k].p[e];
        x[k].p[e] = ffma2(fmul2(c, both(st.factor)), gain[k].p[e], shift[k].p[e]);
      }
      store8(a.h + n * a.h_stride + col[k], x[k]);
    }
  }
}

// Backward.  Column sums of a CTA's rows of request r (dh, dh xh, t yh) go to slot c + r: along the rows c and
// r only grow, one at least at each new pair, so no two pairs share a slot.
constexpr int kSums = 3;

template <typename X, int kVecs, int kThreads, int kCtas, bool kLayer>
__global__ void __launch_bounds__(kThreads, kCtas)
residual_norm_bwd_kernel(const __grid_constant__ ResidualNormArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kMaxStages];
  __shared__ Parley<kThreads / 32> inputs, dots;
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
  if (threadIdx.x == 0) {
    for (Parley<kThreads / 32>* p : {&inputs, &dots}) {
      mbar_init(smem_u32(&p->bar), blockDim.x >> 5);
      p->failed[0] = p->failed[1] = 0;
    }
  }
  ring.start();
  check_offsets(a);

  constexpr int kTold = 6, kDots = 2;
  Talk<kThreads / 32, kTold> row_talk{inputs};
  Talk<kThreads / 32, kDots> dot_talk{dots};
  const float inv_dim = 1.f / dim;
  const float mine = columns_of<kVecs>(threadIdx.x >> 5, dim), theirs = columns_of<kVecs>(threadIdx.x & 31, dim);
  const float inv_mine = mine > 0.f ? 1.f / mine : 0.f;
  int col[kVecs];
  bool own[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    col[k] = (k * blockDim.x + threadIdx.x) * 8;
    own[k] = col[k] < dim;
  }
  Vec8 gain[kVecs], gate[kVecs];
  Vec8 sums[kSums][kVecs] = {};
  const bool want_shift = a.dshift != nullptr;
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
          p[0] = make_float4(s.p[0].x, s.p[0].y, s.p[1].x, s.p[1].y);
          p[1] = make_float4(s.p[2].x, s.p[2].y, s.p[3].x, s.p[3].y);
        }
        sums[j][k] = Vec8{};
      }
  };
  const bool layer = kLayer && a.norm == kNormLayer, branch_layer = kLayer && a.branch_norm == kNormLayer;
  const bool branch = has_y && a.branch_norm != kNormNone;
  // A row is read once and kept as it lies in memory for the second look, where the registers are there for it (29,001
  // rows of 5,120: 357 us against 375; with a layer norm it spills: 20,000 rows 425 against 334).
  constexpr bool kKeep = !kLayer && 65536 / (kThreads * kCtas) > 128;
  Raw8<X> raw_x[kVecs], raw_d[kVecs];
  Raw8<__nv_bfloat16> raw_g[kVecs], raw_y[kVecs];
  auto fetch = [&](int k) {
    if (has_h) raw_x[k].load(reinterpret_cast<const X*>(ring.row(0)) + col[k]);
    if (has_dx) raw_d[k].load(reinterpret_cast<const X*>(ring.row(1)) + col[k]);
    if (has_h) raw_g[k].load(reinterpret_cast<const __nv_bfloat16*>(ring.row(2)) + col[k]);
    if (has_y) raw_y[k].load(reinterpret_cast<const __nv_bfloat16*>(ring.row(3)) + col[k]);
  };
  auto load_x = [&](int k) { return kKeep ? raw_x[k].values() : load8(reinterpret_cast<const X*>(ring.row(0)) + col[k]); };
  auto load_g = [&](int k) {
    return kKeep ? raw_g[k].values() : load8(reinterpret_cast<const __nv_bfloat16*>(ring.row(2)) + col[k]);
  };
  auto load_y = [&](int k) {
    return kKeep ? raw_y[k].values() : load8(reinterpret_cast<const __nv_bfloat16*>(ring.row(3)) + col[k]);
  };
  auto load_d = [&](int k) {
    if (!has_dx) return Vec8{};
    return kKeep ? raw_d[k].values() : load8(reinterpret_cast<const X*>(ring.row(1)) + col[k]);
  };
  Vec8 t[kVecs], y[kVecs];  // (a layer norm) of the row whose dot product is on its way: t gate w_b and yh
  float2 ry = both(1.f);
  // The rest of row n once the dot products are there.
  auto finish = [&](int n) {
    float d[kDots], unused[kDots];
    const bool fine = dot_talk.hear(d, unused);
    lane_sums(d);
    const float2 dot = both(-d[0] * inv_dim), mean = both(branch_layer ? -d[1] * inv_dim : 0.f);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!own[k]) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[k].p[e] = fmul2(ry, ffma2(y[k].p[e], dot, fadd2(t[k].p[e], mean)));
      store8(a.dy + n * a.dy_stride + col[k], t[k]);
    }
    return fine;
  };
  bool fine = true;
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
        for (int e = 0; e < 4; ++e) {
          gain[k].p[e] = fmul2(w.p[e], fadd2(both(1.f), sc.p[e]));
          gate[k].p[e] = fmul2(wb.p[e], g.p[e]);
        }
      }
    }
    // What the row's inputs give: the statistics of both norms and the sums of g and g xh.  Without a layer norm also
    // the branch's dot product, from three sums that need no statistic:
    //   sum t gate w_b y = sum dx' u + rs sum g u + rs dot sum xh u,  u = gate w_b y
    // With one, centring would double them: t is then summed when it is known, in an exchange of its own.
    const bool ok = ring.wait();
    if (kKeep) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        if (own[k]) fetch(k);
    }
    float v[kTold];
    if constexpr (kLayer) {
      float wx = 0.f, wy = 0.f, q[4] = {0.f, 0.f, 0.f, 0.f};
      if (has_h) {
        Vec8 x[kVecs];
        float2 xx = make_float2(0.f, 0.f), gs = xx, gx = xx;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) x[k] = own[k] ? load_x(k) : Vec8{};
        if (layer) wx = warp_mean(x, inv_mine);
        const float2 m = both(-wx);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          if (!own[k]) continue;
          const Vec8 g = load_g(k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c = fadd2(x[k].p[e], m), weighted = fmul2(g.p[e], gain[k].p[e]);
            if (want_shift) sums[0][k].p[e] = fadd2(sums[0][k].p[e], g.p[e]);
            xx = ffma2(c, c, xx);
            gs = fadd2(gs, weighted);
            gx = ffma2(weighted, c, gx);
          }
        }
        q[0] = xx.x + xx.y;
        q[1] = gx.x + gx.y;
        q[3] = gs.x + gs.y;
      }
      if (branch) {
        Vec8 b[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) b[k] = own[k] ? load_y(k) : Vec8{};
        if (branch_layer) wy = warp_mean(b, inv_mine);
        q[2] = lane_squares<true>(b, own, wy);
      }
      lane_sums(q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = q[e];
      v[4] = wx;
      v[5] = wy;
    } else {
      float2 q[kTold] = {};
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!own[k]) continue;
        Vec8 x{}, weighted{};
        if (has_h) {
          x = load_x(k);
          const Vec8 g = load_g(k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            weighted.p[e] = fmul2(g.p[e], gain[k].p[e]);
            if (want_shift) sums[0][k].p[e] = fadd2(sums[0][k].p[e], g.p[e]);
            q[0] = ffma2(x.p[e], x.p[e], q[0]);
            q[1] = ffma2(weighted.p[e], x.p[e], q[1]);
          }
        }
        if (branch) {
          const Vec8 b = load_y(k), d = load_d(k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = fmul2(b.p[e], gate[k].p[e]);
            q[2] = ffma2(b.p[e], b.p[e], q[2]);
            q[3] = ffma2(d.p[e], u, q[3]);
            q[4] = ffma2(weighted.p[e], u, q[4]);
            q[5] = ffma2(x.p[e], u, q[5]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kTold; ++e) v[e] = q[e].x + q[e].y;
      lane_sums(v);
    }
    row_talk.say(v, ok);
    if (kLayer && branch && i > 0) fine = finish(n - 1);  // while the others' sums come in
    float s[kTold], first[kTold];
    fine = row_talk.hear(s, first) && fine;
    if (!fine) break;
    ring.release(i);  // every warp is behind its last read of the row before
    float x_mean = 0.f, y_mean = 0.f, x_square, y_square, x_dot, g_sum = 0.f;  // of the centred rows
    if constexpr (kLayer) {
      const float dx = s[4] - first[4], dy = s[5] - first[5];  // of this lane's warp's means from the first's
      float j[6] = {theirs * dx, fmaf(theirs * dx, dx, s[0]), fmaf(dx, s[3], s[1]),
                    s[3],        theirs * dy,                 fmaf(theirs * dy, dy, s[2])};
      lane_sums(j);
      const float sx = j[0] * inv_dim, sy = j[4] * inv_dim;
      x_mean = first[4] + sx;
      y_mean = first[5] + sy;
      x_square = j[1] - j[0] * sx;
      y_square = j[5] - j[4] * sy;
      x_dot = j[2] - sx * j[3];
      g_sum = j[3];
    } else {
      lane_sums(s);
      x_square = s[0];
      x_dot = s[1];
      y_square = s[2];
    }
    const float factor = rsqrtf(x_square * inv_dim + a.eps), x_mean_dot = factor * x_dot * inv_dim;
    const float2 rs = both(factor), mean = both(layer ? -g_sum * inv_dim : 0.f), dot = both(-x_mean_dot);
    const float y_factor = branch ? rsqrtf(y_square * inv_dim + a.eps) : 1.f;
    ry = both(y_factor);
    float2 ts = make_float2(0.f, 0.f), ty = ts, y_dot = ts;
    if (!kLayer && branch) y_dot = both(-y_factor * inv_dim * (s[3] + factor * (s[4] - x_mean_dot * factor * s[5])));
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!own[k]) continue;
      Vec8 u = load_d(k);
      if (has_h) {
        const Vec8 x = load_x(k), g = load_g(k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 xh = fmul2(kLayer ? fadd2(x.p[e], both(-x_mean)) : x.p[e], rs);
          sums[1][k].p[e] = ffma2(g.p[e], xh, sums[1][k].p[e]);
          const float2 weighted = kLayer ? ffma2(g.p[e], gain[k].p[e], mean) : fmul2(g.p[e], gain[k].p[e]);
          u.p[e] = ffma2(rs, ffma2(xh, dot, weighted), u.p[e]);
        }
      }
      Vec8 scaled = u;
      if (a.residual_scale != 1.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) scaled.p[e] = fmul2(both(a.residual_scale), u.p[e]);
      }
      store8(static_cast<X*>(a.dx) + n * a.dx_stride + col[k], scaled);
      if (!has_y) continue;
      Vec8 z = load_y(k);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z.p[e] = fmul2(kLayer ? fadd2(z.p[e], both(-y_mean)) : z.p[e], ry);
        sums[2][k].p[e] = ffma2(u.p[e], z.p[e], sums[2][k].p[e]);
        u.p[e] = fmul2(u.p[e], gate[k].p[e]);
        if (kLayer) {
          ts = fadd2(ts, u.p[e]);
          ty = ffma2(u.p[e], z.p[e], ty);
        } else if (branch) {
          u.p[e] = fmul2(ry, ffma2(z.p[e], y_dot, u.p[e]));
        }
      }
      if (!kLayer || !branch) store8(a.dy + n * a.dy_stride + col[k], u);
      if (kLayer) {
        t[k] = u;
        y[k] = z;
      }
    }
    ring.advance();
    if (kLayer && branch) {
      float d[kDots] = {ty.x + ty.y, ts.x + ts.y};
      lane_sums(d);
      dot_talk.say(d, true);
    }
  }
  if (kLayer && fine && branch && ring.rows > 0) fine = finish(ring.first + ring.rows - 1);
  if (!fine) {  // a wait ran out
    ring.drain(a.err);
    return;
  }
  flush();
}

// The requests' column sums: their CTAs' slots, in CTA order within each strand, then over the strands.
// A request's terms of the weights' gradients replace its first slot (its own columns of this block alone),
// where weight_sum_kernel adds them over the requests; a single request's are the gradients themselves.
constexpr int kSumColumns = 32, kSumStrands = 32;
__global__ void __launch_bounds__(kSumColumns* kSumStrands)
request_sum_kernel(const __grid_constant__ ResidualNormArgs a, int ctas) {
  __shared__ float part[kSums][kSumStrands][kSumColumns];
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x % kSumColumns, strand = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + lane;
  const bool own = c < a.dim;
  const bool single = a.num_requests == 1;
  const bool wanted[kSums] = {a.dshift != nullptr, a.dscale != nullptr || a.dweight != nullptr,
                              a.dgate != nullptr || a.dbranch_weight != nullptr};
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
#pragma unroll
    for (int j = 0; j < kSums; ++j) {
      if (!wanted[j] || !own) continue;
#pragma unroll 4
      for (int k = lo + strand; k <= hi; k += kSumStrands)
        s[j] += a.partials[(static_cast<size_t>(k + r) * kSums + j) * a.dim + c];
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

// Threads of a row: 8 * kVecs columns each, whole warps.
int row_threads(int dim) { return (dim + 256 * kVecs - 1) / (256 * kVecs) * 32; }

// CTAs of kThreads at most, kCtas of them an SM.
template <typename X, int kThreads, int kCtas, bool kBackward>
cudaError_t launch_rows(const ResidualNormArgs& a, int sms, int* ctas, cudaStream_t stream) {
  constexpr int kSmem = 226 * 1024 / kCtas - 1024 - 128 - 2 * static_cast<int>(sizeof(Parley<kThreads / 32>));
  const bool layer = a.norm == kNormLayer || a.branch_norm == kNormLayer;
  const bool has_h = a.norm != kNormNone, has_y = a.y != nullptr;
  const uint32_t xb = row_place(a.dim * sizeof(X)), yb = row_place(a.dim * 2);
  const uint32_t stage = kBackward ? (has_h ? xb + yb : 0) + (a.dx_out != nullptr ? xb : 0) + (has_y ? yb : 0)
                                   : xb + (has_y ? yb : 0);
  int stages = static_cast<int>(kSmem / stage);
  stages = stages < 1 ? 1 : stages > kMaxStages ? kMaxStages : stages;
  void (*kernel)(const ResidualNormArgs, int);
  if constexpr (kBackward) {
    kernel = layer ? residual_norm_bwd_kernel<X, kVecs, kThreads, kCtas, true>
                   : residual_norm_bwd_kernel<X, kVecs, kThreads, kCtas, false>;
  } else {
    kernel = layer ? residual_norm_kernel<X, kVecs, kThreads, kCtas, true>
                   : residual_norm_kernel<X, kVecs, kThreads, kCtas, false>;
  }
  const cudaError_t e = allow_shared_memory<kSmem>(kernel);
  if (e != cudaSuccess) return e;
  const int resident = sms * kCtas;  // (the backward's workspace has slots for so many)
  *ctas = residual_norm_ctas(a.num_tokens, kBackward ? std::min(resident, kResidualNormMaxBwdCtas) : resident);
  if (kBackward) {
    // A CTA's column sums are written and read again, so no more CTAs than the rows of the fullest need, and past one
    // an SM three rows each (2,000 rows of 512: 15 us, 19 with one or two each; 317 of 2,560: 13, 14.4).
    const int full = (a.num_tokens + *ctas - 1) / *ctas;
    const int rows = std::max(full, std::min(3, (a.num_tokens + sms - 1) / sms));
    *ctas = (a.num_tokens + rows - 1) / rows;
  }
  return launch_programmatic(kernel, dim3(*ctas), dim3(row_threads(a.dim)), stages * stage, stream, a, stages);
}

// A row's threads follow from dim, 16 columns each; so does how many CTAs' registers and rings an SM holds (threads *
// CTAs * registers within 65,536).  The backward keeps three sums and two vectors a column: 320 threads fit once,
// and held to half the registers twice, which spills (600 us and more against 390 at dim 5,120).  The forward keeps
// three vectors and fits twice.
template <typename X>
cudaError_t launch_type(const ResidualNormArgs& a, bool backward, int sms, int* ctas, cudaStream_t stream) {
  if (backward) {
    if (a.dim <= 512) return launch_rows<X, 32, 8, true>(a, sms, ctas, stream);
    if (a.dim <= 1024) return launch_rows<X, 64, 5, true>(a, sms, ctas, stream);
    if (a.dim <= 1536) return launch_rows<X, 96, 4, true>(a, sms, ctas, stream);
    if (a.dim <= 2560) return launch_rows<X, 160, 2, true>(a, sms, ctas, stream);
    if (a.dim <= 5120) return launch_rows<X, 320, 1, true>(a, sms, ctas, stream);
    return launch_rows<X, 512, 1, true>(a, sms, ctas, stream);
  }
  if (a.dim <= 512) return launch_rows<X, 32, 16, false>(a, sms, ctas, stream);
  if (a.dim <= 1024) return launch_rows<X, 64, 8, false>(a, sms, ctas, stream);
  if (a.dim <= 1536) return launch_rows<X, 96, 6, false>(a, sms, ctas, stream);
  if (a.dim <= 2560) return launch_rows<X, 160, 4, false>(a, sms, ctas, stream);
  if (a.dim <= 5120) return launch_rows<X, 320, 2, false>(a, sms, ctas, stream);
  return launch_rows<X, 512, 1, false>(a, sms, ctas, stream);
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
