// RMS norm of queries and keys per head, with the modality-tagged rotation in the same pass, and
// the gradient of both.
//
// Per row x (one token, one head; D values) with weight w and rotation R(phi) of pairs:
//   r = 1 / sqrt(mean(x^2) + eps),   z = x r w,   y = R(phi) z
//   backward: dz = R(-phi) dy,  dw = sum over rows of dz x r,  g = dz w,
//             dx = r (g - x r^2 mean(g x))
//
// Memory-bound: the forward reads x and writes y once, the backward reads x and dy and writes dx
// once; positions and tags are 13 bytes a token.  A row is D / 8 lanes of 16 bytes (a warp holds
// two rows at D = 128, four at 64), so its sums are 4 or 3 shuffle steps and x stays in registers
// between the norm and the rotation.  A warp takes a token, computes the token's (cos, sin) once
// -- each lane a share, traded by shuffles -- keeps them in registers and runs over the heads of Q
// and K; when tokens are few, a token's heads are dealt to several warps.  Warps share nothing but
// the frequency tables, so no barrier separates the loads of one token from those of the next.
// All arithmetic is fp32; the results are rounded to bf16 once.
//
// Angles are kept in turns as a pair of floats (coordinate and frequency both hi + lo), so the
// phase is good to about 1e-7 turns for positions up to 1e7: the product's remainder, itself a float, stays
// under a fifth of a turn there (its three roundings: 2^-25 of it each), and a frequency's pair is off by
// 2^-49 of it, 3e-9 turns.  fp32 radians would lose 1e-3 already at position 10^4.
#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Rows a lane has in flight and CTAs an SM holds with the registers that takes.  The forward of
// 58,758 tokens x 80 heads x 128 takes 369 us so (6.5 TB/s, 96 % of a plain copy's rate); 4 rows
// and 4 CTAs 377 us, 4 and 5 403 us (spills).  The backward of 29,001 tokens takes 295 us (6.0 TB/s,
// 89 %: two reads to a write); 3 rows 324 us, 2 rows 349 us.
constexpr int kFwdUnroll = 8, kFwdCtas = 3;
constexpr int kBwdUnroll = 4, kBwdCtas = 2;
constexpr int kFewUnroll = 1;

struct Tables {  // shared-memory copy of the frequencies: lanes index them apart
  float2 f[3][kMaxPairs];  // text, video, audio (the tags' order)
};

// (cos, sin) of pair j of token n; axis_j: the coordinate that drives the pair in video rows.
__device__ __forceinline__ float2 token_cos_sin(const NormRopeArgs& a, const Tables& tab, int n, int j, int axis_j) {
  const int tg = a.tag[n];
  const float* p = a.pos + 3 * static_cast<size_t>(n);
  const int axis = tg == 1 ? axis_j : 0;
  float ch = p[axis], cl = 0.f;
  if (axis == 0 && a.start_frames != nullptr) {
    int lo = 0, hi = a.num_requests - 1;  // largest r with cu_requests[r] <= n
    if (a.cu_requests == nullptr) hi = 0;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu_requests[mid] <= n) lo = mid; else hi = mid - 1;
    }
    // t + s * hz / fps in two floats: product and quotient with their remainders, then a two-sum
    const float s = a.start_frames[lo];
    const float nh = __fmul_rn(s, a.tab.audio_hz);
    const float nl = fmaf(s, a.tab.audio_hz, -nh);
    const float qh = __fdiv_rn(nh, a.tab.video_fps);
    const float ql = __fdiv_rn(fmaf(-qh, a.tab.video_fps, nh) + nl, a.tab.video_fps);
    const float sum = __fadd_rn(ch, qh);
    const float b = __fsub_rn(sum, ch);
    cl = __fadd_rn(__fsub_rn(ch, __fsub_rn(sum, b)), __fsub_rn(qh, b)) + ql;
    ch = sum;
  }
  const float2 inv = tab.f[tg <= 2 ? tg : 0][j];
  const float turns = __fmul_rn(ch, inv.x);
  const float rest = fmaf(cl, inv.x, fmaf(ch, inv.y, fmaf(ch, inv.x, -turns)));
  float s, c;
  sincospif(2.f * (__fsub_rn(turns, rintf(turns)) + rest), &s, &c);
  return make_float2(c, s);
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Eight values of a row as packed pairs of floats, evens and odds apart: e[0] = (x0, x2),
// e[1] = (x4, x6), o[0] = (x1, x3), o[1] = (x5, x7), so that two rotation pairs share each
// two-lane multiply-add.
struct Row8 {
  float2 e[2], o[2];
};
__device__ __forceinline__ Row8 unpack8(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Row8 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.e[i] = make_float2(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
    r.o[i] = make_float2(__uint_as_float(w[2 * i] & 0xffff0000u),
                         __uint_as_float(w[2 * i + 1] & 0xffff0000u));
  }
  return r;
}
__device__ __forceinline__ uint4 pack8(const Row8& r) {
  return make_uint4(pack_bf16x2(r.e[0].x, r.o[0].x), pack_bf16x2(r.e[0].y, r.o[0].y),
                    pack_bf16x2(r.e[1].x, r.o[1].x), pack_bf16x2(r.e[1].y, r.o[1].y));
}
__device__ __forceinline__ Row8 load_weight(const void* w, int bf16, int col) {
  if (bf16) return unpack8(*(static_cast<const uint4*>(w) + col / 8));
  const float4* p = static_cast<const float4*>(w) + col / 4;
  const float4 a = p[0], b = p[1];
  Row8 r;
  r.e[0] = make_float2(a.x, a.z);
  r.o[0] = make_float2(a.y, a.w);
  r.e[1] = make_float2(b.x, b.z);
  r.o[1] = make_float2(b.y, b.w);
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 minus(float2 v) { return make_float2(-v.x, -v.y); }

// The cosines and sines of this lane's four pairs of a token.
struct CosSin {
  float2 c[2], s[2];  // pairs (0, 1) and (2, 3)
};

// A lane's place: row group g of the warp (kGroups rows at a time), columns [col, col + 8) of it.
template <int D>
struct Lane {
  static constexpr int kLanes = D / 8, kGroups = 32 / kLanes, kOwn = 4 / kGroups;
  int lane, group, col;
  uint32_t axes;  // two bits each: axis of the kOwn pairs whose angle this lane computes
  __device__ __forceinline__ Lane(const NormRopeArgs& a)
      : lane(threadIdx.x & 31), group(lane / kLanes), col(lane % kLanes * 8), axes(0u) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      axes |= static_cast<uint32_t>(a.tab.video_axis[col / 2 + group * kOwn + i]) << (2 * i);
  }
  __device__ __forceinline__ CosSin cos_sin(const NormRopeArgs& a, const Tables& tab, int n) const {
    float2 own[kOwn], all[4];
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      own[i] = token_cos_sin(a, tab, n, col / 2 + group * kOwn + i, (axes >> (2 * i)) & 3u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = lane % kLanes + kLanes * (i / kOwn);
      all[i].x = __shfl_sync(0xffffffffu, own[i % kOwn].x, from);
      all[i].y = __shfl_sync(0xffffffffu, own[i % kOwn].y, from);
    }
    CosSin r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r.c[i] = make_float2(all[2 * i].x, all[2 * i + 1].x);
      r.s[i] = make_float2(all[2 * i].y, all[2 * i + 1].y);
    }
    return r;
  }
};

__device__ __forceinline__ void fill_tables(const NormRopeArgs& a, Tables& tab) {
  if (threadIdx.x < kMaxPairs) {
    tab.f[0][threadIdx.x] = a.tab.text[threadIdx.x];
    tab.f[1][threadIdx.x] = a.tab.video[threadIdx.x];
    tab.f[2][threadIdx.x] = a.tab.audio[threadIdx.x];
  }
  __syncthreads();
}

// Heads of one tensor of token n, kUnroll rows a lane in flight: the warp's part takes batches
// part, part + parts, ... of kGroups * kUnroll heads.  f(x, dy) -> result; called by whole warps,
// with zeros past the last head.
template <int D, int kUnroll, bool kTwo, typename F>
__device__ __forceinline__ void for_heads(const NormRopeTensor& t, const Lane<D>& ln, int n, int part,
                                          int parts, F&& f) {
  constexpr int kBatch = Lane<D>::kGroups * kUnroll;
  const __nv_bfloat16* x = t.x + n * t.x_stride + ln.group * D + ln.col;
  const __nv_bfloat16* dy = kTwo ? t.dy + n * t.dy_stride + ln.group * D + ln.col : nullptr;
  __nv_bfloat16* out = t.out + n * t.out_stride + ln.group * D + ln.col;
  for (int h = part * kBatch; h < t.heads; h += parts * kBatch) {
    uint4 xv[kUnroll], yv[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = h + u * Lane<D>::kGroups;  // of the warp's first row
      xv[u] = yv[u] = make_uint4(0u, 0u, 0u, 0u);
      if (head + ln.group < t.heads) {
        xv[u] = __ldcs(reinterpret_cast<const uint4*>(x + head * D));
        if (kTwo) yv[u] = __ldcs(reinterpret_cast<const uint4*>(dy + head * D));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = h + u * Lane<D>::kGroups;
      if (head >= t.heads) break;  // the whole warp
      const uint4 r = f(xv[u], yv[u]);
      if (head + ln.group < t.heads) __stcs(reinterpret_cast<uint4*>(out + head * D), r);
    }
  }
}

template <int D, bool kRotate, int kUnroll>
__global__ void __launch_bounds__(kThreads, kFwdCtas)
norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int parts) {
  __shared__ Tables tab;
  if (kRotate) fill_tables(a, tab);
  grid_dependency_wait();
  launch_dependents();
  const Lane<D> ln(a);
  const int warps = gridDim.x * kWarps;
  for (int64_t unit = blockIdx.x * kWarps + threadIdx.x / 32;
       unit < static_cast<int64_t>(a.num_tokens) * parts; unit += warps) {
    const int n = static_cast<int>(unit / parts), part = static_cast<int>(unit % parts);
    CosSin cs;
    if (kRotate) cs = ln.cos_sin(a, tab, n);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const NormRopeTensor& t = a.t[k];
      if (t.heads == 0) break;
      const Row8 w = load_weight(t.weight, a.weight_bf16, ln.col);
      for_heads<D, kUnroll, false>(t, ln, n, part, parts, [&](const uint4& xv, const uint4&) {
        Row8 x = unpack8(xv);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) ss = ffma2(x.e[i], x.e[i], ffma2(x.o[i], x.o[i], ss));
        const float2 r = both(rsqrtf(row_sum<D / 8>(ss.x + ss.y) * (1.f / D) + a.eps));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x.e[i] = fmul2(x.e[i], fmul2(r, w.e[i]));
          x.o[i] = fmul2(x.o[i], fmul2(r, w.o[i]));
        }
        if (kRotate) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 e = x.e[i], o = x.o[i];
            x.e[i] = ffma2(e, cs.c[i], fmul2(minus(o), cs.s[i]));
            x.o[i] = ffma2(e, cs.s[i], fmul2(o, cs.c[i]));
          }
        }
        return pack8(x);
      });
    }
  }
}

// Backward.  Warps keep their share of dw in registers (8 columns a lane); the shares of a CTA's
// rows are summed in a fixed order and written as one row of partials, which
// norm_weight_grad_kernel sums in a fixed order: the result does not depend on timing.
template <int D, bool kRotate, int kUnroll>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, int parts) {
  constexpr int kRows = kThreads / (D / 8);
  __shared__ Tables tab;
  __shared__ float part_dw[kRows][D];
  if (kRotate) fill_tables(a, tab);
  grid_dependency_wait();
  launch_dependents();
  const Lane<D> ln(a);
  const int warps = gridDim.x * kWarps;
  Row8 dw[2] = {};
  for (int64_t unit = blockIdx.x * kWarps + threadIdx.x / 32;
       unit < static_cast<int64_t>(a.num_tokens) * parts; unit += warps) {
    const int n = static_cast<int>(unit / parts), part = static_cast<int>(unit % parts);
    CosSin cs;
    if (kRotate) cs = ln.cos_sin(a, tab, n);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const NormRopeTensor& t = a.t[k];
      if (t.heads == 0) break;
      const Row8 w = load_weight(t.weight, a.weight_bf16, ln.col);
      for_heads<D, kUnroll, true>(t, ln, n, part, parts, [&](const uint4& xv, const uint4& yv) {
        Row8 x = unpack8(xv), g = unpack8(yv);
        if (kRotate) {  // R(-phi)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 e = g.e[i], o = g.o[i];
            g.e[i] = ffma2(e, cs.c[i], fmul2(o, cs.s[i]));
            g.o[i] = ffma2(o, cs.c[i], fmul2(minus(e), cs.s[i]));
          }
        }
        float2 ss = make_float2(0.f, 0.f), gx = ss;
        Row8 p;  // dz x
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          p.e[i] = fmul2(g.e[i], x.e[i]);
          p.o[i] = fmul2(g.o[i], x.o[i]);
          ss = ffma2(x.e[i], x.e[i], ffma2(x.o[i], x.o[i], ss));
          gx = ffma2(p.e[i], w.e[i], ffma2(p.o[i], w.o[i], gx));
        }
        const float rs = rsqrtf(row_sum<D / 8>(ss.x + ss.y) * (1.f / D) + a.eps);
        const float2 r = both(rs);
        const float2 m = both(row_sum<D / 8>(gx.x + gx.y) * (-1.f / D) * rs * rs);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          dw[k].e[i] = ffma2(p.e[i], r, dw[k].e[i]);
          dw[k].o[i] = ffma2(p.o[i], r, dw[k].o[i]);
          x.e[i] = fmul2(r, ffma2(x.e[i], m, fmul2(g.e[i], w.e[i])));
          x.o[i] = fmul2(r, ffma2(x.o[i], m, fmul2(g.o[i], w.o[i])));
        }
        return pack8(x);
      });
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (a.t[k].heads == 0) break;
    __syncthreads();
    float* mine = &part_dw[threadIdx.x / (D / 8)][ln.col];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mine[4 * i] = dw[k].e[i].x;
      mine[4 * i + 1] = dw[k].o[i].x;
      mine[4 * i + 2] = dw[k].e[i].y;
      mine[4 * i + 3] = dw[k].o[i].y;
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) s += part_dw[i][threadIdx.x];
      a.partials[(static_cast<size_t>(blockIdx.x) * 2 + k) * D + threadIdx.x] = s;
    }
  }
}

// dw[k][c] = sum of the CTAs' partials, in CTA order within each of 32 strands, then over strands.
constexpr int kStrands = 32;
__global__ void __launch_bounds__(8 * kStrands)
norm_weight_grad_kernel(const float* __restrict__ partials, int num_partials, int head_dim,
                        float* __restrict__ dw_q, float* __restrict__ dw_k) {
  __shared__ float s[kStrands][8];
  grid_dependency_wait();
  launch_dependents();
  const int c = blockIdx.x * 8 + threadIdx.x % 8, strand = threadIdx.x / 8;
  float v = 0.f;
  for (int i = strand; i < num_partials; i += kStrands)
    v += partials[static_cast<size_t>(i) * 2 * head_dim + c];
  s[strand][threadIdx.x % 8] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kStrands; ++i) v += s[i][threadIdx.x];
    float* out = c < head_dim ? dw_q : dw_k;
    if (out != nullptr) out[c < head_dim ? c : c - head_dim] = v;
  }
}

template <int D, bool kRotate, int kUnroll>
cudaError_t launch_unroll(const NormRopeArgs& a, int sms, bool backward, cudaStream_t stream) {
  const int ctas = sms * (backward ? kBwdCtas : kFwdCtas);
  // a token is dealt to one warp when the tokens alone fill the GPU's warps, else to as many as
  // fill them, up to one batch of heads a warp
  constexpr int kBatch = Lane<D>::kGroups * kUnroll;
  const int64_t n = a.num_tokens, warps = static_cast<int64_t>(ctas) * kWarps;
  const int heads = a.t[0].heads > a.t[1].heads ? a.t[0].heads : a.t[1].heads;
  const int64_t most = (heads + kBatch - 1) / kBatch, want = n > 0 ? (warps + n - 1) / n : 1;
  const int parts = static_cast<int>(want < most ? want : most);
  const int64_t need = (n * parts + kWarps - 1) / kWarps;
  int grid = static_cast<int>(need < ctas ? need : ctas);
  if (!backward)
    return launch_programmatic(norm_rope_kernel<D, kRotate, kUnroll>, dim3(grid), dim3(kThreads), 0,
                               stream, a, parts);
  if (grid > kNormBwdMaxCtas) grid = kNormBwdMaxCtas;
  if (grid > 0) {
    const cudaError_t e = launch_programmatic(norm_rope_bwd_kernel<D, kRotate, kUnroll>, dim3(grid),
                                              dim3(kThreads), 0, stream, a, parts);
    if (e != cudaSuccess) return e;
  }
  // with no rows the weights' gradient is zero: the sum over no partials
  const int columns = a.t[1].heads > 0 ? 2 * D : D;
  return launch_programmatic(norm_weight_grad_kernel, dim3(columns / 8), dim3(8 * kStrands), 0, stream,
                             static_cast<const float*>(a.partials), grid, D, a.t[0].dw, a.t[1].dw);
}

template <int D>
cudaError_t launch_d(const NormRopeArgs& a, int sms, bool backward, cudaStream_t stream) {
  // Few rows: one step of rows for each warp that the GPU holds, or less.  Then a warp takes one
  // step, so that nothing runs in turn (one token x 48 heads: 3.8 us against 5.1 us at eight rows
  // a lane); with more rows than that a warp would compute a token's angles again at each step
  // (the gradient of 320 tokens x 48 heads: 10.4 us so, 7.7 us at four rows a lane).
  const int heads = a.t[0].heads > a.t[1].heads ? a.t[0].heads : a.t[1].heads;
  const int64_t steps = (heads + Lane<D>::kGroups - 1) / Lane<D>::kGroups;
  const bool few = a.num_tokens * steps <= sms * (backward ? kBwdCtas : kFwdCtas) * kWarps;
  if (a.pos != nullptr) {
    if (few) return launch_unroll<D, true, kFewUnroll>(a, sms, backward, stream);
    return backward ? launch_unroll<D, true, kBwdUnroll>(a, sms, true, stream)
                    : launch_unroll<D, true, kFwdUnroll>(a, sms, false, stream);
  }
  if (few) return launch_unroll<D, false, kFewUnroll>(a, sms, backward, stream);
  return backward ? launch_unroll<D, false, kBwdUnroll>(a, sms, true, stream)
                  : launch_unroll<D, false, kFwdUnroll>(a, sms, false, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, bool backward, cudaStream_t stream) {
  if (!backward && a.num_tokens <= 0) return cudaSuccess;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  return head_dim == 128 ? launch_d<128>(a, sms, backward, stream) : launch_d<64>(a, sms, backward, stream);
}

}  // namespace h3
