// RMS norm of queries and keys per head, with the modality-tagged rotation in the same pass, and
// the gradient of both.
//
// Per row x (one token, one head; D values) with weight w and rotation R(phi) of pairs:
//   r = 1 / sqrt(mean(x^2) + eps),   z = x r w,   y = R(phi) z
//   backward: dz = R(-phi) dy,  dw = sum over rows of dz x r,  g = dz w,
//             dx = r (g - x r^2 mean(g x))
//
// Memory-bound: the forward reads x and writes y once, the backward reads x and dy and writes dx
// once; positions and tags are 13 bytes a token.  A row is D / 8 lanes of 16 bytes, so its sums
// are 3 or 4 shuffle steps and x never leaves registers between the norm and the rotation.  The
// (cos, sin) of a token's pairs are computed once by the CTA into shared memory and serve all
// heads of Q and K.  All arithmetic is fp32; the results are rounded to bf16 once.
//
// Angles are kept in turns as a pair of floats (coordinate and frequency both hi + lo), so the
// phase is good to about 1e-7 turns whatever the position; fp32 radians would lose 1e-3 already at
// position 10^4.
#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens of a CTA's group

// (cos, sin) of pair j of token n.
__device__ __forceinline__ float2 token_cos_sin(const NormRopeArgs& a, int n, int j) {
  const int tg = a.tag[n];
  const float* p = a.pos + 3 * static_cast<size_t>(n);
  const int axis = tg == 1 ? a.tab.video_axis[j] : 0;
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
  const float2 inv = tg == 1 ? a.tab.video[j] : (tg == 2 ? a.tab.audio[j] : a.tab.text[j]);
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

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load_weight(const void* w, int bf16, int col, float (&out)[8]) {
  if (bf16) {
    unpack8(*(static_cast<const uint4*>(w) + col / 8), out);
  } else {
    const float4* p = static_cast<const float4*>(w) + col / 4;
    const float4 a = p[0], b = p[1];
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
  }
}

// Rows of one tensor for a group of tokens [tok0, tok0 + ntok): row slot s takes rows s, s + R, ...
// of the group's ntok * heads rows; f(x, dy, cs pointer) -> result, kUnroll rows' loads in flight.
template <int D, int kUnroll, bool kTwo, typename F>
__device__ __forceinline__ void for_rows(const NormRopeTensor& t, int tok0, int ntok, F&& f) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = kThreads / kLanes;
  const int slot = threadIdx.x / kLanes, col = (threadIdx.x % kLanes) * 8;
  const int rows = ntok * t.heads;
  int ti = 0, h = slot;  // token of the group and head of the next row
  while (h >= t.heads && ti < ntok) { h -= t.heads; ++ti; }
  // every thread makes the same number of steps: the row sums shuffle across whole warps
  for (int base = 0; base < rows; base += kRows * kUnroll) {
    uint4 x[kUnroll], y[kUnroll];
    int tok[kUnroll], head[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      tok[u] = ti;
      head[u] = h;
      x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
      if (ti < ntok) {
        const size_t n = static_cast<size_t>(tok0 + ti);
        x[u] = __ldcs(reinterpret_cast<const uint4*>(t.x + n * t.x_stride + h * D + col));
        if (kTwo) y[u] = __ldcs(reinterpret_cast<const uint4*>(t.dy + n * t.dy_stride + h * D + col));
      }
      h += kRows;
      while (h >= t.heads && ti < ntok) { h -= t.heads; ++ti; }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (base + u * kRows >= rows) break;  // uniform: no row of the CTA is left
      const uint4 r = f(x[u], y[u], min(tok[u], ntok - 1));  // zeros past the last row
      if (tok[u] < ntok)
        __stcs(reinterpret_cast<uint4*>(t.out + static_cast<size_t>(tok0 + tok[u]) * t.out_stride +
                                        head[u] * D + col), r);
    }
  }
}

template <int D, bool kRotate>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int group) {
  __shared__ __align__(16) float2 cs[kMaxTokens][D / 2];
  grid_dependency_wait();
  launch_dependents();
  const int tok0 = blockIdx.x * group;
  const int ntok = min(group, a.num_tokens - tok0);
  const int pair0 = (threadIdx.x % (D / 8)) * 4;
  if (kRotate) {
    for (int i = threadIdx.x; i < ntok * (D / 2); i += kThreads)
      cs[i / (D / 2)][i % (D / 2)] = token_cos_sin(a, tok0 + i / (D / 2), i % (D / 2));
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const NormRopeTensor& t = a.t[k];
    if (t.heads == 0) break;
    float w[8];
    load_weight(t.weight, a.weight_bf16, pair0 * 2, w);
    for_rows<D, 4, false>(t, tok0, ntok, [&](const uint4& xv, const uint4&, int ti) {
      float x[8];
      unpack8(xv, x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      const float r = rsqrtf(row_sum<D / 8>(ss) * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
      if (kRotate) {
        const float4* c = reinterpret_cast<const float4*>(&cs[ti][pair0]);
        const float4 c01 = c[0], c23 = c[1];
        const float cc[8] = {c01.x, c01.y, c01.z, c01.w, c23.x, c23.y, c23.z, c23.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = x[2 * i], q = x[2 * i + 1], co = cc[2 * i], si = cc[2 * i + 1];
          x[2 * i] = fmaf(p, co, -q * si);
          x[2 * i + 1] = fmaf(p, si, q * co);
        }
      }
      return pack8(x);
    });
  }
}

// Backward.  CTAs loop over token groups and keep their share of dw in registers (8 columns a
// thread); the shares of a CTA's row slots are summed in slot order and written as one row of
// partials, which norm_weight_grad_kernel sums in CTA order: the result does not depend on timing.
template <int D, bool kRotate>
__global__ void __launch_bounds__(kThreads)
norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, int group) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = kThreads / kLanes;
  __shared__ __align__(16) float2 cs[kMaxTokens][D / 2];
  __shared__ float part[kRows][D];
  grid_dependency_wait();
  launch_dependents();
  const int pair0 = (threadIdx.x % kLanes) * 4;
  float w[2][8], dw[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (a.t[k].heads > 0) load_weight(a.t[k].weight, a.weight_bf16, pair0 * 2, w[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.f;
  }
  for (int tok0 = blockIdx.x * group; tok0 < a.num_tokens; tok0 += gridDim.x * group) {
    const int ntok = min(group, a.num_tokens - tok0);
    if (kRotate) {
      __syncthreads();  // the previous group's rotations are done
      for (int i = threadIdx.x; i < ntok * (D / 2); i += kThreads)
        cs[i / (D / 2)][i % (D / 2)] = token_cos_sin(a, tok0 + i / (D / 2), i % (D / 2));
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (a.t[k].heads == 0) break;
      for_rows<D, 2, true>(a.t[k], tok0, ntok, [&](const uint4& xv, const uint4& yv, int ti) {
        float x[8], g[8];
        unpack8(xv, x);
        unpack8(yv, g);
        if (kRotate) {
          const float4* c = reinterpret_cast<const float4*>(&cs[ti][pair0]);
          const float4 c01 = c[0], c23 = c[1];
          const float cc[8] = {c01.x, c01.y, c01.z, c01.w, c23.x, c23.y, c23.z, c23.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // R(-phi)
            const float p = g[2 * i], q = g[2 * i + 1], co = cc[2 * i], si = cc[2 * i + 1];
            g[2 * i] = fmaf(p, co, q * si);
            g[2 * i + 1] = fmaf(q, co, -p * si);
          }
        }
        float ss = 0.f, gx = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(x[i], x[i], ss);
          gx = fmaf(g[i] * w[k][i], x[i], gx);
        }
        const float r = rsqrtf(row_sum<kLanes>(ss) * (1.f / D) + a.eps);
        const float m = row_sum<kLanes>(gx) * (1.f / D) * r * r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[k][i] = fmaf(g[i] * x[i], r, dw[k][i]);
          x[i] = r * fmaf(-x[i], m, g[i] * w[k][i]);
        }
        return pack8(x);
      });
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (a.t[k].heads == 0) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x / kLanes][pair0 * 2 + i] = dw[k][i];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) s += part[i][threadIdx.x];
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

// Tokens of a CTA's group: one while that still leaves SMs idle (a token's rows are at most a few
// steps of the CTA), else four, which computes 256 angles at once.
int group_tokens(int num_tokens, int sms) { return num_tokens < 4 * kMaxTokens * sms ? 1 : kMaxTokens; }

template <int D>
cudaError_t launch_d(const NormRopeArgs& a, int sms, bool backward, cudaStream_t stream) {
  const int group = group_tokens(a.num_tokens, sms);
  const int groups = (a.num_tokens + group - 1) / group;
  if (!backward) {
    auto* kernel = a.pos != nullptr ? norm_rope_kernel<D, true> : norm_rope_kernel<D, false>;
    return launch_programmatic(kernel, dim3(groups), dim3(kThreads), 0, stream, a, group);
  }
  const int grid = groups < kNormBwdMaxCtas ? groups : kNormBwdMaxCtas;
  if (grid > 0) {
    auto* kernel = a.pos != nullptr ? norm_rope_bwd_kernel<D, true> : norm_rope_bwd_kernel<D, false>;
    const cudaError_t e = launch_programmatic(kernel, dim3(grid), dim3(kThreads), 0, stream, a, group);
    if (e != cudaSuccess) return e;
  }
  // with no rows the weights' gradient is zero: the sum over no partials
  const int columns = a.t[1].heads > 0 ? 2 * D : D;
  return launch_programmatic(norm_weight_grad_kernel, dim3(columns / 8), dim3(8 * kStrands), 0, stream,
                             static_cast<const float*>(a.partials), grid, D, a.t[0].dw, a.t[1].dw);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, bool backward, cudaStream_t stream) {
  if (!backward && a.num_tokens <= 0) return cudaSuccess;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  return head_dim == 128 ? launch_d<128>(a, sms, backward, stream) : launch_d<64>(a, sms, backward, stream);
}

}  // namespace h3
