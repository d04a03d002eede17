// Rows of keys and values into a paged cache, and back out of it.  Row i of segment g stands at position
// start[g] + i of the segment's sequence: page table[g][position / page], row position % page of it.
//
// A bf16 cache holds the rows as they are.  An e4m3 cache holds, for each row (a token of a key head, D
// values), a power of two and D values rounded to e4m3: 2^e with the least e for which the row's largest
// magnitude is at most 448 * 2^e, so no value saturates and none but the smallest lose bits to e4m3's
// subnormals; e4m3 is a floating type, so a finer scale would gain nothing.  A value is off by half an e4m3
// step, 2^-4 of itself at most (or 2^-10 * 2^e below 2^-6 * 2^e), and q * 2^e is exact in bf16: what is
// read back is what the cache holds.  A row with a NaN in it is marked by its scale and reads back as NaN
// throughout, so no reader has to look for NaN among the values.
//
// Memory-bound: each row is read once and written once.  A row is D / 8 lanes of eight values; a warp takes
// a token, finds its page once and runs over the heads of K and V with kUnroll rows a lane in flight; when
// tokens are few, a token's heads are dealt to several warps.
#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "paged_segments.cuh"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 4, kCtas = 6;

// Where a packed row stands in the cache.
struct Place {
  bool ok;
  size_t page;
  int row;
};
__device__ __forceinline__ Place place_of(const KvCacheArgs& a, int n) {
  int lo = 0, hi = a.num_segments - 1;  // largest g with cu[g] <= n
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= n) lo = mid; else hi = mid - 1;
  }
  Place p{false, 0, 0};
  const int begin = a.cu[lo];
  if (begin > n || n >= a.cu[lo + 1]) return p;  // behind the last segment (or offsets out of order)
  const int64_t at = static_cast<int64_t>(a.start[lo]) + (n - begin);
  const int64_t page = at >> a.table.page_shift;
  if (begin < 0 || at < 0 || page >= a.table.per_segment) {
    record_error(a.err, kErrBadCuSeqlens);
    return p;
  }
  const int id = page_id(a.table, lo, static_cast<int>(page));
  if (!page_ok(a.table, id)) {
    record_error(a.err, kErrBadPage);
    return p;
  }
  return Place{true, static_cast<size_t>(id), static_cast<int>(at & ((1 << a.table.page_shift) - 1))};
}

// The first warp of the grid looks over the offsets: they start at 0, do not fall, end within the capacity.
__device__ __forceinline__ void check_offsets(const KvCacheArgs& a) {
  if (blockIdx.x != 0 || threadIdx.x >= 32) return;
  bool bad = threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.num_segments] > a.capacity);
  for (int g = threadIdx.x; g < a.num_segments; g += 32) bad |= a.cu[g + 1] < a.cu[g];
  if (bad) record_error(a.err, kErrBadCuSeqlens);
}

template <int D, bool kE4m3, bool kWrite>
__global__ void __launch_bounds__(kThreads, kCtas) kv_cache_kernel(const __grid_constant__ KvCacheArgs a, int parts) {
  constexpr int kLanes = D / 8, kGroups = 32 / kLanes, kBatch = kGroups * kUnroll;
  grid_dependency_wait();
  launch_dependents();
  check_offsets(a);
  const int lane = threadIdx.x & 31, group = lane / kLanes, col = lane % kLanes * 8;
  const int rows = 2 * a.heads;  // K's, then V's
  const int warps = gridDim.x * kWarps;
  for (int64_t unit = blockIdx.x * kWarps + threadIdx.x / 32; unit < static_cast<int64_t>(a.capacity) * parts;
       unit += warps) {
    const int n = static_cast<int>(unit / parts), part = static_cast<int>(unit % parts);
    const Place at = place_of(a, n);
    if (!at.ok) continue;
    for (int j0 = part * kBatch; j0 < rows; j0 += parts * kBatch) {
      uint4 in[kUnroll];
      uint32_t byte[kUnroll];
      auto packed = [&](int j) {  // row j of the token
        const bool is_v = j >= a.heads;
        return (is_v ? a.v + n * a.v_stride : a.k + n * a.k_stride) + (is_v ? j - a.heads : j) * D + col;
      };
      auto cached = [&](int j) {  // its row in the cache
        return (at.page * a.heads + (j >= a.heads ? j - a.heads : j)) << a.table.page_shift | at.row;
      };
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int j = j0 + u * kGroups + group;
        in[u] = make_uint4(0u, 0u, 0u, 0u);
        byte[u] = 127u;
        if (j >= rows) continue;
        if (kWrite) {
          in[u] = __ldcs(reinterpret_cast<const uint4*>(packed(j)));
        } else if (kE4m3) {
          const size_t c = cached(j);
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(j >= a.heads ? a.v_cache : a.k_cache) +
                                                          c * D + col);
          in[u].x = w.x;
          in[u].y = w.y;
          byte[u] = (j >= a.heads ? a.v_scale : a.k_scale)[c];
        } else {
          in[u] = *reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(j >= a.heads ? a.v_cache : a.k_cache) + cached(j) * D + col);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int j = j0 + u * kGroups + group;
        if (j0 + u * kGroups >= rows) break;  // the whole warp
        if (!kE4m3) {
          if (j >= rows) continue;
          if (kWrite)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(j >= a.heads ? a.v_cache : a.k_cache) + cached(j) * D +
                                      col) = in[u];
          else
            __stcs(reinterpret_cast<uint4*>(packed(j)), in[u]);
          continue;
        }
        const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
        if (kWrite) {
          float x[8];
          uint32_t most = 0u;  // the largest magnitude's bits: their order is the values', NaN above all
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            most = max(most, max(w[i] << 16 & 0x7fffffffu, w[i] & 0x7fff0000u));
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
          // most = 1.m * 2^(b - 127) <= 448 * 2^e = 1.75 * 2^(8 + e)
          const int b = static_cast<int>(most >> 23);
          const int e = min(max(b - 127 - 8 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0), kScaleMin), kScaleMax);
          const float inv = scale_of(127 - e);
          uint2 q;
          q.x = e4m3x2_pack(x[0] * inv, x[1] * inv) | e4m3x2_pack(x[2] * inv, x[3] * inv) << 16;
          q.y = e4m3x2_pack(x[4] * inv, x[5] * inv) | e4m3x2_pack(x[6] * inv, x[7] * inv) << 16;
          if (j >= rows) continue;
          const size_t c = cached(j);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(j >= a.heads ? a.v_cache : a.k_cache) + c * D + col) = q;
          if (col == 0) (j >= a.heads ? a.v_scale : a.k_scale)[c] = static_cast<uint8_t>(most > 0x7f800000u ? kScaleNan : e + 127);
        } else {
          if (j >= rows) continue;
          const float s = scale_of(byte[u]);
          uint32_t r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = e4m3x2_floats(w[i / 2] >> (16 * (i & 1)) & 0xffffu);
            r[i] = pack_bf16x2(f.x * s, f.y * s);
          }
          __stcs(reinterpret_cast<uint4*>(packed(j)), make_uint4(r[0], r[1], r[2], r[3]));
        }
      }
    }
  }
}

template <int D, bool kE4m3>
cudaError_t launch(const KvCacheArgs& a, bool write, int sms, cudaStream_t stream) {
  constexpr int kBatch = 32 / (D / 8) * kUnroll;
  const int64_t n = a.capacity, warps = static_cast<int64_t>(sms) * kCtas * kWarps;
  const int64_t most = (2 * a.heads + kBatch - 1) / kBatch, want = (warps + n - 1) / n;
  const int parts = static_cast<int>(want < most ? want : most);
  const int64_t need = (n * parts + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(need < sms * kCtas ? need : sms * kCtas);
  return launch_programmatic(write ? kv_cache_kernel<D, kE4m3, true> : kv_cache_kernel<D, kE4m3, false>, dim3(grid),
                             dim3(kThreads), 0, stream, a, parts);
}

}  // namespace

cudaError_t launch_kv_cache(const KvCacheArgs& a, int head_dim, bool write, cudaStream_t stream) {
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (a.k_scale != nullptr)
    return head_dim == 128 ? launch<128, true>(a, write, sms, stream) : launch<64, true>(a, write, sms, stream);
  return head_dim == 128 ? launch<128, false>(a, write, sms, stream) : launch<64, false>(a, write, sms, stream);
}

}  // namespace h3
