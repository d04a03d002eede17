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
// Memory-bound: each row is read once and written once.  A row is D / 8 lanes of eight values; a warp
// takes a token, finds its page once and runs over the heads of K and V with kRowsAhead rows a lane in flight; when
// tokens are few, a token's heads are dealt to several warps.  Three windows of 12,000 to 14,690 rows of 40 heads x
// 128 written into and read back from an e4m3 cache: 376 us for both, 89 % of a plain copy's rate (8 rows ahead, 3 or 6 CTAs an SM, or
// four tokens a warp: no faster).  The magnitudes of two values are compared in one instruction, and no value is
// looked at for NaN: its bits are the largest.
#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "paged_segments.cuh"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRowsAhead = 4, kCtas = 4;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Eight e4m3 values times s in bf16 (exactly: s is a power of two).
__device__ __forceinline__ uint4 e4m3x8_bf16(uint2 w, float s) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_floats((i < 2 ? w.x : w.y) >> (16 * (i & 1)) & 0xffffu);
    r[i] = pack_bf16x2(f.x * s, f.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Where a packed row stands in the cache.
struct Place {
  bool ok;
  size_t row;  // of the first head's, counting rows of D values
};
__device__ __forceinline__ Place place_of(const KvCacheArgs& a, int n) {
  int lo = 0, hi = a.num_segments - 1;  // largest g with cu[g] <= n
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= n) lo = mid; else hi = mid - 1;
  }
  Place p{false, 0};
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
  return Place{true, (static_cast<size_t>(id) * a.heads << a.table.page_shift) +
                         static_cast<size_t>(at & ((1 << a.table.page_shift) - 1))};
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
  constexpr int kLanes = D / 8, kGroups = 32 / kLanes, kBatch = kGroups * kRowsAhead;
  grid_dependency_wait();
  launch_dependents();
  check_offsets(a);
  const int lane = threadIdx.x & 31, group = lane / kLanes, col = lane % kLanes * 8;
  const int batches = (a.heads + kBatch - 1) / kBatch;  // of heads; K's, then V's
  const int warps = gridDim.x * kWarps, shift = a.table.page_shift;
  for (int64_t unit = blockIdx.x * kWarps + threadIdx.x / 32; unit < static_cast<int64_t>(a.capacity) * parts;
       unit += warps) {
    const int n = static_cast<int>(unit / parts), part = static_cast<int>(unit % parts);
    const Place at = place_of(a, n);
    if (!at.ok) continue;
    for (int b = part; b < 2 * batches; b += parts) {
      const bool is_v = b >= batches;
      const int h0 = (is_v ? b - batches : b) * kBatch + group;  // this lane's first head
      __nv_bfloat16* packed = (is_v ? a.v + n * a.v_stride : a.k + n * a.k_stride) + h0 * D + col;
      const size_t first = at.row + (static_cast<size_t>(h0) << shift);  // its row in the cache
      uint8_t* cache = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (first * D + col) * (kE4m3 ? 1 : 2);
      uint8_t* scale = kE4m3 ? (is_v ? a.v_scale : a.k_scale) + first : nullptr;
      const size_t step = static_cast<size_t>(kGroups) << shift;  // rows to the lane's next head
      uint4 in[kRowsAhead];
      uint32_t byte[kRowsAhead];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        in[u] = make_uint4(0u, 0u, 0u, 0u);
        byte[u] = 127u;
        if (h0 + u * kGroups >= a.heads) continue;
        if (kWrite) {
          in[u] = __ldcs(reinterpret_cast<const uint4*>(packed + u * kGroups * D));
        } else if (kE4m3) {
          const uint2 w = *reinterpret_cast<const uint2*>(cache + u * step * D);
          in[u].x = w.x;
          in[u].y = w.y;
          byte[u] = scale[u * step];
        } else {
          in[u] = *reinterpret_cast<const uint4*>(cache + u * step * D * 2);
        }
      }
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const bool here = h0 + u * kGroups < a.heads;
        if (h0 - group + u * kGroups >= a.heads) break;  // the whole warp
        const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
        if (!kE4m3) {
          if (!here) continue;
          if (kWrite)
            *reinterpret_cast<uint4*>(cache + u * step * D * 2) = in[u];
          else
            __stcs(reinterpret_cast<uint4*>(packed + u * kGroups * D), in[u]);
        } else if (kWrite) {
          // the largest magnitude's bits, of evens and odds at once: their order is the values', NaN above all
          uint32_t most = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                    max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) most = max_u16x2(most, __shfl_xor_sync(0xffffffffu, most, o));
          most = max(most & 0xffffu, most >> 16);
          // 1.m * 2^(b - 127) <= 448 * 2^e = 1.75 * 2^(8 + e)
          const int e = min(max(static_cast<int>(most >> 7) - 127 - 8 + ((most & 0x7fu) > 0x60u ? 1 : 0), kScaleMin),
                            kScaleMax);
          const float2 inv = make_float2(scale_of(127 - e), scale_of(127 - e));
          uint32_t q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = fmul2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), inv);
            q[i] = e4m3x2_pack(x.x, x.y);
          }
          if (!here) continue;
          *reinterpret_cast<uint2*>(cache + u * step * D) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
          if (col == 0) scale[u * step] = static_cast<uint8_t>(most > 0x7f80u ? kScaleNan : e + 127);
        } else {
          if (!here) continue;
          __stcs(reinterpret_cast<uint4*>(packed + u * kGroups * D), e4m3x8_bf16(make_uint2(w[0], w[1]), scale_of(byte[u])));
        }
      }
    }
  }
}

template <int D, bool kE4m3, bool kWrite>
cudaError_t launch(const KvCacheArgs& a, int sms, cudaStream_t stream) {
  constexpr int kBatch = 32 / (D / 8) * kRowsAhead;
  const int64_t n = a.capacity, warps = static_cast<int64_t>(sms) * kCtas * kWarps;
  const int64_t most = 2 * ((a.heads + kBatch - 1) / kBatch), want = (warps + n - 1) / n;
  const int parts = static_cast<int>(want < most ? want : most);
  const int64_t need = (n * parts + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(need < sms * kCtas ? need : sms * kCtas);
  return launch_programmatic(kv_cache_kernel<D, kE4m3, kWrite>, dim3(grid), dim3(kThreads), 0, stream, a, parts);
}

template <int D, bool kE4m3>
cudaError_t launch(const KvCacheArgs& a, bool write, int sms, cudaStream_t stream) {
  return write ? launch<D, kE4m3, true>(a, sms, stream) : launch<D, kE4m3, false>(a, sms, stream);
}

// An e4m3 cache's pages as bf16, for a call that reads each of them many times.  A warp takes 16 rows of a (slot, key
// head) of K or V: eight bytes a lane and load, all of them under way before the first is used.  The warps count the
// pages in use alone, 32 segments at once, so loose bounds cost nothing.
template <int D>
__global__ void __launch_bounds__(kThreads) paged_unpack_kernel(const __grid_constant__ PagedUnpackArgs a) {
  constexpr int kRows = 16, kLoads = kRows * D / (32 * 8), kLanes = D / 8;
  grid_dependency_wait();
  launch_dependents();
  const int lane = threadIdx.x & 31, shift = a.seg.table.page_shift, heads = a.seg.num_kv_heads;
  const uint32_t parts = 2u << (shift - 4), units = heads * parts;  // of a slot
  const uint32_t warps = gridDim.x * kWarps;
  uint32_t at = blockIdx.x * kWarps + threadIdx.x / 32, before = 0;  // this warp's unit, those of earlier segments
  for (int g0 = 0; g0 < a.seg.num_segments; g0 += 32) {
    int used = 0;  // (the plan records what is wrong with a segment, and skips one past the slots)
    if (g0 + lane < a.seg.num_segments) {
      const PagedSegment s = checked_paged_segment(a.seg, g0 + lane, nullptr);
      if (s.rows > 0 && s.used <= static_cast<int64_t>(a.per_segment) << shift) used = s.used;
    }
    const uint32_t mine = ((used + (1 << shift) - 1) >> shift) * units;
    uint32_t end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, end, 31);
    for (; at - before < all; at += warps) {
      const uint32_t in = at - before;
      const int l = __popc(__ballot_sync(0xffffffffu, end <= in));  // the lane whose segment it is
      const int g = g0 + l, tokens = __shfl_sync(0xffffffffu, used, l);
      const uint32_t rest = in - __shfl_sync(0xffffffffu, end - mine, l);
      const uint32_t p = rest / units, unit = rest - p * units, head = unit / parts, part = unit - head * parts;
      const size_t slot = static_cast<size_t>(g) * a.per_segment + p;
      if (unit == 0 && lane == 0) a.table[slot] = static_cast<int>(slot);
      const int row = static_cast<int>(part / 2) * kRows;
      if (static_cast<int64_t>(p << shift) + row >= tokens) continue;
      int id = page_id(a.seg.table, g, p);
      if (!page_ok(a.seg.table, id)) {
        record_error(a.err, kErrBadPage);
        id = 0;
      }
      const size_t from = (static_cast<size_t>(id) * heads + head << shift) + row;
      const size_t to = (slot * heads + head << shift) + row;
      const uint8_t* in8 = (part & 1 ? a.v : a.k) + from * D + lane * 8;
      const uint8_t* scale = (part & 1 ? a.v_scale : a.k_scale) + from + lane / kLanes;
      __nv_bfloat16* out = (part & 1 ? a.v_out : a.k_out) + to * D + lane * 8;
      uint2 w[kLoads];
      uint32_t byte[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        w[i] = __ldcs(reinterpret_cast<const uint2*>(in8 + i * 256));
        byte[i] = scale[i * (32 / kLanes)];
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        *reinterpret_cast<uint4*>(out + i * 256) = e4m3x8_bf16(w[i], scale_of(byte[i]));
    }
    before += all;
  }
}

}  // namespace

cudaError_t launch_paged_unpack(const PagedUnpackArgs& a, int head_dim, cudaStream_t stream) {
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const uint64_t units = static_cast<uint64_t>(a.seg.num_segments) * a.per_segment * a.seg.num_kv_heads *
                         (2u << (a.seg.table.page_shift - 4));
  const uint64_t need = (units + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(need < static_cast<uint64_t>(8 * sms) ? need : 8 * sms);
  return launch_programmatic(head_dim == 128 ? paged_unpack_kernel<128> : paged_unpack_kernel<64>, dim3(grid),
                             dim3(kThreads), 0, stream, a);
}

cudaError_t launch_kv_cache(const KvCacheArgs& a, int head_dim, bool write, cudaStream_t stream) {
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (a.k_scale != nullptr)
    return head_dim == 128 ? launch<128, true>(a, write, sms, stream) : launch<64, true>(a, write, sms, stream);
  return head_dim == 128 ? launch<128, false>(a, write, sms, stream) : launch<64, false>(a, write, sms, stream);
}

}  // namespace h3
