// C ABI of libh3attn: argument validation, tensor-map construction, kernel launch.
//
// Nothing here allocates device memory.  The one piece of library-owned device state is the
// error word below (a static __device__ variable, 4 bytes per device), where kernels record the
// first device-side problem they meet (bad cu_seqlens, bad permutation entry, a timed-out wait).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "h3attn.h"
#include "h3_internal.h"

// Scratch for h3_varlen_attn_fwd_noalloc: the attention work plan lives in this fixed array
// instead of a caller-provided workspace.  Every device that loads the library holds it (132 KB,
// enough for H3_NOALLOC_MAX_SEGMENTS segments) until the process exits.  It is shared by all
// calls on a device.
constexpr int kNoallocScratchBytes = 132 * 1024;
static_assert(h3::attn_plan_bytes(H3_NOALLOC_MAX_SEGMENTS) <= kNoallocScratchBytes,
              "the no-alloc array must hold the plan of H3_NOALLOC_MAX_SEGMENTS segments");
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoallocScratchBytes];

namespace {

__device__ unsigned int g_device_error;

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
unsigned int* g_err_ptr[kMaxDevices] = {};

// Device address of g_device_error on the current device (looked up once per device).
unsigned int* device_error_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_err_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
    g_err_ptr[dev] = static_cast<unsigned int*>(p);
  }
  return g_err_ptr[dev];
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled_fn() {
  static EncodeTiledFn fn = nullptr;
  static bool tried = false;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!tried) {
    tried = true;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// A map of `rank` dimensions; elements outside read as zero.  The driver wants a context that is current in the
// calling thread, and a thread that has made no such runtime call yet (a worker, an engine's backward thread) has
// none: it then gets its device's and the map is made again.
bool encode_map(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int rank,
                const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  auto encode = [&] {
    return enc(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}
// bf16, 128-byte swizzle
bool encode_bf16_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box) {
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base, rank, dims, strides, box);
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 3-D view {D, H, rows} of a bf16 [rows, H, D] tensor; box {64, box_heads, box_rows}, 128-byte swizzle.
// row_stride: elements between rows (0: heads * head_dim).
bool make_qkv_map(CUtensorMap* m, const void* base, int rows, int heads, int head_dim,
                  int64_t row_stride = 0, int box_heads = 1, int box_rows = 128) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2,
                                 (row_stride > 0 ? static_cast<cuuint64_t>(row_stride)
                                                 : static_cast<cuuint64_t>(heads) * head_dim) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  return encode_bf16_map(m, base, 3, dims, strides, box);
}

// 5-D view {D, heads, W, H, T} of a bf16 [T*H*W, heads, D] tensor in row-major token order; box
// {64, 1, win_w, win_h, frames} (one 128-row tile of a window), 128-byte swizzle.  Coordinates
// outside the grid (edge windows) read as zero.
bool make_window_map(CUtensorMap* m, const void* base, const int32_t grid[3], const int32_t win[3],
                     int frames, int heads, int head_dim) {
  const cuuint64_t row = static_cast<cuuint64_t>(heads) * head_dim * 2;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(grid[2]), static_cast<cuuint64_t>(grid[1]),
                              static_cast<cuuint64_t>(grid[0])};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(head_dim) * 2, row, row * grid[2],
                                 row * grid[2] * grid[1]};
  const cuuint32_t box[5] = {64, 1, static_cast<cuuint32_t>(win[2]), static_cast<cuuint32_t>(win[1]),
                             static_cast<cuuint32_t>(frames)};
  return encode_bf16_map(m, base, 5, dims, strides, box);
}

// 3-D view {D, page, pages * heads} of a paged cache; a box is a page's rows of a head, 128 at most: of 64 bf16 values
// (128-byte swizzle), or of all D e4m3 values (a swizzle as wide as they are).
bool make_cache_map(CUtensorMap* m, const void* base, bool e4m3, int64_t planes, int page_size, int head_dim) {
  const cuuint64_t row = static_cast<cuuint64_t>(head_dim) * (e4m3 ? 1 : 2);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {row, row * page_size};
  const cuuint32_t rows = static_cast<cuuint32_t>(page_size < 128 ? page_size : 128);
  const cuuint32_t box[3] = {e4m3 ? static_cast<cuuint32_t>(head_dim) : 64u, rows, 1};
  if (!e4m3) return encode_bf16_map(m, base, 3, dims, strides, box);
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    base, 3, dims, strides, box);
}

bool device_is_sm103() {
  static std::atomic<int> cached[kMaxDevices];  // 0 until looked up; then 1 (no) or 2 (yes)
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  const int known = cached[dev].load(std::memory_order_relaxed);
  if (known != 0) return known == 2;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return false;
  const bool yes = major == 10 && minor == 3;
  cached[dev].store(yes ? 2 : 1, std::memory_order_relaxed);
  return yes;
}

h3_status from_cuda(cudaError_t e) { return e == cudaSuccess ? H3_OK : H3_ERR_CUDA; }

void* g_noalloc_ptr[kMaxDevices] = {};

// Device address of g_noalloc_scratch on the current device.  The name of a __device__ array in
// host code is only a host-side stand-in, so the real address is looked up once per device with
// that device current; nullptr on failure.
void* noalloc_scratch_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) return nullptr;
    g_noalloc_ptr[dev] = p;
  }
  return g_noalloc_ptr[dev];
}

std::atomic<uint64_t> g_wait_limit_ns{0};  // 0: the default
std::atomic<int32_t> g_stall_after{-1};    // negative: never

}  // namespace

namespace h3 {
uint64_t wait_limit_ns() {
  const uint64_t v = g_wait_limit_ns.load(std::memory_order_relaxed);
  return v == 0 ? kDefaultWaitLimitNs : v;
}
uint32_t stall_after_tiles() {
  const int32_t v = g_stall_after.load(std::memory_order_relaxed);
  return v < 0 ? 0xffffffffu : static_cast<uint32_t>(v);
}
}  // namespace h3

extern "C" {

int32_t h3_version(void) { return 100; }

uint64_t h3_set_wait_limit_ns(uint64_t nanoseconds) {
  const uint64_t prev = h3::wait_limit_ns();
  g_wait_limit_ns.store(nanoseconds, std::memory_order_relaxed);
  return prev;
}

int32_t h3_debug_stall_loads(int32_t tiles) {
  return g_stall_after.exchange(tiles < 0 ? -1 : tiles, std::memory_order_relaxed);
}

const char* h3_status_string(h3_status s) {
  switch (s) {
    case H3_OK: return "ok";
    case H3_ERR_NULL: return "a required pointer is NULL";
    case H3_ERR_INVALID_ARG: return "a size or scalar argument is out of range";
    case H3_ERR_BAD_CU_SEQLENS:
      return "cu_seqlens is not 0-based and non-decreasing within capacity, or a segment exceeds "
             "max_seqlen";
    case H3_ERR_UNSUPPORTED: return "unsupported head_dim or device (needs sm_103a, D in {64,128})";
    case H3_ERR_WORKSPACE: return "workspace missing or too small";
    case H3_ERR_CUDA: return "a CUDA runtime or driver call failed";
    case H3_ERR_TIMEOUT: return "a bounded wait inside a kernel ran out";
    case H3_ERR_MISALIGNED: return "a device pointer or row size is not 16-byte aligned";
    case H3_ERR_BAD_PERM: return "a permutation entry is out of range";
    case H3_ERR_BAD_BLOCK_INDEX: return "a selected block index is out of range";
    case H3_ERR_SMEM_LAYOUT: return "a kernel's shared memory does not start on a 1024-byte boundary";
    case H3_ERR_BAD_PAGE: return "a page id of a block table is out of range";
  }
  return "unknown status";
}

h3_status h3_get_device_error(h3_stream_t stream) {
  unsigned int* p = device_error_ptr();
  if (p == nullptr) return H3_ERR_CUDA;
  unsigned int host = 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&host, p, sizeof(host), cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return H3_ERR_CUDA;
  if (cudaMemsetAsync(p, 0, sizeof(unsigned int), st) != cudaSuccess) return H3_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return H3_ERR_CUDA;
  return static_cast<h3_status>(host);
}

h3_status h3_rope_apply(const void* q_in, void* q_out, const void* k_in, void* k_out,
                        int32_t num_tokens, int32_t num_heads, int32_t head_dim,
                        const float* pos, const uint8_t* tag, const int32_t* cu_requests,
                        int32_t num_requests, const float* start_frames,
                        const h3_rope_cfg* cfg, h3_stream_t stream) {
  if (q_in == nullptr || q_out == nullptr || pos == nullptr || tag == nullptr) return H3_ERR_NULL;
  if ((k_in == nullptr) != (k_out == nullptr)) return H3_ERR_NULL;
  if (num_tokens < 0 || num_heads <= 0) return H3_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return H3_ERR_UNSUPPORTED;
  if (cu_requests != nullptr && num_requests <= 0) return H3_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_tokens) * num_heads * head_dim / 8 > INT32_MAX)
    return H3_ERR_INVALID_ARG;
  if (!aligned16(q_in) || !aligned16(q_out) || (k_in && (!aligned16(k_in) || !aligned16(k_out))))
    return H3_ERR_MISALIGNED;

  h3_rope_cfg c{};
  if (cfg != nullptr) c = *cfg;
  const double base_t = c.base_text > 0 ? c.base_text : 10000.0;
  const double base_v = c.base_video > 0 ? c.base_video : 10000.0;
  const double base_a = c.base_audio > 0 ? c.base_audio : 10000.0;
  int dt = c.video_dims_t, dh = c.video_dims_h, dw = c.video_dims_w;
  if (dt == 0 && dh == 0 && dw == 0) {
    dt = head_dim / 2;
    dh = head_dim / 4;
    dw = head_dim / 4;
  }
  if (dt < 0 || dh < 0 || dw < 0 || dt + dh + dw != head_dim || (dt | dh | dw) & 1)
    return H3_ERR_INVALID_ARG;

  // Frequency ladders, fp64 on the host, rounded once to fp32: theta_j = base^(-2j/d).
  h3::RopeTables tab{};
  const int P = head_dim / 2;
  for (int j = 0; j < P; ++j) {
    tab.inv_text[j] = static_cast<float>(std::pow(base_t, -2.0 * j / head_dim));
    tab.inv_audio[j] = static_cast<float>(std::pow(base_a, -2.0 * j / head_dim));
    int axis, jl, d;
    if (j < dt / 2) { axis = 0; jl = j; d = dt; }
    else if (j < (dt + dh) / 2) { axis = 1; jl = j - dt / 2; d = dh; }
    else { axis = 2; jl = j - (dt + dh) / 2; d = dw; }
    tab.video_axis[j] = static_cast<uint8_t>(axis);
    tab.inv_video[j] = static_cast<float>(std::pow(base_v, -2.0 * jl / d));
  }
  tab.audio_hz = c.audio_hz > 0 ? c.audio_hz : 40.f;
  tab.video_fps = c.video_fps > 0 ? c.video_fps : 24.f;

  const int nreq = cu_requests ? num_requests : 1;
  return from_cuda(h3::launch_rope(q_in, q_out, k_in, k_out, num_tokens, num_heads, head_dim, pos,
                                   tag, cu_requests, nreq, start_frames, tab,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

// ---- norm of Q and K rows with the rotation -------------------------------------------------------

namespace {

bool make_norm_tables(const h3_rope_cfg* cfg, int head_dim, h3::NormRopeTables* tab) {
  h3_rope_cfg c{};
  if (cfg != nullptr) c = *cfg;
  int dims[3] = {c.video_dims_t, c.video_dims_h, c.video_dims_w};
  if (dims[0] == 0 && dims[1] == 0 && dims[2] == 0) {
    dims[0] = head_dim / 2;
    dims[1] = dims[2] = head_dim / 4;
  }
  int sum = 0;
  for (int d : dims) {
    if (d < 0 || d > head_dim || d % 2 != 0) return false;
    sum += d;
  }
  if (sum != head_dim) return false;
  // base^(-2j/d) / (2 pi) for j in [0, d/2), each split into two floats; the ladder is a running
  // product in fp64 (relative error under 1e-14 after 64 steps)
  auto ladder = [](float base, int d, float2* out) {
    if (d == 0) return;
    const double step = std::pow(base > 0 ? static_cast<double>(base) : 10000.0, -2.0 / d);
    double f = 1.0 / 6.283185307179586476925286766559;
    for (int j = 0; j < d / 2; ++j, f *= step) {
      const float hi = static_cast<float>(f);
      out[j] = make_float2(hi, static_cast<float>(f - hi));
    }
  };
  ladder(c.base_text, head_dim, tab->text);
  ladder(c.base_audio, head_dim, tab->audio);
  for (int axis = 0, j = 0; axis < 3; ++axis) {
    ladder(c.base_video, dims[axis], tab->video + j);
    for (int i = 0; i < dims[axis] / 2; ++i, ++j) tab->video_axis[j] = static_cast<uint8_t>(axis);
  }
  tab->audio_hz = c.audio_hz > 0 ? c.audio_hz : 40.f;
  tab->video_fps = c.video_fps > 0 ? c.video_fps : 24.f;
  return true;
}

// Checks shared by the forward and the backward, and the arguments common to both.
h3_status norm_rope_args(const h3_qk_norm_desc* d, const void* q, const void* k, const void* q_weight,
                         const void* k_weight, const float* pos, const uint8_t* tag,
                         const int32_t* cu_requests, int32_t num_requests, const float* start_frames,
                         const h3_rope_cfg* cfg, h3::NormRopeArgs* a) {
  if (d == nullptr || q == nullptr || q_weight == nullptr) return H3_ERR_NULL;
  if ((pos == nullptr) != (tag == nullptr)) return H3_ERR_NULL;
  if (k != nullptr && k_weight == nullptr) return H3_ERR_NULL;
  if (d->num_tokens < 0 || d->num_q_heads <= 0 || d->num_q_heads > 65535 || d->num_k_heads < 0 ||
      d->num_k_heads > 65535 || (k != nullptr) != (d->num_k_heads > 0))
    return H3_ERR_INVALID_ARG;
  if (d->weight_type != H3_WEIGHT_F32 && d->weight_type != H3_WEIGHT_BF16) return H3_ERR_INVALID_ARG;
  if (!(d->eps <= 0.f || std::isfinite(d->eps))) return H3_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return H3_ERR_UNSUPPORTED;
  if (cu_requests != nullptr && num_requests <= 0) return H3_ERR_INVALID_ARG;
  if (!aligned16(q) || (k != nullptr && !aligned16(k)) || !aligned16(q_weight) ||
      (k != nullptr && !aligned16(k_weight)))
    return H3_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(cu_requests) |
       reinterpret_cast<uintptr_t>(start_frames)) & 3u)
    return H3_ERR_MISALIGNED;
  if (pos != nullptr && !make_norm_tables(cfg, d->head_dim, &a->tab)) return H3_ERR_INVALID_ARG;
  a->num_tokens = d->num_tokens;
  a->weight_bf16 = d->weight_type == H3_WEIGHT_BF16;
  a->eps = d->eps > 0.f ? d->eps : 1e-6f;
  a->pos = pos;
  a->tag = tag;
  a->cu_requests = cu_requests;
  a->num_requests = cu_requests != nullptr ? num_requests : 1;
  a->start_frames = start_frames;
  a->t[0].heads = d->num_q_heads;
  a->t[0].x = static_cast<const __nv_bfloat16*>(q);
  a->t[0].weight = q_weight;
  a->t[1].heads = d->num_k_heads;
  a->t[1].x = static_cast<const __nv_bfloat16*>(k);
  a->t[1].weight = k_weight;
  return H3_OK;
}

// A token stride in elements: 0 selects contiguous rows; else at least a row, whole 16-byte units.
h3_status token_stride(int64_t stride, int heads, int head_dim, int64_t* out) {
  const int64_t row = static_cast<int64_t>(heads) * head_dim;
  if (stride == 0) stride = row;
  if (stride < row || stride > INT32_MAX) return H3_ERR_INVALID_ARG;
  if (stride % 8 != 0) return H3_ERR_MISALIGNED;
  *out = stride;
  return H3_OK;
}

}  // namespace

h3_status h3_qk_norm_rope(const h3_qk_norm_desc* desc, const void* q, void* q_out, const void* k,
                          void* k_out, const void* q_weight, const void* k_weight, const float* pos,
                          const uint8_t* tag, const int32_t* cu_requests, int32_t num_requests,
                          const float* start_frames, const h3_rope_cfg* cfg, h3_stream_t stream) {
  h3::NormRopeArgs a{};
  h3_status st = norm_rope_args(desc, q, k, q_weight, k_weight, pos, tag, cu_requests, num_requests,
                                start_frames, cfg, &a);
  if (st != H3_OK) return st;
  if (q_out == nullptr || (k != nullptr) != (k_out != nullptr)) return H3_ERR_NULL;
  if (!aligned16(q_out) || !aligned16(k_out)) return H3_ERR_MISALIGNED;
  const int D = desc->head_dim;
  if ((st = token_stride(desc->q_stride, a.t[0].heads, D, &a.t[0].x_stride)) != H3_OK ||
      (st = token_stride(desc->k_stride, a.t[1].heads, D, &a.t[1].x_stride)) != H3_OK ||
      (st = token_stride(desc->q_out_stride, a.t[0].heads, D, &a.t[0].out_stride)) != H3_OK ||
      (st = token_stride(desc->k_out_stride, a.t[1].heads, D, &a.t[1].out_stride)) != H3_OK)
    return st;
  a.t[0].out = static_cast<__nv_bfloat16*>(q_out);
  a.t[1].out = static_cast<__nv_bfloat16*>(k_out);
  if (desc->num_tokens == 0) return H3_OK;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  return from_cuda(h3::launch_norm_rope(a, D, false, reinterpret_cast<cudaStream_t>(stream)));
}

size_t h3_qk_norm_rope_bwd_workspace_size(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? h3::norm_bwd_workspace_bytes(head_dim) : 0;
}

h3_status h3_qk_norm_rope_bwd(const h3_qk_norm_desc* desc, const void* dq_out, const void* dk_out,
                              const void* q, const void* k, const void* q_weight,
                              const void* k_weight, const float* pos, const uint8_t* tag,
                              const int32_t* cu_requests, int32_t num_requests,
                              const float* start_frames, const h3_rope_cfg* cfg, void* dq, void* dk,
                              float* dq_weight, float* dk_weight, void* workspace,
                              size_t workspace_bytes, h3_stream_t stream) {
  h3::NormRopeArgs a{};
  h3_status st = norm_rope_args(desc, q, k, q_weight, k_weight, pos, tag, cu_requests, num_requests,
                                start_frames, cfg, &a);
  if (st != H3_OK) return st;
  const bool has_k = k != nullptr;
  if (dq_out == nullptr || dq == nullptr || dq_weight == nullptr || has_k != (dk_out != nullptr) ||
      has_k != (dk != nullptr) || has_k != (dk_weight != nullptr))
    return H3_ERR_NULL;
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk) ||
      ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u))
    return H3_ERR_MISALIGNED;
  const int D = desc->head_dim;
  if ((st = token_stride(desc->q_stride, a.t[0].heads, D, &a.t[0].x_stride)) != H3_OK ||
      (st = token_stride(desc->k_stride, a.t[1].heads, D, &a.t[1].x_stride)) != H3_OK ||
      (st = token_stride(desc->q_out_stride, a.t[0].heads, D, &a.t[0].dy_stride)) != H3_OK ||
      (st = token_stride(desc->k_out_stride, a.t[1].heads, D, &a.t[1].dy_stride)) != H3_OK ||
      (st = token_stride(desc->dq_stride, a.t[0].heads, D, &a.t[0].out_stride)) != H3_OK ||
      (st = token_stride(desc->dk_stride, a.t[1].heads, D, &a.t[1].out_stride)) != H3_OK)
    return st;
  if (workspace == nullptr || workspace_bytes < h3::norm_bwd_workspace_bytes(D))
    return H3_ERR_WORKSPACE;
  if (!aligned16(workspace)) return H3_ERR_MISALIGNED;
  a.t[0].dy = static_cast<const __nv_bfloat16*>(dq_out);
  a.t[1].dy = static_cast<const __nv_bfloat16*>(dk_out);
  a.t[0].out = static_cast<__nv_bfloat16*>(dq);
  a.t[1].out = static_cast<__nv_bfloat16*>(dk);
  a.t[0].dw = dq_weight;
  a.t[1].dw = dk_weight;
  a.partials = static_cast<float*>(workspace);
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  return from_cuda(h3::launch_norm_rope(a, D, true, reinterpret_cast<cudaStream_t>(stream)));
}

// ---- gated residual and modulated norm ------------------------------------------------------------

namespace {

bool residual_norm_sizes_ok(const h3_residual_norm_desc* d) {
  return d->num_tokens >= 0 && d->dim > 0 && d->num_requests > 0;
}

// A row stride in elements of `bytes` each: 0 selects contiguous rows; else at least a row, whole 16-byte units.
h3_status row_stride(int64_t stride, int dim, int bytes, int64_t* out) {
  if (stride == 0) stride = dim;
  if (stride < dim || stride > INT32_MAX) return H3_ERR_INVALID_ARG;
  if (stride * bytes % 16 != 0) return H3_ERR_MISALIGNED;
  *out = stride;
  return H3_OK;
}

bool all_aligned16(std::initializer_list<const void*> pointers) {
  return std::all_of(pointers.begin(), pointers.end(), aligned16);
}

// Checks shared by the forward and the backward, and the arguments common to both.
h3_status residual_norm_args(const h3_residual_norm_desc* d, const void* y, const void* weight,
                             const void* branch_weight, const void* scale, const void* shift, const void* gate,
                             const int32_t* cu_requests, h3::ResidualNormArgs* a) {
  if (d == nullptr) return H3_ERR_NULL;
  if (!residual_norm_sizes_ok(d) || d->norm < H3_NORM_NONE || d->norm > H3_NORM_LAYER ||
      d->branch_norm < H3_NORM_NONE || d->branch_norm > H3_NORM_LAYER)
    return H3_ERR_INVALID_ARG;
  for (int32_t t : {d->stream_type, d->weight_type, d->mod_type})
    if (t != H3_TYPE_F32 && t != H3_TYPE_BF16) return H3_ERR_INVALID_ARG;
  if (!(d->eps <= 0.f || std::isfinite(d->eps)) || !std::isfinite(d->residual_scale)) return H3_ERR_INVALID_ARG;
  if (cu_requests == nullptr && d->num_requests != 1) return H3_ERR_INVALID_ARG;
  if (d->dim % 8 != 0 || d->dim > h3::kResidualNormMaxDim) return H3_ERR_UNSUPPORTED;
  // nothing to do, or something that would not be used
  if (d->norm == H3_NORM_NONE && (y == nullptr || weight != nullptr || scale != nullptr || shift != nullptr))
    return H3_ERR_INVALID_ARG;
  if (y == nullptr && (d->branch_norm != H3_NORM_NONE || branch_weight != nullptr || gate != nullptr ||
                       d->residual_scale != 1.f))
    return H3_ERR_INVALID_ARG;
  if (!all_aligned16({y, weight, branch_weight, scale, shift, gate}) || (reinterpret_cast<uintptr_t>(cu_requests) & 3u))
    return H3_ERR_MISALIGNED;
  const int mod = d->mod_type == H3_TYPE_F32 ? 4 : 2;
  h3_status st;
  if ((st = row_stride(d->y_stride, d->dim, 2, &a->y_stride)) != H3_OK ||
      (st = row_stride(d->scale_stride, d->dim, mod, &a->scale_stride)) != H3_OK ||
      (st = row_stride(d->shift_stride, d->dim, mod, &a->shift_stride)) != H3_OK ||
      (st = row_stride(d->gate_stride, d->dim, mod, &a->gate_stride)) != H3_OK)
    return st;
  a->num_tokens = d->num_tokens;
  a->dim = d->dim;
  a->num_requests = d->num_requests;
  a->norm = d->norm;
  a->branch_norm = d->branch_norm;
  a->x_fp32 = d->stream_type == H3_TYPE_F32;
  a->weight_bf16 = d->weight_type == H3_TYPE_BF16;
  a->mod_bf16 = d->mod_type == H3_TYPE_BF16;
  a->eps = d->eps > 0.f ? d->eps : 1e-6f;
  a->residual_scale = d->residual_scale;
  a->y = static_cast<const __nv_bfloat16*>(y);
  a->weight = weight;
  a->branch_weight = branch_weight;
  a->scale = scale;
  a->shift = shift;
  a->gate = gate;
  a->cu_requests = cu_requests;
  return H3_OK;
}

}  // namespace

h3_status h3_residual_norm(const h3_residual_norm_desc* desc, const void* x, const void* y, const void* weight,
                           const void* branch_weight, const void* scale, const void* shift, const void* gate,
                           const int32_t* cu_requests, void* x_out, void* h, h3_stream_t stream) {
  h3::ResidualNormArgs a{};
  h3_status st = residual_norm_args(desc, y, weight, branch_weight, scale, shift, gate, cu_requests, &a);
  if (st != H3_OK) return st;
  if (x == nullptr || (y != nullptr) != (x_out != nullptr) || (a.norm != h3::kNormNone) != (h != nullptr))
    return H3_ERR_NULL;
  if (!all_aligned16({x, x_out, h})) return H3_ERR_MISALIGNED;
  const int stream_bytes = a.x_fp32 ? 4 : 2;
  if ((st = row_stride(desc->x_stride, a.dim, stream_bytes, &a.x_stride)) != H3_OK ||
      (st = row_stride(desc->x_out_stride, a.dim, stream_bytes, &a.x_out_stride)) != H3_OK ||
      (st = row_stride(desc->h_stride, a.dim, 2, &a.h_stride)) != H3_OK)
    return st;
  a.x = x;
  a.x_out = x_out;
  a.h = static_cast<__nv_bfloat16*>(h);
  if (a.num_tokens == 0) return H3_OK;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  a.err = device_error_ptr();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_residual_norm(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

size_t h3_residual_norm_bwd_workspace_size(const h3_residual_norm_desc* d) {
  if (d == nullptr || !residual_norm_sizes_ok(d)) return 0;
  return h3::residual_norm_bwd_bytes(d->num_tokens, d->num_requests, d->dim);
}

h3_status h3_residual_norm_bwd(const h3_residual_norm_desc* desc, const void* dx_out, const void* dh,
                               const void* x_out, const void* y, const void* weight, const void* branch_weight,
                               const void* scale, const void* gate, const int32_t* cu_requests, void* dx, void* dy,
                               float* dweight, float* dbranch_weight, float* dscale, float* dshift, float* dgate,
                               void* workspace, size_t workspace_bytes, h3_stream_t stream) {
  h3::ResidualNormArgs a{};
  h3_status st = residual_norm_args(desc, y, weight, branch_weight, scale, nullptr, gate, cu_requests, &a);
  if (st != H3_OK) return st;
  const bool has_h = a.norm != h3::kNormNone, has_y = y != nullptr;
  if (has_h != (dh != nullptr) || (has_h && x_out == nullptr) || dx == nullptr || has_y != (dy != nullptr))
    return H3_ERR_NULL;
  if (!has_h && dx_out == nullptr) return H3_ERR_NULL;
  if ((!has_h && (dweight != nullptr || dscale != nullptr || dshift != nullptr)) ||
      (!has_y && (dbranch_weight != nullptr || dgate != nullptr)))
    return H3_ERR_INVALID_ARG;
  if (!all_aligned16({dx_out, dh, x_out, dx, dy, workspace}) ||
      ((reinterpret_cast<uintptr_t>(dweight) | reinterpret_cast<uintptr_t>(dbranch_weight) |
        reinterpret_cast<uintptr_t>(dscale) | reinterpret_cast<uintptr_t>(dshift) |
        reinterpret_cast<uintptr_t>(dgate)) & 3u))
    return H3_ERR_MISALIGNED;
  const int stream_bytes = a.x_fp32 ? 4 : 2;
  if ((st = row_stride(desc->x_out_stride, a.dim, stream_bytes, &a.x_stride)) != H3_OK ||
      (st = row_stride(desc->dx_out_stride, a.dim, stream_bytes, &a.dx_out_stride)) != H3_OK ||
      (st = row_stride(desc->dx_stride, a.dim, stream_bytes, &a.dx_stride)) != H3_OK ||
      (st = row_stride(desc->dh_stride, a.dim, 2, &a.dh_stride)) != H3_OK ||
      (st = row_stride(desc->dy_stride, a.dim, 2, &a.dy_stride)) != H3_OK)
    return st;
  if (workspace == nullptr || workspace_bytes < h3_residual_norm_bwd_workspace_size(desc)) return H3_ERR_WORKSPACE;
  a.x = x_out;
  a.dx_out = dx_out;
  a.dh = static_cast<const __nv_bfloat16*>(dh);
  a.dx = dx;
  a.dy = static_cast<__nv_bfloat16*>(dy);
  a.dweight = dweight;
  a.dbranch_weight = dbranch_weight;
  a.dscale = dscale;
  a.dshift = dshift;
  a.dgate = dgate;
  a.partials = static_cast<float*>(workspace);
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  a.err = device_error_ptr();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_residual_norm(a, true, reinterpret_cast<cudaStream_t>(stream)));
}

// ---- paged key/value cache --------------------------------------------------------------------------

namespace {

int page_shift_of(int32_t page_size) {  // -1: not a page size
  for (int shift = 4; shift <= 8; ++shift)
    if (page_size == 1 << shift) return shift;
  return -1;
}

h3_status kv_cache_call(const h3_kv_cache_desc* d, const void* k, const void* v, const void* k_cache,
                        const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                        const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* start, bool write,
                        h3_stream_t stream) {
  if (d == nullptr) return H3_ERR_NULL;
  if (d->num_segments < 0 || d->num_segments > 65535 || d->capacity < 0 || d->num_heads <= 0 ||
      d->num_heads > 65535 || d->num_pages < 0 || d->max_pages < 0 ||
      (d->cache_type != H3_TYPE_BF16 && d->cache_type != H3_TYPE_E4M3) || page_shift_of(d->page_size) < 0)
    return H3_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return H3_ERR_UNSUPPORTED;
  const bool e4m3 = d->cache_type == H3_TYPE_E4M3;
  h3::KvCacheArgs a{};
  h3_status st;
  if ((st = token_stride(d->k_stride, d->num_heads, d->head_dim, &a.k_stride)) != H3_OK ||
      (st = token_stride(d->v_stride, d->num_heads, d->head_dim, &a.v_stride)) != H3_OK)
    return st;
  if (e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr)) return H3_ERR_NULL;
  if (!all_aligned16({k, v, k_cache, v_cache}) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(cu_seqlens) |
        reinterpret_cast<uintptr_t>(start)) & 3u))
    return H3_ERR_MISALIGNED;
  if (d->num_segments == 0 || d->capacity == 0) return H3_OK;
  if (k == nullptr || v == nullptr || cu_seqlens == nullptr || start == nullptr ||
      (d->max_pages > 0 && block_table == nullptr) || (d->num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)))
    return H3_ERR_NULL;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  a.k = static_cast<__nv_bfloat16*>(const_cast<void*>(k));
  a.v = static_cast<__nv_bfloat16*>(const_cast<void*>(v));
  a.k_cache = const_cast<void*>(k_cache);
  a.v_cache = const_cast<void*>(v_cache);
  a.k_scale = const_cast<uint8_t*>(k_scale);
  a.v_scale = const_cast<uint8_t*>(v_scale);
  a.table = h3::PagedTable{block_table, d->max_pages, d->num_pages, page_shift_of(d->page_size)};
  a.cu = cu_seqlens;
  a.start = start;
  a.num_segments = d->num_segments;
  a.capacity = d->capacity;
  a.heads = d->num_heads;
  a.err = device_error_ptr();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_kv_cache(a, d->head_dim, write, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

h3_status h3_kv_cache_write(const h3_kv_cache_desc* desc, const void* k, const void* v, void* k_cache, void* v_cache,
                            uint8_t* k_scale, uint8_t* v_scale, const int32_t* block_table, const int32_t* cu_seqlens,
                            const int32_t* start, h3_stream_t stream) {
  return kv_cache_call(desc, k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, start, true, stream);
}

h3_status h3_kv_cache_read(const h3_kv_cache_desc* desc, const void* k_cache, const void* v_cache,
                           const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table,
                           const int32_t* cu_seqlens, const int32_t* start, void* k, void* v, h3_stream_t stream) {
  return kv_cache_call(desc, k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, start, false, stream);
}

// ---- attention over a paged cache -------------------------------------------------------------------

namespace {

bool paged_sizes_ok(const h3_paged_attn_desc* d) {
  return d->num_segments >= 0 && d->num_segments <= 65535 && d->max_seqlen_q >= 0 && d->max_seqlen_k >= 0 &&
         d->capacity_q >= 0 && d->max_seqlen_q <= d->capacity_q && d->num_q_heads > 0 && d->num_q_heads <= 65535 &&
         d->num_kv_heads > 0 && d->num_q_heads % d->num_kv_heads == 0 && d->num_q_heads / d->num_kv_heads <= 128 &&
         (d->cache_type == H3_TYPE_BF16 || d->cache_type == H3_TYPE_E4M3) && page_shift_of(d->page_size) >= 0 &&
         d->num_pages >= 0 && d->max_pages >= 0 && d->causal_block >= 0 && d->capacity_q <= 1 << 29 &&
         // work items are counted in 32 bits, and a page's rows of a head are one coordinate of a tensor map
         (static_cast<int64_t>(d->capacity_q) / (128 / (d->num_q_heads / d->num_kv_heads)) + d->num_segments) *
                 d->num_kv_heads <= INT32_MAX &&
         static_cast<int64_t>(d->num_pages) * d->num_kv_heads <= INT32_MAX;
}

// Few rows per segment take the key-streaming kernel: its 16-row tile holds all of a key head's rows.
bool paged_few_rows(const h3_paged_attn_desc* d) {
  return static_cast<int64_t>(d->max_seqlen_q) * (d->num_q_heads / d->num_kv_heads) <= h3::kPagedTokenRows;
}

// Bytes for the least workspace: a plan and, of long segments, the chunks' partial results.
size_t paged_least_bytes(const h3_paged_attn_desc* d) {
  const int group = d->num_q_heads / d->num_kv_heads;
  if (paged_few_rows(d)) return h3::paged_token_bytes(d->max_seqlen_q * group, d->head_dim);
  return h3::paged_plan_bytes(d->capacity_q, d->num_segments, 128 / group) +
         (d->max_seqlen_k >= h3::kSplitMinSeqlen ? h3::paged_split_bytes(d->head_dim) : 0);
}

// An e4m3 cache is unpacked to bf16 first when more than kUnpackRows rows of a key head read each key (a third pair of
// query tiles would convert it again) and the bf16 pages fit kUnpackMost bytes.  Converted as read against unpacked
// first, 8 key heads x 128: 2 x 512 rows over 20,000 tokens 118 / 130 us, 600 rows 161 / 151, 2,048 rows 358 / 321;
// with 40 query heads 4 x 512 rows over 12,000 tokens 561 / 397; x 64: 16 x 512 rows over 4,000 tokens 132 / 138, 800
// rows 210 / 198.
constexpr int kUnpackRows = 512;
constexpr size_t kUnpackMost = size_t{4} << 30;
int paged_unpack_pages(const h3_paged_attn_desc* d) {  // slots of a segment
  const int64_t pages = (static_cast<int64_t>(d->max_seqlen_k) + d->page_size - 1) / d->page_size;
  return static_cast<int>(pages < d->max_pages ? pages : d->max_pages);
}
size_t paged_unpack_bytes(const h3_paged_attn_desc* d) {  // 0: tiles are converted as they are read
  const int64_t slots = static_cast<int64_t>(paged_unpack_pages(d)) * d->num_segments;
  if (d->cache_type != H3_TYPE_E4M3 || d->num_pages == 0 || slots == 0 || slots > INT32_MAX / d->num_kv_heads ||
      static_cast<int64_t>(d->max_seqlen_q) * (d->num_q_heads / d->num_kv_heads) <= kUnpackRows)
    return 0;
  const size_t bytes = 4 * h3::paged_unpack_cache_elements(slots, d->num_kv_heads, d->page_size, d->head_dim);
  return bytes <= kUnpackMost ? h3::paged_unpack_table_bytes(slots) + bytes : 0;
}

}  // namespace

size_t h3_paged_attn_workspace_size(const h3_paged_attn_desc* d) {
  if (d == nullptr || !paged_sizes_ok(d) || d->num_segments == 0 || d->max_seqlen_q == 0) return 0;
  if (d->head_dim != 64 && d->head_dim != 128) return 0;
  const size_t least = paged_least_bytes(d), unpack = paged_unpack_bytes(d);
  return unpack == 0 ? least : (least + 255) / 256 * 256 + unpack;
}

h3_status h3_paged_attn_fwd(const h3_paged_attn_desc* d, const void* q, const void* k_cache, const void* v_cache,
                            const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table,
                            const int32_t* cu_seqlens_q, const int32_t* seqused_k, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, h3_stream_t stream) {
  if (d == nullptr) return H3_ERR_NULL;
  if (!paged_sizes_ok(d) || !(d->softmax_scale <= 0.f || std::isfinite(d->softmax_scale))) return H3_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return H3_ERR_UNSUPPORTED;
  const bool e4m3 = d->cache_type == H3_TYPE_E4M3;
  if (e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr)) return H3_ERR_NULL;
  int64_t q_stride;
  const h3_status st = token_stride(d->q_stride, d->num_q_heads, d->head_dim, &q_stride);
  if (st != H3_OK) return st;
  if (!all_aligned16({q, k_cache, v_cache, k_scale, v_scale, o, workspace}) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(cu_seqlens_q) |
        reinterpret_cast<uintptr_t>(seqused_k) | reinterpret_cast<uintptr_t>(lse)) & 3u))
    return H3_ERR_MISALIGNED;
  if (d->num_segments == 0 || d->max_seqlen_q == 0) return H3_OK;
  if (q == nullptr || o == nullptr || cu_seqlens_q == nullptr || seqused_k == nullptr ||
      (d->max_pages > 0 && block_table == nullptr) || (d->num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)))
    return H3_ERR_NULL;
  const size_t need = paged_least_bytes(d), unpack = paged_unpack_bytes(d), unpack_at = (need + 255) / 256 * 256;
  if (workspace == nullptr || workspace_bytes < need) return H3_ERR_WORKSPACE;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  unsigned int* err = device_error_ptr();
  if (err == nullptr) return H3_ERR_CUDA;
  const int group = d->num_q_heads / d->num_kv_heads;
  const float scale = d->softmax_scale > 0.f ? d->softmax_scale : static_cast<float>(1.0 / std::sqrt(d->head_dim));
  const h3::PagedSegments seg{cu_seqlens_q, seqused_k,
                              h3::PagedTable{block_table, d->max_pages, d->num_pages, page_shift_of(d->page_size)},
                              d->num_segments, d->max_seqlen_q, d->max_seqlen_k, d->capacity_q, d->num_q_heads,
                              d->num_kv_heads, d->causal_block};
  if (paged_few_rows(d)) {
    h3::PagedTokenArgs t{};
    t.seg = seg;
    t.q = static_cast<const __nv_bfloat16*>(q);
    t.q_stride = q_stride;
    t.k = k_cache;
    t.v = v_cache;
    t.k_scale = k_scale;
    t.v_scale = v_scale;
    t.o = static_cast<__nv_bfloat16*>(o);
    t.lse = lse;
    t.scale = scale;
    t.max_rows = d->max_seqlen_q * group;
    t.joins = static_cast<int4*>(workspace);
    t.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + h3::paged_token_joins_bytes());
    t.err = err;
    return from_cuda(h3::launch_paged_token(t, d->head_dim, reinterpret_cast<cudaStream_t>(stream)));
  }

  h3::PagedTileArgs a{};
  // no page at all: any valid map will do, every row is masked
  const bool none = d->num_pages == 0;
  a.seg = seg;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const void *keys = none ? q : k_cache, *values = none ? q : v_cache;
  if (unpack > 0 && workspace_bytes >= unpack_at + unpack) {
    h3::PagedUnpackArgs u{};
    u.seg = seg;
    u.k = static_cast<const uint8_t*>(k_cache);
    u.v = static_cast<const uint8_t*>(v_cache);
    u.k_scale = k_scale;
    u.v_scale = v_scale;
    u.per_segment = paged_unpack_pages(d);
    const int slots = u.per_segment * d->num_segments;
    uint8_t* at = static_cast<uint8_t*>(workspace) + unpack_at;
    u.table = reinterpret_cast<int32_t*>(at);
    u.k_out = reinterpret_cast<__nv_bfloat16*>(at + h3::paged_unpack_table_bytes(slots));
    u.v_out = u.k_out + h3::paged_unpack_cache_elements(slots, d->num_kv_heads, d->page_size, d->head_dim);
    u.err = err;
    const cudaError_t e = h3::launch_paged_unpack(u, d->head_dim, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return H3_ERR_CUDA;
    // from here on a bf16 cache of the slots
    keys = u.k_out;
    values = u.v_out;
    a.k_scale = a.v_scale = nullptr;
    a.seg.table.pages = u.table;
    a.seg.table.per_segment = u.per_segment;
    a.seg.table.num_pages = slots;
  }
  const bool bytes = a.k_scale != nullptr;
  const int64_t planes = none ? 1 : static_cast<int64_t>(a.seg.table.num_pages) * d->num_kv_heads;
  if (!make_qkv_map(&a.tmap_q, q, d->capacity_q, d->num_q_heads, d->head_dim, q_stride, group, 128 / group) ||
      !make_cache_map(&a.tmap_k, keys, bytes, planes, none ? 1 : d->page_size, d->head_dim) ||
      !make_cache_map(&a.tmap_v, values, bytes, planes, none ? 1 : d->page_size, d->head_dim))
    return H3_ERR_CUDA;
  a.o = o;
  a.wide = aligned32(o);
  a.lse = lse;
  a.scale = scale;
  a.workspace = workspace;
  if (d->max_seqlen_k >= h3::kSplitMinSeqlen)
    a.split_area = static_cast<uint8_t*>(workspace) + h3::paged_plan_bytes(d->capacity_q, d->num_segments, 128 / group);
  a.err = err;
  a.wait_limit_ns = h3::wait_limit_ns();
  a.stall_after_tiles = h3::stall_after_tiles();
  return from_cuda(h3::launch_paged_attn(a, d->head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

size_t h3_varlen_attn_workspace_size(int32_t num_segments, int32_t num_heads, int32_t max_seqlen,
                                     int32_t head_dim) {
  (void)num_heads;
  if (num_segments <= 0) return 0;
  return h3::attn_workspace_bytes(num_segments, max_seqlen, head_dim);
}

h3_status h3_varlen_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int32_t* cu_seqlens, int32_t num_segments, int32_t max_seqlen,
                             int32_t capacity, int32_t num_heads, int32_t head_dim,
                             float softmax_scale, void* workspace, size_t workspace_bytes,
                             h3_stream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || cu_seqlens == nullptr)
    return H3_ERR_NULL;
  if (num_segments < 0 || num_segments > 65535 || max_seqlen < 0 || capacity < 0 ||
      num_heads <= 0 || num_heads > 65535)
    return H3_ERR_INVALID_ARG;
  if (max_seqlen > capacity) return H3_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return H3_ERR_UNSUPPORTED;
  if (!(softmax_scale <= 0.f || std::isfinite(softmax_scale))) return H3_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return H3_ERR_MISALIGNED;
  // the plan is required; the split area after it is used when the workspace holds it
  const size_t need = num_segments > 0 ? h3::attn_plan_bytes(num_segments) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return H3_ERR_WORKSPACE;
  if (workspace != nullptr && !aligned16(workspace)) return H3_ERR_MISALIGNED;
  // work items are counted in 32 bits: (capacity / 256 + segments) * heads must fit
  if ((static_cast<int64_t>(capacity) / 256 + num_segments) * num_heads > INT32_MAX)
    return H3_ERR_INVALID_ARG;
  if (num_segments == 0 || max_seqlen == 0 || capacity == 0) return H3_OK;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;

  h3::AttnArgs a{};
  if (!make_qkv_map(&a.tmap_q, q, capacity, num_heads, head_dim) ||
      !make_qkv_map(&a.tmap_k, k, capacity, num_heads, head_dim) ||
      !make_qkv_map(&a.tmap_v, v, capacity, num_heads, head_dim))
    return H3_ERR_CUDA;
  a.o = o;
  a.lse = lse;
  a.cu_seqlens = cu_seqlens;
  a.num_segments = num_segments;
  a.max_seqlen = max_seqlen;
  a.capacity = capacity;
  a.num_heads = num_heads;
  a.head_dim = head_dim;
  a.scale = softmax_scale > 0.f ? softmax_scale : static_cast<float>(1.0 / std::sqrt(head_dim));
  a.workspace = workspace;
  if (max_seqlen >= h3::kSplitMinSeqlen && workspace_bytes >= need + h3::attn_split_bytes(head_dim))
    a.split_area = static_cast<uint8_t*>(workspace) + need;
  a.err = device_error_ptr();
  a.wait_limit_ns = h3::wait_limit_ns();
  a.stall_after_tiles = h3::stall_after_tiles();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_attn_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

h3_status h3_varlen_attn_fwd_noalloc(const void* q, const void* k, const void* v, void* o,
                                     float* lse, const int32_t* cu_seqlens, int32_t num_segments,
                                     int32_t max_seqlen, int32_t capacity, int32_t num_heads,
                                     int32_t head_dim, float softmax_scale, h3_stream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || cu_seqlens == nullptr)
    return H3_ERR_NULL;
  if (num_segments < 0 || num_segments > 65535 || max_seqlen < 0 || capacity < 0 ||
      num_heads <= 0 || num_heads > 65535)
    return H3_ERR_INVALID_ARG;
  if (max_seqlen > capacity) return H3_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return H3_ERR_UNSUPPORTED;
  if (!(softmax_scale <= 0.f || std::isfinite(softmax_scale))) return H3_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return H3_ERR_MISALIGNED;
  // the plan must fit the fixed array: refuse more segments than it was sized for
  if (num_segments > H3_NOALLOC_MAX_SEGMENTS ||
      h3::attn_plan_bytes(num_segments) > static_cast<size_t>(kNoallocScratchBytes))
    return H3_ERR_WORKSPACE;
  if ((static_cast<int64_t>(capacity) / 256 + num_segments) * num_heads > INT32_MAX)
    return H3_ERR_INVALID_ARG;
  if (num_segments == 0 || max_seqlen == 0 || capacity == 0) return H3_OK;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;

  void* scratch = noalloc_scratch_ptr();
  if (scratch == nullptr) return H3_ERR_CUDA;
  h3::AttnArgs a{};
  if (!make_qkv_map(&a.tmap_q, q, capacity, num_heads, head_dim) ||
      !make_qkv_map(&a.tmap_k, k, capacity, num_heads, head_dim) ||
      !make_qkv_map(&a.tmap_v, v, capacity, num_heads, head_dim))
    return H3_ERR_CUDA;
  a.o = o;
  a.lse = lse;
  a.cu_seqlens = cu_seqlens;
  a.num_segments = num_segments;
  a.max_seqlen = max_seqlen;
  a.capacity = capacity;
  a.num_heads = num_heads;
  a.head_dim = head_dim;
  a.scale = softmax_scale > 0.f ? softmax_scale : static_cast<float>(1.0 / std::sqrt(head_dim));
  a.workspace = scratch;  // the plan kernel rewrites every word the attention kernel reads
  a.err = device_error_ptr();
  a.wait_limit_ns = h3::wait_limit_ns();
  a.stall_after_tiles = h3::stall_after_tiles();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_attn_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

// ---- cross attention -------------------------------------------------------------------------------

namespace {

bool cross_sizes_ok(const h3_cross_attn_desc* d) {
  return d->num_segments >= 0 && d->num_segments <= 65535 && d->max_seqlen_q >= 0 &&
         d->max_seqlen_k >= 0 && d->capacity_q >= 0 && d->capacity_k >= 0 &&
         d->max_seqlen_q <= d->capacity_q && d->max_seqlen_k <= d->capacity_k && d->num_q_heads > 0 &&
         d->num_q_heads <= 65535 && d->num_kv_heads > 0 && d->num_q_heads % d->num_kv_heads == 0;
}

// Checks shared by the forward and the backward; strides are returned in elements.
h3_status check_cross(const h3_cross_attn_desc* d, const void* q, const void* k, const void* v,
                      const int32_t* cu_q, const int32_t* cu_k, const int32_t* seqused_k,
                      int64_t strides[3]) {
  if (d == nullptr || q == nullptr || cu_q == nullptr || cu_k == nullptr) return H3_ERR_NULL;
  if (!cross_sizes_ok(d)) return H3_ERR_INVALID_ARG;
  if (d->capacity_k > 0 && (k == nullptr || v == nullptr)) return H3_ERR_NULL;
  if (d->head_dim != 64 && d->head_dim != 128) return H3_ERR_UNSUPPORTED;
  if (!(d->softmax_scale <= 0.f || std::isfinite(d->softmax_scale))) return H3_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) ||
      ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k) |
        reinterpret_cast<uintptr_t>(seqused_k)) & 3u))
    return H3_ERR_MISALIGNED;
  h3_status st;
  if ((st = token_stride(d->q_stride, d->num_q_heads, d->head_dim, &strides[0])) != H3_OK ||
      (st = token_stride(d->k_stride, d->num_kv_heads, d->head_dim, &strides[1])) != H3_OK ||
      (st = token_stride(d->v_stride, d->num_kv_heads, d->head_dim, &strides[2])) != H3_OK)
    return st;
  // work items are counted in 32 bits
  if ((static_cast<int64_t>(d->capacity_q) / 128 + d->num_segments) * d->num_q_heads > INT32_MAX ||
      (static_cast<int64_t>(d->capacity_k) / 128 + d->num_segments) * d->num_q_heads > INT32_MAX)
    return H3_ERR_INVALID_ARG;
  return H3_OK;
}

float cross_scale(const h3_cross_attn_desc* d) {
  return d->softmax_scale > 0.f ? d->softmax_scale : static_cast<float>(1.0 / std::sqrt(d->head_dim));
}

}  // namespace

namespace {

// Few rows per segment take the key-streaming kernel: its 16-row tile holds all of a key head's
// rows, so K and V are read once.  One row more and the tile kernel reads them once for each pair of query
// heads (both sides measured in cross_token_kernel.cu).
bool cross_few_rows(const h3_cross_attn_desc* d) {
  return static_cast<int64_t>(d->max_seqlen_q) * (d->num_q_heads / d->num_kv_heads) <= h3::kCrossTokenRows;
}

h3::CrossSegments cross_segments(const h3_cross_attn_desc* d, const int32_t* cu_q, const int32_t* cu_k,
                                 const int32_t* seqused_k) {
  return h3::CrossSegments{cu_q, cu_k, seqused_k, d->num_segments, d->max_seqlen_q, d->max_seqlen_k,
                           d->capacity_q, d->capacity_k, d->num_q_heads, d->num_kv_heads};
}

}  // namespace

size_t h3_varlen_cross_attn_workspace_size(const h3_cross_attn_desc* d) {
  if (d == nullptr || !cross_sizes_ok(d) || d->num_segments == 0) return 0;
  if (cross_few_rows(d)) return h3::cross_token_bytes(cross_segments(d, nullptr, nullptr, nullptr), d->head_dim);
  return h3::attn_workspace_bytes(d->num_segments, d->max_seqlen_k, d->head_dim);
}

h3_status h3_varlen_cross_attn_fwd(const h3_cross_attn_desc* d, const void* q, const void* k,
                                   const void* v, void* o, float* lse, const int32_t* cu_seqlens_q,
                                   const int32_t* cu_seqlens_k, const int32_t* seqused_k,
                                   void* workspace, size_t workspace_bytes, h3_stream_t stream) {
  int64_t strides[3];
  const h3_status st = check_cross(d, q, k, v, cu_seqlens_q, cu_seqlens_k, seqused_k, strides);
  if (st != H3_OK) return st;
  if (o == nullptr) return H3_ERR_NULL;
  if (!aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return H3_ERR_MISALIGNED;
  const size_t need = h3_varlen_cross_attn_workspace_size(d);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return H3_ERR_WORKSPACE;
  if (!aligned16(workspace)) return H3_ERR_MISALIGNED;
  if (d->num_segments == 0 || d->max_seqlen_q == 0) return H3_OK;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;

  if (cross_few_rows(d)) {
    h3::CrossTokenArgs t{};
    t.seg = cross_segments(d, cu_seqlens_q, cu_seqlens_k, seqused_k);
    t.q = static_cast<const __nv_bfloat16*>(q);
    t.k = static_cast<const __nv_bfloat16*>(k);
    t.v = static_cast<const __nv_bfloat16*>(v);
    t.q_stride = strides[0];
    t.k_stride = strides[1];
    t.v_stride = strides[2];
    t.o = static_cast<__nv_bfloat16*>(o);
    t.lse = lse;
    t.scale = cross_scale(d);
    t.max_rows = d->max_seqlen_q * (d->num_q_heads / d->num_kv_heads);
    h3::cross_token_split(t.seg, &t.chunk_keys, &t.chunks);
    t.partials = static_cast<float*>(workspace);
    t.err = device_error_ptr();
    if (t.err == nullptr) return H3_ERR_CUDA;
    return from_cuda(h3::launch_cross_token(t, d->head_dim, reinterpret_cast<cudaStream_t>(stream)));
  }

  h3::CrossArgs a{};
  // no keys at all: any valid map will do, its rows are masked
  const bool none = d->capacity_k == 0;
  if (!make_qkv_map(&a.tmap_q, q, d->capacity_q, d->num_q_heads, d->head_dim, strides[0]) ||
      !make_qkv_map(&a.tmap_k, none ? q : k, none ? d->capacity_q : d->capacity_k,
                    none ? d->num_q_heads : d->num_kv_heads, d->head_dim, strides[none ? 0 : 1]) ||
      !make_qkv_map(&a.tmap_v, none ? q : v, none ? d->capacity_q : d->capacity_k,
                    none ? d->num_q_heads : d->num_kv_heads, d->head_dim, strides[none ? 0 : 2]))
    return H3_ERR_CUDA;
  a.seg = cross_segments(d, cu_seqlens_q, cu_seqlens_k, seqused_k);
  a.o = o;
  a.wide = aligned32(o);
  a.lse = lse;
  a.scale = cross_scale(d);
  a.workspace = workspace;
  if (d->max_seqlen_k >= h3::kSplitMinSeqlen)
    a.split_area = static_cast<uint8_t*>(workspace) + h3::attn_plan_bytes(d->num_segments);
  a.err = device_error_ptr();
  a.wait_limit_ns = h3::wait_limit_ns();
  a.stall_after_tiles = h3::stall_after_tiles();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_cross_attn(a, d->head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

size_t h3_varlen_cross_attn_bwd_workspace_size(const h3_cross_attn_desc* d) {
  if (d == nullptr || !cross_sizes_ok(d) || d->num_segments == 0) return 0;
  return h3::cross_bwd_workspace(cross_segments(d, nullptr, nullptr, nullptr), d->head_dim).bytes;
}

h3_status h3_varlen_cross_attn_bwd(const h3_cross_attn_desc* d, const void* dout, const void* q,
                                   const void* k, const void* v, const void* o, const float* lse,
                                   const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                                   const int32_t* seqused_k, void* dq, void* dk, void* dv,
                                   void* workspace, size_t workspace_bytes, h3_stream_t stream) {
  if (d == nullptr || cu_seqlens_q == nullptr || cu_seqlens_k == nullptr) return H3_ERR_NULL;
  if (!cross_sizes_ok(d)) return H3_ERR_INVALID_ARG;
  const bool none_q = d->capacity_q == 0, none_k = d->capacity_k == 0;
  if (!none_q && (dout == nullptr || q == nullptr || o == nullptr || lse == nullptr || dq == nullptr))
    return H3_ERR_NULL;
  if (!none_k && (dk == nullptr || dv == nullptr)) return H3_ERR_NULL;
  if (none_q && none_k) return d->head_dim == 64 || d->head_dim == 128 ? H3_OK : H3_ERR_UNSUPPORTED;
  int64_t strides[3];
  // a side without rows may be NULL: the other side's tensor stands in for the checks
  h3_status st = check_cross(d, none_q ? k : q, none_k ? q : k, none_k ? q : v, cu_seqlens_q, cu_seqlens_k,
                             seqused_k, strides);
  if (st != H3_OK) return st;
  if (!aligned16(dout) || !aligned16(o) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return H3_ERR_MISALIGNED;
  h3::CrossBwdArgs a{};
  if ((st = token_stride(d->dq_stride, d->num_q_heads, d->head_dim, &a.dq_stride)) != H3_OK ||
      (st = token_stride(d->dk_stride, d->num_kv_heads, d->head_dim, &a.dk_stride)) != H3_OK ||
      (st = token_stride(d->dv_stride, d->num_kv_heads, d->head_dim, &a.dv_stride)) != H3_OK)
    return st;
  const size_t need = h3_varlen_cross_attn_bwd_workspace_size(d);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return H3_ERR_WORKSPACE;
  if (!aligned16(workspace)) return H3_ERR_MISALIGNED;
  if (d->num_segments == 0) return H3_OK;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;

  // a side without rows is never read: any valid map will do
  const int cap_q = none_q ? d->capacity_k : d->capacity_q, cap_k = none_k ? d->capacity_q : d->capacity_k;
  const int hq = none_q ? d->num_kv_heads : d->num_q_heads, hk = none_k ? d->num_q_heads : d->num_kv_heads;
  if (!make_qkv_map(&a.tmap_q, none_q ? k : q, cap_q, hq, d->head_dim, strides[none_q ? 1 : 0]) ||
      !make_qkv_map(&a.tmap_do, none_q ? k : dout, cap_q, hq, d->head_dim, none_q ? strides[1] : 0) ||
      !make_qkv_map(&a.tmap_k, none_k ? q : k, cap_k, hk, d->head_dim, strides[none_k ? 0 : 1]) ||
      !make_qkv_map(&a.tmap_v, none_k ? q : v, cap_k, hk, d->head_dim, strides[none_k ? 0 : 2]))
    return H3_ERR_CUDA;
  a.seg = cross_segments(d, cu_seqlens_q, cu_seqlens_k, seqused_k);
  a.o = o;
  a.dout = dout;
  a.lse = lse;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.wide = aligned32(dq) && aligned32(dk) && aligned32(dv) &&
           (a.dq_stride | a.dk_stride | a.dv_stride) % 16 == 0;
  a.scale = cross_scale(d);
  const h3::CrossBwdWorkspace w = h3::cross_bwd_workspace(a.seg, d->head_dim);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  a.plan = reinterpret_cast<uint32_t*>(base);
  a.delta = reinterpret_cast<float*>(base + w.delta);
  a.partials = reinterpret_cast<float*>(base + w.partials);
  a.partials_q = reinterpret_cast<float*>(base + w.partials_q);
  a.slots = w.slots;
  a.err = device_error_ptr();
  a.wait_limit_ns = h3::wait_limit_ns();
  a.stall_after_tiles = h3::stall_after_tiles();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_cross_bwd(a, d->head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

h3_status h3_window_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int32_t grid[3], const int32_t win[3], const int32_t shift[3],
                             int32_t num_heads, int32_t head_dim, float softmax_scale,
                             h3_stream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || grid == nullptr ||
      win == nullptr || shift == nullptr)
    return H3_ERR_NULL;
  const int32_t nwin = h3_window_count(grid, win, shift);
  if (nwin < 0 || num_heads <= 0) return H3_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return H3_ERR_UNSUPPORTED;
  // a 128-row tile is whole frames of a window, and a window is at most two tiles
  const int per_frame = win[1] * win[2];
  if (per_frame > 128 || 128 % per_frame != 0 || win[0] * per_frame > 256 || win[1] > 256 ||
      win[2] > 256)
    return H3_ERR_UNSUPPORTED;
  if (!(softmax_scale <= 0.f || std::isfinite(softmax_scale))) return H3_ERR_INVALID_ARG;
  const int64_t n = static_cast<int64_t>(grid[0]) * grid[1] * grid[2];
  if (n > INT32_MAX / 2 || static_cast<int64_t>(nwin) * num_heads > INT32_MAX)
    return H3_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return H3_ERR_MISALIGNED;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;

  h3::AttnArgs a{};
  a.mode = h3::kAttnModeWindow;
  const int frames = 128 / per_frame;
  for (int ax = 0; ax < 3; ++ax) {
    a.wg.L[ax] = grid[ax];
    a.wg.w[ax] = win[ax];
    a.wg.s[ax] = shift[ax];
    a.wg.nwin[ax] = (grid[ax] + shift[ax] + win[ax] - 1) / win[ax];
  }
  a.wg.frames_per_tile = frames;
  if (!make_window_map(&a.tmap_q, q, grid, win, frames, num_heads, head_dim) ||
      !make_window_map(&a.tmap_k, k, grid, win, frames, num_heads, head_dim) ||
      !make_window_map(&a.tmap_v, v, grid, win, frames, num_heads, head_dim))
    return H3_ERR_CUDA;
  // half-height boxes for edge windows with at most half their rows along H inside the grid
  a.wg.half_h = win[1] % 2 == 0 ? 1 : 0;
  if (a.wg.half_h) {
    const int32_t half_win[3] = {win[0], win[1] / 2, win[2]};
    if (!make_window_map(&a.tmap_q2, q, grid, half_win, 2 * frames, num_heads, head_dim) ||
        !make_window_map(&a.tmap_k2, k, grid, half_win, 2 * frames, num_heads, head_dim) ||
        !make_window_map(&a.tmap_v2, v, grid, half_win, 2 * frames, num_heads, head_dim))
      return H3_ERR_CUDA;
  }
  a.o = o;
  a.lse = lse;
  a.capacity = static_cast<int>(n);  // LSE row stride: [heads, T*H*W]
  a.num_heads = num_heads;
  a.head_dim = head_dim;
  a.scale = softmax_scale > 0.f ? softmax_scale : static_cast<float>(1.0 / std::sqrt(head_dim));
  a.err = device_error_ptr();
  a.wait_limit_ns = h3::wait_limit_ns();
  a.stall_after_tiles = h3::stall_after_tiles();
  if (a.err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_attn_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

// ---- continuation window ------------------------------------------------------------------------

h3_status h3_continuation_make_plan(const h3_continuation_cfg* c, h3_continuation_plan* p) {
  if (c == nullptr || p == nullptr) return H3_ERR_NULL;
  if (c->text_rows < 0 || c->clip_video_frames < 0 || c->clip_audio_rows < 0 || c->frame_h <= 0 ||
      c->frame_w <= 0 || c->new_video_frames < 0 || c->new_audio_rows < 0 || c->tail_frames < 0 ||
      c->frames_per_latent <= 0)
    return H3_ERR_INVALID_ARG;
  const int64_t g0 = static_cast<int64_t>(c->clip_video_frames) - c->tail_frames;
  if (g0 < 0 || c->new_video_frames < c->tail_frames) return H3_ERR_INVALID_ARG;
  const int64_t s = g0 * c->frames_per_latent;
  if (s > INT32_MAX / 40) return H3_ERR_INVALID_ARG;
  const int64_t cut = std::min<int64_t>(s * 40 / 24, c->clip_audio_rows);  // floor(s * 40 / 24)
  const int64_t ref_audio = c->clip_audio_rows - cut;
  if (c->new_audio_rows < ref_audio) return H3_ERR_INVALID_ARG;
  const int64_t hw = static_cast<int64_t>(c->frame_h) * c->frame_w;
  const int64_t rows[5] = {c->text_rows, ref_audio, c->tail_frames * hw, c->new_audio_rows,
                           c->new_video_frames * hw};
  int64_t off = 0;
  for (int k = 0; k < 5; ++k) {
    p->group_offset[k] = static_cast<int32_t>(off);
    off += rows[k];
    if (off > INT32_MAX) return H3_ERR_INVALID_ARG;
    p->group_rows[k] = static_cast<int32_t>(rows[k]);
  }
  p->group_offset[5] = static_cast<int32_t>(off);
  p->num_rows = static_cast<int32_t>(off);
  p->tail_start = static_cast<int32_t>(g0);
  p->start_frame = static_cast<int32_t>(s);
  p->audio_cut = static_cast<int32_t>(cut);
  p->keep_video_from = c->tail_frames;
  p->keep_audio_from = static_cast<int32_t>(ref_audio);
  if (g0 + c->new_video_frames > INT32_MAX || cut + c->new_audio_rows > INT32_MAX)
    return H3_ERR_INVALID_ARG;
  p->out_video_frames = static_cast<int32_t>(g0 + c->new_video_frames);
  p->out_audio_rows = static_cast<int32_t>(cut + c->new_audio_rows);
  return H3_OK;
}

h3_status h3_continuation_pack(const h3_continuation_cfg* cfg, const void* text,
                               const void* clip_video, const void* clip_audio,
                               const void* new_video, const void* new_audio, int32_t row_bytes,
                               void* rows, float* pos, uint8_t* tag, uint8_t* target,
                               h3_stream_t stream) {
  if (cfg == nullptr || rows == nullptr || pos == nullptr || tag == nullptr || target == nullptr)
    return H3_ERR_NULL;
  h3_continuation_plan p;
  const h3_status st = h3_continuation_make_plan(cfg, &p);
  if (st != H3_OK) return st;
  if (row_bytes <= 0 || row_bytes % 16 != 0) return H3_ERR_INVALID_ARG;
  const void* src[5] = {text, clip_audio, clip_video, new_audio, new_video};
  for (int k = 0; k < 5; ++k) {
    if (p.group_rows[k] > 0 && src[k] == nullptr) return H3_ERR_NULL;
    if (src[k] != nullptr && !aligned16(src[k])) return H3_ERR_MISALIGNED;
  }
  if (static_cast<int64_t>(p.num_rows) * row_bytes / 16 > INT64_MAX / 4) return H3_ERR_INVALID_ARG;
  if (!aligned16(rows) || (reinterpret_cast<uintptr_t>(pos) & 3u)) return H3_ERR_MISALIGNED;
  const int64_t hw = static_cast<int64_t>(cfg->frame_h) * cfg->frame_w;
  const int64_t first[5] = {0, p.audio_cut, static_cast<int64_t>(p.tail_start) * hw, 0, 0};
  h3::ContinuationGeom g;
  for (int k = 0; k < 5; ++k) g.offset[k] = p.group_offset[k];
  g.num_rows = p.num_rows;
  g.frame_h = cfg->frame_h;
  g.frame_w = cfg->frame_w;
  return from_cuda(h3::launch_continuation_pack(g, src, first, row_bytes, rows, pos, tag, target,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

h3_status h3_continuation_append(const h3_continuation_cfg* cfg, const void* new_video,
                                 const void* new_audio, int32_t row_bytes, void* clip_video,
                                 int64_t clip_video_capacity_rows, void* clip_audio,
                                 int64_t clip_audio_capacity_rows, h3_stream_t stream) {
  if (cfg == nullptr) return H3_ERR_NULL;
  h3_continuation_plan p;
  const h3_status st = h3_continuation_make_plan(cfg, &p);
  if (st != H3_OK) return st;
  if (row_bytes <= 0 || row_bytes % 16 != 0) return H3_ERR_INVALID_ARG;
  const int64_t hw = static_cast<int64_t>(cfg->frame_h) * cfg->frame_w;
  const int64_t v_rows = (static_cast<int64_t>(cfg->new_video_frames) - p.keep_video_from) * hw;
  const int64_t a_rows = static_cast<int64_t>(cfg->new_audio_rows) - p.keep_audio_from;
  if ((v_rows > 0 && (new_video == nullptr || clip_video == nullptr)) ||
      (a_rows > 0 && (new_audio == nullptr || clip_audio == nullptr)))
    return H3_ERR_NULL;
  if (static_cast<int64_t>(p.out_video_frames) * hw > clip_video_capacity_rows && v_rows > 0)
    return H3_ERR_INVALID_ARG;
  if (p.out_audio_rows > clip_audio_capacity_rows && a_rows > 0) return H3_ERR_INVALID_ARG;
  for (const void* ptr : {new_video, new_audio, static_cast<const void*>(clip_video),
                          static_cast<const void*>(clip_audio)})
    if (ptr != nullptr && !aligned16(ptr)) return H3_ERR_MISALIGNED;
  const char* nv = static_cast<const char*>(new_video);
  const char* na = static_cast<const char*>(new_audio);
  char* cv = static_cast<char*>(clip_video);
  char* ca = static_cast<char*>(clip_audio);
  const void* src[2] = {v_rows > 0 ? nv + p.keep_video_from * hw * row_bytes : nullptr,
                        a_rows > 0 ? na + static_cast<int64_t>(p.keep_audio_from) * row_bytes : nullptr};
  void* dst[2] = {v_rows > 0 ? cv + cfg->clip_video_frames * hw * row_bytes : nullptr,
                  a_rows > 0 ? ca + static_cast<int64_t>(cfg->clip_audio_rows) * row_bytes : nullptr};
  const int64_t bytes[2] = {v_rows > 0 ? v_rows * row_bytes : 0, a_rows > 0 ? a_rows * row_bytes : 0};
  return from_cuda(h3::launch_copy_ranges(src, dst, bytes, reinterpret_cast<cudaStream_t>(stream)));
}

h3_status h3_masked_row_update(void* dst, const void* src, const uint8_t* mask, int32_t num_rows,
                               int32_t row_bytes, h3_stream_t stream) {
  if (num_rows < 0 || row_bytes <= 0 || row_bytes % 16 != 0) return H3_ERR_INVALID_ARG;
  if (num_rows == 0) return H3_OK;
  if (dst == nullptr || src == nullptr || mask == nullptr) return H3_ERR_NULL;
  if (!aligned16(dst) || !aligned16(src)) return H3_ERR_MISALIGNED;
  return from_cuda(h3::launch_masked_row_update(dst, src, mask, num_rows, row_bytes,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

// ---- VSA ----------------------------------------------------------------------------------------

int32_t h3_vsa_block_count(const int32_t grid[3], const int32_t block[3]) {
  if (grid == nullptr || block == nullptr) return -1;
  int64_t n = 1;
  for (int a = 0; a < 3; ++a) {
    if (grid[a] <= 0 || block[a] <= 0) return -1;
    n *= (static_cast<int64_t>(grid[a]) + block[a] - 1) / block[a];
  }
  return n > INT32_MAX ? -1 : static_cast<int32_t>(n);
}

namespace {

// Shared checks of the VSA calls: a 64-token block (one half of a 128-row tile), a grid whose
// rows and blocks fit the kernels' int32 indexing.
h3_status vsa_geometry(const int32_t grid[3], const int32_t block[3], int32_t num_heads,
                       int32_t head_dim, h3::VsaGeom* g) {
  const int32_t nblk = h3_vsa_block_count(grid, block);
  if (nblk < 0 || num_heads <= 0) return H3_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return H3_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(block[0]) * block[1] * block[2] != 64) return H3_ERR_UNSUPPORTED;
  const int64_t n = static_cast<int64_t>(grid[0]) * grid[1] * grid[2];
  if (n > INT32_MAX / 2 || static_cast<int64_t>(nblk) * num_heads > INT32_MAX / 4)
    return H3_ERR_INVALID_ARG;
  for (int a = 0; a < 3; ++a) {
    g->L[a] = grid[a];
    g->b[a] = block[a];
    g->nb[a] = (grid[a] + block[a] - 1) / block[a];
  }
  return H3_OK;
}

}  // namespace

size_t h3_vsa_select_workspace_size(const int32_t grid[3], const int32_t block[3],
                                    int32_t num_heads, int32_t head_dim) {
  h3::VsaGeom g;
  if (vsa_geometry(grid, block, num_heads, head_dim, &g) != H3_OK) return 0;
  return h3::vsa_pool_bytes(g.nb[0] * g.nb[1] * g.nb[2], num_heads, head_dim);
}

h3_status h3_vsa_select(const void* q, const void* k, const int32_t grid[3],
                        const int32_t block[3], int32_t num_heads, int32_t head_dim,
                        int32_t topk, float softmax_scale, float* scores, int32_t* block_idx,
                        void* workspace, size_t workspace_bytes, h3_stream_t stream) {
  if (q == nullptr || k == nullptr || grid == nullptr || block == nullptr || scores == nullptr ||
      block_idx == nullptr)
    return H3_ERR_NULL;
  h3::VsaGeom g;
  const h3_status st = vsa_geometry(grid, block, num_heads, head_dim, &g);
  if (st != H3_OK) return st;
  const int64_t nblk = static_cast<int64_t>(g.nb[0]) * g.nb[1] * g.nb[2];
  if (topk < 1 || topk > nblk) return H3_ERR_INVALID_ARG;
  if (nblk * nblk * num_heads > (static_cast<int64_t>(1) << 40)) return H3_ERR_INVALID_ARG;
  if (!(softmax_scale <= 0.f || std::isfinite(softmax_scale))) return H3_ERR_INVALID_ARG;
  if (workspace == nullptr ||
      workspace_bytes < h3::vsa_pool_bytes(static_cast<int>(nblk), num_heads, head_dim))
    return H3_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(scores) & 3u) || (reinterpret_cast<uintptr_t>(block_idx) & 3u))
    return H3_ERR_MISALIGNED;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  const float scale =
      softmax_scale > 0.f ? softmax_scale : static_cast<float>(1.0 / std::sqrt(head_dim));
  return from_cuda(h3::launch_vsa_select(q, k, g, num_heads, head_dim, topk, scale, scores,
                                         block_idx, workspace,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

size_t h3_vsa_attn_workspace_size(const int32_t grid[3], const int32_t block[3],
                                  int32_t num_heads, int32_t topk) {
  h3::VsaGeom g;
  if (grid == nullptr || block == nullptr ||
      vsa_geometry(grid, block, num_heads, 128, &g) != H3_OK)
    return 0;
  const int nblk = g.nb[0] * g.nb[1] * g.nb[2];
  if (topk < 1 || topk > nblk) return 0;
  return h3::vsa_schedule_bytes(nblk, num_heads, topk);
}

h3_status h3_vsa_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                          const int32_t grid[3], const int32_t block[3], int32_t num_heads,
                          int32_t head_dim, const int32_t* block_idx, int32_t topk,
                          float softmax_scale, void* workspace, size_t workspace_bytes,
                          h3_stream_t stream) {
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || grid == nullptr ||
      block == nullptr || block_idx == nullptr)
    return H3_ERR_NULL;
  h3::VsaGeom g;
  const h3_status st = vsa_geometry(grid, block, num_heads, head_dim, &g);
  if (st != H3_OK) return st;
  const int64_t nblk = static_cast<int64_t>(g.nb[0]) * g.nb[1] * g.nb[2];
  if (topk < 1 || topk > nblk || nblk > static_cast<int64_t>(h3::kVsaBlockMask))
    return H3_ERR_INVALID_ARG;
  if (!(softmax_scale <= 0.f || std::isfinite(softmax_scale))) return H3_ERR_INVALID_ARG;
  const size_t need = h3::vsa_schedule_bytes(static_cast<int>(nblk), num_heads, topk);
  if (workspace == nullptr || workspace_bytes < need) return H3_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(workspace) ||
      (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) ||
      (reinterpret_cast<uintptr_t>(block_idx) & 3u))
    return H3_ERR_MISALIGNED;
  if (!device_is_sm103()) return H3_ERR_UNSUPPORTED;
  unsigned int* err = device_error_ptr();
  if (err == nullptr) return H3_ERR_CUDA;

  h3::AttnArgs a{};
  a.mode = h3::kAttnModeVsa;
  for (int ax = 0; ax < 3; ++ax) {
    a.wg.L[ax] = grid[ax];
    a.wg.w[ax] = block[ax];
    a.wg.s[ax] = 0;
    a.wg.nwin[ax] = g.nb[ax];
  }
  a.wg.topk = topk;
  const size_t pairs = static_cast<size_t>(num_heads) * h3::vsa_pairs(static_cast<int>(nblk));
  a.vsa_steps = static_cast<const uint2*>(workspace);
  a.vsa_counts = reinterpret_cast<const int2*>(static_cast<const uint8_t*>(workspace) +
                                              (pairs * topk * 8 + 255) / 256 * 256);
  // one block (bw x bh x bt = 64 rows) per box
  if (!make_window_map(&a.tmap_q, q, grid, block, block[0], num_heads, head_dim) ||
      !make_window_map(&a.tmap_k, k, grid, block, block[0], num_heads, head_dim) ||
      !make_window_map(&a.tmap_v, v, grid, block, block[0], num_heads, head_dim))
    return H3_ERR_CUDA;
  a.o = o;
  a.lse = lse;
  a.capacity = grid[0] * grid[1] * grid[2];  // LSE row stride: [heads, T*H*W]
  a.num_heads = num_heads;
  a.head_dim = head_dim;
  a.scale = softmax_scale > 0.f ? softmax_scale : static_cast<float>(1.0 / std::sqrt(head_dim));
  a.err = err;
  a.wait_limit_ns = h3::wait_limit_ns();
  a.stall_after_tiles = h3::stall_after_tiles();
  // the pairs' key/value schedule, then the attention that follows it (same stream)
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t ce = h3::launch_vsa_schedule(block_idx, static_cast<int>(nblk), num_heads,
                                                 topk, workspace, err, cs);
  if (ce != cudaSuccess) return from_cuda(ce);
  return from_cuda(h3::launch_attn_fwd(a, cs));
}

int32_t h3_window_count(const int32_t grid[3], const int32_t win[3], const int32_t shift[3]) {
  if (grid == nullptr || win == nullptr || shift == nullptr) return -1;
  int64_t n = 1;
  for (int a = 0; a < 3; ++a) {
    if (grid[a] <= 0 || win[a] <= 0 || shift[a] < 0 || shift[a] >= win[a]) return -1;
    n *= (static_cast<int64_t>(grid[a]) + shift[a] + win[a] - 1) / win[a];
  }
  return n > INT32_MAX ? -1 : static_cast<int32_t>(n);
}

h3_status h3_window_pack(const int32_t grid[3], const int32_t win[3], const int32_t shift[3],
                         int32_t* perm, int32_t* cu_seqlens, const void* const* src,
                         void* const* dst, int32_t num_tensors, int32_t row_bytes,
                         h3_stream_t stream) {
  if (grid == nullptr || win == nullptr || shift == nullptr || perm == nullptr ||
      cu_seqlens == nullptr)
    return H3_ERR_NULL;
  if (num_tensors < 0 || num_tensors > h3::kMaxPackTensors) return H3_ERR_INVALID_ARG;
  if (num_tensors > 0 && (src == nullptr || dst == nullptr)) return H3_ERR_NULL;
  const int32_t nwin = h3_window_count(grid, win, shift);
  if (nwin < 0) return H3_ERR_INVALID_ARG;
  const int64_t n = static_cast<int64_t>(grid[0]) * grid[1] * grid[2];
  if (n > INT32_MAX / 2) return H3_ERR_INVALID_ARG;
  h3::PackPtrs ptrs{};
  if (num_tensors > 0) {
    if (row_bytes <= 0 || (row_bytes & 15)) return H3_ERR_MISALIGNED;
    for (int i = 0; i < num_tensors; ++i) {
      if (src[i] == nullptr || dst[i] == nullptr) return H3_ERR_NULL;
      if (!aligned16(src[i]) || !aligned16(dst[i])) return H3_ERR_MISALIGNED;
      ptrs.src[i] = src[i];
      ptrs.dst[i] = dst[i];
    }
  }
  h3::WindowGeom g{};
  for (int a = 0; a < 3; ++a) {
    g.L[a] = grid[a];
    g.w[a] = win[a];
    g.s[a] = shift[a];
    g.nwin[a] = (grid[a] + shift[a] + win[a] - 1) / win[a];
  }
  return from_cuda(h3::launch_window_pack(g, perm, cu_seqlens, ptrs, num_tensors, row_bytes,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

h3_status h3_window_unpack(const int32_t* perm, int32_t num_tokens, const void* src, void* dst,
                           int32_t row_bytes, h3_stream_t stream) {
  if (perm == nullptr || src == nullptr || dst == nullptr) return H3_ERR_NULL;
  if (num_tokens < 0) return H3_ERR_INVALID_ARG;
  if (row_bytes <= 0 || (row_bytes & 15)) return H3_ERR_MISALIGNED;
  if (!aligned16(src) || !aligned16(dst)) return H3_ERR_MISALIGNED;
  unsigned int* err = device_error_ptr();
  if (err == nullptr) return H3_ERR_CUDA;
  return from_cuda(h3::launch_window_unpack(perm, num_tokens, src, dst, row_bytes, err,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
