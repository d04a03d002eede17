// Segments of a paged cache on the device: the one check of their offsets, and the look-up of a page.
#pragma once

#include "h3_internal.h"
#include "sm103_ptx.cuh"

namespace h3 {

// Page p of segment g.  An id out of range is recorded; the caller skips it, or reads page 0 in its place.
__device__ __forceinline__ int page_id(const PagedTable& t, int g, int p) {
  return t.pages[static_cast<size_t>(g) * t.per_segment + p];
}
__device__ __forceinline__ bool page_ok(const PagedTable& t, int id) { return id >= 0 && id < t.num_pages; }

// Two e4m3 values (the low and the high byte) as floats.
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(pair)));
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
// Two floats rounded to e4m3 (to even; past the largest value to it), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_pack(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^e of a row's biased exponent
__device__ __forceinline__ float scale_of(uint32_t biased) { return __uint_as_float(biased << 23); }

}  // namespace h3
