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

struct PagedSegment {
  int q0, rows;  // query rows
  int used;      // cached tokens, of which the rows are the last
};

// Segment g; one that is out of range has neither rows nor keys, and is recorded.
__device__ __forceinline__ PagedSegment checked_paged_segment(const PagedSegments& s, int g, unsigned int* err) {
  const int a = s.cu_q[g], b = s.cu_q[g + 1], used = s.used[g];
  const bool ordered = a >= 0 && a <= b && b <= s.capacity_q && (g > 0 || a == 0);
  const int64_t room = s.table.num_pages > 0 ? static_cast<int64_t>(s.table.per_segment) << s.table.page_shift : 0;
  if (!ordered || b - a > s.max_seqlen_q || used < 0 || used > room || used > kPagedMaxTokens) {
    record_error(err, kErrBadCuSeqlens);
    return PagedSegment{0, 0, 0};
  }
  if (used > s.max_seqlen_k) record_error(err, kErrBadCuSeqlens);  // computed all the same
  return PagedSegment{a, b - a, used};
}

// Keys that row i of a segment sees.  Its position, used - rows + i, is negative when there are more rows than
// tokens; such a row sees none.
__device__ __forceinline__ int row_limit(const PagedSegment& s, int i, int block) {
  if (block == 0) return s.used;
  const int p = s.used - s.rows + i;
  if (p < 0) return 0;
  const int rest = block - p % block;  // to the end of the row's block
  return s.used - p <= rest ? s.used : p + rest;
}

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
// Bytes `pick` and `pick` + 1 of a word of e4m3 as a pair of bf16 that stand for the values times 2^(7 - 127), a
// subnormal e4m3 being a subnormal bf16: the seven low bits go to bits 4 to 10 and the sign from there to bit 15.  With
// b = s 2^7 + r that is 16 b + 240 s 2^7: a byte permutation, a mask and two multiply-adds.  The multiply-adds leave
// the ALU free, which the softmax needs too (1,042 us; with a shift and masks in their place 1,056).
template <int kPick>
__device__ __forceinline__ uint32_t e4m3_pair_bits(uint32_t w) {
  const uint32_t b = __byte_perm(w, 0u, kPick == 0 ? 0x4140 : 0x4342);  // a byte in each half
  uint32_t wide, r;
  asm("mul.lo.u32 %0, %1, 16;" : "=r"(wide) : "r"(b));
  asm("mad.lo.u32 %0, %1, 240, %2;" : "=r"(r) : "r"(b & 0x00800080u), "r"(wide));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Two e4m3 bytes (the low or the high half of a word) as a pair of f16, which holds each exactly.
template <int kHalf>
__device__ __forceinline__ uint32_t e4m3_pair_f16(uint32_t w) {
  uint32_t r;
  if (kHalf == 0)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// 2^e of a row's biased exponent; NaN for kScaleNan, which marks a row that held a NaN
__device__ __forceinline__ float scale_of(uint32_t biased) {
  return __uint_as_float(biased == kScaleNan ? 0x7fffffffu : biased << 23);
}

// e itself as a float, NaN likewise
__device__ __forceinline__ float scale_log2_of(uint32_t biased) {
  const float e = __uint_as_float(0x4b000000u | biased) - (8388608.f + 127.f);  // 2^23 + biased, exactly
  return biased == kScaleNan ? __uint_as_float(0x7fffffffu) : e;
}

}  // namespace h3
