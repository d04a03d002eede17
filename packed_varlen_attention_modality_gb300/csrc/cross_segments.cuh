// Segments of a cross attention call on the device, and the one check of what their offsets may say.
#pragma once

#include "h3_internal.h"
#include "sm103_ptx.cuh"

namespace h3 {

struct CrossSegment {
  int q0, rows;        // query rows
  int k0, keys, used;  // key rows, and how many of them are used
};

// Segment g as the offsets say it, for segments that have passed checked_cross_segment().
__device__ __forceinline__ CrossSegment cross_segment(const CrossSegments& s, int g) {
  CrossSegment r;
  r.q0 = s.cu_q[g];
  r.rows = s.cu_q[g + 1] - r.q0;
  r.k0 = s.cu_k[g];
  r.keys = s.cu_k[g + 1] - r.k0;
  r.used = s.seqused_k != nullptr ? s.seqused_k[g] : r.keys;
  return r;
}

// Segment g; one that is out of range has neither rows nor keys, and is recorded.
__device__ __forceinline__ CrossSegment checked_cross_segment(const CrossSegments& s, int g, unsigned int* err) {
  const int a = s.cu_q[g], b = s.cu_q[g + 1], ka = s.cu_k[g], kb = s.cu_k[g + 1];
  const bool ordered = a >= 0 && a <= b && b <= s.capacity_q && ka >= 0 && ka <= kb && kb <= s.capacity_k &&
                       (g > 0 || (a == 0 && ka == 0));
  const int rows = ordered ? b - a : 0, keys = ordered ? kb - ka : 0;
  const int used = s.seqused_k != nullptr ? s.seqused_k[g] : keys;
  if (!ordered || rows > s.max_seqlen_q || used < 0 || used > keys) {
    record_error(err, kErrBadCuSeqlens);
    return CrossSegment{0, 0, 0, 0, 0};
  }
  if (used > s.max_seqlen_k) record_error(err, kErrBadCuSeqlens);  // computed all the same
  return CrossSegment{a, rows, ka, keys, used};
}

}  // namespace h3
