// Device helpers shared by the paged-cache kernels.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace ds {

constexpr unsigned kFlagBadPage = 0x8u;  // mirrored in ds_layer.h

// The sequence that owns packed row t: the number of ends cu[1 .. B] that are
// <= t, B where the row is behind the last sequence.  All 32 lanes take part:
// 32 probes a step, so 1024 sequences take two dependent loads.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer is in lo .. lo + n
  while (n > 32) {
    const int step = (n + 31) >> 5;
    const int i = (lane + 1) * step;
    const bool le = i <= n && cu[lo + i] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    n = min(n - c * step, step);
  }
  const bool le = lane < n && cu[lo + lane + 1] <= t;
  return lo + __popc(__ballot_sync(0xffffffffu, le));
}

// Row index (of [num_pages][kv_heads][page_size] rows) of position pos of
// sequence b for head 0, or -1 with a flag in *why where there is none.
__device__ __forceinline__ long long page_row(const PagedView& c, int b, int pos, unsigned* why) {
  const int pi = pos >> c.page_shift;
  if (pi >= c.table_stride) {
    *why = kFlagCacheOverflow;
    return -1;
  }
  const int page = c.table[(size_t)b * c.table_stride + pi];
  if (page < 0 || page >= c.num_pages) {
    *why = kFlagBadPage;
    return -1;
  }
  return ((long long)page * c.kv_heads << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// min / max that return NaN where an operand is NaN (a row that holds one
// must not lose it to the quantiser).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace ds
