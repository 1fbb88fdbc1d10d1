// gdn_scan_device.h -- what the scan's kernels share: a segment's tokens and
// 64-bit wave sums.
#pragma once
#include "gdn_layer.h"

namespace gdn {

struct SegRange {
  int n, s, ns;     // sequence, segment within it, segments of the sequence
  int64_t row0;     // first token of the segment (global row)
  int len;          // its tokens
  int c0;           // its first chunk within the sequence
};
__device__ __forceinline__ bool seg_range(const SeqInfo& seq, const SegDesc* segs, const int* seg_first, int j,
                                          SegRange& r) {
  const SegDesc d = seq.seg_of(segs, j);
  if (d.n < 0) return false;  // the device cu_seqlens disagrees with the plan: nothing is written
  r.n = d.n;
  r.s = d.s;
  r.ns = seq.nseg_of(seg_first, d.n);
  const int t0 = min(d.c_begin * CH, seq.len(d.n)), t1 = min(d.c_end * CH, seq.len(d.n));
  r.row0 = seq.start(d.n) + t0;
  r.len = t1 - t0;
  r.c0 = d.c_begin;
  return true;
}

// The plan marks every segment when the device cu_seqlens disagrees with the
// host copy that sized the work.
__device__ __forceinline__ bool plan_invalid(const SeqInfo& seq, const SegDesc* segs) {
  return seq.cu && segs[0].n < 0;
}

__device__ __forceinline__ double wave_sum_d(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

}  // namespace gdn
