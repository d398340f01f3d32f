// Device helpers of the cross attention kernels: segments, slots.
#pragma once

#include "cross.h"
#include "retention.cuh"

namespace mhla {

struct CrossSegment {
  int seq;   // sequence, -1: no such segment
  int row0;  // first token row (within the sequence's batch entry when dense)
  int len;   // tokens of the segment
  int nseg;  // segments of the sequence
};

__device__ __forceinline__ void cross_range(const CrossSide& s, int i, int* lo, int* hi) {
  if (s.cu != nullptr) {
    *lo = min(max(s.cu[i], 0), s.T);
    *hi = min(max(s.cu[i + 1], *lo), s.T);
  } else {
    *lo = 0;
    *hi = s.lens != nullptr ? min(max(s.lens[i], 0), s.N) : s.N;
  }
}
// The number of a sequence's first segment.  Packed: lo / L + i, which leaves every sequence its ceil(len / L) numbers
// (the next one's is at least lo / L + len / L + i + 1) and needs no sum over the sequences before; offsets out of order
// stay below T / L + B all the same.
__device__ __forceinline__ int cross_first(const CrossSide& s, int i, int lo) {
  return s.cu != nullptr ? lo / s.L + i : i * ret_pieces(s.N, s.L);
}

// Segment number k (whole block; scratch: one int of shared memory).
__device__ __forceinline__ CrossSegment cross_segment(const CrossSide& s, int k, int* scratch) {
  CrossSegment g;
  if (s.cu == nullptr) {
    g.nseg = ret_pieces(s.N, s.L);
    g.seq = k / g.nseg;
    int lo, hi;
    cross_range(s, g.seq, &lo, &hi);
    g.row0 = (k - g.seq * g.nseg) * s.L;
    g.len = min(max(hi - g.row0, 0), s.L);
    return g;
  }
  if (threadIdx.x == 0) *scratch = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < s.B; i += blockDim.x) {
    int lo, hi;
    cross_range(s, i, &lo, &hi);
    const int first = cross_first(s, i, lo);
    if (k >= first && k - first < ret_pieces(hi - lo, s.L)) atomicMax(scratch, i);
  }
  __syncthreads();
  g.seq = *scratch;
  if (g.seq < 0) return g;
  int lo, hi;
  cross_range(s, g.seq, &lo, &hi);
  g.nseg = ret_pieces(hi - lo, s.L);
  g.row0 = lo + (k - cross_first(s, g.seq, lo)) * s.L;
  g.len = min(max(hi - g.row0, 0), s.L);
  return g;
}

// Element (sequence, head, 0, 0) of a tensor; packed sequences share batch entry 0.
__device__ __forceinline__ long long cross_base(const CrossSide& s, const RetTensor& t, int seq, int h) {
  return (s.cu == nullptr ? (long long)seq * t.sb : 0ll) + (long long)h * t.sh;
}

// 1 / den: 0 where no token counts (den = 0 with eps = 0 and nothing summed), so that such rows are zeros.  A den below 2^-120
// counts as 0 too: the reciprocal of one below 2^-128 is infinite, and zeros times it not a number; and y . dy / den, which the
// gradients go through, passes the largest number for |y . dy| = 2^8 at 2^-120.
constexpr float kLeastDen = 0x1p-120f;
__device__ __forceinline__ float cross_inverse(float den) { return fabsf(den) < kLeastDen ? 0.f : 1.f / den; }

}  // namespace mhla
