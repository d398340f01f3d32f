// Device helpers shared by the retention kernels: decays, feature maps, segments, slots.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "retention.h"

namespace mhla {

constexpr int kFeatIdentity = 3;  // beside the kinds of phi_k

__device__ __forceinline__ float ret_phi(float x, int feature) {
  if (feature == kFeatIdentity) return x;
  if (feature == 1) return x > 0.f ? x : (x == x ? 0.f : x);  // (not-a-number stays)
  // without a branch for the sign: neighbouring lanes differ in it
  const float e = expf(feature == 0 && x > 0.f ? 0.f : x);
  return feature == 0 && x > 0.f ? x + 1.f : e;
}
// phi'(x): 1 for the identity; ELU + 1: 1 for x > 0, e^x otherwise; ReLU: 1 for x > 0; exp: e^x
__device__ __forceinline__ float ret_dphi(float x, int feature) {
  if (feature == kFeatIdentity) return 1.f;
  if (feature == 1) return x > 0.f ? 1.f : 0.f;
  return feature == 0 && x > 0.f ? 1.f : expf(x);
}

// Two products / multiply-adds in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return r;
}

// log2(gamma).  From 1/2 on gamma - 1 is exact, so decays close to 1 keep their digits; below it gamma - 1 would be
// rounded (1e-5 off by 0.1 %, 2e-8 taken as 0), so gamma is m 2^e with m in [1/2, 1).  One logarithm for both: every
// block waits for it (with log2f beside log1pf 64 heads of 8192 tokens 101.7 us, so 100.9).  gamma = 0 gives -inf.
__device__ __forceinline__ float decay_log2(float gamma) {
  int e = 0;
  const float m = gamma < 0.5f ? frexpf(gamma, &e) : gamma;
  return fmaf(log1pf(m - 1.f), 1.4426950408889634f, (float)e);
}

// gamma^n for n >= 0 from lg = log2(gamma).  Relative error: the logarithm within 1.75 steps, its product with n
// rounded, so 2.25 x 2^-23 n |lg| ln 2, and the exponential's own 2^-21: about 2^-18 where the power is 2^-32, less
// where it is larger.  gamma^0 = 1 for every gamma, 0 among them.
__device__ __forceinline__ float decay_pow(float lg, int n) { return n == 0 ? 1.f : exp2f(lg * (float)n); }

// Programmatic dependent launch: a kernel of a call starts while the one before it drains; what it reads of
// that one's results comes behind grid_dependency_wait().  The inputs do not: the first kernel of a call is
// an ordinary launch.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename Args>
cudaError_t launch_dependent(void (*kernel)(Args), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, bool dependent,
                             const Args& args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = dependent ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args);
  note_launch();
  return e;
}

struct Segment {
  int seq;     // sequence, -1: no such segment
  int seg;     // its number within the sequence
  int nseg;    // segments of the sequence
  int w0;      // of a sequence of two segments or more: the workspace's first state of it
  int row0;    // first token row (within the sequence's batch entry when dense)
  int len;     // tokens of the segment
  int all;     // tokens of the sequence
};

// Which segments a kernel's blocks go over.
enum SegmentKind {
  SEG_ALL = 0,    // every segment
  SEG_INNER = 1,  // nseg - 1 of each sequence: those that enter another one (numbered from 0)
  SEG_SPLIT = 2   // one for each sequence of two segments or more
};

// Tokens [lo, hi) of packed sequence i.  Offsets outside [0, T] or out of order are clamped, so that
// whatever cu holds, no row outside the tensors is touched.
__device__ __forceinline__ void packed_range(const RetArgs& a, int i, int* lo, int* hi) {
  *lo = min(max(a.cu[i], 0), a.T);
  *hi = min(max(a.cu[i + 1], *lo), a.T);
}
__device__ __forceinline__ int packed_segments(const RetArgs& a, int i) {
  int lo, hi;
  packed_range(a, i, &lo, &hi);
  return ret_pieces(hi - lo, a.L);
}

__device__ __forceinline__ int segments_of_kind(int nseg, SegmentKind kind) {
  return kind == SEG_ALL ? nseg : kind == SEG_INNER ? max(nseg - 1, 0) : nseg >= 2 ? 1 : 0;
}

// Sum of two counts of segments, capped: offsets out of order may claim 2^31 segments and more, and a place that
// wrapped would lie outside the workspace.  Every number that counts (blocks of a grid, states of the workspace) is
// below the cap: a call has at most 2^31 / 3.
constexpr unsigned kMostSegments = 1u << 30;
__device__ __forceinline__ int add_capped(int a, int b) { return (int)min((unsigned)a + (unsigned)b, kMostSegments - 1); }

constexpr int kOrdered = 64;  // packed sequences up to so many are taken longest first: two a lane of one warp

// Number k of the call's segments, of at most kOrdered packed sequences taken in the order of their lengths, the
// longest first: blocks start in the order of their numbers, and a long sequence started last would run alone.  More
// sequences are taken as they come.  On both sides of the limit, 64 sequences of 40,000 tokens, one of 4000 among them,
// 16 heads, and the same with one of a single token more: prompts with d = 128 232 us, 285 with the long one first and 310
// with it last; d = 64 126, 177 and 204; gradients 468, 492 and 512, d = 64 265, 337 and 362.  (The counts fit: 64
// sequences of at most 2^31 - 128 tokens in segments of 64 or more are below 2^31 segments.)
__device__ __forceinline__ Segment find_ordered(const RetArgs& a, int k, int* scratch) {
  const int tid = threadIdx.x;
  int lo = 0, hi = 0;
  if (tid < a.B) {
    packed_range(a, tid, &lo, &hi);
    scratch[tid] = hi - lo;
  }
  __syncthreads();
  if (tid < a.B) {
    const int mine = hi - lo;
    int at = 0;
    for (int i = 0; i < a.B; ++i) at += scratch[i] > mine || (scratch[i] == mine && i < tid);
    scratch[kOrdered + at] = tid;
  }
  __syncthreads();
  Segment s;
  s.seq = -1;
  if (tid < 32) {  // the first warp: places 2 lane, 2 lane + 1 of the order
    int q[2], m[2], n = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = 2 * tid + i < a.B ? scratch[kOrdered + 2 * tid + i] : 0;
      m[i] = 2 * tid + i < a.B ? ret_pieces(scratch[q[i]], a.L) : 0;
      n += m[i];
    }
    int first = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, first, o);
      if (tid >= o) first += u;
    }
    first -= n;
    // states of the split sequences before sequence 2 tid, 2 tid + 1 (in their own order)
    int w[2], v = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = 2 * tid + i < a.B ? ret_pieces(scratch[2 * tid + i], a.L) : 0;
      w[i] = w[i] >= 2 ? w[i] : 0;
      v += w[i];
    }
    int before = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, before, o);
      if (tid >= o) before += u;
    }
    before -= v;
    const bool one = k >= first && k < first + n;
    const unsigned who = __ballot_sync(0xffffffffu, one);
    if (who != 0) {
      const int src = __ffs(who) - 1, hit = k - first >= m[0] ? 1 : 0;
      s.seq = __shfl_sync(0xffffffffu, hit ? q[1] : q[0], src);
      s.nseg = __shfl_sync(0xffffffffu, hit ? m[1] : m[0], src);
      s.seg = __shfl_sync(0xffffffffu, k - first - (hit ? m[0] : 0), src);
      const int even = __shfl_sync(0xffffffffu, before, s.seq >> 1), first_w = __shfl_sync(0xffffffffu, w[0], s.seq >> 1);
      s.w0 = even + (s.seq & 1 ? first_w : 0);
    }
    __syncwarp();
    if (tid == 0) {
      scratch[kOrdered] = s.seq;
      scratch[kOrdered + 1] = s.nseg;
      scratch[kOrdered + 2] = s.seg;
      scratch[kOrdered + 3] = s.w0;
    }
  }
  __syncthreads();
  s.seq = scratch[kOrdered];
  s.nseg = scratch[kOrdered + 1];
  s.seg = scratch[kOrdered + 2];
  s.w0 = scratch[kOrdered + 3];
  __syncthreads();
  if (s.seq < 0) return s;
  packed_range(a, s.seq, &lo, &hi);
  s.all = hi - lo;
  s.row0 = lo + s.seg * a.L;
  s.len = min(a.L, s.all - s.seg * a.L);
  if (s.nseg >= 2 && s.w0 + s.nseg > a.W) s.seq = -1;  // (offsets out of order, as below)
  return s;
}

// Number k of the call's segments of a kind (whole block; scratch: 2 kOrdered ints of shared memory).  Packed sequences'
// segments are numbered sequence after sequence: thread t counts those of B / blockDim.x sequences, a block-wide scan
// finds the thread whose range holds k.  An empty sequence has none.
__device__ __forceinline__ Segment find_segment(const RetArgs& a, int k, SegmentKind kind, int* scratch) {
  Segment s;
  int lo = 0;
  if (a.cu != nullptr && kind == SEG_ALL && a.B <= kOrdered) return find_ordered(a, k, scratch);
  if (a.cu == nullptr) {
    s.nseg = ret_pieces(a.N, a.L);
    const int per = segments_of_kind(s.nseg, kind);
    s.seq = per > 0 && k < a.B * per ? k / per : -1;
    if (s.seq < 0) return s;
    s.seg = k - s.seq * per;
    s.w0 = s.seq * s.nseg;
    s.all = a.N;
  } else {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int i0 = min(tid * per, a.B), i1 = min(i0 + per, a.B);
    int n = 0, m = 0;  // of the kind, of split sequences
    for (int i = i0; i < i1; ++i) {
      const int q = packed_segments(a, i);
      n = add_capped(n, segments_of_kind(q, kind));
      m = add_capped(m, q >= 2 ? q : 0);
    }
    int in = n, im = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, in, o), v = __shfl_up_sync(0xffffffffu, im, o);
      if (lane >= o) {
        in = add_capped(in, u);
        im = add_capped(im, v);
      }
    }
    if (lane == 31) {
      scratch[warp] = in;
      scratch[32 + warp] = im;
    }
    if (tid == 0) scratch[64] = -1;
    __syncthreads();
    // the sums before this thread (not in - n: capped sums have no difference)
    int first = __shfl_up_sync(0xffffffffu, in, 1), w0 = __shfl_up_sync(0xffffffffu, im, 1);
    if (lane == 0) first = w0 = 0;
    for (int w = 0; w < warp; ++w) {
      first = add_capped(first, scratch[w]);
      w0 = add_capped(w0, scratch[32 + w]);
    }
    if (k >= first && k < first + n) {
      for (int i = i0; i < i1; ++i) {
        const int q = packed_segments(a, i), c = segments_of_kind(q, kind);
        if (k < first + c) {
          scratch[64] = i;
          scratch[65] = k - first;
          scratch[66] = w0;
          break;
        }
        first = add_capped(first, c);
        w0 = add_capped(w0, q >= 2 ? q : 0);
      }
    }
    __syncthreads();
    s.seq = scratch[64];
    s.seg = scratch[65];
    s.w0 = scratch[66];
    __syncthreads();
    if (s.seq < 0) return s;
    int hi;
    packed_range(a, s.seq, &lo, &hi);
    s.nseg = packed_segments(a, s.seq);
    s.all = hi - lo;
    if (s.nseg >= 2 && s.w0 + s.nseg > a.W) {  // (offsets out of order may claim more than the workspace has)
      s.seq = -1;
      return s;
    }
  }
  s.row0 = lo + s.seg * a.L;
  s.len = max(0, min(a.L, s.all - s.seg * a.L));
  return s;
}
// The segment of an inner one (SEG_INNER) in a pass's direction: forward all but the last, reverse all but the first.
__device__ __forceinline__ void inner_segment(const RetArgs& a, Segment& s, int reverse) {
  if (reverse == 0) return;
  s.seg += 1;
  s.row0 += a.L;
  s.len = max(0, min(a.L, s.all - s.seg * a.L));
}

// Base of sequence seq, head h: packed sequences share batch entry 0.
__device__ __forceinline__ long long ret_base(const RetArgs& a, const RetTensor& t, int seq, int h) {
  return (a.cu == nullptr ? (long long)seq * t.sb : 0ll) + (long long)h * t.sh;
}

// The slot of sequence `seq`, -1 for none: out of range, or already taken by a sequence before it
// (whole block; at most B compares).
__device__ __forceinline__ int ret_slot(const int* slots, int n_slots, int seq) {
  if (slots == nullptr) return seq < n_slots ? seq : -1;
  const int s = slots[seq];
  bool taken = false;
  for (int i = threadIdx.x; i < seq; i += blockDim.x) taken |= slots[i] == s;
  return __syncthreads_or(taken) || s < 0 || s >= n_slots ? -1 : s;
}

// The state entering a segment of head h (null: zero); slot: the sequence's state slot, -1 for none.  The states in
// the workspace are there behind grid_dependency_wait().
__device__ __forceinline__ const float* entering_state(const RetArgs& a, const RetPass& p, const Segment& sg, int h,
                                                       int slot) {
  const size_t dd = (size_t)a.d * a.d;
  if (sg.nseg > 1) return a.seg + (((size_t)p.sum * a.W + sg.w0 + sg.seg) * a.H + h) * dd;
  return a.load && slot >= 0 ? a.states + ((size_t)slot * a.H + h) * dd : nullptr;
}

}  // namespace mhla
