// Internal interfaces of the retention operators (linear attention with a decay for each head).
//
// Everything is one kind of pass over a sequence,
//   out_t = scale * sum_{s <= t} gamma^(t-s) (a_t . b_s) c_s        (reverse: s >= t, gamma^(s-t)),
// the forward with a = phi(q), b = phi(k), c = v, and the three gradients
//   dphi(q): a = dy, b = v, c = phi(k);                  reverse  dphi(k): a = v, b = dy, c = phi(q);
//   reverse  dv: a = phi(k), b = phi(q), c = dy
// ("Linear Attention notes" §七 for the recurrence S_t = gamma S_{t-1} + phi(k_t) v_t^T; the gradients
// are its chain rule).  The sequences are cut into segments of L tokens; a pass over a segment starts
// from the state entering it, X = sum over the tokens before it of gamma^(distance) b c^T.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "mhla.h"

namespace mhla {

constexpr int kRetMaxPasses = 3;
// SMs of a GB300: what the segments' plan and the copies' grid count on.  A constant, so that a workspace's size
// depends on the sizes alone and can be asked for without a device; with another count the results are the same
// and the last round of blocks is filled less well.
constexpr int kRetSms = 152;
// Tokens of a call at most: a chunk's last row (128 tokens), in the sequence or behind it, has an int of its own.
constexpr long long kRetMaxTokens = (1ll << 31) - 128;

// Pieces of `size` tokens that `len` tokens take.  (len + size - 1 would pass 2^31 in the longest sequences.)
__host__ __device__ __forceinline__ int ret_pieces(int len, int size) { return len > 0 ? (len - 1) / size + 1 : 0; }

struct RetTensor {
  const void* p;                // element (0, 0, 0, 0) of [B, H, N, d], d contiguous
  long long sb, sh, sn;         // strides in elements
  int feature;                  // feature map applied when read (3 = identity)
};

struct RetPass {
  RetTensor a, b, c;
  RetTensor x;                  // out is multiplied by phi'(x); x.p null: by nothing
  RetTensor out;
  int reverse;
  int sum;                      // index of the pass's set of segment states in the workspace ...
  int sum_t;                    // ... and whether they are that set's transposes
};

struct RetArgs {
  RetPass pass[kRetMaxPasses];
  int npass;                    // passes
  int nsum;                     // sets of segment states; set i is made by the pass with sum = i, sum_t = 0
  int B, H, N, T, d;            // B sequences; dense: of N tokens each (T = B N); packed: of T tokens in all (N = T)
  const int* cu;                // packed: [B + 1] offsets; dense: null
  const float* gamma;           // [H]
  float scale;
  float* states;                // [n_slots][H][d][d] or null: the forward's state in (load) and out
  const int* slots;             // [B] or null (sequence i uses slot i)
  int n_slots, load;
  int L;                        // tokens of a segment (a multiple of 128; fp32: of 64)
  int G;                        // segments in all; of those, segments that enter another one; sequences of two
  int inner, split;             // segments or more (packed: at most)
  int W;                        // segments of such sequences (packed: at most)
  float* seg;                   // [nsum][W][H][d][d] their states; null when no sequence has two segments
  unsigned* status;             // the workspace's status word
};

// ---- tensor-core passes (bf16)
cudaError_t tc_retention_launch(const RetArgs& a, cudaStream_t st);
// Limit of every bounded device-side wait of these (0 restores the default 0.5 s).
void tc_retention_set_wait_limit(unsigned long long ns);
// ---- SIMT passes (fp32)
cudaError_t simt_retention_launch(const RetArgs& a, cudaStream_t st);
// Turns the segments' own sums into the states entering them (both kernel families).
cudaError_t retention_scan_launch(const RetArgs& a, cudaStream_t st);

cudaError_t retention_step_launch(int B, int H, int d, mhla_dtype dt, const RetTensor& q, const RetTensor& k,
                                  const RetTensor& v, const RetTensor& out, const float* gamma, float scale,
                                  float* states, const int* slots, int n_slots, cudaStream_t st);
cudaError_t retention_copy_launch(float* states, long long slot_elems, int n_slots, const int* src, const int* dst,
                                  int n, cudaStream_t st);

}  // namespace mhla
