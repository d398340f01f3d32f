// Internal interfaces of linear cross attention: an encoder's tokens summed up as S = sum phi(k) v^T, z = sum phi(k),
// and read by queries of another number ("Linear Attention notes" §三 with keys and values of another sequence).
#pragma once

#include <cuda_runtime.h>

#include "mhla.h"
#include "retention.h"

namespace mhla {

// One side's tokens, queries or keys, as sequences cut into segments of L tokens.
struct CrossSide {
  int B, N, T;       // B sequences; dense: of N tokens each; packed: of T tokens in all (N = T)
  const int* cu;     // packed: [B + 1] offsets; dense: null
  const int* lens;   // dense: [B] tokens of each, or null (N)
  int L;             // tokens of a segment
  int segs;          // segments at most: dense B ceil(N / L); packed T / L + B
};

struct CrossArgs {
  RetTensor q, k, v, y;            // feature maps in q.feature, k.feature
  RetTensor dy, dq, dk, dv;        // backward
  CrossSide qs, ks;
  int H, Hk, d;
  float *S, *z;                    // [n_slots or B][Hk][d][d], [..][Hk][d]
  const int* slots;                // [B] or null (sequence i uses slot i)
  int n_slots;
  int normalise;
  float eps;
  float* part;                     // partial sums: [segs][heads][d * d + d] (heads: Hk of the keys, H of the queries)
  float* dS;                       // backward: [B][Hk][d * d + d], dS then dz
  unsigned* status;                // the workspace's status word
};

// ---- SIMT kernels (every type and width)
cudaError_t simt_cross_states_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st);
cudaError_t simt_cross_read_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st);
cudaError_t simt_cross_backward_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st);
// one query a row (N = 1, dense)
cudaError_t cross_step_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st);
// The sums over segments (and, backward, over the query heads of a key head): what the segments' kernels left in part.
cudaError_t cross_join_launch(const CrossArgs& a, bool backward, cudaStream_t st);

// Whether the segments' kernel of the states has to be joined: not where every sequence is one segment.
__host__ __device__ inline bool cross_joined(const CrossSide& s) { return s.cu != nullptr || s.N == 0 || s.N > s.L; }

}  // namespace mhla
