// Internal interfaces of the gated scan, h_t = a_t h_{t-1} + b_t with a gate for every token and channel.
#pragma once

#include <cuda_runtime.h>

#include "mhla.h"
#include "retention.h"

namespace mhla {

// Tokens between two states that the forward keeps for the backward pass.  64: 1/32 of a bf16 tensor's bytes, and a
// multiple of every kernel's rows a warp.
constexpr int kScanKept = 64;

// Tokens of a sequence (packed: of a call) at most: a row of a tile that ends behind them has an int of its own.
constexpr long long kScanMaxTokens = (1ll << 31) - 1024;
// Channels at most: a block's last channel, in the row or behind it, has an int of its own.
constexpr int kScanMaxChannels = (int)((1ll << 31) - 1024);

struct ScanArgs {
  RetTensor x, g, y;            // [B, 1, N, D] (sh unused)
  RetTensor dy, dx, dg;         // backward
  int B, N, D;                  // B sequences; dense: of N tokens each; packed: of N tokens in all
  const int* cu;                // packed: [B + 1] offsets; dense: null
  int gate;                     // a gated_scan_gate
  float* states;                // [n_slots][D] or null
  const int* slots;             // [B] or null (sequence i uses slot i)
  int n_slots, load;
  float* kept;                  // [batch][ceil(N / kScanKept)][D]: the state before token kScanKept i; forward: may be null
  const float* h0;              // backward: [B][D] the start, or null (zero)
  const float* dh_last;         // backward: [B][D] the gradient of the last state, or null (zero)
  float* dh0;                   // backward: [B][D] the gradient of the start, or null
};

cudaError_t gated_scan_forward_launch(const ScanArgs& a, mhla_dtype dt, cudaStream_t st);
cudaError_t gated_scan_backward_launch(const ScanArgs& a, mhla_dtype dt, cudaStream_t st);
cudaError_t gated_scan_step_launch(const ScanArgs& a, mhla_dtype dt, cudaStream_t st);

}  // namespace mhla
