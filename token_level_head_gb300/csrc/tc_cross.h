// Linear cross attention on the tensor cores: bf16, d = 64 or 128.
#pragma once

#include "cross.h"

namespace mhla {

bool tc_cross_supported(int d, mhla_dtype dt);
cudaError_t tc_cross_states_launch(const CrossArgs& a, cudaStream_t st);
cudaError_t tc_cross_read_launch(const CrossArgs& a, cudaStream_t st);
cudaError_t tc_cross_backward_launch(const CrossArgs& a, cudaStream_t st);
// Limit of every bounded device-side wait of these (0 restores the default 0.5 s).
void tc_cross_set_wait_limit(unsigned long long ns);

}  // namespace mhla
