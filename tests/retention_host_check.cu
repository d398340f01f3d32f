// The host side of the retention entries (csrc/retention_api.cu) with launches that only note their arguments: a
// call that passes every check can be made with addresses of no memory, on a machine without a GPU.
#include "retention_api.cu"

namespace mhla {
namespace {
RetArgs last;
long long calls = 0;
}  // namespace
cudaError_t tc_retention_launch(const RetArgs& a, cudaStream_t) {
  last = a;
  ++calls;
  return cudaSuccess;
}
cudaError_t simt_retention_launch(const RetArgs& a, cudaStream_t) {
  last = a;
  ++calls;
  return cudaSuccess;
}
cudaError_t retention_step_launch(int, int, int, mhla_dtype, const RetTensor&, const RetTensor&, const RetTensor&,
                                  const RetTensor&, const float*, float, float*, const int*, int, cudaStream_t) {
  ++calls;
  return cudaSuccess;
}
cudaError_t retention_copy_launch(float*, long long, int, const int*, const int*, int, cudaStream_t) {
  ++calls;
  return cudaSuccess;
}
}  // namespace mhla

extern "C" long long check_calls() { return mhla::calls; }
// The last passes' plan: L, G, inner, split, W, nsum, first byte behind the workspace's states.
extern "C" void check_plan(long long* out) {
  const mhla::RetArgs& a = mhla::last;
  const long long states = a.seg ? 1ll * a.nsum * a.W * a.H * a.d * a.d * 4 : 0;
  const long long v[7] = {a.L, a.G, a.inner, a.split, a.W, a.nsum, (long long)mhla::kWorkspacePrefix + states};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
}
