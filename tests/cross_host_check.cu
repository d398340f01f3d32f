// The host side of the cross attention's entries (csrc/cross_api.cu) with launches that only note their arguments: a call
// that passes every check can be made with addresses of no memory, on a machine without a GPU.
#include "cross_api.cu"

namespace mhla {
namespace {
CrossArgs last;
long long calls[4];  // states, read, backward, join
cudaError_t note(int what, const CrossArgs& a) {
  last = a;
  ++calls[what];
  return cudaSuccess;
}
}  // namespace
bool tc_cross_supported(int d, mhla_dtype dt) { return dt == MHLA_BF16 && (d == 64 || d == 128); }
cudaError_t tc_cross_states_launch(const CrossArgs& a, cudaStream_t) { return note(0, a); }
cudaError_t tc_cross_read_launch(const CrossArgs& a, cudaStream_t) { return note(1, a); }
cudaError_t tc_cross_backward_launch(const CrossArgs& a, cudaStream_t) { return note(2, a); }
cudaError_t simt_cross_states_launch(const CrossArgs& a, mhla_dtype, cudaStream_t) { return note(0, a); }
cudaError_t simt_cross_read_launch(const CrossArgs& a, mhla_dtype, cudaStream_t) { return note(1, a); }
cudaError_t simt_cross_backward_launch(const CrossArgs& a, mhla_dtype, cudaStream_t) { return note(2, a); }
cudaError_t cross_step_launch(const CrossArgs& a, mhla_dtype, cudaStream_t) { return note(1, a); }
cudaError_t cross_join_launch(const CrossArgs& a, bool, cudaStream_t) { return note(3, a); }
}  // namespace mhla

extern "C" void check_calls(long long* out) {
  for (int i = 0; i < 4; ++i) {
    out[i] = mhla::calls[i];
    mhla::calls[i] = 0;
  }
}
// Of the last launch: segments of the queries and of the keys, bytes of the workspace with its parts (and, backward, dS).
extern "C" void check_plan(long long* out, int backward) {
  const mhla::CrossArgs& a = mhla::last;
  const long long E = 1ll * a.d * a.d + a.d;
  const long long parts = backward ? 1ll * a.qs.segs * a.H + 1ll * a.qs.B * a.Hk : 1ll * a.ks.segs * a.Hk;
  out[0] = a.qs.segs;
  out[1] = a.ks.segs;
  out[2] = (long long)mhla::kWorkspacePrefix + parts * E * 4;
}
