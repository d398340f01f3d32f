// C-ABI entry points of the gated scan: argument validation and dispatch.  The operations are documented in
// include/mhla.h.
#include "common.cuh"
#include "gated_scan.h"
#include "internal.h"
#include "strided.h"

namespace mhla {
namespace {

struct Sizes {
  Extent e;          // of a token tensor
  size_t rows_bytes; // of a [B, D] fp32 tensor
  size_t cu_bytes, slot_bytes;
};

mhla_status sizes_of(Sizes* s, int B, int N, int D, const int* cu, mhla_dtype dt, int gate, bool* empty) {
  *empty = false;
  if (B < 0 || N < 0 || D < 0 || (dt != MHLA_F32 && dt != MHLA_BF16) || gate < GATED_SCAN_SIGMOID || gate > GATED_SCAN_DECAY)
    return MHLA_ERR_INVALID_ARG;
  const int es = dt == MHLA_F32 ? 4 : 2;
  if (D % (16 / es) != 0 || !aligned(cu, 4)) return MHLA_ERR_INVALID_ARG;
  *empty = B == 0 || N == 0 || D == 0;
  if (N > kScanMaxTokens || D > kScanMaxChannels) return MHLA_ERR_UNSUPPORTED;
  if ((Wide)B * D * 4 > kNoMemory) return MHLA_ERR_INVALID_ARG;
  if ((long long)B * ((D + 31) / 32) > 0x7fffffffll / 16) return MHLA_ERR_UNSUPPORTED;  // the blocks are numbered
  s->e = {cu ? 1 : B, 1, N, D, es};
  s->rows_bytes = (size_t)B * D * 4;
  s->cu_bytes = cu ? ((size_t)B + 1) * 4 : 0;
  s->slot_bytes = (size_t)B * 4;
  return MHLA_OK;
}

bool kept_bytes(size_t* n, const Extent& e) {
  const Wide w = (Wide)e.b * ret_pieces((int)e.n, kScanKept) * e.d * 4;
  *n = (size_t)w;
  return w <= kNoMemory;
}

}  // namespace
}  // namespace mhla

using namespace mhla;

extern "C" {

long long gated_scan_checkpoint_rows(int B, int N) {
  return B < 0 || N < 0 || N > kScanMaxTokens ? 0 : (long long)B * ret_pieces(N, kScanKept);
}

mhla_status gated_scan_forward(const void* x, const mhla_strides* x_strides, const void* g, const mhla_strides* g_strides,
                               void* y, const mhla_strides* y_strides, int B, int N, int D, const int* cu_seqlens,
                               float* states, const int* slots, int n_slots, int load_state, float* checkpoints,
                               mhla_dtype dt, int gate, void* stream) {
  if (load_state != 0 && load_state != 1) return MHLA_ERR_INVALID_ARG;
  if (states == nullptr ? (slots != nullptr || load_state != 0) : n_slots < 0) return MHLA_ERR_INVALID_ARG;
  Sizes s;
  bool empty;
  const mhla_status st = sizes_of(&s, B, N, D, cu_seqlens, dt, gate, &empty);
  if (st != MHLA_OK || empty) return st;
  ScanArgs a{};
  const Extent& e = s.e;
  if (!make_tensor(&a.x, x, x_strides, e) || !make_tensor(&a.g, g, g_strides, e) || !make_tensor(&a.y, y, y_strides, e) ||
      !injective(a.y, e) || !disjoint(a.y, a.x, e) || !disjoint(a.y, a.g, e))
    return MHLA_ERR_INVALID_ARG;
  const Wide pool = states ? (Wide)n_slots * D * 4 : 0;
  size_t kb;
  if (pool > kNoMemory || !kept_bytes(&kb, e) || !aligned(states, 16) || !aligned(slots, 4) || !aligned(checkpoints, 16))
    return MHLA_ERR_INVALID_ARG;
  const Region r[] = {{x, span_bytes(a.x, e), false}, {g, span_bytes(a.g, e), false}, {y, span_bytes(a.y, e), true},
                      {states, (size_t)pool, true}, {checkpoints, checkpoints ? kb : 0, true},
                      {cu_seqlens, s.cu_bytes, false}, {slots, slots ? s.slot_bytes : 0, false}};
  if (clash(r, 3)) return MHLA_ERR_INVALID_ARG;
  a.B = B;
  a.N = N;
  a.D = D;
  a.cu = cu_seqlens;
  a.gate = gate;
  a.states = states;
  a.slots = slots;
  a.n_slots = n_slots;
  a.load = load_state;
  a.kept = checkpoints;
  return from_cuda(gated_scan_forward_launch(a, dt, static_cast<cudaStream_t>(stream)));
}

mhla_status gated_scan_backward(const void* x, const mhla_strides* x_strides, const void* g,
                                const mhla_strides* g_strides, const void* dy, const mhla_strides* dy_strides,
                                const float* checkpoints, void* dx, const mhla_strides* dx_strides, void* dg,
                                const mhla_strides* dg_strides, int B, int N, int D, const int* cu_seqlens,
                                const float* h0, const float* dh_last, float* dh0, mhla_dtype dt, int gate, void* stream) {
  Sizes s;
  bool empty;
  const mhla_status st = sizes_of(&s, B, N, D, cu_seqlens, dt, gate, &empty);
  if (st != MHLA_OK) return st;
  if (!aligned(h0, 16) || !aligned(dh_last, 16) || !aligned(dh0, 16)) return MHLA_ERR_INVALID_ARG;
  if (dh0 != nullptr && (!apart(dh0, s.rows_bytes, h0, s.rows_bytes) || !apart(dh0, s.rows_bytes, dh_last, s.rows_bytes)))
    return MHLA_ERR_INVALID_ARG;
  if (empty) {  // without tokens the last state is the start
    if (N != 0 || dh0 == nullptr || s.rows_bytes == 0) return MHLA_OK;
    return from_cuda(dh_last ? cudaMemcpyAsync(dh0, dh_last, s.rows_bytes, cudaMemcpyDeviceToDevice, static_cast<cudaStream_t>(stream))
                             : cudaMemsetAsync(dh0, 0, s.rows_bytes, static_cast<cudaStream_t>(stream)));
  }
  ScanArgs a{};
  const Extent& e = s.e;
  RetTensor* in[3] = {&a.x, &a.g, &a.dy};
  RetTensor* out[2] = {&a.dx, &a.dg};
  if (!make_tensor(&a.x, x, x_strides, e) || !make_tensor(&a.g, g, g_strides, e) || !make_tensor(&a.dy, dy, dy_strides, e) ||
      !make_tensor(&a.dx, dx, dx_strides, e) || !make_tensor(&a.dg, dg, dg_strides, e) || !disjoint(a.dx, a.dg, e))
    return MHLA_ERR_INVALID_ARG;
  for (const RetTensor* o : out) {
    if (!injective(*o, e)) return MHLA_ERR_INVALID_ARG;
    for (const RetTensor* i : in)
      if (!disjoint(*o, *i, e)) return MHLA_ERR_INVALID_ARG;
  }
  size_t kb;
  if (checkpoints == nullptr || !aligned(checkpoints, 16) || !kept_bytes(&kb, e)) return MHLA_ERR_INVALID_ARG;
  const Region r[] = {{x, span_bytes(a.x, e), false}, {g, span_bytes(a.g, e), false}, {dy, span_bytes(a.dy, e), false},
                      {dx, span_bytes(a.dx, e), true}, {dg, span_bytes(a.dg, e), true}, {checkpoints, kb, false},
                      {h0, h0 ? s.rows_bytes : 0, false}, {dh_last, dh_last ? s.rows_bytes : 0, false},
                      {dh0, dh0 ? s.rows_bytes : 0, true}, {cu_seqlens, s.cu_bytes, false}};
  if (clash(r, 5)) return MHLA_ERR_INVALID_ARG;
  a.B = B;
  a.N = N;
  a.D = D;
  a.cu = cu_seqlens;
  a.gate = gate;
  a.kept = const_cast<float*>(checkpoints);
  a.h0 = h0;
  a.dh_last = dh_last;
  a.dh0 = dh0;
  return from_cuda(gated_scan_backward_launch(a, dt, static_cast<cudaStream_t>(stream)));
}

mhla_status gated_scan_step(const void* x, const mhla_strides* x_strides, const void* g, const mhla_strides* g_strides,
                            float* states, const int* slots, int n_slots, void* out, const mhla_strides* out_strides,
                            int B, int D, mhla_dtype dt, int gate, void* stream) {
  Sizes s;
  bool empty;
  const mhla_status st = sizes_of(&s, B, 1, D, nullptr, dt, gate, &empty);
  if (st != MHLA_OK) return st;
  if (n_slots < 0) return MHLA_ERR_INVALID_ARG;
  if (empty) return MHLA_OK;
  ScanArgs a{};
  const Extent& e = s.e;
  if (!make_tensor(&a.x, x, x_strides, e) || !make_tensor(&a.g, g, g_strides, e) || !make_tensor(&a.y, out, out_strides, e) ||
      !injective(a.y, e) || !disjoint(a.y, a.x, e) || !disjoint(a.y, a.g, e))
    return MHLA_ERR_INVALID_ARG;
  const Wide pool = (Wide)n_slots * D * 4;
  if (states == nullptr || !aligned(states, 16) || !aligned(slots, 4) || pool > kNoMemory) return MHLA_ERR_INVALID_ARG;
  const Region r[] = {{x, span_bytes(a.x, e), false}, {g, span_bytes(a.g, e), false}, {out, span_bytes(a.y, e), true},
                      {states, (size_t)pool, true}, {slots, slots ? s.slot_bytes : 0, false}};
  if (clash(r, 3)) return MHLA_ERR_INVALID_ARG;
  a.B = B;
  a.N = 1;
  a.D = D;
  a.gate = gate;
  a.states = states;
  a.slots = slots;
  a.n_slots = n_slots;
  return from_cuda(gated_scan_step_launch(a, dt, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
