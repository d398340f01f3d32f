// C-ABI entry points of linear cross attention: argument validation, the segments and dispatch.  The operations are
// documented in include/mhla.h.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "cross.h"
#include "internal.h"
#include "strided.h"
#include "tc_cross.h"

namespace mhla {
namespace {

// The kernels that a call runs on, as far as the segments go: a segment's tokens are a multiple of `unit`, and `slots`
// blocks (a segment of a head each) fill the SMs.  The FP32 kernels' unit is half of a tile of theirs: forward and gradients
// of 2003 queries and 1501 keys of 6 heads, d = 64, with segments of 128 tokens 99 us, of 64 72, of 32 64.
struct Kind {
  int unit, slots;
};
Kind kind_of(int d, bool tc) { return tc ? Kind{128, (d == 64 ? 2 : 1) * kRetSms} : Kind{32, (d == 128 ? 2 : 6) * kRetSms}; }

// Reads (three blocks an SM on the tensor cores with d = 64) leave no parts, so their segments need no room.
Kind read_kind(int d, bool tc) { return tc ? Kind{128, (d == 64 ? 3 : 1) * kRetSms} : Kind{64, (d == 128 ? 2 : 4) * kRetSms}; }

// The length of a segment: so many tokens that the blocks fill the SMs, and no fewer than a tile.
int segment_length(const CrossSide& s, int heads, const Kind& k) {
  const long long most = 1ll << 23;
  long long L;
  if (s.cu != nullptr) {
    L = ((long long)s.T * heads + k.slots - 1) / k.slots;
  } else {
    const long long pieces = std::max(1ll, k.slots / std::max(1ll, (long long)s.B * heads));
    L = (s.N + pieces - 1) / pieces;
  }
  return (int)std::max((long long)k.unit, std::min((L + k.unit - 1) / k.unit * k.unit, most));
}
// Cuts a side; false where the segments cannot be numbered.  A side without a token has none (packed too): its tensors may
// have no address, and the joins of no parts give the zeros.
bool cut_side(CrossSide* s, int B, int N, const int* cu, const int* lens, int heads, const Kind& k) {
  *s = {B, N, cu ? N : 0, cu, lens, 0, 0};
  s->L = segment_length(*s, heads, k);
  const long long segs = N == 0 ? 0 : cu ? (long long)N / s->L + B : (long long)B * ret_pieces(N, s->L);
  s->segs = (int)std::min(segs, 0x7fffffffll);
  return segs * std::max(heads, 1) <= 0x7fffffffll;
}

long long entry(int d) { return (long long)d * d + d; }
bool fits(Wide bytes) { return bytes <= kNoMemory; }

// Floats behind the prefix of a workspace: the segments' parts, and backward the gradients of the sums.
Wide part_floats(const CrossSide& s, int heads, int d) { return (Wide)s.segs * heads * entry(d); }

bool sizes_ok(int B, int H, int Hk, int N, int d) {
  return B >= 0 && H >= 0 && Hk >= 0 && N >= 0 && valid_d(d) && (Hk > 0 ? H % Hk == 0 : H == 0);
}
bool options_ok(const mhla_options* o, float eps) {
  if (!std::isfinite(eps) || eps < 0.f) return false;
  if (o == nullptr) return true;
  if (o->feature < MHLA_PHI_ELU1 || o->feature > MHLA_PHI_IDENTITY || (o->normalise != 0 && o->normalise != 1) || o->gamma != 1.f)
    return false;
  return o->feature != MHLA_PHI_IDENTITY || o->normalise == 0;  // (a denominator of any sign)
}
int feature_of(const mhla_options* o) { return o ? o->feature : MHLA_PHI_ELU1; }

mhla_status check_side(int B, int N, bool packed, const int* cu, const int* lens) {
  if (cu != nullptr && lens != nullptr) return MHLA_ERR_INVALID_ARG;
  if (!aligned(cu, 4) || !aligned(lens, 4)) return MHLA_ERR_INVALID_ARG;
  const long long tokens = packed ? N : (long long)B * N;
  return tokens > kRetMaxTokens ? MHLA_ERR_UNSUPPORTED : MHLA_OK;
}

struct Sums {  // S and z
  size_t s_bytes, z_bytes;
};
bool check_sums(Sums* b, const float* S, const float* z, long long n_slots, int Hk, int d) {
  const Wide s = (Wide)n_slots * Hk * d * d * 4;
  if (n_slots < 0 || !fits(s)) return false;
  b->s_bytes = (size_t)s;
  b->z_bytes = (size_t)n_slots * Hk * d * 4;
  return S != nullptr && z != nullptr && aligned(S, 16) && aligned(z, 16);
}

}  // namespace
}  // namespace mhla

using namespace mhla;

extern "C" {

size_t linattn_cross_workspace_bytes(int B, int H, int Hk, int tokens_q, int tokens_k, int d, int backward) {
  if (!sizes_ok(B, H, Hk, tokens_q, d) || tokens_k < 0 || tokens_q > kRetMaxTokens || tokens_k > kRetMaxTokens ||
      (backward != 0 && backward != 1))
    return 0;
  if (B == 0 || Hk == 0) return kWorkspacePrefix;
  Wide n = 0;
  static const int some = 0;  // (packed: an address that is not looked at)
  for (int i = 0; i < 4; ++i) {
    const bool packed = i % 2 != 0;
    const Kind kind = kind_of(d, i / 2 != 0);
    CrossSide s;
    if (packed || tokens_k % B == 0) {
      if (!cut_side(&s, B, packed ? tokens_k : tokens_k / B, packed ? &some : nullptr, nullptr, Hk, kind)) continue;
      n = std::max(n, part_floats(s, Hk, d));
    }
    if (backward && (packed || tokens_q % B == 0)) {
      if (!cut_side(&s, B, packed ? tokens_q : tokens_q / B, packed ? &some : nullptr, nullptr, H, kind)) continue;
      n = std::max(n, part_floats(s, H, d) + (Wide)B * Hk * entry(d));
    }
  }
  return fits(n * 4) ? kWorkspacePrefix + (size_t)(n * 4) : 0;
}

mhla_status linattn_cross_states(const void* k, const mhla_strides* k_strides, const void* v, const mhla_strides* v_strides,
                                 float* S, float* z, int B, int Hk, int N, int d, const int* cu_seqlens, const int* lens,
                                 const int* slots, int n_slots, mhla_dtype dt, const mhla_options* opt, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!sizes_ok(B, Hk, Hk, N, d) || (dt != MHLA_F32 && dt != MHLA_BF16) || !options_ok(opt, 0.f)) return MHLA_ERR_INVALID_ARG;
  if (B == 0 || Hk == 0) return MHLA_OK;
  mhla_status st = check_side(B, N, cu_seqlens != nullptr, cu_seqlens, lens);
  if (st != MHLA_OK) return st;
  CrossArgs a{};
  Sums sb;
  if (!check_sums(&sb, S, z, n_slots, Hk, d) || !aligned(slots, 4)) return MHLA_ERR_INVALID_ARG;
  if (!cut_side(&a.ks, B, N, cu_seqlens, lens, Hk, kind_of(d, tc_cross_supported(d, dt))) || (long long)B * Hk * (entry(d) / 128 + 1) > 0x7fffffffll)
    return MHLA_ERR_UNSUPPORTED;
  const size_t part = cross_joined(a.ks) ? (size_t)part_floats(a.ks, Hk, d) * 4 : 0;
  if (!workspace || !aligned(workspace, 256) || !fits(part_floats(a.ks, Hk, d) * 4) || workspace_bytes < kWorkspacePrefix + part)
    return MHLA_ERR_INVALID_ARG;
  const Extent e{cu_seqlens ? 1 : B, Hk, N, d, dt == MHLA_F32 ? 4 : 2};
  const size_t cb = cu_seqlens ? ((size_t)B + 1) * 4 : 0, lb = lens ? (size_t)B * 4 : 0, tb = slots ? (size_t)B * 4 : 0;
  size_t kb = 0, vb = 0;
  if (N > 0) {
    if (!make_tensor(&a.k, k, k_strides, e) || !make_tensor(&a.v, v, v_strides, e)) return MHLA_ERR_INVALID_ARG;
    kb = span_bytes(a.k, e);
    vb = span_bytes(a.v, e);
  }
  const Region r[] = {{k, kb, false}, {v, vb, false}, {cu_seqlens, cb, false}, {lens, lb, false}, {slots, tb, false},
                      {S, sb.s_bytes, true}, {z, sb.z_bytes, true}, {workspace, kWorkspacePrefix + part, true}};
  if (clash(r, 5)) return MHLA_ERR_INVALID_ARG;
  a.k.feature = feature_of(opt);
  a.H = a.Hk = Hk;
  a.d = d;
  a.S = S;
  a.z = z;
  a.slots = slots;
  a.n_slots = n_slots;
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWorkspacePrefix);
  a.status = &static_cast<WorkspaceHeader*>(workspace)->status;
  cudaError_t err = cudaSuccess;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.ks.segs > 0) err = tc_cross_supported(d, dt) ? tc_cross_states_launch(a, s) : simt_cross_states_launch(a, dt, s);
  if (err == cudaSuccess && cross_joined(a.ks)) err = cross_join_launch(a, false, s);
  return from_cuda(err);
}

mhla_status linattn_cross_read(const void* q, const mhla_strides* q_strides, const float* S, const float* z, void* y,
                               const mhla_strides* y_strides, int B, int H, int Hk, int N, int d, const int* cu_seqlens,
                               const int* slots, int n_slots, mhla_dtype dt, const mhla_options* opt, float eps,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(B, H, Hk, N, d) || (dt != MHLA_F32 && dt != MHLA_BF16) || !options_ok(opt, eps)) return MHLA_ERR_INVALID_ARG;
  if (B == 0 || H == 0 || N == 0) return MHLA_OK;
  const mhla_status st = check_side(B, N, cu_seqlens != nullptr, cu_seqlens, nullptr);
  if (st != MHLA_OK) return st;
  CrossArgs a{};
  Sums sb;
  if (!check_sums(&sb, S, z, n_slots, Hk, d) || !aligned(slots, 4)) return MHLA_ERR_INVALID_ARG;
  if (!cut_side(&a.qs, B, N, cu_seqlens, nullptr, H, read_kind(d, tc_cross_supported(d, dt)))) return MHLA_ERR_UNSUPPORTED;
  const bool step = N == 1 && cu_seqlens == nullptr;
  if (!(step && workspace == nullptr) && (!workspace || !aligned(workspace, 256) || workspace_bytes < kWorkspacePrefix)) return MHLA_ERR_INVALID_ARG;
  const Extent e{cu_seqlens ? 1 : B, H, N, d, dt == MHLA_F32 ? 4 : 2};
  if (!make_tensor(&a.q, q, q_strides, e) || !make_tensor(&a.y, y, y_strides, e) || !injective(a.y, e) || !disjoint(a.y, a.q, e))
    return MHLA_ERR_INVALID_ARG;
  const size_t cb = cu_seqlens ? ((size_t)B + 1) * 4 : 0, tb = slots ? (size_t)B * 4 : 0;
  const Region r[] = {{q, span_bytes(a.q, e), false}, {y, span_bytes(a.y, e), true}, {S, sb.s_bytes, false},
                      {z, sb.z_bytes, false}, {cu_seqlens, cb, false}, {slots, tb, false},
                      {workspace, kWorkspacePrefix, true}};
  if (clash(r, 2)) return MHLA_ERR_INVALID_ARG;
  a.q.feature = feature_of(opt);
  a.H = H;
  a.Hk = Hk;
  a.d = d;
  a.S = const_cast<float*>(S);
  a.z = const_cast<float*>(z);
  a.slots = slots;
  a.n_slots = n_slots;
  a.normalise = opt ? opt->normalise : 1;
  a.eps = eps;
  if (step) {
    if ((long long)B * Hk > 0x7fffffffll) return MHLA_ERR_UNSUPPORTED;
    return from_cuda(cross_step_launch(a, dt, static_cast<cudaStream_t>(stream)));
  }
  a.status = &static_cast<WorkspaceHeader*>(workspace)->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(tc_cross_supported(d, dt) ? tc_cross_read_launch(a, s) : simt_cross_read_launch(a, dt, s));
}

mhla_status linattn_cross_backward(const void* q, const mhla_strides* q_strides, const void* k, const mhla_strides* k_strides,
                                   const void* v, const mhla_strides* v_strides, const float* S, const float* z,
                                   const void* dy, const mhla_strides* dy_strides, void* dq, const mhla_strides* dq_strides,
                                   void* dk, const mhla_strides* dk_strides, void* dv, const mhla_strides* dv_strides, int B,
                                   int H, int Hk, int Nq, int Nk, int d, const int* cu_seqlens_q, const int* cu_seqlens_k,
                                   const int* lens, mhla_dtype dt, const mhla_options* opt, float eps, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!sizes_ok(B, H, Hk, Nq, d) || Nk < 0 || (dt != MHLA_F32 && dt != MHLA_BF16) || !options_ok(opt, eps))
    return MHLA_ERR_INVALID_ARG;
  if (H == 0) Nq = 0;  // no query head is no query: dk and dv become zeros
  if (B == 0 || Hk == 0 || (Nq == 0 && Nk == 0)) return MHLA_OK;
  mhla_status st = check_side(B, Nq, cu_seqlens_q != nullptr, cu_seqlens_q, nullptr);
  if (st == MHLA_OK) st = check_side(B, Nk, cu_seqlens_k != nullptr, cu_seqlens_k, lens);
  if (st != MHLA_OK) return st;
  CrossArgs a{};
  Sums sb;
  if (!check_sums(&sb, S, z, B, Hk, d)) return MHLA_ERR_INVALID_ARG;
  const Kind kind = kind_of(d, tc_cross_supported(d, dt));
  if (!cut_side(&a.qs, B, Nq, cu_seqlens_q, nullptr, H, kind) || !cut_side(&a.ks, B, Nk, cu_seqlens_k, lens, Hk, kind) ||
      (long long)B * Hk * (entry(d) / 128 + 1) > 0x7fffffffll)
    return MHLA_ERR_UNSUPPORTED;
  const Wide parts = part_floats(a.qs, H, d), need = (parts + (Wide)B * Hk * entry(d)) * 4;
  if (!workspace || !aligned(workspace, 256) || !fits(need) || workspace_bytes < kWorkspacePrefix + (size_t)need)
    return MHLA_ERR_INVALID_ARG;
  const int es = dt == MHLA_F32 ? 4 : 2;
  const Extent eq{cu_seqlens_q ? 1 : B, H, Nq, d, es}, ek{cu_seqlens_k ? 1 : B, Hk, Nk, d, es};
  size_t nq[3] = {}, nk[4] = {};
  if (Nq > 0) {
    if (!make_tensor(&a.q, q, q_strides, eq) || !make_tensor(&a.dy, dy, dy_strides, eq) || !make_tensor(&a.dq, dq, dq_strides, eq) ||
        !injective(a.dq, eq) || !disjoint(a.dq, a.q, eq) || !disjoint(a.dq, a.dy, eq))
      return MHLA_ERR_INVALID_ARG;
    nq[0] = span_bytes(a.q, eq);
    nq[1] = span_bytes(a.dy, eq);
    nq[2] = span_bytes(a.dq, eq);
  }
  if (Nk > 0) {
    if (!make_tensor(&a.k, k, k_strides, ek) || !make_tensor(&a.v, v, v_strides, ek) || !make_tensor(&a.dk, dk, dk_strides, ek) ||
        !make_tensor(&a.dv, dv, dv_strides, ek) || !injective(a.dk, ek) || !injective(a.dv, ek) || !disjoint(a.dk, a.k, ek) ||
        !disjoint(a.dk, a.v, ek) || !disjoint(a.dv, a.k, ek) || !disjoint(a.dv, a.v, ek) || !disjoint(a.dk, a.dv, ek))
      return MHLA_ERR_INVALID_ARG;
    nk[0] = span_bytes(a.k, ek);
    nk[1] = span_bytes(a.v, ek);
    nk[2] = span_bytes(a.dk, ek);
    nk[3] = span_bytes(a.dv, ek);
  }
  const size_t cq = cu_seqlens_q ? ((size_t)B + 1) * 4 : 0, ck = cu_seqlens_k ? ((size_t)B + 1) * 4 : 0, lb = lens ? (size_t)B * 4 : 0;
  // the two sides' token tensors against each other, and everything else
  const Region side[] = {{q, nq[0], false}, {dy, nq[1], false}, {dq, nq[2], true}, {k, nk[0], false}, {v, nk[1], false},
                         {dk, nk[2], true}, {dv, nk[3], true}};
  for (int i = 3; i < 7; ++i)
    for (int j = 0; j < 3; ++j)
      if ((side[i].written || side[j].written) && !apart(side[i].p, side[i].n, side[j].p, side[j].n)) return MHLA_ERR_INVALID_ARG;
  const Region r[] = {side[0], side[1], side[2], side[3], side[4], side[5], side[6], {S, sb.s_bytes, false},
                      {z, sb.z_bytes, false}, {cu_seqlens_q, cq, false}, {cu_seqlens_k, ck, false}, {lens, lb, false},
                      {workspace, kWorkspacePrefix + (size_t)need, true}};
  if (clash(r, 7)) return MHLA_ERR_INVALID_ARG;
  a.q.feature = a.k.feature = feature_of(opt);
  a.H = H;
  a.Hk = Hk;
  a.d = d;
  a.S = const_cast<float*>(S);
  a.z = const_cast<float*>(z);
  a.n_slots = B;
  a.normalise = opt ? opt->normalise : 1;
  a.eps = eps;
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWorkspacePrefix);
  a.dS = a.part + (size_t)parts;
  a.status = &static_cast<WorkspaceHeader*>(workspace)->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(tc_cross_supported(d, dt) ? tc_cross_backward_launch(a, s) : simt_cross_backward_launch(a, dt, s));
}

}  // extern "C"
