// C-ABI entry points of the retention operators: argument validation, the plan of the segments and
// dispatch.  The operations are documented in include/mhla.h.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "retention.h"
#include "strided.h"

namespace mhla {
namespace {

constexpr int kMaxPairs = 1024;

bool options_ok(const retention_options* opt) {
  return opt == nullptr ||
         (opt->feature >= MHLA_PHI_ELU1 && opt->feature <= MHLA_PHI_IDENTITY && std::isfinite(opt->scale));
}

// ---- segments
struct Plan {
  int L;         // tokens of a segment
  long long G;   // segments
  long long inner, splits, W;  // segments that enter another one, sequences of two or more, segments of those
  size_t bytes;  // workspace
  bool split;    // some sequence may have two segments
  bool fits;     // the grids' blocks can be numbered
};

// The length of a segment: the n chunks of 128 tokens (fp32: halves count) for which a call is estimated to take least, in
// units of a chunk's time in a pass:
//   pass   (rounds of blocks) (n + start)
//   split  (rounds) (n + start) sum  +  a state for each segment, written and read by the sums' kernel, the scan and
//          the pass  +  two more launches
// where a round is `slots` blocks.  Packed sequences, of unknown lengths, take their work over the slots and half a
// block for the tail; four times the mean counts as their longest.  The costs are measured ones.  bf16: a chunk takes
// 3.1 us (d = 64: in each of two blocks an SM), a block 2.5 chunks to start, the sum of a chunk 0.45 of its pass, a
// segment's state 2 chunks, two launches 8 us; a block that returns a state (exact) takes half as long again for about
// 8 chunks: its segment, the last one, is better short.  fp32: a chunk takes 26 us (two blocks an SM, but d = 128; a
// third one waits, one by itself takes 0.86 of that), a block 0.3 chunks to start, a sum 0.35.
// What it picks is within 5 % of the best of a sweep of segment lengths (us of whole calls, the pick first): 8 heads of
// 65,536 tokens 3584: 152, 3456: 168, 4096: 182, 2048: 207; 64 heads of 8192 2176: 101, 2304: 101, 2048: 106, 1024: 116, 4096:
// 148; 24 packed sequences of 20,011 tokens 4096: 133, 2048: 152, 1024: 172; gradients of 64 heads of 4096 tokens 4096: 104,
// 1408: 110, 1024: 127, 2048: 131; of 12 packed sequences of 16,384 tokens 5376: 162, 4096: 164, 2048: 204; fp32: 12 heads of
// 4096 tokens 192: 80, 64: 86, 128: 88, 256: 96; 24 heads of 6000 320: 180, 512: 173, 192: 182, 64: 209; gradients of 8 heads of
// 500 tokens 64: 31, 128: 49.
// One length serves all packed sequences, of which the host knows the mean alone.  Where no cut is picked, sequences of up
// to kUncut tokens or four times the mean are left whole and longer ones are cut at that length.  kUncut is a middle; with
// 1024 / 4096 / 8192 in its place, 16 heads, d = 128: 60 sequences of 40,000 tokens, the longest 4000, 266 / 227 / 224 us,
// the longest 16,000, 266 / 267 / 301; 24 of 20,011, the longest 6000, 159 / 155 / 183, 12,000, 148 / 170 / 303.  With few
// heads short pieces would be better, and long ones with gradients: 4 heads, d = 64, 60 sequences of 20,011, the longest 12,000,
// 57 / 130 / 218; gradients with 16 heads, d = 128, of 60 sequences of 40,000, the longest 8000, 508 / 503 / 450.
constexpr int kUncut = 4096;
Plan make_plan(int B, int H, long long tokens, int d, mhla_dtype dt, bool packed, bool backward, bool exact) {
  const bool f32 = dt == MHLA_F32;
  const int N = packed ? (int)tokens : (int)(tokens / B), npass = backward ? 3 : 1, nsum = backward ? 2 : 1;
  const int unit = f32 ? 64 : 128;  // tokens that a length is counted in below
  const double slots = d == 128 ? kRetSms : 2.0 * kRetSms, chunk = unit / 128.0;
  const double fixed = 8.0 / (f32 ? 26.0 : 3.1);
  const double start = f32 ? 0.3 : 2.5, sum = f32 ? 0.35 : 0.45, state = f32 ? 0.2 : 2.0;
  const double slow = exact && !f32 ? 0.5 : 0.0;
  const int cols = f32 && d == 128 ? 2 : 1;  // blocks that share a segment
  const auto rounds = [&](double blocks) {
    if (!f32 || d == 128) return std::ceil(blocks / slots);
    return blocks <= slots / 2 ? 0.86 : std::ceil(2 * blocks / slots) / 2;
  };
  const long long all = (tokens + unit - 1) / unit, most = ((long long)N + unit - 1) / unit;
  const double longest = packed ? std::min<double>((double)most, 4.0 * all / B) : (double)most;
  double best = 1e300;
  long long pick = most;
  for (long long n = 1; n <= most; n = n < 64 ? n + 1 : n < most ? std::min(n + n / 16, most) : n + 1) {
    double cost;
    if (packed) {
      const double more = n < longest ? (double)all / n : 0.0;  // segments beyond one a sequence
      const double work = (all * chunk + 0.5 * B) * H * cols, blocks = ((double)B + more) * H * cols;
      cost = (work + blocks * start) * npass / slots + 0.5 * (std::min<double>(n, longest) * chunk + start);
      if (n < most) cost += fixed + (more > 0 ? (work + blocks * start) * nsum * sum / slots + more * H * nsum * state / slots : 0);
    } else {
      const long long segs = (most + n - 1) / n;
      const double blocks = (double)B * H * segs * cols, rest = (most - (segs - 1) * n) * chunk, end = rest + slow * std::min(rest, 8.0);
      cost = rounds(blocks * npass) * (std::max(std::min(n, most) * chunk, end) + start);
      if (segs > 1)
        cost += rounds((double)B * H * (segs - 1) * cols * nsum) * (n * chunk + start) * sum + fixed +
                (double)B * H * segs * nsum * state / slots;
    }
    if (cost < best) {
      best = cost;
      pick = n;
    }
  }
  if (packed && pick >= longest) pick = std::max<long long>(kUncut / unit, (long long)longest);
  Plan p;
  p.L = (int)std::max<long long>(std::min<long long>(pick, 1 << 23) * unit, unit);
  p.G = packed ? tokens / p.L + B : (long long)B * ret_pieces(N, p.L);
  p.split = N > p.L;
  p.inner = packed ? tokens / p.L : p.G - B;  // (an inner segment is a full one)
  p.splits = packed ? std::min<long long>(B, p.inner) : B;
  p.W = packed ? std::min(p.G, 2 * p.inner) : p.G;  // (nseg <= 2 (nseg - 1))
  p.fits = p.G * H <= 0x7fffffffll / 3 && (long long)B * H <= 0x7fffffffll / 3;
  p.bytes = kWorkspacePrefix + (p.split && p.fits ? (size_t)nsum * p.W * H * d * d * sizeof(float) : 0);
  return p;
}

bool sizes_ok(int B, int H, int N, int d) { return B >= 0 && H >= 0 && N >= 0 && valid_d(d); }

// What retention_forward and retention_backward have in common; *empty: nothing to do.
mhla_status begin(RetArgs* a, Plan* plan, Extent* e, const float* gamma, int B, int H, int N, int d, const int* cu,
                  mhla_dtype dt, const retention_options* opt, bool backward, bool exact, void* ws, size_t ws_bytes,
                  bool* empty) {
  *empty = false;
  if (!sizes_ok(B, H, N, d) || (dt != MHLA_F32 && dt != MHLA_BF16) || !options_ok(opt)) return MHLA_ERR_INVALID_ARG;
  if (B == 0 || H == 0 || N == 0) {
    *empty = true;
    return MHLA_OK;
  }
  const long long tokens = cu ? N : (long long)B * N;
  if (tokens > kRetMaxTokens) return MHLA_ERR_UNSUPPORTED;
  if (!gamma || !aligned(gamma, 4) || !aligned(cu, 4)) return MHLA_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return MHLA_ERR_INVALID_ARG;
  *plan = make_plan(B, H, tokens, d, dt, cu != nullptr, backward, exact);
  if (!plan->fits) return MHLA_ERR_UNSUPPORTED;
  if (ws_bytes < plan->bytes) return MHLA_ERR_INVALID_ARG;
  *e = {cu ? 1 : B, H, N, d, dt == MHLA_F32 ? 4 : 2};
  *a = RetArgs{};
  a->B = B;
  a->H = H;
  a->N = N;
  a->T = (int)tokens;
  a->d = d;
  a->cu = cu;
  a->gamma = gamma;
  a->scale = opt ? opt->scale : 1.f;
  a->L = plan->L;
  a->G = (int)plan->G;
  a->inner = (int)plan->inner;
  a->split = (int)plan->splits;
  a->W = (int)plan->W;
  a->seg = plan->split ? reinterpret_cast<float*>(static_cast<char*>(ws) + kWorkspacePrefix) : nullptr;
  a->status = &static_cast<WorkspaceHeader*>(ws)->status;
  return MHLA_OK;
}

RetTensor mapped(RetTensor t, int feature) {
  t.feature = feature;
  return t;
}

}  // namespace
}  // namespace mhla

using namespace mhla;

extern "C" {

size_t retention_workspace_bytes(int B, int H, int tokens, int d, int backward) {
  if (!sizes_ok(B, H, tokens, d) || tokens > kRetMaxTokens || (backward != 0 && backward != 1)) return 0;
  if (B == 0 || H == 0 || tokens == 0) return kWorkspacePrefix;
  size_t n = 0;
  for (mhla_dtype dt : {MHLA_F32, MHLA_BF16})
    for (bool exact : {false, true}) {
      if (exact && backward) continue;
      for (bool packed : {true, false}) {
        if (!packed && tokens % B != 0) continue;
        const Plan p = make_plan(B, H, tokens, d, dt, packed, backward != 0, exact);
        if (p.fits) n = std::max(n, p.bytes);
      }
    }
  return n;
}

mhla_status retention_forward(const void* q, const mhla_strides* q_strides, const void* k,
                              const mhla_strides* k_strides, const void* v, const mhla_strides* v_strides,
                              const float* gamma, void* y, const mhla_strides* y_strides, int B, int H, int N, int d,
                              const int* cu_seqlens, float* states, const int* slots, int n_slots, int load_state,
                              mhla_dtype dt, const retention_options* opt, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (load_state != 0 && load_state != 1) return MHLA_ERR_INVALID_ARG;
  if (states == nullptr ? (slots != nullptr || load_state != 0) : n_slots < 0) return MHLA_ERR_INVALID_ARG;
  RetArgs a;
  Plan plan;
  Extent e;
  bool empty;
  const mhla_status st = begin(&a, &plan, &e, gamma, B, H, N, d, cu_seqlens, dt, opt, false, states != nullptr,
                               workspace, workspace_bytes, &empty);
  if (st != MHLA_OK || empty) return st;
  RetTensor tq, tk, tv, ty;
  if (!make_tensor(&tq, q, q_strides, e) || !make_tensor(&tk, k, k_strides, e) || !make_tensor(&tv, v, v_strides, e) ||
      !make_tensor(&ty, y, y_strides, e) || !injective(ty, e))
    return MHLA_ERR_INVALID_ARG;
  size_t sb;
  if (!pool_bytes(&sb, states ? n_slots : 0, H, d) || !aligned(states, 16) || !aligned(slots, 4))
    return MHLA_ERR_INVALID_ARG;
  for (const RetTensor* t : {&tq, &tk, &tv, &ty}) {
    const size_t n = (size_t)span(*t, e) * e.es;
    if (t != &ty && !disjoint(ty, *t, e)) return MHLA_ERR_INVALID_ARG;
    if (!apart(t->p, n, states, sb) || !apart(t->p, n, workspace, plan.bytes)) return MHLA_ERR_INVALID_ARG;
  }
  const size_t yb = (size_t)span(ty, e) * e.es, gb = (size_t)H * 4, cb = (size_t)(B + 1) * 4, lb = (size_t)B * 4;
  if (!apart(states, sb, workspace, plan.bytes) || !apart(gamma, gb, y, yb) || !apart(gamma, gb, states, sb) ||
      !apart(gamma, gb, workspace, plan.bytes) || !apart(cu_seqlens, cb, y, yb) || !apart(cu_seqlens, cb, states, sb) ||
      !apart(cu_seqlens, cb, workspace, plan.bytes) || !apart(slots, lb, y, yb) || !apart(slots, lb, states, sb) ||
      !apart(slots, lb, workspace, plan.bytes))
    return MHLA_ERR_INVALID_ARG;
  const int f = opt ? opt->feature : MHLA_PHI_IDENTITY;
  a.npass = a.nsum = 1;
  a.pass[0].a = mapped(tq, f);
  a.pass[0].b = mapped(tk, f);
  a.pass[0].c = tv;
  a.pass[0].out = ty;
  a.states = states;
  a.slots = slots;
  a.n_slots = n_slots;
  a.load = load_state;
  return from_cuda(dt == MHLA_BF16 ? tc_retention_launch(a, static_cast<cudaStream_t>(stream))
                                   : simt_retention_launch(a, static_cast<cudaStream_t>(stream)));
}

mhla_status retention_backward(const void* q, const mhla_strides* q_strides, const void* k,
                               const mhla_strides* k_strides, const void* v, const mhla_strides* v_strides,
                               const float* gamma, const void* dy, const mhla_strides* dy_strides, void* dq,
                               const mhla_strides* dq_strides, void* dk, const mhla_strides* dk_strides, void* dv,
                               const mhla_strides* dv_strides, int B, int H, int N, int d, const int* cu_seqlens,
                               mhla_dtype dt, const retention_options* opt, void* workspace, size_t workspace_bytes,
                               void* stream) {
  RetArgs a;
  Plan plan;
  Extent e;
  bool empty;
  const mhla_status st = begin(&a, &plan, &e, gamma, B, H, N, d, cu_seqlens, dt, opt, true, false, workspace,
                               workspace_bytes, &empty);
  if (st != MHLA_OK || empty) return st;
  RetTensor in[4], out[3];
  const void* ip[4] = {q, k, v, dy};
  void* op[3] = {dq, dk, dv};
  const mhla_strides* is[4] = {q_strides, k_strides, v_strides, dy_strides};
  const mhla_strides* os[3] = {dq_strides, dk_strides, dv_strides};
  const size_t gb = (size_t)H * 4, cb = (size_t)(B + 1) * 4;
  for (int i = 0; i < 4; ++i) {
    if (!make_tensor(&in[i], ip[i], is[i], e)) return MHLA_ERR_INVALID_ARG;
    if (!apart(ip[i], (size_t)span(in[i], e) * e.es, workspace, plan.bytes)) return MHLA_ERR_INVALID_ARG;
  }
  if (!apart(gamma, gb, workspace, plan.bytes) || !apart(cu_seqlens, cb, workspace, plan.bytes))
    return MHLA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (!make_tensor(&out[i], op[i], os[i], e) || !injective(out[i], e)) return MHLA_ERR_INVALID_ARG;
    const size_t n = (size_t)span(out[i], e) * e.es;
    for (int j = 0; j < 4; ++j)
      if (!disjoint(out[i], in[j], e)) return MHLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (!disjoint(out[i], out[j], e)) return MHLA_ERR_INVALID_ARG;
    if (!apart(op[i], n, workspace, plan.bytes) || !apart(op[i], n, gamma, gb) || !apart(op[i], n, cu_seqlens, cb))
      return MHLA_ERR_INVALID_ARG;
  }
  const int f = opt ? opt->feature : MHLA_PHI_IDENTITY;
  const RetTensor fq = mapped(in[0], f), fk = mapped(in[1], f);
  const bool deriv = f != MHLA_PHI_IDENTITY;
  a.npass = 3;
  a.nsum = 2;
  RetPass& pq = a.pass[0];
  pq.a = in[3];
  pq.b = in[2];
  pq.c = fk;
  if (deriv) pq.x = fq;
  pq.out = out[0];
  RetPass& pk = a.pass[1];
  pk.a = in[2];
  pk.b = in[3];
  pk.c = fq;
  if (deriv) pk.x = fk;
  pk.out = out[1];
  pk.reverse = 1;
  pk.sum = 1;
  RetPass& pv = a.pass[2];  // its state, sum phi(q) dy^T, is the transpose of the one above
  pv.a = fk;
  pv.b = fq;
  pv.c = in[3];
  pv.out = out[2];
  pv.reverse = 1;
  pv.sum = 1;
  pv.sum_t = 1;
  return from_cuda(dt == MHLA_BF16 ? tc_retention_launch(a, static_cast<cudaStream_t>(stream))
                                   : simt_retention_launch(a, static_cast<cudaStream_t>(stream)));
}

mhla_status retention_step(const void* q, const mhla_strides* q_strides, const void* k, const mhla_strides* k_strides,
                           const void* v, const mhla_strides* v_strides, const float* gamma, float* states,
                           const int* slots, int n_slots, void* out, const mhla_strides* out_strides, int B, int H,
                           int d, mhla_dtype dt, const retention_options* opt, void* stream) {
  if (!sizes_ok(B, H, 1, d) || (dt != MHLA_F32 && dt != MHLA_BF16) || !options_ok(opt) || n_slots < 0)
    return MHLA_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return MHLA_OK;
  if ((long long)B * H > 0x7fffffffll) return MHLA_ERR_UNSUPPORTED;
  if (!gamma || !states || !aligned(gamma, 4) || !aligned(states, 16) || !aligned(slots, 4))
    return MHLA_ERR_INVALID_ARG;
  const Extent e{B, H, 1, d, dt == MHLA_F32 ? 4 : 2};
  RetTensor tq, tk, tv, to;
  if (!make_tensor(&tq, q, q_strides, e) || !make_tensor(&tk, k, k_strides, e) || !make_tensor(&tv, v, v_strides, e) ||
      !make_tensor(&to, out, out_strides, e) || !injective(to, e))
    return MHLA_ERR_INVALID_ARG;
  const size_t ob = (size_t)span(to, e) * e.es;
  size_t sb;
  if (!pool_bytes(&sb, n_slots, H, d)) return MHLA_ERR_INVALID_ARG;
  for (const RetTensor* t : {&tq, &tk, &tv, &to}) {
    if (t != &to && !disjoint(to, *t, e)) return MHLA_ERR_INVALID_ARG;
    if (!apart(t->p, (size_t)span(*t, e) * e.es, states, sb)) return MHLA_ERR_INVALID_ARG;
  }
  if (!apart(gamma, (size_t)H * 4, states, sb) || !apart(slots, (size_t)B * 4, states, sb) ||
      !apart(gamma, (size_t)H * 4, out, ob) || !apart(slots, (size_t)B * 4, out, ob))
    return MHLA_ERR_INVALID_ARG;
  const int f = opt ? opt->feature : MHLA_PHI_IDENTITY;
  return from_cuda(retention_step_launch(B, H, d, dt, mapped(tq, f), mapped(tk, f), tv, to, gamma,
                                         opt ? opt->scale : 1.f, states, slots, n_slots,
                                         static_cast<cudaStream_t>(stream)));
}

mhla_status retention_copy_states(float* states, int n_slots, int H, int d, const int* src, const int* dst, int n,
                                  void* stream) {
  if (!sizes_ok(n_slots, H, 0, d) || n < 0) return MHLA_ERR_INVALID_ARG;
  if (n_slots == 0 || H == 0 || n == 0) return MHLA_OK;
  if (n > kMaxPairs) return MHLA_ERR_UNSUPPORTED;
  if (!states || !src || !dst || !aligned(states, 16) || !aligned(src, 4) || !aligned(dst, 4))
    return MHLA_ERR_INVALID_ARG;
  const long long slot = (long long)H * d * d;
  if (slot / 32 > 0x7fffffffll) return MHLA_ERR_UNSUPPORTED;
  size_t sb;
  if (!pool_bytes(&sb, n_slots, H, d) || !apart(states, sb, src, (size_t)n * 4) || !apart(states, sb, dst, (size_t)n * 4))
    return MHLA_ERR_INVALID_ARG;
  return from_cuda(retention_copy_launch(states, slot, n_slots, src, dst, n, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
