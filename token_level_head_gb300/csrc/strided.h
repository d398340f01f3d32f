// Host side of strided tensors: their checks and overlaps (the argument checks of the entries that take strides).
#pragma once

#include <algorithm>
#include <cstdint>
#include <cstdlib>

#include "retention.h"

namespace mhla {
namespace {

inline bool valid_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline mhla_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA; }

// ---- token tensors
struct Extent {  // of a tensor: B x H x N rows of d elements
  long long b, h, n, d;
  int es;
};

// Bytes of no GPU's memory, virtual addresses included: what spans more is no tensor, and its sizes are not
// multiplied in 64 bits.
constexpr long long kNoMemory = 1ll << 48;
using Wide = __int128;

inline Wide wide_span(const RetTensor& t, const Extent& e) {
  return (Wide)(e.b - 1) * t.sb + (Wide)(e.h - 1) * t.sh + (Wide)(e.n - 1) * t.sn + e.d;
}
inline long long span(const RetTensor& t, const Extent& e) { return (long long)wide_span(t, e); }

// Fills t; false if the pointer, the alignment, the strides or the size are not valid.
inline bool make_tensor(RetTensor* t, const void* p, const mhla_strides* st, const Extent& e) {
  if (p == nullptr || !aligned(p, 16)) return false;
  t->p = p;
  if (st == nullptr && (Wide)e.b * e.h * e.n * e.d * e.es > kNoMemory) return false;
  t->sb = st ? st->b : e.h * e.n * e.d;
  t->sh = st ? st->h : e.n * e.d;
  t->sn = st ? st->n : e.d;
  if (e.b <= 1) t->sb = 0;  // the stride of a single entry is not looked at
  if (e.h <= 1) t->sh = 0;
  if (e.n <= 1) t->sn = 0;
  const long long q = 16 / e.es, most = 1ll << 38;  // 2^40 bytes
  for (long long s : {t->sb, t->sh, t->sn})
    if (s < 0 || s % q != 0 || s >= most) return false;
  if (t->sn == 0 && e.n > 1) return false;  // rows of their own, so that a tile can be loaded by TMA
  if (wide_span(*t, e) * e.es > kNoMemory) return false;
  t->feature = MHLA_PHI_IDENTITY;
  return true;
}

// Bytes of a pool of states; false if no memory holds it.
inline bool pool_bytes(size_t* bytes, long long n_slots, int H, int d) {
  const Wide n = (Wide)n_slots * H * d * d * sizeof(float);
  *bytes = (size_t)n;
  return n <= kNoMemory;
}

struct Dim {
  long long stride, extent;
};
inline void sorted_dims(const RetTensor& t, const Extent& e, Dim* d) {
  d[0] = {t.sb, e.b};
  d[1] = {t.sh, e.h};
  d[2] = {t.sn, e.n};
  std::sort(d, d + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
}

// No two rows of the tensor overlap (sufficient: each stride spans what is inside it).
inline bool injective(const RetTensor& t, const Extent& e) {
  Dim d[3];
  sorted_dims(t, e, d);
  long long inner = e.d;
  for (const Dim& x : d) {
    if (x.extent <= 1) continue;
    if (x.stride < inner) return false;
    inner = (x.extent - 1) * x.stride + inner;
  }
  return true;
}

// Is there a combination of index differences with |delta + sum| < width?  dims[0 .. n): strides
// ascending, each spanning what is inside it, so only the two multiples around delta can be near.
inline bool meet(long long delta, const Dim* dims, int n, long long width) {
  while (n > 0 && dims[n - 1].extent <= 1) --n;
  if (n == 0) return std::llabs(delta) < width;
  const Dim& x = dims[n - 1];
  const long long q = delta / x.stride;
  for (long long c = q - 1; c <= q + 1; ++c)
    if (std::llabs(c) < x.extent && meet(delta - c * x.stride, dims, n - 1, width)) return true;
  return false;
}

// An output against another tensor: apart in memory, or interleaved with the same strides (slices of one
// fused tensor) without a common element.
inline bool disjoint(const RetTensor& o, const RetTensor& t, const Extent& e) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(o.p), b = reinterpret_cast<uintptr_t>(t.p);
  if (a >= b + span(t, e) * e.es || b >= a + span(o, e) * e.es) return true;
  if (o.sb != t.sb || o.sh != t.sh || o.sn != t.sn || !injective(o, e)) return false;
  const long long diff = (long long)(b - a);
  if (diff % e.es != 0) return false;
  Dim d[3];
  sorted_dims(o, e, d);
  return !meet(diff / e.es, d, 3, e.d);
}

inline bool apart(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an == 0 || bn == 0 || a == nullptr || b == nullptr || x >= y + bn || y >= x + an;
}

struct Region {
  const void* p;
  size_t n;
  bool written;
};
// Does one of the regions from `first` on overlap one before it, one of the two written?  (The token tensors, before
// `first`, may be interleaved slices of one tensor: disjoint() answers for them.)
template <int n>
bool clash(const Region (&r)[n], int first) {
  for (int i = first; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if ((r[i].written || r[j].written) && !apart(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
  return false;
}

inline size_t span_bytes(const RetTensor& t, const Extent& e) { return (size_t)span(t, e) * e.es; }

}  // namespace
}  // namespace mhla
