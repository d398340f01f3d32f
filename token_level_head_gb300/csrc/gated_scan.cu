// The gated scan: h_t = a_t h_{t-1} + b_t with a gate a_t of its own for every token and channel, its gradients and
// its single-token step ("Linear Attention notes" §七, the gated update S_t = G_t . S_{t-1} + ..., for a vector state).
//
// Two runs of tokens with (A, B) and (A', B'), h -> A h + B, one behind the other are (A A', A' B + B'), so a tile of
// tokens is folded by every thread over its own few rows, over the row groups of a warp by shuffles, over the warps
// through shared memory; then every thread knows the state before its rows and runs them once more.  The gradient
// runs the same way from the end: c_t = a_t (dy_t + c_{t+1}), G_t = dy_t + c_{t+1}.
//
// Bound: memory (forward 3 tensors, backward 5), next to it the instructions of the gates and of two passes over a tile (an
// SM that two blocks fill issues in half of its cycles; the rest are the waits of a tile for the one before).  A block takes a
// tile of rows and LW lanes of channels; tiles behind one another are taken by the blocks of a cluster, which exchange their
// (A, B) through distributed shared memory, and a cluster walks along the sequence.  So x and g are read once and no memory,
// flag or wait is shared between clusters.
// Measured, whole calls: 65,536 x 1024 bf16, log, 79 us (5.1 TB/s); 77 x 1024 bf16 8; forward and backward of 4 x 8192 x 1024
// bf16, sigmoid, 126 (4.3 TB/s), of 20,011 packed x 384 fp32, decay, 74 (3.3 TB/s); the step of 256 x 8192 bf16 8.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "gated_scan.h"
#include "retention.cuh"

namespace mhla {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;  // of the tiles,
constexpr int kBlock = kThreads + 32;                  // and a warp that carries the state over the tiles (exchange)
constexpr int kMostBlocks = 16;                        // of a cluster
constexpr int P = 1, V = 2 * P;  // channels of a thread: a pair, so that a warp of bf16 has a row of 128 bytes to itself

// A thread's rows of a tile and the lanes of 128 bytes of channels.  Half of the values for fp32, whose tiles are as many bytes.
template <typename T>
struct Tile;
template <>
struct Tile<__nv_bfloat16> {
  static constexpr int R = 16, WIDE = 32;
};
template <>
struct Tile<float> {
  static constexpr int R = 8, WIDE = 16;
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// N pairs of channels as they lie in memory.
template <typename T, int N>
struct Io;
template <>
struct Io<float, 1> {
  using Raw = uint2;
};
template <>
struct Io<float, 2> {
  using Raw = uint4;
};
template <>
struct Io<__nv_bfloat16, 1> {
  using Raw = unsigned;
};
template <>
struct Io<__nv_bfloat16, 2> {
  using Raw = uint2;
};
__device__ __forceinline__ float2 bf16_pair(unsigned u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void unpack(unsigned u, float2 (&f)[1]) {
  f[0] = bf16_pair(u);
}
template <typename T>
__device__ __forceinline__ void unpack(const uint2& u, float2 (&f)[1]) {
  f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
}
template <typename T>
__device__ __forceinline__ void unpack(const uint2& u, float2 (&f)[2]) {
  f[0] = bf16_pair(u.x);
  f[1] = bf16_pair(u.y);
}
template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void store(float* p, const float2 (&f)[1]) { *reinterpret_cast<float2*>(p) = f[0]; }
__device__ __forceinline__ void store(float* p, const float2 (&f)[2]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&f)[1]) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0].x, f[0].y);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&f)[2]) {
  __nv_bfloat162 r[2] = {__floats2bfloat162_rn(f[0].x, f[0].y), __floats2bfloat162_rn(f[1].x, f[1].y)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(r);
}
__device__ __forceinline__ void load_f(const float* p, float2 (&f)[1]) { f[0] = *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void load_f(const float* p, float2 (&f)[2]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = make_float2(v.x, v.y);
  f[1] = make_float2(v.z, v.w);
}
template <int N>
__device__ __forceinline__ void fill(float2 (&f)[N], float v) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = both(v);
}

__device__ __forceinline__ float exp2_of(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
// exp(x).  bf16 tensors: the hardware's base-2 exponential of x log2 e (log2 e = 1.4426950408889634), off by
// 2^-22 and |x| 1.25 2^-24 at most (the product's and the constant's rounding); fp32: expf.  Measured over all bf16 log gates:
// 2^-22.9 of a gate at most up to |g| = 2, and 1.25 steps of 2^-24 (7.5e-8) for |g| < 2^-9, whose memories multiply it; a bf16
// gate's own half step is more from |g| = 2^-15 on, and nearer to 1 no 32-bit gate says more than a step.  (The series
// 1 + g + .. + g^5 / 120 for |g| < 1/16 halves the latter, with 65,536 x 1024 106 us instead of 79.)  Not-a-number stays.
template <typename T>
__device__ __forceinline__ float2 exp_of(float2 x) {
  if (sizeof(T) == 4) return make_float2(expf(x.x), expf(x.y));
  const float2 t = mul2(x, both(1.4426950408889634f));
  return make_float2(exp2_of(t.x), exp2_of(t.y));
}
__device__ __forceinline__ float rcp_of(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// a = e rest where e < 2: a comparison and a product under it (both forms and a selection: 129 us instead of 126 for the forward
// and backward of 4 x 8192 x 1024).
__device__ __forceinline__ void small_gate(float& a, float e, float rest) {
  asm("{\n\t.reg .pred p;\n\tsetp.lt.f32 p, %1, 0f40000000;\n\t@p mul.f32 %0, %1, %2;\n\t}" : "+f"(a) : "f"(e), "f"(rest));
}

struct Gate {
  float2 a;     // the gate
  float2 rest;  // sigmoid: 1 - a, the factor of x
};
// sigmoid, with e = exp(g): 1 - a = 1 / (1 + e), which needs no case for either end.  a = e / (1 + e) below 2/3, so that a small
// gate has all its digits (what fades is off by 2^-21 of itself, bf16 and by |g| 2^-23; a = 1 - (1 - a) throughout was off by
// 5e-4 at g = -10 and zero from -17 on); from there 1 - (1 - a), so that gates near 1 are rounded once (a long memory
// multiplies thousands of them, and their errors).  Not-a-number stays.
template <typename T, int GATE>
__device__ __forceinline__ Gate gate_of(float2 g) {
  Gate k;
  if (GATE == GATED_SCAN_DECAY) {
    k.a = add2(g, both(0.f));  // (-0, which stands for a cut, see kCut, becomes 0)
  } else if (GATE == GATED_SCAN_LOG) {
    k.a = exp_of<T>(g);
  } else {
    const float2 e = exp_of<T>(g), d = add2(e, both(1.f));
    k.rest = make_float2(rcp_of(d.x), rcp_of(d.y));
    k.a = fma2(k.rest, both(-1.f), both(1.f));
    small_gate(k.a.x, e.x, k.rest.x);
    small_gate(k.a.y, e.y, k.rest.y);
  }
  return k;
}
template <int GATE>
__device__ __forceinline__ float2 input_of(float2 x, float2 rest) {
  return GATE == GATED_SCAN_SIGMOID ? mul2(rest, x) : x;
}

// ---- rows of a tile: which are tokens, and where sequences begin and end
struct Marks {
  unsigned live, first, last;  // bit r: row r of the thread
};
__device__ __forceinline__ void tile_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }  // the kThreads of the tiles
__device__ __forceinline__ bool tile_sync_or(bool any) {  // and whether one of them has `any`
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((unsigned)any)
      : "memory");
  return r != 0;
}
static_assert(kThreads == 256, "the barrier's count");

// Packed sequences: bits of the tile's rows row0 .., a word for the kR rows of a thread, and the sequences of the rows that
// have one (a row that begins one and ends one is the same's; find_slots makes slots of them).  Sets by the tile, as a later tile's are made while the state
// that enters this one is on its way.  Offsets outside [0, N] are clamped; out of order they mark rows of the tile all the
// same and nothing else.
template <int GROUPS, int ROWS>
struct MarkRows {
  unsigned first[GROUPS], last[GROUPS];
  int seq[ROWS];
};
template <>
struct MarkRows<0, 0> {};  // dense
// (the tiles' threads, between two of their barriers each: cleared, then set)
template <int GROUPS, int ROWS>
__device__ __forceinline__ void clear_marks(MarkRows<GROUPS, ROWS>& m) {
  for (int i = threadIdx.x; i < GROUPS; i += kThreads) m.first[i] = m.last[i] = 0;
  for (int i = threadIdx.x; i < ROWS; i += kThreads) m.seq[i] = 0;
}
// (Whether the thread has set one.)
template <int GROUPS, int ROWS>
__device__ __forceinline__ bool set_marks(const ScanArgs& p, int row0, MarkRows<GROUPS, ROWS>& m) {
  constexpr int kR = ROWS / GROUPS;
  bool any = false;
  for (int i = threadIdx.x; i < p.B; i += kThreads) {
    const int lo = min(max(p.cu[i], 0), p.N), hi = min(max(p.cu[i + 1], lo), p.N);
    if (lo == hi) continue;
    const int f = lo - row0, l = hi - 1 - row0;
    if (f >= 0 && f < ROWS) {
      atomicOr(&m.first[f / kR], 1u << f % kR);
      atomicMax(&m.seq[f], i);
      any = true;
    }
    if (l >= 0 && l < ROWS) {
      atomicOr(&m.last[l / kR], 1u << l % kR);
      atomicMax(&m.seq[l], i);
      any = true;
    }
  }
  return any;
}

// The slots of packed sequences, -1 for none: out of range, or the slot of a sequence before.  The slots of the sequences that
// begin or end in the tile go into a table (open addressing, half full at most); one pass over the slots up to the tile's last
// sequence, shared by the tiles' threads as set_marks's pass over the offsets is, then finds the first sequence with each.
// (With every thread looking through the slots before its own sequences': 65,536 x 256 bf16 as 4096 sequences 4239 us, so 175,
// without slots 143; a dense batch of 1024 x 64 rows, where a block looks once, 793, so 68.)
template <int ROWS>
struct SlotTable {
  int key[2 * ROWS], first[2 * ROWS];  // a slot (-1: free), the first sequence with it
  int end;                             // behind the last sequence of the tile
};
template <>
struct SlotTable<0> {};  // dense
// m.seq becomes the slots.  (The tiles' threads, behind set_marks, with a barrier of theirs since the call before; `any`: what
// set_marks gave.)
template <int GROUPS, int ROWS>
__device__ __noinline__ void find_slots(const int* slots, int n_slots, bool any, MarkRows<GROUPS, ROWS>& m,
                                        SlotTable<ROWS>& t) {
  constexpr int kR = ROWS / GROUPS, SIZE = 2 * ROWS;
  static_assert(ROWS <= kThreads && (SIZE & (SIZE - 1)) == 0, "a thread a row, a table of a power of two");
  const auto place = [](int s) { return (int)((unsigned)s * 2654435769u >> 16) % SIZE; };  // (2^32 over the golden ratio)
  for (int i = threadIdx.x; i < SIZE; i += kThreads) {
    t.key[i] = -1;
    t.first[i] = 0x7fffffff;
  }
  if (threadIdx.x == 0) t.end = 0;
  if (!tile_sync_or(any)) return;
  const int r = threadIdx.x;
  int seq = -1, slot = -1, at = 0;
  if (r < ROWS && ((m.first[r / kR] | m.last[r / kR]) >> r % kR & 1u)) {
    seq = m.seq[r];
    slot = slots[seq];
    atomicMax(&t.end, seq + 1);
    if (slot >= n_slots || slot < 0) slot = -1;
    if (slot >= 0)
      for (at = place(slot);; at = (at + 1) % SIZE) {
        const int was = atomicCAS(&t.key[at], -1, slot);
        if (was == -1 || was == slot) break;
      }
  }
  tile_sync();
  constexpr int U = 4;  // loads in flight
  const int end = t.end;
  for (int i0 = threadIdx.x; i0 < end; i0 += U * kThreads) {
    int s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = i0 + u * kThreads < end ? slots[i0 + u * kThreads] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s[u] < 0) continue;
      for (int a = place(s[u]); t.key[a] != -1; a = (a + 1) % SIZE)
        if (t.key[a] == s[u]) {
          atomicMin(&t.first[a], i0 + u * kThreads);
          break;
        }
    }
  }
  tile_sync();
  if (seq >= 0) m.seq[r] = slot >= 0 && t.first[at] == seq ? slot : -1;
}
// (A call, as it is rare: in the rows' loops its code would stand sixteen times over.)
__device__ __noinline__ int slot_at(const int* place, bool given, int n_slots) {
  const int s = *place;
  return given || s < n_slots ? s : -1;
}
// The slot of dense sequence i, as above (all of the tiles' threads).
__device__ __forceinline__ int find_slot(const int* slots, int n_slots, int i) {
  if (slots == nullptr) return i < n_slots ? i : -1;
  const int s = slots[i];
  bool taken = false;
#pragma unroll 4
  for (int j = threadIdx.x; j < i; j += kThreads) taken |= slots[j] == s;
  return tile_sync_or(taken) || s < 0 || s >= n_slots ? -1 : s;
}
// The thread's kR rows from `row` on; rows in [lo, hi) are tokens.
template <int kR>
__device__ __forceinline__ unsigned live_rows(int row, int lo, int hi) {
  constexpr unsigned all = (1u << kR) - 1;
  const int skip = min(max(lo - row, 0), kR), n = min(max(hi - row, 0), kR);
  return all >> (kR - n) & all << skip;
}
template <int kR>
__device__ __forceinline__ Marks dense_marks(int row, int hi) {
  Marks k;
  k.live = live_rows<kR>(row, 0, hi);
  k.first = row == 0 ? 1u : 0u;
  k.last = hi > row && hi - row <= kR ? 1u << (hi - 1 - row) : 0u;
  return k;
}
template <int kR, int GROUPS, int ROWS>
__device__ __forceinline__ Marks packed_marks(const MarkRows<GROUPS, ROWS>& m, int group, int row, int lo, int hi) {
  Marks k;
  k.live = live_rows<kR>(row, lo, hi);
  k.first = m.first[group] & k.live;
  k.last = m.last[group] & k.live;
  return k;
}

// ---- runs of rows, h -> A h + B
// Packed rows: where a sequence starts (backwards: ends) within a run, nothing of h goes on, not even not-a-number.  Such
// a run has A = -0, which no product of gates >= 0 gives, and which any such gate behind it leaves as it is (gates of -0 are
// taken as 0).
constexpr float kCut = -0.f;
template <bool PACKED>
__device__ __forceinline__ bool is_cut(float A) {
  return PACKED && __float_as_uint(A) == 0x80000000u;
}
// The run's effect on h.
template <bool PACKED>
__device__ __forceinline__ float carry_on(float A, float B, float h) {
  return is_cut<PACKED>(A) ? B : fmaf(A, h, B);
}
template <bool PACKED>
__device__ __forceinline__ float2 carry_on(float2 A, float2 B, float2 h) {
  const float2 r = fma2(A, h, B);
  return make_float2(is_cut<PACKED>(A.x) ? B.x : r.x, is_cut<PACKED>(A.y) ? B.y : r.y);
}
// A of a run with A, behind one with `before`.
template <bool PACKED>
__device__ __forceinline__ float join(float A, float before) {
  return is_cut<PACKED>(A) ? A : A * before;
}
template <bool PACKED>
__device__ __forceinline__ float2 join(float2 A, float2 before) {
  const float2 r = mul2(A, before);
  return make_float2(is_cut<PACKED>(A.x) ? A.x : r.x, is_cut<PACKED>(A.y) ? A.y : r.y);
}

// ---- the scan of a block's tile over its threads
template <bool REVERSE>
__device__ __forceinline__ float2 shift(float2 v, int o) {
  return make_float2(REVERSE ? __shfl_down_sync(0xffffffffu, v.x, o) : __shfl_up_sync(0xffffffffu, v.x, o),
                     REVERSE ? __shfl_down_sync(0xffffffffu, v.y, o) : __shfl_up_sync(0xffffffffu, v.y, o));
}
// Row groups lie LW lanes apart.  (A, B) of the thread's rows becomes that of the row groups before it in the warp
// (after it, if REVERSE), and (wA, wB), valid in the warp's last row group (first), that of the whole warp.
template <int LW, bool REVERSE, bool PACKED>
__device__ __forceinline__ void scan_warp(float2 (&A)[P], float2 (&B)[P], float2 (&wA)[P], float2 (&wB)[P], int lane) {
  if (LW == 32) {  // one row group
#pragma unroll
    for (int i = 0; i < P; ++i) {
      wA[i] = A[i];
      wB[i] = B[i];
      A[i] = both(1.f);
      B[i] = both(0.f);
    }
    return;
  }
  const int place = REVERSE ? 31 - lane : lane;
#pragma unroll
  for (int o = LW; o < 16; o <<= 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 ua = shift<REVERSE>(A[i], o), ub = shift<REVERSE>(B[i], o);
      if (place >= o) {
        B[i] = carry_on<PACKED>(A[i], B[i], ub);
        A[i] = join<PACKED>(A[i], ua);
      }
    }
  }
  // the step over half a warp: with two row groups it is the only one, and gives what lies before
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float2 ua = shift<REVERSE>(A[i], 16), ub = shift<REVERSE>(B[i], 16);
    wA[i] = place >= 16 ? join<PACKED>(A[i], ua) : A[i];
    wB[i] = place >= 16 ? carry_on<PACKED>(A[i], B[i], ub) : B[i];
    const float2 pa = LW == 16 ? ua : shift<REVERSE>(wA[i], LW), pb = LW == 16 ? ub : shift<REVERSE>(wB[i], LW);
    A[i] = place >= LW ? pa : both(1.f);
    B[i] = place >= LW ? pb : both(0.f);
  }
}

template <typename T, int LW>
struct ScanShared {
  static constexpr int CW = V * LW;
  float wa[2][kWarps][CW], wb[2][kWarps][CW];  // A, B of the warps, by the tile's parity; then of what lies before them
  float ba[2][CW], bb[2][CW];                  // of the block, which the cluster's others read
  float carry[2][CW];                          // the state entering the block's tile
};

// What goes on from tile to tile, in a warp of its own: as it has no other stores, the release of the cluster's barrier
// waits for none (with the state carried by warps of the tiles each round waited for their outputs to arrive in L2).  Blocks
// read one another's A, B behind that barrier (each writing them to all: 65,536 x 1024 80 us against 79, 20,011 packed x 384 76
// against 73); a place is written again two tiles later, behind another one.  The block's warps have A, B in s.wa, s.wb and wait
// for s.carry.  The warp also leaves what lies before each of them in s.wa, s.wb (every warp for itself over up to seven
// others: 65,536 x 1024 85 us against 81).
// (Two barriers each, by the tile's parity: one side may be a tile ahead of the other.)
__device__ __forceinline__ void block_sync(int par) { asm volatile("bar.sync %0, 288;" ::"r"(2 + par) : "memory"); }
__device__ __forceinline__ void block_arrive(int par) { asm volatile("bar.arrive %0, 288;" ::"r"(2 + par) : "memory"); }
__device__ __forceinline__ void carry_sync(int par) { asm volatile("bar.sync %0, 288;" ::"r"(4 + par) : "memory"); }
__device__ __forceinline__ void carry_arrive(int par) { asm volatile("bar.arrive %0, 288;" ::"r"(4 + par) : "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
static_assert(kBlock == 288, "the barriers' counts");

// The warps of the tiles: s.wa, s.wb[par] of a tile are written.  The tile before must have passed give_wait.
__device__ __forceinline__ void give(int par, bool clustered) {
  block_arrive(par);
  if (clustered) cluster_arrive_relaxed();
}
__device__ __forceinline__ void give_wait(bool clustered) {
  if (clustered) cluster_wait();
}
// The carrying warp: all rounds of tiles.
template <typename T, int LW, bool REVERSE, bool PACKED>
__device__ __forceinline__ void carry_tiles(ScanShared<T, LW>& s, int rounds, int n, int rank) {
  constexpr int CW = ScanShared<T, LW>::CW, K = (CW + 31) / 32;
  const int lane = threadIdx.x & 31;
  float running[K];
#pragma unroll
  for (int k = 0; k < K; ++k) running[k] = 0.f;
  for (int t = 0, par = 0; t < rounds; ++t, par ^= 1) {
    block_sync(par);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = lane + 32 * k;
      if (CW % 32 != 0 && c >= CW) continue;
      float A = 1.f, B = 0.f, fa[kWarps], fb[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        fa[w] = s.wa[par][w][c];
        fb[w] = s.wb[par][w][c];
      }
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {  // what a warp had becomes what lies before it in the block
        const int w = REVERSE ? kWarps - 1 - i : i;
        s.wa[par][w][c] = A;
        s.wb[par][w][c] = B;
        B = carry_on<PACKED>(fa[w], fb[w], B);
        A = join<PACKED>(fa[w], A);
      }
      if (n == 1) {
        s.carry[par][c] = running[k];
        running[k] = carry_on<PACKED>(A, B, running[k]);
      } else {
        s.ba[par][c] = A;
        s.bb[par][c] = B;
      }
    }
    if (n == 1) {
      __syncwarp();
      carry_arrive(par);
      continue;
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = lane + 32 * k;
      if (CW % 32 != 0 && c >= CW) continue;
      float h = running[k], mine = h;
      cg::cluster_group cl = cg::this_cluster();
#pragma unroll
      for (int j = 0; j < kMostBlocks; j += 8) {
        if (j >= n) break;
        float A[8], B[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (j + i >= n) continue;
          A[i] = cl.map_shared_rank(&s.ba[par][0], j + i)[c];
          B[i] = cl.map_shared_rank(&s.bb[par][0], j + i)[c];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (j + i == rank) mine = h;
          if (j + i < n) h = carry_on<PACKED>(A[i], B[i], h);
        }
      }
      s.carry[par][c] = mine;
      running[k] = h;
    }
    __syncwarp();
    carry_arrive(par);
  }
}
// The state before the warp, once the carrying warp has been there.
template <typename T, int LW, bool PACKED>
__device__ __forceinline__ void state_before(const ScanShared<T, LW>& s, int par, int cl, int warp, float2 (&h)[P]) {
  float2 A[P], B[P];
  load_f(&s.carry[par][cl], h);
  load_f(&s.wa[par][warp][cl], A);
  load_f(&s.wb[par][warp][cl], B);
#pragma unroll
  for (int j = 0; j < P; ++j) h[j] = carry_on<PACKED>(A[j], B[j], h[j]);
}
// h over the warps from `from` on, up to the warp.
template <int CW, bool PACKED>
__device__ __forceinline__ void over_warps(const float (&wa)[kWarps][CW], const float (&wb)[kWarps][CW], int cl, int warp,
                                           int from, float2 (&h)[P]) {
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w >= from && w < warp) {
      float2 A[P], B[P];
      load_f(&wa[w][cl], A);
      load_f(&wb[w][cl], B);
#pragma unroll
      for (int j = 0; j < P; ++j) h[j] = carry_on<PACKED>(A[j], B[j], h[j]);
    }
  }
}

// ---- tiles in shared memory
// A tile's ROWS rows of CW channels of one tensor.  Rows of 64 bytes are read two row groups at a time: in every other group
// neighbouring rows change places, so that the two lie in banks of their own.
template <typename T, int LW>
struct Stage {
  static constexpr int CW = V * LW, kR = Tile<T>::R, ROWS = kThreads / LW * kR, PIECES = CW * (int)sizeof(T) / 16;
  static constexpr bool SWAP = LW < Tile<T>::WIDE;
  static constexpr int ELEMS = ROWS * CW;
  static __device__ __forceinline__ int at(int row) { return (SWAP ? row ^ (row / kR & 1) : row) * CW; }
  // The copy of rows [row0, row0 + ROWS) and channels from c0 on (D - c0 at most), asynchronously; zeros for rows outside
  // [lo, hi) and channels behind D.
  static __device__ __forceinline__ void fetch(T* to, const T* from, long long sn, long long row0, int lo, int hi, int c0,
                                               int D) {
    constexpr int N = ROWS * PIECES / kThreads, STEP = kThreads / PIECES;
    static_assert(!SWAP || STEP % (2 * kR) == 0, "the rows of a thread's copies change places alike");
    const int piece = threadIdx.x % PIECES, r = threadIdx.x / PIECES;
    const int c = piece * (16 / (int)sizeof(T));
    const bool on = c0 + c < D;
    const T* src = from + (on ? c0 + c : 0);
    unsigned dst = (unsigned)__cvta_generic_to_shared(to + at(r) + c);
    if (on && row0 >= lo && row0 + ROWS <= hi) {
      src += (row0 + r) * sn;
      const long long step = STEP * sn;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        src += step;
        dst += STEP * CW * (int)sizeof(T);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long row = row0 + r + i * STEP;
      const bool ok = on && row >= lo && row < hi;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src + (ok ? row * sn : 0)), "r"(ok ? 16 : 0)
                   : "memory");
      dst += STEP * CW * (int)sizeof(T);
    }
  }
};
// Row r of a thread's rows, from its first row's place; delta: the way to the neighbour where rows have changed places.
template <int CW, typename T>
__device__ __forceinline__ const T* row_at(const T* first, int r, int delta) {
  return first + r * CW + (r & 1 ? -delta : delta);
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
__device__ __forceinline__ void copies_wait0() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// ---- forward
// A tile's rows twice, from shared memory: folded into (A, B) while the state that enters the tile before is on its way, and
// run with that state.  The gates are taken both times: kept in registers they would cost the second block of an SM (one
// block an SM: 212 us and more for the forward and backward of 4 x 8192 x 1024, where two took 139; four of half the threads 145).
// The look ahead, when it came: log gates of 65,536 x 1024 109 us against 125 without it; sigmoid gates of 4 x 8192 x 1024 58
// against 53, as its clusters fill the SMs and the waits are another block's to fill.
// Plain rows, without a look at their marks: with the sigmoid below 139 us to 127 for the forward and backward of 4 x 8192 x
// 1024.  Four channels a thread and half of the rows (fewer addresses, one more shuffle): 134 against 127.
template <typename T, int GATE, int LW, bool PACKED>
__global__ void __launch_bounds__(kBlock, 2) gated_scan_forward_kernel(const __grid_constant__ ScanArgs p, int cluster) {
  using Raw = typename Io<T, P>::Raw;
  using St = Stage<T, LW>;
  constexpr int kR = St::kR, CW = St::CW, ROWS = St::ROWS, GROUPS = 32 / LW;
  __shared__ __align__(16) ScanShared<T, LW> s;
  __shared__ MarkRows<PACKED ? ROWS / kR : 0, PACKED ? ROWS : 0> marks[3];
  __shared__ SlotTable<PACKED ? ROWS : 0> table;
  __shared__ int dense_slot;
  launch_dependents();
  grid_dependency_wait();  // (every kernel here is launched while the one before it in the stream drains)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % cluster), chain = (int)(blockIdx.x / cluster);
  const int cols = (p.D + CW - 1) / CW, batch = chain / cols, c0 = (chain % cols) * CW;
  const int cl = (tid % LW) * V, c = c0 + cl;         // the thread's channels
  const int r0 = (warp * GROUPS + lane / LW) * kR;    // and rows of the tile
  constexpr unsigned kAll = (1u << kR) - 1;           // (plain: a thread's rows that are all tokens, of one sequence's middle)
  const int delta = St::SWAP && (r0 / kR & 1) ? CW : 0;
  const bool on = c < p.D;
  const T* x = static_cast<const T*>(p.x.p) + (long long)batch * p.x.sb;
  const T* g = static_cast<const T*>(p.g.p) + (long long)batch * p.g.sb;
  T* y = static_cast<T*>(const_cast<void*>(p.y.p)) + (long long)batch * p.y.sb + c;
  int lo = 0, hi = p.N;
  if (PACKED) {
    lo = min(max(p.cu[0], 0), p.N);
    hi = min(max(p.cu[p.B], lo), p.N);
  }
  const int tiles = ret_pieces(p.N, ROWS), kept_rows = ret_pieces(p.N, kScanKept);
  if (tid >= kThreads) {
    carry_tiles<T, LW, false, PACKED>(s, ret_pieces(tiles, cluster), cluster, rank);
    if (cluster > 1) cg::this_cluster().sync();  // no block ends while another one reads its shared memory
    return;
  }
  extern __shared__ __align__(128) uint8_t raw[];  // (16 bytes off a multiple of 128: 65,536 x 1024 105 us instead of 79)
  T* stage = reinterpret_cast<T*>(raw);  // [3][x, g]
  const int rounds = ret_pieces(tiles, cluster);
  const auto fetch = [&](int i) {  // the block's tile of round i
    const int t = i * cluster + rank;
    T* to = stage + i % 3 * 2 * St::ELEMS;
    if (i < rounds && t < tiles) {
      St::fetch(to, x, p.x.sn, (long long)t * ROWS, lo, hi, c0, p.D);
      St::fetch(to + St::ELEMS, g, p.g.sn, (long long)t * ROWS, lo, hi, c0, p.D);
    }
    copies_commit();
  };
  // a and b of the thread's row r
  const auto row_of = [&](const T* sx, int r, float2 (&a)[P], float2 (&b)[P]) {
    float2 gv[P], xv[P];
    unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sx, r, delta)), xv);
    unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sx, r, delta) + St::ELEMS), gv);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const Gate k = gate_of<T, GATE>(gv[i]);
      a[i] = k.a;
      b[i] = input_of<GATE>(xv[i], k.rest);
    }
  };
  // The slot of the sequence that row r of the thread's in the tile of round i begins or ends, and the start of it.
  const auto slot_of = [&](int i, int r) {
    if constexpr (PACKED) return slot_at(&marks[i % 3].seq[r0 + r], p.slots != nullptr, p.n_slots);
    return slot_at(&dense_slot, true, 0);
  };
  const auto start_of = [&](int i, int r, float2 (&h)[P]) {
    fill(h, 0.f);
    const int slot = slot_of(i, r);
    if (slot >= 0) load_f(p.states + (long long)slot * p.D + c, h);
  };
  // What is known of a tile before the state that enters it.
  struct Ahead {
    Marks m;
    int row;                 // the thread's first
    float2 A[P], B[P];       // of the row groups of the warp before the thread's
    float2 h0[P];            // the start of the last sequence that begins in the thread's rows: its slot may be written (by
  };                         // the thread with its last token) before the rows are run once more; the others' are not
  // (whole block; the tile of round i has landed for every thread)
  const auto look = [&](int i, Ahead& n) {
    const int par = i & 1, row0 = (int)min(((long long)i * cluster + rank) * ROWS, (long long)p.N);
    n.row = row0 + r0;
    if constexpr (PACKED)
      n.m = packed_marks<kR>(marks[i % 3], r0 / kR, n.row, lo, hi);
    else
      n.m = dense_marks<kR>(n.row, hi);
    const T* sx = stage + i % 3 * 2 * St::ELEMS + r0 * CW + cl;
    float2 wA[P], wB[P];
    fill(n.A, 1.f);
    fill(n.B, 0.f);
    const auto fold = [&](auto plain) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float2 a[P], b[P];
        row_of(sx, r, a, b);
        if constexpr (!plain) {
          if (p.load && on && n.m.first >> r & 1) {
            start_of(i, r, n.h0);
#pragma unroll
            for (int k = 0; k < P; ++k) b[k] = fma2(a[k], n.h0[k], b[k]);
          }
          if (!(n.m.live >> r & 1)) continue;
          if (PACKED && (n.m.first >> r & 1)) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
              n.B[k] = b[k];
              n.A[k] = both(kCut);
            }
            continue;
          }
        }
#pragma unroll
        for (int k = 0; k < P; ++k) {
          n.B[k] = fma2(a[k], n.B[k], b[k]);
          n.A[k] = mul2(n.A[k], a[k]);
        }
      }
    };
    if (n.m.live == kAll && n.m.first == 0)
      fold(std::true_type());
    else
      fold(std::false_type());
    scan_warp<LW, false, PACKED>(n.A, n.B, wA, wB, lane);
    if (lane / LW == GROUPS - 1) {
      store(&s.wa[par][warp][cl], wA);
      store(&s.wb[par][warp][cl], wB);
    }
  };
  const auto row0_of = [&](int i) { return (int)min(((long long)i * cluster + rank) * ROWS, (long long)p.N); };
  fetch(0);
  fetch(1);
  Ahead next;
  const auto mark = [&](int i) {
    if constexpr (PACKED) {
      const bool any = set_marks(p, row0_of(i), marks[i % 3]);
      if (p.slots != nullptr) find_slots(p.slots, p.n_slots, any, marks[i % 3], table);
    }
  };
  if constexpr (PACKED) {
    clear_marks(marks[0]);
    clear_marks(marks[1]);
    tile_sync();
    mark(0);
    tile_sync();
    mark(1);
  } else if (p.states != nullptr && (rank == 0 || rank == (tiles - 1) % cluster)) {  // the sequence begins or ends here
    const int slot = find_slot(p.slots, p.n_slots, batch);
    if (tid == 0) dense_slot = slot;
  }
  copies_wait1();
  tile_sync();
  look(0, next);
  give(0, cluster > 1);
  for (int i = 0; i < rounds; ++i) {
    const int par = i & 1;
    const Ahead now = next;
    if (i + 1 < rounds) {  // while the state that enters this tile is on its way, the next one
      copies_wait0();
      tile_sync();  // every thread's part of it is there, the buffer after it has been read
      fetch(i + 2);
      if constexpr (PACKED) clear_marks(marks[(i + 2) % 3]);
      look(i + 1, next);
    }
    give_wait(cluster > 1);
    if (i + 1 < rounds) give(par ^ 1, cluster > 1);
    if constexpr (PACKED) {
      if (i + 2 < rounds) {
        tile_sync();
        mark(i + 2);
      }
    }
    carry_sync(par);
    float2 h[P];
    state_before<T, LW, PACKED>(s, par, cl, warp, h);
#pragma unroll
    for (int k = 0; k < P; ++k) h[k] = carry_on<PACKED>(now.A[k], now.B[k], h[k]);
    const int row = now.row;
    if (p.kept != nullptr && on && row < p.N && row % kScanKept == 0)
      store(p.kept + ((long long)batch * kept_rows + row / kScanKept) * p.D + c, h);
    const T* sx = stage + i % 3 * 2 * St::ELEMS + r0 * CW + cl;
    T* py = y + row * p.y.sn;
    const unsigned out = on ? now.m.live : 0, ends = p.states != nullptr && on ? now.m.last : 0;
    const auto run = [&](auto plain) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float2 a[P], b[P];
        row_of(sx, r, a, b);
        bool cut = false;
        if constexpr (!plain) {
          if (p.load && on && now.m.first >> r & 1) {
            float2 h0[P];
            if (now.m.first >> r == 1) {
#pragma unroll
              for (int k = 0; k < P; ++k) h0[k] = now.h0[k];
            } else {
              start_of(i, r, h0);
            }
#pragma unroll
            for (int k = 0; k < P; ++k) b[k] = fma2(a[k], h0[k], b[k]);
          }
          cut = PACKED && (now.m.first >> r & 1);
        }
#pragma unroll
        for (int k = 0; k < P; ++k) h[k] = cut ? b[k] : fma2(a[k], h[k], b[k]);
        if (plain || out >> r & 1) store(py, h);
        py += p.y.sn;
        if constexpr (!plain) {
          if (ends >> r & 1) {
            const int slot = slot_of(i, r);
            if (slot >= 0) store(p.states + (long long)slot * p.D + c, h);
          }
        }
      }
    };
    if (out == kAll && now.m.first == 0 && ends == 0)
      run(std::true_type());
    else
      run(std::false_type());
  }
  if (cluster > 1) cg::this_cluster().sync();  // no block ends while another one reads its shared memory
}

// ---- backward
// A thread's rows three times: the runs of both directions; G from the last row on; h from the first row on, with what
// goes out.  The gates of the first two stay in registers, the third takes them again.
template <typename T, int GATE, int LW, bool PACKED>
__global__ void __launch_bounds__(kBlock, 2) gated_scan_backward_kernel(const __grid_constant__ ScanArgs p, int cluster) {
  using Raw = typename Io<T, P>::Raw;
  using St = Stage<T, LW>;
  constexpr int kR = St::kR, CW = St::CW, ROWS = St::ROWS, GROUPS = 32 / LW;
  constexpr int PER = kScanKept / (GROUPS * kR) > 1 ? kScanKept / (GROUPS * kR) : 1;  // warps of a kept state
  static_assert((GROUPS * kR * PER) % kScanKept == 0 && kWarps % PER == 0, "a kept state at the first row of every PER warps");
  __shared__ __align__(16) ScanShared<T, LW> s;
  __shared__ MarkRows<PACKED ? ROWS / kR : 0, PACKED ? ROWS : 0> marks[2];
  launch_dependents();
  grid_dependency_wait();  // (every kernel here is launched while the one before it in the stream drains)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % cluster), chain = (int)(blockIdx.x / cluster);
  const int cols = (p.D + CW - 1) / CW, batch = chain / cols, c0 = (chain % cols) * CW;
  const int cl = (tid % LW) * V, c = c0 + cl;
  const int r0 = (warp * GROUPS + lane / LW) * kR;
  constexpr unsigned kAll = (1u << kR) - 1;  // (plain: as in the forward)
  const int delta = St::SWAP && (r0 / kR & 1) ? CW : 0;
  const bool on = c < p.D;
  const T* x = static_cast<const T*>(p.x.p) + (long long)batch * p.x.sb;
  const T* g = static_cast<const T*>(p.g.p) + (long long)batch * p.g.sb;
  const T* dy = static_cast<const T*>(p.dy.p) + (long long)batch * p.dy.sb;
  T* dx = static_cast<T*>(const_cast<void*>(p.dx.p)) + (long long)batch * p.dx.sb + c;
  T* dg = static_cast<T*>(const_cast<void*>(p.dg.p)) + (long long)batch * p.dg.sb + c;
  int lo = 0, hi = p.N;
  if (PACKED) {
    lo = min(max(p.cu[0], 0), p.N);
    hi = min(max(p.cu[p.B], lo), p.N);
    // a sequence without tokens: its last state is its start
    if (p.dh0 != nullptr && rank == 0 && tid < kThreads)
      for (int i = tid / LW; i < p.B; i += kThreads / LW) {
        const int l = min(max(p.cu[i], 0), p.N);
        if (on && min(p.cu[i + 1], p.N) <= l) {
          float2 f[P];
          fill(f, 0.f);
          if (p.dh_last != nullptr) load_f(p.dh_last + (long long)i * p.D + c, f);
          store(p.dh0 + (long long)i * p.D + c, f);
        }
      }
  }
  const int tiles = ret_pieces(p.N, ROWS), kept_rows = ret_pieces(p.N, kScanKept);
  if (tid >= kThreads) {
    carry_tiles<T, LW, true, PACKED>(s, ret_pieces(tiles, cluster), cluster, rank);
    if (cluster > 1) cg::this_cluster().sync();  // no block ends while another one reads its shared memory
    return;
  }
  extern __shared__ __align__(128) uint8_t raw[];
  T* stage = reinterpret_cast<T*>(raw);  // [2][x, g, dy]
  const auto fetch = [&](int t, int buf) {
    T* to = stage + buf * 3 * St::ELEMS;
    if (t >= 0) {
      St::fetch(to, x, p.x.sn, (long long)t * ROWS, lo, hi, c0, p.D);
      St::fetch(to + St::ELEMS, g, p.g.sn, (long long)t * ROWS, lo, hi, c0, p.D);
      St::fetch(to + 2 * St::ELEMS, dy, p.dy.sn, (long long)t * ROWS, lo, hi, c0, p.D);
    }
    copies_commit();
  };
  fetch(tiles - 1 - rank, 0);
  if constexpr (PACKED) {
    clear_marks(marks[0]);
    tile_sync();
    set_marks(p, tiles - 1 - rank >= 0 ? (tiles - 1 - rank) * ROWS : p.N, marks[0]);
  }
  int par = 0;
  for (int t0 = 0; t0 < tiles; t0 += cluster, par ^= 1) {
    // tiles from the last one on; a cluster's last round may hold tiles before the first: without rows
    const int t = tiles - 1 - (t0 + rank);
    const int row0 = t >= 0 ? t * ROWS : p.N;
    float2 h[P];
    fill(h, 0.f);
    const int from = warp / PER * PER, krow = row0 + from * GROUPS * kR;
    if (on && krow < p.N) load_f(p.kept + ((long long)batch * kept_rows + krow / kScanKept) * p.D + c, h);
    copies_wait0();
    tile_sync();
    fetch(t - cluster, par ^ 1);
    if constexpr (PACKED) clear_marks(marks[par ^ 1]);
    const T *sx = stage + par * 3 * St::ELEMS + r0 * CW + cl, *sg = sx + St::ELEMS, *sd = sg + St::ELEMS;
    Marks m;
    if constexpr (PACKED)
      m = packed_marks<kR>(marks[par], r0 / kR, row0 + r0, lo, hi);
    else
      m = dense_marks<kR>(row0 + r0, hi);
    const auto sequence_of = [&](int r) {
      if constexpr (PACKED) return marks[par].seq[r0 + r];
      return batch;
    };
    const unsigned first = m.first, last = m.last;
    // the start of a sequence that begins in row r, the gradient behind one that ends there
    const auto start = [&](int r, float2 (&f)[P]) {
      fill(f, 0.f);
      if (p.h0 != nullptr && on) load_f(p.h0 + (long long)sequence_of(r) * p.D + c, f);
    };
    const auto end = [&](int r, float2 (&f)[P]) {
      fill(f, 0.f);
      if (p.dh_last != nullptr && on) load_f(p.dh_last + (long long)sequence_of(r) * p.D + c, f);
    };
    // the thread's rows backwards, c -> rA c + rB
    float2 a[kR][P], rA[P], rB[P], wA[P], wB[P];
    fill(rA, 1.f);
    fill(rB, 0.f);
    const bool is_plain = m.live == kAll && on && (first | last) == 0;
    const auto fold = [&](auto plain) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float2 gv[P], d[P];
        unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sg, r, delta)), gv);
        unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sd, r, delta)), d);
#pragma unroll
        for (int i = 0; i < P; ++i) a[r][i] = gate_of<T, GATE>(gv[i]).a;
        // row r acts before the rows so far, c -> rA (a (dy + c)) + rB
        if constexpr (plain) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            rB[i] = fma2(rA[i], mul2(a[r][i], d[i]), rB[i]);
            rA[i] = mul2(rA[i], a[r][i]);
          }
        } else {
          if (last >> r & 1) {
            float2 e[P];
            end(r, e);
#pragma unroll
            for (int i = 0; i < P; ++i) d[i] = add2(d[i], e[i]);
          }
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (!(m.live >> r & 1)) a[r][i] = both(1.f);
            rB[i] = carry_on<PACKED>(rA[i], rB[i], mul2(a[r][i], d[i]));
            rA[i] = join<PACKED>(rA[i], PACKED && (last >> r & 1) ? both(kCut) : a[r][i]);
          }
        }
      }
    };
    if (is_plain)
      fold(std::true_type());
    else
      fold(std::false_type());
    scan_warp<LW, true, PACKED>(rA, rB, wA, wB, lane);
    if (lane / LW == 0) {
      store(&s.wa[par][warp][cl], wA);
      store(&s.wb[par][warp][cl], wB);
    }
    give(par, cluster > 1);
    // and forwards, h -> fA h + fB, while the gradient that enters the tile is on its way.  b = x - a x here: off by 2^-24 of x,
    // as h is anyway
    if constexpr (PACKED) {
      if (t0 + cluster < tiles) {
        tile_sync();
        set_marks(p, t - cluster >= 0 ? (t - cluster) * ROWS : p.N, marks[par ^ 1]);
      }
    }
    float2 fA[P], fB[P];
    fill(fA, 1.f);
    fill(fB, 0.f);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float2 xv[P];
      unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sx, r, delta)), xv);
      if (!is_plain && first >> r & 1) {
        start(r, fB);
        if (PACKED) fill(fA, kCut);  // (dense: the state before the first row is zero)
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 b = GATE == GATED_SCAN_SIGMOID ? fma2(a[r][i], make_float2(-xv[i].x, -xv[i].y), xv[i]) : xv[i];
        fB[i] = fma2(a[r][i], fB[i], b);
        fA[i] = mul2(fA[i], a[r][i]);
      }
    }
    scan_warp<LW, false, PACKED>(fA, fB, wA, wB, lane);
    if (PER > 1) {
      if (lane / LW == GROUPS - 1) {
        store(&s.wa[par ^ 1][warp][cl], wA);  // (the tile before's have been read)
        store(&s.wb[par ^ 1][warp][cl], wB);
      }
      tile_sync();
      over_warps<CW, PACKED>(s.wa[par ^ 1], s.wb[par ^ 1], cl, warp, from, h);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) h[i] = carry_on<PACKED>(fA[i], fB[i], h[i]);
    give_wait(cluster > 1);
    carry_sync(par);
    float2 k[P];
    state_before<T, LW, PACKED>(s, par, cl, warp, k);
#pragma unroll
    for (int i = 0; i < P; ++i) k[i] = carry_on<PACKED>(rA[i], rB[i], k[i]);
    const unsigned out = on ? m.live : 0, starts = p.dh0 != nullptr && on ? first : 0;
    const long long row = (long long)row0 + r0;
    T *px = dx + row * p.dx.sn, *pg = dg + row * p.dg.sn;
    const auto run = [&](auto plain) {
      float2 G[kR][P];
#pragma unroll
      for (int r = kR - 1; r >= 0; --r) {
        float2 d[P];
        unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sd, r, delta)), d);
        if constexpr (!plain) {
          if (last >> r & 1) end(r, k);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          G[r][i] = add2(d[i], k[i]);
          k[i] = mul2(a[r][i], G[r][i]);
        }
        if constexpr (!plain) {
          if (starts >> r & 1)
            store(p.dh0 + (long long)sequence_of(r) * p.D + c, k);
        }
      }
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float2 gv[P], xv[P], ox[P], og[P];
        unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sg, r, delta)), gv);
        unpack<T>(*reinterpret_cast<const Raw*>(row_at<CW>(sx, r, delta)), xv);
        if constexpr (!plain) {
          if (first >> r & 1) start(r, h);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const Gate gt = gate_of<T, GATE>(gv[i]);
          if (GATE == GATED_SCAN_SIGMOID) {
            ox[i] = mul2(gt.rest, G[r][i]);
            og[i] = mul2(mul2(gt.a, ox[i]), fma2(xv[i], both(-1.f), h[i]));
            h[i] = fma2(gt.a, h[i], mul2(gt.rest, xv[i]));
          } else {
            ox[i] = G[r][i];
            og[i] = mul2(GATE == GATED_SCAN_LOG ? mul2(gt.a, G[r][i]) : G[r][i], h[i]);
            h[i] = fma2(gt.a, h[i], xv[i]);
          }
        }
        if (plain || out >> r & 1) {
          store(px, ox);
          store(pg, og);
        }
        px += p.dx.sn;
        pg += p.dg.sn;
      }
    };
    if (is_plain)
      run(std::true_type());
    else
      run(std::false_type());
  }
  if (cluster > 1) cg::this_cluster().sync();
}

// ---- one token for every row: a block a row and a run of channels
// Bound by the call (launch 2 to 3 us, the binding 4): 256 x 8192 bf16 8 us, of it 4.3 the floor of its 29 MB.
constexpr int kStepPairs = 2;
template <typename T, int GATE>
__global__ void __launch_bounds__(128) gated_scan_step_kernel(const __grid_constant__ ScanArgs p) {
  using Raw = typename Io<T, kStepPairs>::Raw;
  constexpr int P = kStepPairs, V = 2 * P;
  launch_dependents();
  grid_dependency_wait();
  const int runs = (p.D + 128 * V - 1) / (128 * V);
  const int b = (int)(blockIdx.x / runs), c = ((int)(blockIdx.x % runs) * 128 + threadIdx.x) * V;
  const bool on = c < p.D;
  Raw qx{}, qg{};
  if (on) {
    qx = *reinterpret_cast<const Raw*>(static_cast<const T*>(p.x.p) + (long long)b * p.x.sb + c);
    qg = *reinterpret_cast<const Raw*>(static_cast<const T*>(p.g.p) + (long long)b * p.g.sb + c);
  }
  const int slot = ret_slot(p.slots, p.n_slots, b);
  if (!on || slot < 0) return;
  float* state = p.states + (long long)slot * p.D + c;
  float2 h[P], xv[P], gv[P];
  load_f(state, h);
  unpack<T>(qx, xv);
  unpack<T>(qg, gv);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const Gate k = gate_of<T, GATE>(gv[i]);
    h[i] = fma2(k.a, h[i], input_of<GATE>(xv[i], k.rest));
  }
  store(state, h);
  store(static_cast<T*>(const_cast<void*>(p.y.p)) + (long long)b * p.y.sb + c, h);
}

// ---- host
// Blocks of a cluster: as many as there are places for with all clusters running at once, which the SMs of the processing
// clusters decide (a cluster has to lie within one), so the driver is asked, once a kernel and device.  Forward and backward
// of 20,011 packed x 384 fp32 (24 chains): 6 blocks 115 us, 8 blocks 88, 10 blocks 77, 11, of which one cluster has to wait for
// the others, 125; 4 x 8192 x 1024 bf16 (64 chains): 4 blocks 140, 8, in two turns, 157.
class ClusterFit {
 public:
  // The most blocks, up to `most`, of which `chains` clusters run at once; 1 if none do.
  int blocks(int dev, const void* kernel, int smem, long long chains, int most) {
    if (most <= 1 || dev >= kDevices) return 1;
    if (!known_[dev].load(std::memory_order_acquire)) ask(dev, kernel, smem);
    int n = most;
    while (n > 1 && fit_[dev][n] < chains) --n;
    return n;
  }

 private:
  void ask(int dev, const void* kernel, int smem) {
    std::lock_guard<std::mutex> lk(mu_);
    if (!known_[dev].load(std::memory_order_relaxed)) {
      // (more than 8 blocks are not portable; every cluster of a kernel here may have them)
      const bool large = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
      for (int n = 2; n <= kMostBlocks; ++n) {
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim = {(unsigned)n, 1, 1};
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)n);
        cfg.blockDim = dim3(kBlock);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        int k = 0;
        if ((n > 8 && !large) || cudaOccupancyMaxActiveClusters(&k, kernel, &cfg) != cudaSuccess) k = 0;
        fit_[dev][n] = (unsigned short)std::min(k, 65535);
      }
      (void)cudaGetLastError();  // (a size that is refused has no clusters)
      known_[dev].store(true, std::memory_order_release);
    }
  }

  static constexpr int kDevices = 16;
  std::mutex mu_;
  std::atomic<bool> known_[kDevices] = {};
  unsigned short fit_[kDevices][kMostBlocks + 1] = {};
};

struct Plan {
  long long chains;
  int cluster;
  long long turns;  // tiles that a place on an SM takes, one behind the other
};
template <typename T, int GATE, int LW, bool PACKED>
struct Scan {
  static constexpr int CW = V * LW, ROWS = kThreads / LW * Tile<T>::R;
  static constexpr int kSmem = 6 * Stage<T, LW>::ELEMS * (int)sizeof(T);  // forward three tiles of two tensors, backward two of three
  using Kernel = void (*)(ScanArgs, int);
  static Kernel kernel(bool backward) {
    return backward ? gated_scan_backward_kernel<T, GATE, LW, PACKED> : gated_scan_forward_kernel<T, GATE, LW, PACKED>;
  }
  static cudaError_t plan(const ScanArgs& a, bool backward, int dev, Plan* p) {
    static SmemOptIn opt[2];
    static ClusterFit fit[2];
    const int tiles = ret_pieces(a.N, ROWS);
    p->chains = (PACKED ? 1ll : a.B) * ((a.D + CW - 1) / CW);
    const cudaError_t e = opt[backward].ensure((const void*)kernel(backward), kSmem);
    if (e != cudaSuccess) return e;
    p->cluster = fit[backward].blocks(dev, (const void*)kernel(backward), kSmem, p->chains, std::min(kMostBlocks, tiles));
    const long long places = 2ll * kRetSms;
    p->turns = (p->cluster > 1 ? 1 : (p->chains + places - 1) / places) * ret_pieces(tiles, p->cluster);
    return p->chains * p->cluster > 0x7fffffffll ? cudaErrorInvalidValue : cudaSuccess;
  }
  static cudaError_t launch(const ScanArgs& a, bool backward, const Plan& p, cudaStream_t st) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {(unsigned)p.cluster, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.chains * p.cluster));
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel(backward), a, p.cluster);
    note_launch();
    return e;
  }
};

// The lanes of a row, 128 bytes of channels or 64: those with which a place on an SM takes fewer tiles, and 128 where it is the
// same (a tile has as many bytes either way).  128 bytes against 64: 4 x 8192 x 1024 bf16 (64 chains of 128 bytes, 16 tiles
// each way) 140 us against 147; 65,536 x 1024 bf16 (16 chains) 160 against 91; 20,011 x 384 fp32 (12 chains) 132 against 88.
// 32 bytes, where 64 fill the SMs too: 111 against 100.
template <typename T, int GATE, bool PACKED>
cudaError_t launch_gate(const ScanArgs& a, bool backward, cudaStream_t st) {
  using Wide = Scan<T, GATE, Tile<T>::WIDE, PACKED>;
  using Narrow = Scan<T, GATE, Tile<T>::WIDE / 2, PACKED>;
  Plan w, n{};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = Wide::plan(a, backward, dev, &w);
  if (e == cudaSuccess && w.turns > 1) e = Narrow::plan(a, backward, dev, &n);
  if (e != cudaSuccess) return e;
  return w.turns > 1 && n.turns < w.turns ? Narrow::launch(a, backward, n, st) : Wide::launch(a, backward, w, st);
}

template <typename T, bool PACKED>
cudaError_t launch_gated(const ScanArgs& a, bool backward, cudaStream_t st) {
  switch (a.gate) {
    case GATED_SCAN_DECAY: return launch_gate<T, GATED_SCAN_DECAY, PACKED>(a, backward, st);
    case GATED_SCAN_LOG: return launch_gate<T, GATED_SCAN_LOG, PACKED>(a, backward, st);
    default: return launch_gate<T, GATED_SCAN_SIGMOID, PACKED>(a, backward, st);
  }
}

template <typename T>
cudaError_t launch_type(const ScanArgs& a, bool backward, cudaStream_t st) {
  return a.cu != nullptr ? launch_gated<T, true>(a, backward, st) : launch_gated<T, false>(a, backward, st);
}

template <typename T, int GATE>
cudaError_t launch_step(const ScanArgs& a, cudaStream_t st) {
  const int run = 128 * 2 * kStepPairs;
  return launch_dependent(gated_scan_step_kernel<T, GATE>, dim3((unsigned)((long long)a.B * ((a.D + run - 1) / run))), 128, 0, st, true, a);
}

template <typename T>
cudaError_t launch_step_type(const ScanArgs& a, cudaStream_t st) {
  switch (a.gate) {
    case GATED_SCAN_DECAY: return launch_step<T, GATED_SCAN_DECAY>(a, st);
    case GATED_SCAN_LOG: return launch_step<T, GATED_SCAN_LOG>(a, st);
    default: return launch_step<T, GATED_SCAN_SIGMOID>(a, st);
  }
}

}  // namespace

cudaError_t gated_scan_forward_launch(const ScanArgs& a, mhla_dtype dt, cudaStream_t st) {
  return dt == MHLA_BF16 ? launch_type<__nv_bfloat16>(a, false, st) : launch_type<float>(a, false, st);
}
cudaError_t gated_scan_backward_launch(const ScanArgs& a, mhla_dtype dt, cudaStream_t st) {
  return dt == MHLA_BF16 ? launch_type<__nv_bfloat16>(a, true, st) : launch_type<float>(a, true, st);
}
cudaError_t gated_scan_step_launch(const ScanArgs& a, mhla_dtype dt, cudaStream_t st) {
  return dt == MHLA_BF16 ? launch_step_type<__nv_bfloat16>(a, st) : launch_step_type<float>(a, st);
}

}  // namespace mhla
