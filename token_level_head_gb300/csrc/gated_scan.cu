// The gated scan: h_t = a_t h_{t-1} + b_t with a gate a_t of its own for every token and channel, its gradients and
// its single-token step ("Linear Attention notes" §七, the gated update S_t = G_t . S_{t-1} + ..., for a vector state).
//
// Two runs of tokens with (A, B) and (A', B'), h -> A h + B, one behind the other are (A A', A' B + B'), so a tile of
// tokens is folded by every thread over its own few rows, over the row groups of a warp by shuffles, over the warps
// through shared memory; then every thread knows the state before its rows and runs them once more.  The gradient
// runs the same way from the end: c_t = a_t (dy_t + c_{t+1}), G_t = dy_t + c_{t+1}.
//
// Bound: memory (forward 3 tensors, backward 5; about 20 instructions a value).  A block takes a tile of kRows rows and
// LW * 16 bytes of channels; tiles behind one another are taken by the blocks of a cluster (up to 16), which exchange
// their (A, B) through distributed shared memory, and a cluster walks along the sequence.  So x and g are read once and
// no memory, flag or wait is shared between clusters.
#include <cooperative_groups.h>

#include "gated_scan.h"
#include "retention.cuh"

namespace mhla {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int V = 4;  // channels of a thread

// A thread's rows of a tile and the lanes that lie beside one another: 128 bytes of channels, 128 rows a block.
template <typename T>
struct Tile;
template <>
struct Tile<__nv_bfloat16> {
  using Raw = uint2;
  static constexpr int R = 8, LW = 16;
};
template <>
struct Tile<float> {
  using Raw = uint4;
  static constexpr int R = 4, LW = 8;
};

__device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x);
  f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z);
  f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint2& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[4]) {
  __nv_bfloat162 r[2] = {__floats2bfloat162_rn(f[0], f[1]), __floats2bfloat162_rn(f[2], f[3])};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(r);
}
__device__ __forceinline__ void load_f(const float* p, float (&f)[4]) {
  *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(p);
}

// a and 1 - a of a gate.  sigmoid: from exp(-|g|), so that neither 1 + e overflows nor the smaller of the two is a
// difference of nearly equal numbers; the larger is 1 - the smaller, rounded once (a long memory multiplies thousands of
// gates near 1, and their errors).
template <int GATE>
__device__ __forceinline__ void gate_of(float g, float* a, float* rest) {
  if (GATE == GATED_SCAN_DECAY) {
    *a = g;
    *rest = 1.f;
  } else if (GATE == GATED_SCAN_LOG) {
    *a = expf(g);
    *rest = 1.f;
  } else {
    const float e = expf(-fabsf(g));
    const float s = __fdividef(e, 1.f + e), l = 1.f - s;
    *a = g > 0.f ? l : s;
    *rest = g > 0.f ? s : l;
  }
}

// ---- rows of a tile: which are tokens, and where sequences begin and end
struct Marks {
  unsigned live, first, last;  // bit r: row r of the thread
};

template <int ROWS>
struct MarkRows {
  int first[ROWS], last[ROWS];  // packed: 1 + the sequence whose first / last token the row is, 0: none
};

// Packed sequences: marks of the tile's rows row0 .. row0 + ROWS - 1 (whole block).  Offsets outside [0, N] are clamped;
// out of order they mark rows of the tile all the same and nothing else.
template <int ROWS>
__device__ __forceinline__ void mark_rows(const ScanArgs& p, int row0, MarkRows<ROWS>& m) {
  __syncthreads();  // (the marks of the tile before have been read)
  for (int i = threadIdx.x; i < ROWS; i += kThreads) m.first[i] = m.last[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.B; i += kThreads) {
    const int lo = min(max(p.cu[i], 0), p.N), hi = min(max(p.cu[i + 1], lo), p.N);
    if (lo == hi) continue;
    const int f = lo - row0, l = hi - 1 - row0;
    if (f >= 0 && f < ROWS) atomicMax(&m.first[f], i + 1);
    if (l >= 0 && l < ROWS) atomicMax(&m.last[l], i + 1);
  }
  __syncthreads();
}

// The thread's rows r0 .. r0 + kR - 1, lo <= row < hi: tokens.
template <int kR, int ROWS>
__device__ __forceinline__ Marks marks_of(const ScanArgs& p, const MarkRows<ROWS>* m, int row0, int r0, int lo, int hi) {
  Marks k{0, 0, 0};
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int row = row0 + r0 + r;
    if (row >= lo && row < hi) k.live |= 1u << r;
    if (m != nullptr) {
      if (m->first[r0 + r] != 0) k.first |= 1u << r;
      if (m->last[r0 + r] != 0) k.last |= 1u << r;
    } else {
      if (row == 0) k.first |= 1u << r;
      if (row == hi - 1) k.last |= 1u << r;
    }
  }
  return k;
}

// The slot of sequence i, -1 for none: out of range, or the slot of a sequence before it (one thread).
__device__ __noinline__ int slot_of(const int* slots, int n_slots, int i) {
  if (slots == nullptr) return i < n_slots ? i : -1;
  const int s = slots[i];
  if (s < 0 || s >= n_slots) return -1;
  for (int j = 0; j < i; ++j)
    if (slots[j] == s) return -1;
  return s;
}

// ---- runs of rows, h -> A h + B
// Packed rows: where a sequence starts (backwards: ends) within a run, nothing of h goes on, not even not-a-number.  Such
// a run has A = -0, which no product of gates >= 0 gives.
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
// A of a run with A, behind one with `before`.
template <bool PACKED>
__device__ __forceinline__ float join(float A, float before) {
  return is_cut<PACKED>(A) ? A : A * before;
}

// ---- the scan of a block's tile over its threads
// Row groups lie LW lanes apart.  (A, B) of the thread's rows becomes that of the row groups before it in the warp
// (after it, if REVERSE), and (wA, wB), valid in the warp's last row group (first), that of the whole warp.
template <int LW, bool REVERSE, bool PACKED>
__device__ __forceinline__ void scan_warp(float (&A)[V], float (&B)[V], float (&wA)[V], float (&wB)[V], int lane) {
  const int place = REVERSE ? 31 - lane : lane;
#pragma unroll
  for (int o = LW; o < 32; o <<= 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float ua = REVERSE ? __shfl_down_sync(0xffffffffu, A[v], o) : __shfl_up_sync(0xffffffffu, A[v], o);
      const float ub = REVERSE ? __shfl_down_sync(0xffffffffu, B[v], o) : __shfl_up_sync(0xffffffffu, B[v], o);
      if (place >= o) {
        B[v] = carry_on<PACKED>(A[v], B[v], ub);
        A[v] = join<PACKED>(A[v], ua);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    wA[v] = A[v];
    wB[v] = B[v];
    const float ua = REVERSE ? __shfl_down_sync(0xffffffffu, A[v], LW) : __shfl_up_sync(0xffffffffu, A[v], LW);
    const float ub = REVERSE ? __shfl_down_sync(0xffffffffu, B[v], LW) : __shfl_up_sync(0xffffffffu, B[v], LW);
    A[v] = place >= LW ? ua : 1.f;
    B[v] = place >= LW ? ub : 0.f;
  }
}

template <int CW>
struct ScanShared {
  float2 warp[2][kWarps][CW];  // (A, B) of the warps, by the tile's parity
  float2 block[2][kMaxCluster][CW];  // of the cluster's blocks, which write them here
  float carry[2][CW];          // the state entering the block's tile
};

// The state entering the block's tile, for every channel, in s.carry[par] (whole block), and in `running` (threads
// below CW: a channel each) that behind the cluster's tiles.  The warps' (A, B) are in s.warp[par].
template <int CW, bool REVERSE, bool PACKED>
__device__ __forceinline__ void exchange(ScanShared<CW>& s, int par, float* running, bool clustered) {
  const int c = threadIdx.x;
  if (!clustered) {
    // the tile's entering state was written for this parity one tile ago; fold the next one meanwhile
    if (c < CW) s.carry[par][c] = *running;
    __syncthreads();
    if (c < CW) {
      float h = *running;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 f = s.warp[par][REVERSE ? kWarps - 1 - w : w][c];
        h = carry_on<PACKED>(f.x, f.y, h);
      }
      *running = h;
    }
    return;
  }
  cg::cluster_group cl = cg::this_cluster();
  const int n = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  __syncthreads();
  if (c < CW) {
    float A = 1.f, B = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 f = s.warp[par][REVERSE ? kWarps - 1 - w : w][c];
      B = carry_on<PACKED>(f.x, f.y, B);
      A = join<PACKED>(f.x, A);
    }
    for (int i = 0; i < n; ++i) cl.map_shared_rank(&s.block[par][rank][0], i)[c] = make_float2(A, B);
  }
  cl.sync();
  if (c < CW) {
    float h = *running;
    for (int i = 0; i < n; ++i) {
      if (i == rank) s.carry[par][c] = h;
      const float2 f = s.block[par][i][c];
      h = carry_on<PACKED>(f.x, f.y, h);
    }
    *running = h;
  }
  __syncthreads();
}

// ---- forward
template <typename T, int GATE, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) gated_scan_forward_kernel(const __grid_constant__ ScanArgs p, int cluster) {
  using Raw = typename Tile<T>::Raw;
  constexpr int LW = Tile<T>::LW, kR = Tile<T>::R, CW = V * LW, ROWS = kThreads / LW * kR, GROUPS = 32 / LW;
  __shared__ ScanShared<CW> s;
  __shared__ MarkRows<PACKED ? ROWS : 1> marks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % cluster), chain = (int)(blockIdx.x / cluster);
  const int cols = (p.D + CW - 1) / CW, batch = chain / cols, c0 = (chain % cols) * CW;
  const int cl = (tid % LW) * V, c = c0 + cl;         // the thread's channels
  const int r0 = (warp * GROUPS + lane / LW) * kR;    // and rows of the tile
  const bool on = c < p.D;
  const T* x = static_cast<const T*>(p.x.p) + (long long)batch * p.x.sb + c;
  const T* g = static_cast<const T*>(p.g.p) + (long long)batch * p.g.sb + c;
  T* y = static_cast<T*>(const_cast<void*>(p.y.p)) + (long long)batch * p.y.sb + c;
  int lo = 0, hi = p.N;
  if (PACKED) {
    lo = min(max(p.cu[0], 0), p.N);
    hi = min(max(p.cu[p.B], lo), p.N);
  }
  const int tiles = ret_pieces(p.N, ROWS), kept_rows = ret_pieces(p.N, kScanKept);
  float running = 0.f;
  Raw nx[kR], ng[kR];
  const auto fetch = [&](int t) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const long long row = (long long)t * ROWS + r0 + r;
      const bool ok = on && t < tiles && row >= lo && row < hi;
      nx[r] = ok ? *reinterpret_cast<const Raw*>(x + row * p.x.sn) : Raw{};
      ng[r] = ok ? *reinterpret_cast<const Raw*>(g + row * p.g.sn) : Raw{};
    }
  };
  fetch(rank);
  if (cluster > 1) cg::this_cluster().sync();  // every block runs: its shared memory may be written
  int par = 0;
  for (int t0 = 0; t0 < tiles; t0 += cluster, par ^= 1) {
    const int t = t0 + rank, row0 = (int)min((long long)t * ROWS, (long long)p.N);
    if (PACKED) mark_rows(p, row0, marks);
    const Marks m = marks_of<kR>(p, PACKED ? &marks : nullptr, row0, r0, lo, hi);
    float a[kR][V], b[kR][V];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float gv[V];
      unpack(nx[r], b[r]);
      unpack(ng[r], gv);
      const bool live = m.live >> r & 1;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rest;
        gate_of<GATE>(gv[v], &a[r][v], &rest);
        if (GATE == GATED_SCAN_SIGMOID) b[r][v] *= rest;
        if (!live) {
          a[r][v] = 1.f;
          b[r][v] = 0.f;
        }
      }
    }
    fetch(t + cluster);
    if (m.first & m.live) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if ((m.first & m.live) >> r & 1) {
          const int seq = PACKED ? marks.first[r0 + r] - 1 : batch;
          const int slot = p.load && on ? slot_of(p.slots, p.n_slots, seq) : -1;
          float h[V];
          if (slot >= 0) load_f(p.states + (long long)slot * p.D + c, h);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (slot >= 0) b[r][v] = fmaf(a[r][v], h[v], b[r][v]);
            if (PACKED) a[r][v] = kCut;  // (dense: nothing comes before)
          }
        }
    }
    float A[V], B[V], wA[V], wB[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] = a[0][v];
      B[v] = b[0][v];
#pragma unroll
      for (int r = 1; r < kR; ++r) {
        B[v] = carry_on<PACKED>(a[r][v], b[r][v], B[v]);
        A[v] = join<PACKED>(a[r][v], A[v]);
      }
    }
    scan_warp<LW, false, PACKED>(A, B, wA, wB, lane);
    if (lane / LW == GROUPS - 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) s.warp[par][warp][cl + v] = make_float2(wA[v], wB[v]);
    }
    exchange<CW, false, PACKED>(s, par, &running, cluster > 1);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = s.carry[par][cl + v];
      for (int w = 0; w < warp; ++w) {
        const float2 f = s.warp[par][w][cl + v];
        h[v] = carry_on<PACKED>(f.x, f.y, h[v]);
      }
      h[v] = carry_on<PACKED>(A[v], B[v], h[v]);
    }
    const int row = row0 + r0;
    if (p.kept != nullptr && on && row < p.N && row % kScanKept == 0)
      store(p.kept + ((long long)batch * kept_rows + row / kScanKept) * p.D + c, h);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = carry_on<PACKED>(a[r][v], b[r][v], h[v]);
      if (on && m.live >> r & 1) {
        store(y + (long long)(row + r) * p.y.sn, h);
        if (p.states != nullptr && m.last >> r & 1) {
          const int slot = slot_of(p.slots, p.n_slots, PACKED ? marks.last[r0 + r] - 1 : batch);
          if (slot >= 0) store(p.states + (long long)slot * p.D + c, h);
        }
      }
    }
  }
  if (cluster > 1) cg::this_cluster().sync();  // no block ends while another one reads its shared memory
}

// ---- backward
template <typename T, int GATE, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) gated_scan_backward_kernel(const __grid_constant__ ScanArgs p, int cluster) {
  using Raw = typename Tile<T>::Raw;
  constexpr int LW = Tile<T>::LW, kR = Tile<T>::R, CW = V * LW, ROWS = kThreads / LW * kR, GROUPS = 32 / LW;
  constexpr int PER = kScanKept / (GROUPS * kR) > 1 ? kScanKept / (GROUPS * kR) : 1;  // warps of a kept state
  static_assert((GROUPS * kR * PER) % kScanKept == 0, "a kept state at the first row of every PER warps");
  __shared__ ScanShared<CW> s;
  __shared__ float2 fwd[2][kWarps][CW];
  __shared__ MarkRows<PACKED ? ROWS : 1> marks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % cluster), chain = (int)(blockIdx.x / cluster);
  const int cols = (p.D + CW - 1) / CW, batch = chain / cols, c0 = (chain % cols) * CW;
  const int cl = (tid % LW) * V, c = c0 + cl;
  const int r0 = (warp * GROUPS + lane / LW) * kR;
  const bool on = c < p.D;
  const T* x = static_cast<const T*>(p.x.p) + (long long)batch * p.x.sb + c;
  const T* g = static_cast<const T*>(p.g.p) + (long long)batch * p.g.sb + c;
  const T* dy = static_cast<const T*>(p.dy.p) + (long long)batch * p.dy.sb + c;
  T* dx = static_cast<T*>(const_cast<void*>(p.dx.p)) + (long long)batch * p.dx.sb + c;
  T* dg = static_cast<T*>(const_cast<void*>(p.dg.p)) + (long long)batch * p.dg.sb + c;
  int lo = 0, hi = p.N;
  if (PACKED) {
    lo = min(max(p.cu[0], 0), p.N);
    hi = min(max(p.cu[p.B], lo), p.N);
    // a sequence without tokens: its last state is its start
    if (p.dh0 != nullptr && rank == 0)
      for (int i = tid / LW; i < p.B; i += kThreads / LW) {
        const int l = min(max(p.cu[i], 0), p.N);
        if (on && p.cu[i + 1] <= l) {
          float f[V] = {};
          if (p.dh_last != nullptr) load_f(p.dh_last + (long long)i * p.D + c, f);
          store(p.dh0 + (long long)i * p.D + c, f);
        }
      }
  }
  const int tiles = ret_pieces(p.N, ROWS), kept_rows = ret_pieces(p.N, kScanKept);
  float running = 0.f;
  if (cluster > 1) cg::this_cluster().sync();
  int par = 0;
  for (int t0 = 0; t0 < tiles; t0 += cluster, par ^= 1) {
    // tiles from the last one on; a cluster's last round may hold tiles before the first: without rows
    const int t = tiles - 1 - (t0 + rank);
    const int row0 = t >= 0 ? t * ROWS : p.N;
    Raw qx[kR], qg[kR], qd[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const long long row = (long long)row0 + r0 + r;
      const bool ok = on && row >= lo && row < hi;
      qx[r] = ok ? *reinterpret_cast<const Raw*>(x + row * p.x.sn) : Raw{};
      qg[r] = ok ? *reinterpret_cast<const Raw*>(g + row * p.g.sn) : Raw{};
      qd[r] = ok ? *reinterpret_cast<const Raw*>(dy + row * p.dy.sn) : Raw{};
    }
    float hin[V] = {};
    const int krow = row0 + warp / PER * PER * GROUPS * kR;
    if (on && krow < p.N) load_f(p.kept + ((long long)batch * kept_rows + krow / kScanKept) * p.D + c, hin);
    if (PACKED) mark_rows(p, row0, marks);
    const Marks m = marks_of<kR>(p, PACKED ? &marks : nullptr, row0, r0, lo, hi);
    const unsigned first = m.first & m.live, last = m.last & m.live;
    // the start of a sequence that begins in row r, the gradient behind one that ends there
    const auto start = [&](int r, float (&f)[V]) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = 0.f;
      if (p.h0 != nullptr && on) load_f(p.h0 + (long long)(PACKED ? marks.first[r0 + r] - 1 : batch) * p.D + c, f);
    };
    const auto end = [&](int r, float (&f)[V]) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = 0.f;
      if (p.dh_last != nullptr && on) load_f(p.dh_last + (long long)(PACKED ? marks.last[r0 + r] - 1 : batch) * p.D + c, f);
    };
    const auto gates = [&](int r, float (&a)[V], float (&rest)[V], float (&xv)[V]) {
      float gv[V];
      unpack(qx[r], xv);
      unpack(qg[r], gv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gate_of<GATE>(gv[v], &a[v], &rest[v]);
        if (!(m.live >> r & 1)) a[v] = 1.f;
      }
    };
    // the thread's rows: h -> fA h + fB forwards, c -> rA c + rB backwards
    float fA[V], fB[V], rA[V], rB[V], wA[V], wB[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      fA[v] = rA[v] = 1.f;
      fB[v] = rB[v] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float a[V], rest[V], xv[V], d[V];
      gates(r, a, rest, xv);
      unpack(qd[r], d);
      float h[V], e[V];
      if (first >> r & 1) start(r, h);
      if (last >> r & 1) end(r, e);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // forwards: rows in order
        if (first >> r & 1) {
          fB[v] = h[v];
          if (PACKED) fA[v] = kCut;  // (dense: the state before the first row is zero)
        }
        fB[v] = fmaf(a[v], fB[v], GATE == GATED_SCAN_SIGMOID ? rest[v] * xv[v] : xv[v]);
        fA[v] *= a[v];
        // backwards: row r acts before the rows so far, c -> rA (a (dy + c)) + rB
        const float ad = last >> r & 1 ? a[v] * (d[v] + e[v]) : a[v] * d[v];
        rB[v] = carry_on<PACKED>(rA[v], rB[v], ad);
        rA[v] = join<PACKED>(rA[v], PACKED && (last >> r & 1) ? kCut : a[v]);
      }
    }
    scan_warp<LW, false, PACKED>(fA, fB, wA, wB, lane);
    if (PER > 1 && lane / LW == GROUPS - 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) fwd[par][warp][cl + v] = make_float2(wA[v], wB[v]);
    }
    scan_warp<LW, true, PACKED>(rA, rB, wA, wB, lane);
    if (lane / LW == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) s.warp[par][warp][cl + v] = make_float2(wA[v], wB[v]);
    }
    exchange<CW, true, PACKED>(s, par, &running, cluster > 1);
    float k[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (PER > 1)
        for (int w = warp / PER * PER; w < warp; ++w) {
          const float2 f = fwd[par][w][cl + v];
          hin[v] = carry_on<PACKED>(f.x, f.y, hin[v]);
        }
      hin[v] = carry_on<PACKED>(fA[v], fB[v], hin[v]);
      k[v] = s.carry[par][cl + v];
      for (int w = kWarps - 1; w > warp; --w) {
        const float2 f = s.warp[par][w][cl + v];
        k[v] = carry_on<PACKED>(f.x, f.y, k[v]);
      }
      k[v] = carry_on<PACKED>(rA[v], rB[v], k[v]);
    }
    // h_{t-1} of every row, then the rows from the last one on
    float before[kR][V];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float a[V], rest[V], xv[V];
      gates(r, a, rest, xv);
      if (first >> r & 1) start(r, hin);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        before[r][v] = hin[v];
        hin[v] = fmaf(a[v], hin[v], GATE == GATED_SCAN_SIGMOID ? rest[v] * xv[v] : xv[v]);
      }
    }
#pragma unroll
    for (int r = kR - 1; r >= 0; --r) {
      if (!(m.live >> r & 1)) continue;
      float a[V], rest[V], xv[V], d[V], ox[V], og[V];
      gates(r, a, rest, xv);
      unpack(qd[r], d);
      if (last >> r & 1) end(r, k);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float G = d[v] + k[v];
        k[v] = a[v] * G;
        if (GATE == GATED_SCAN_DECAY) {
          ox[v] = G;
          og[v] = G * before[r][v];
        } else if (GATE == GATED_SCAN_LOG) {
          ox[v] = G;
          og[v] = k[v] * before[r][v];
        } else {
          ox[v] = rest[v] * G;
          og[v] = a[v] * ox[v] * (before[r][v] - xv[v]);
        }
      }
      if (on) {
        const long long row = (long long)row0 + r0 + r;
        store(dx + row * p.dx.sn, ox);
        store(dg + row * p.dg.sn, og);
        if (p.dh0 != nullptr && first >> r & 1)
          store(p.dh0 + (long long)(PACKED ? marks.first[r0 + r] - 1 : batch) * p.D + c, k);
      }
    }
  }
  if (cluster > 1) cg::this_cluster().sync();
}

// ---- one token for every row: a block a row and a run of channels
template <typename T, int GATE>
__global__ void __launch_bounds__(128) gated_scan_step_kernel(const __grid_constant__ ScanArgs p) {
  using Raw = typename Tile<T>::Raw;
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
  float h[V], xv[V], gv[V];
  load_f(state, h);
  unpack(qx, xv);
  unpack(qg, gv);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a, rest;
    gate_of<GATE>(gv[v], &a, &rest);
    h[v] = fmaf(a, h[v], GATE == GATED_SCAN_SIGMOID ? rest * xv[v] : xv[v]);
  }
  store(state, h);
  store(static_cast<T*>(const_cast<void*>(p.y.p)) + (long long)b * p.y.sb + c, h);
}

// ---- host
// Blocks of a cluster: as many as the SMs need (two blocks each) and the tiles give, a power of two.
int cluster_of(long long chains, int tiles) {
  int n = 1;
  while (n < kMaxCluster && chains * n < 2 * kRetSms && n < tiles) n *= 2;
  return n;
}

template <typename T, int GATE, bool PACKED>
cudaError_t launch_scan(const ScanArgs& a, bool backward, cudaStream_t st) {
  constexpr int CW = V * Tile<T>::LW, ROWS = kThreads / Tile<T>::LW * Tile<T>::R;
  void (*kernel)(ScanArgs, int) =
      backward ? gated_scan_backward_kernel<T, GATE, PACKED> : gated_scan_forward_kernel<T, GATE, PACKED>;
  const long long chains = (PACKED ? 1ll : a.B) * ((a.D + CW - 1) / CW);
  const int n = cluster_of(chains, ret_pieces(a.N, ROWS));
  if (chains * n > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {(unsigned)n, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(chains * n));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = n > 1 ? 1 : 0;
  if (n > 8) {
    static std::once_flag once[2][64];  // (an attribute of the kernel on each device)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::call_once(once[backward][dev & 63], [&] {
      e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, n);
  note_launch();
  return e;
}

template <typename T, int GATE>
cudaError_t launch_gate(const ScanArgs& a, bool backward, cudaStream_t st) {
  return a.cu != nullptr ? launch_scan<T, GATE, true>(a, backward, st) : launch_scan<T, GATE, false>(a, backward, st);
}

template <typename T>
cudaError_t launch_type(const ScanArgs& a, bool backward, cudaStream_t st) {
  switch (a.gate) {
    case GATED_SCAN_DECAY: return launch_gate<T, GATED_SCAN_DECAY>(a, backward, st);
    case GATED_SCAN_LOG: return launch_gate<T, GATED_SCAN_LOG>(a, backward, st);
    default: return launch_gate<T, GATED_SCAN_SIGMOID>(a, backward, st);
  }
}

template <typename T, int GATE>
cudaError_t launch_step(const ScanArgs& a, cudaStream_t st) {
  const int run = 128 * V;
  gated_scan_step_kernel<T, GATE><<<(unsigned)((long long)a.B * ((a.D + run - 1) / run)), 128, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
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
