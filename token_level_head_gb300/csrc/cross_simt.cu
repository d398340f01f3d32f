// Linear cross attention on the FP32 units, for every type and width; the single query; the sums over segments.
//
//   S = sum_j phi(k_j) v_j^T, z = sum_j phi(k_j);   den = phi(q) . z + eps, y = phi(q) S / den
//   u = S dy, dden = -(phi(q) . u) / den^2;         dq = phi'(q) (u / den + dden z)
//   dS = sum_t (phi(q_t) / den_t) dy_t^T, dz = sum_t phi(q_t) dden_t
//   dk = phi'(k) (dS v + dz), dv = dS^T phi(k)
//
// Products of 64 (32) token rows with a d x d matrix in shared memory: 256 threads as 16 x 16, each with d / 16 columns
// (vectors of up to four) and rows 16 apart.  Bound by FP32 issue: 4 d^2 flop a token forward, 8 d^2 backward.
#include "cross.cuh"

namespace mhla {
namespace {

constexpr int kThreads = 256;

template <int D>
struct Simt {
  static constexpr int CN = D / 16;              // columns of a thread
  static constexpr int VEC = CN < 4 ? CN : 4;    // of a vector
  static constexpr int LD = D + 4;               // floats of a row in shared memory
  __device__ static __forceinline__ int col(int t, int j) { return j / VEC * (16 * VEC) + t * VEC + j % VEC; }
};

template <int N>
__device__ __forceinline__ void load_vec(const float* p, float* f) {
  if (N == 4) *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(p);
  if (N == 2) *reinterpret_cast<float2*>(f) = *reinterpret_cast<const float2*>(p);
  if (N == 1) f[0] = p[0];
}

// acc[i][j] += sum_k a[ty + 16 i][k] b[k][col(j)]
template <int D, int RN>
__device__ __forceinline__ void rows_times(float (&acc)[RN][Simt<D>::CN], const float* a, const float* b, int ty, int tx) {
  using S = Simt<D>;
#pragma unroll 2
  for (int k = 0; k < D; k += 4) {
    float x[RN][4];
#pragma unroll
    for (int i = 0; i < RN; ++i) load_vec<4>(a + (ty + 16 * i) * S::LD + k, x[i]);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float w[S::CN];
#pragma unroll
      for (int j = 0; j < S::CN; j += S::VEC) load_vec<S::VEC>(b + (k + m) * S::LD + S::col(tx, j), w + j);
#pragma unroll
      for (int i = 0; i < RN; ++i)
#pragma unroll
        for (int j = 0; j < S::CN; ++j) acc[i][j] = fmaf(x[i][m], w[j], acc[i][j]);
    }
  }
}
// acc[i][j] += sum_t a[t][col(ty, i)] b[t][col(tx, j)] over `rows` tokens
template <int D>
__device__ __forceinline__ void outer_sum(float (&acc)[Simt<D>::CN][Simt<D>::CN], const float* a, const float* b, int rows,
                                          int ty, int tx) {
  using S = Simt<D>;
#pragma unroll 4
  for (int t = 0; t < rows; ++t) {
    float x[S::CN], w[S::CN];
#pragma unroll
    for (int j = 0; j < S::CN; j += S::VEC) {
      load_vec<S::VEC>(a + t * S::LD + S::col(ty, j), x + j);
      load_vec<S::VEC>(b + t * S::LD + S::col(tx, j), w + j);
    }
#pragma unroll
    for (int i = 0; i < S::CN; ++i)
#pragma unroll
      for (int j = 0; j < S::CN; ++j) acc[i][j] = fmaf(x[i], w[j], acc[i][j]);
  }
}

// n of ROWS rows of a tensor to shared memory (zeros behind them), phi applied (feature) and, if raw is given, as they are.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void load_rows(float* to, const T* from, long long sn, int n, int feature, float* raw = nullptr) {
  constexpr int V = 16 / sizeof(T), PIECES = D / V, N = (ROWS * PIECES + kThreads - 1) / kThreads;
  uint4 u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {  // (all loads in flight)
    const int at = threadIdx.x + i * kThreads, r = at / PIECES, c = at % PIECES * V;
    u[i] = r < n ? *reinterpret_cast<const uint4*>(from + (long long)r * sn + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = threadIdx.x + i * kThreads, r = at / PIECES, c = at % PIECES * V;
    if (r >= ROWS) continue;
    const T* e = reinterpret_cast<const T*>(&u[i]);
    float f[V];
#pragma unroll
    for (int x = 0; x < V; ++x) f[x] = to_f(e[x]);
    if (raw)
#pragma unroll
      for (int x = 0; x < V; x += 4)
        *reinterpret_cast<float4*>(raw + r * Simt<D>::LD + c + x) = make_float4(f[x], f[x + 1], f[x + 2], f[x + 3]);
#pragma unroll
    for (int x = 0; x < V; ++x) f[x] = r < n ? ret_phi(f[x], feature) : 0.f;
#pragma unroll
    for (int x = 0; x < V; x += 4)
      *reinterpret_cast<float4*>(to + r * Simt<D>::LD + c + x) = make_float4(f[x], f[x + 1], f[x + 2], f[x + 3]);
  }
}
// A d x d fp32 matrix to shared memory, as it is and transposed (either may be null).
template <int D>
__device__ __forceinline__ void load_matrix(float* to, float* turned, const float* from) {
  constexpr int N = (D * D / 4 + kThreads - 1) / kThreads, BATCH = N < 4 ? N : 4;
#pragma unroll 1
  for (int b = 0; b < N; b += BATCH) {
    float4 v[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int at = (threadIdx.x + (b + i) * kThreads) * 4;
      if (at < D * D) v[i] = *reinterpret_cast<const float4*>(from + at);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int at = (threadIdx.x + (b + i) * kThreads) * 4, r = at / D, c = at % D;
      if (at >= D * D) continue;
      if (to) *reinterpret_cast<float4*>(to + r * Simt<D>::LD + c) = v[i];
      if (turned) {
        turned[c * Simt<D>::LD + r] = v[i].x;
        turned[(c + 1) * Simt<D>::LD + r] = v[i].y;
        turned[(c + 2) * Simt<D>::LD + r] = v[i].z;
        turned[(c + 3) * Simt<D>::LD + r] = v[i].w;
      }
    }
  }
}
// The thread's columns of a row.
template <int D, typename T>
__device__ __forceinline__ void store_cols(T* row, int tx, const float (&f)[Simt<D>::CN]) {
  using S = Simt<D>;
#pragma unroll
  for (int j = 0; j < S::CN; j += S::VEC) {
    T v[S::VEC];
#pragma unroll
    for (int x = 0; x < S::VEC; ++x) v[x] = from_f<T>(f[j + x]);
    T* to = row + S::col(tx, j);
    if (sizeof(v) == 16) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(v);
    if (sizeof(v) == 8) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(v);
    if (sizeof(v) == 4) *reinterpret_cast<unsigned*>(to) = *reinterpret_cast<const unsigned*>(v);
    if (sizeof(v) == 2) *to = v[0];
  }
}

// ---- states: a block sums up a segment of a key head
constexpr int kSumRows = 32;
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_states_kernel(const __grid_constant__ CrossArgs p) {
  launch_dependents();
  grid_dependency_wait();  // (every kernel here is launched while the one before it in the stream drains)
  using S = Simt<D>;
  extern __shared__ float sm[];
  __shared__ int scratch;
  float *fk = sm, *v = sm + kSumRows * S::LD;
  const int h = blockIdx.x % p.Hk, k = blockIdx.x / p.Hk, tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const CrossSegment g = cross_segment(p.ks, k, &scratch);
  if (g.seq < 0) return;
  const T* kp = static_cast<const T*>(p.k.p) + cross_base(p.ks, p.k, g.seq, h) + (long long)g.row0 * p.k.sn;
  const T* vp = static_cast<const T*>(p.v.p) + cross_base(p.ks, p.v, g.seq, h) + (long long)g.row0 * p.v.sn;
  float acc[S::CN][S::CN] = {}, zs = 0.f;
  for (int t = 0; t < g.len; t += kSumRows) {
    const int n = min(kSumRows, g.len - t);
    __syncthreads();
    load_rows<T, D, kSumRows>(fk, kp + (long long)t * p.k.sn, p.k.sn, n, p.k.feature);
    load_rows<T, D, kSumRows>(v, vp + (long long)t * p.v.sn, p.v.sn, n, kFeatIdentity);
    __syncthreads();
    outer_sum<D>(acc, fk, v, n, ty, tx);
    if (tid < D)
      for (int r = 0; r < n; ++r) zs += fk[r * S::LD + tid];
  }
  float *so, *zo;
  if (cross_joined(p.ks) && g.nseg != 1) {
    so = p.part + ((size_t)k * p.Hk + h) * (D * D + D);
    zo = so + D * D;
  } else {
    const int slot = ret_slot(p.slots, p.n_slots, g.seq);
    if (slot < 0) return;
    so = p.S + ((size_t)slot * p.Hk + h) * D * D;
    zo = p.z + ((size_t)slot * p.Hk + h) * D;
  }
#pragma unroll
  for (int i = 0; i < S::CN; ++i) store_cols<D>(so + S::col(ty, i) * D, tx, acc[i]);
  if (tid < D) zo[tid] = zs;
}

// ---- sums over segments: a block has 32 runs of four elements of a sequence's key head, and eight threads share a run's
// parts, so that few sums of many segments (one long sequence) are read by enough threads at once (4 heads of 74 segments,
// d = 128: 44 us with a thread an element).  The order is fixed: a thread's parts, then the eight.
constexpr int kJoinRuns = 32, kJoinShare = 8, kJoinThreads = kJoinRuns * kJoinShare;
__global__ void __launch_bounds__(kJoinThreads) cross_join_kernel(const __grid_constant__ CrossArgs p, int backward) {
  __shared__ float4 sums[kJoinShare][kJoinRuns];
  const CrossSide& s = backward ? p.qs : p.ks;
  const int E = p.d * p.d + p.d, per = (E / 4 + kJoinRuns - 1) / kJoinRuns;
  const int run = threadIdx.x % kJoinRuns, share = threadIdx.x / kJoinRuns;
  const int x = ((int)(blockIdx.x % per) * kJoinRuns + run) * 4;
  const long long u = blockIdx.x / per;
  const int h = (int)(u % p.Hk), seq = (int)(u / p.Hk);
  launch_dependents();
  grid_dependency_wait();
  int lo, hi;
  cross_range(s, seq, &lo, &hi);
  const int first = cross_first(s, seq, lo), n = s.cu != nullptr ? ret_pieces(hi - lo, s.L) : ret_pieces(s.N, s.L);
  const int slot = backward ? seq : ret_slot(p.slots, p.n_slots, seq);
  if (slot < 0 || (!backward && n == 1)) return;  // (the whole block)
  const int G = backward ? p.H / p.Hk : 1, heads = backward ? p.H : p.Hk;
  const float* part = p.part + ((size_t)first * heads + (size_t)h * G) * E + x;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const int all = n * G;
  if (x < E) {
#pragma unroll 4
    for (int i = share; i < all; i += kJoinShare) {
      const float4 v = *reinterpret_cast<const float4*>(part + ((size_t)(i / G) * heads + i % G) * E);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
  }
  sums[share][run] = sum;
  __syncthreads();
  if (share != 0 || x >= E) return;
#pragma unroll
  for (int i = 1; i < kJoinShare; ++i) {
    const float4 v = sums[i][run];
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  float* to = backward          ? p.dS + ((size_t)seq * p.Hk + h) * E + x
              : x < p.d * p.d ? p.S + ((size_t)slot * p.Hk + h) * p.d * p.d + x
                              : p.z + ((size_t)slot * p.Hk + h) * p.d + x - p.d * p.d;
  *reinterpret_cast<float4*>(to) = sum;
}

// ---- read: a block reads the sums by a segment of a query head
constexpr int kReadRows = 64;
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_read_kernel(const __grid_constant__ CrossArgs p) {
  launch_dependents();
  grid_dependency_wait();  // (every kernel here is launched while the one before it in the stream drains)
  using S = Simt<D>;
  constexpr int RN = kReadRows / 16;
  extern __shared__ float sm[];
  __shared__ int scratch;
  __shared__ float z[D], inv[kReadRows];
  float *mat = sm, *fq = sm + D * S::LD;
  const int h = blockIdx.x % p.H, k = blockIdx.x / p.H, tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const CrossSegment g = cross_segment(p.qs, k, &scratch);
  if (g.seq < 0) return;
  const int slot = p.slots != nullptr ? p.slots[g.seq] : g.seq;
  if (slot < 0 || slot >= p.n_slots) return;
  const size_t unit = (size_t)slot * p.Hk + h / (p.H / p.Hk);
  load_matrix<D>(mat, nullptr, p.S + unit * D * D);
  if (tid < D) z[tid] = p.z[unit * D + tid];
  const T* qp = static_cast<const T*>(p.q.p) + cross_base(p.qs, p.q, g.seq, h) + (long long)g.row0 * p.q.sn;
  T* yp = static_cast<T*>(const_cast<void*>(p.y.p)) + cross_base(p.qs, p.y, g.seq, h) + (long long)g.row0 * p.y.sn;
  for (int t = 0; t < g.len; t += kReadRows) {
    const int n = min(kReadRows, g.len - t);
    __syncthreads();
    load_rows<T, D, kReadRows>(fq, qp + (long long)t * p.q.sn, p.q.sn, n, p.q.feature);
    __syncthreads();
    if (p.normalise) {  // four threads a row
      const int r = tid / 4;
      float den = 0.f;
      for (int c = tid % 4; c < D; c += 4) den = fmaf(fq[r * S::LD + c], z[c], den);
      den += __shfl_xor_sync(0xffffffffu, den, 1);
      den += __shfl_xor_sync(0xffffffffu, den, 2);
      if (tid % 4 == 0) inv[r] = cross_inverse(den + p.eps);
      __syncthreads();
    }
    float acc[RN][S::CN] = {};
    rows_times<D, RN>(acc, fq, mat, ty, tx);
#pragma unroll
    for (int i = 0; i < RN; ++i) {
      const int r = ty + 16 * i;
      if (r >= n) continue;
      if (p.normalise)
#pragma unroll
        for (int j = 0; j < S::CN; ++j) acc[i][j] *= inv[r];
      store_cols<D>(yp + (long long)(t + r) * p.y.sn, tx, acc[i]);
    }
  }
}

// ---- backward over the queries: dq, and a segment's part of dS and dz
constexpr int kBackRows = 32;
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_backward_query_kernel(const __grid_constant__ CrossArgs p) {
  launch_dependents();
  grid_dependency_wait();  // (every kernel here is launched while the one before it in the stream drains)
  using S = Simt<D>;
  constexpr int RN = kBackRows / 16, E = D * D + D;
  extern __shared__ float sm[];
  __shared__ int scratch;
  __shared__ float z[D], inv[kBackRows], dd[kBackRows];
  float *mat = sm, *fq = mat + D * S::LD, *q = fq + kBackRows * S::LD, *dy = q + kBackRows * S::LD, *u = dy + kBackRows * S::LD;
  const int h = blockIdx.x % p.H, k = blockIdx.x / p.H, tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const CrossSegment g = cross_segment(p.qs, k, &scratch);
  if (g.seq < 0) return;
  const size_t unit = (size_t)g.seq * p.Hk + h / (p.H / p.Hk);
  load_matrix<D>(nullptr, mat, p.S + unit * D * D);
  if (tid < D) z[tid] = p.z[unit * D + tid];
  const T* qp = static_cast<const T*>(p.q.p) + cross_base(p.qs, p.q, g.seq, h) + (long long)g.row0 * p.q.sn;
  const T* dyp = static_cast<const T*>(p.dy.p) + cross_base(p.qs, p.dy, g.seq, h) + (long long)g.row0 * p.dy.sn;
  T* dqp = static_cast<T*>(const_cast<void*>(p.dq.p)) + cross_base(p.qs, p.dq, g.seq, h) + (long long)g.row0 * p.dq.sn;
  float acc[S::CN][S::CN] = {}, dz = 0.f;
  for (int t = 0; t < g.len; t += kBackRows) {
    const int n = min(kBackRows, g.len - t);
    __syncthreads();
    load_rows<T, D, kBackRows>(fq, qp + (long long)t * p.q.sn, p.q.sn, n, p.q.feature, q);
    load_rows<T, D, kBackRows>(dy, dyp + (long long)t * p.dy.sn, p.dy.sn, n, kFeatIdentity);
    __syncthreads();
    float ur[RN][S::CN] = {};
    rows_times<D, RN>(ur, dy, mat, ty, tx);  // u[t][c] = sum_e dy[t][e] S[c][e]
#pragma unroll
    for (int i = 0; i < RN; ++i) store_cols<D>(u + (ty + 16 * i) * S::LD, tx, ur[i]);
    __syncthreads();
    {  // eight threads a row: den and phi(q) . u
      const int r = tid / 8;
      float den = 0.f, s = 0.f;
      for (int c = tid % 8; c < D; c += 8) {
        den = fmaf(fq[r * S::LD + c], z[c], den);
        s = fmaf(fq[r * S::LD + c], u[r * S::LD + c], s);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        den += __shfl_xor_sync(0xffffffffu, den, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
      }
      if (tid % 8 == 0) {
        const float w = p.normalise ? cross_inverse(den + p.eps) : 1.f;
        inv[r] = w;
        dd[r] = p.normalise ? -s * w * w : 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RN; ++i) {
      const int r = ty + 16 * i;
      if (r >= n) continue;
      float o[S::CN];
#pragma unroll
      for (int j = 0; j < S::CN; ++j) {
        const int c = S::col(tx, j);
        o[j] = ret_dphi(q[r * S::LD + c], p.q.feature) * fmaf(dd[r], z[c], ur[i][j] * inv[r]);
      }
      store_cols<D>(dqp + (long long)(t + r) * p.dq.sn, tx, o);
    }
    if (tid < D)
      for (int r = 0; r < n; ++r) dz = fmaf(fq[r * S::LD + tid], dd[r], dz);
    __syncthreads();
    for (int i = tid; i < kBackRows * D; i += kThreads) fq[i / D * S::LD + i % D] *= inv[i / D];
    __syncthreads();
    outer_sum<D>(acc, fq, dy, n, ty, tx);
  }
  float* out = p.part + ((size_t)k * p.H + h) * E;
#pragma unroll
  for (int i = 0; i < S::CN; ++i) store_cols<D>(out + S::col(ty, i) * D, tx, acc[i]);
  if (tid < D) out[D * D + tid] = dz;
}

// ---- backward over the keys: dk and dv; dense rows behind a sequence's tokens become zeros
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_backward_key_kernel(const __grid_constant__ CrossArgs p) {
  launch_dependents();
  grid_dependency_wait();  // (every kernel here is launched while the one before it in the stream drains)
  using S = Simt<D>;
  constexpr int RN = kBackRows / 16, E = D * D + D;
  extern __shared__ float sm[];
  __shared__ int scratch;
  __shared__ float dz[D];
  float *mat = sm, *mat_t = mat + D * S::LD, *fk = mat_t + D * S::LD, *kr = fk + kBackRows * S::LD, *v = kr + kBackRows * S::LD;
  const int h = blockIdx.x % p.Hk, k = blockIdx.x / p.Hk, tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const CrossSegment g = cross_segment(p.ks, k, &scratch);
  if (g.seq < 0) return;
  const T* kp = static_cast<const T*>(p.k.p) + cross_base(p.ks, p.k, g.seq, h) + (long long)g.row0 * p.k.sn;
  const T* vp = static_cast<const T*>(p.v.p) + cross_base(p.ks, p.v, g.seq, h) + (long long)g.row0 * p.v.sn;
  T* dkp = static_cast<T*>(const_cast<void*>(p.dk.p)) + cross_base(p.ks, p.dk, g.seq, h) + (long long)g.row0 * p.dk.sn;
  T* dvp = static_cast<T*>(const_cast<void*>(p.dv.p)) + cross_base(p.ks, p.dv, g.seq, h) + (long long)g.row0 * p.dv.sn;
  const int rows = p.ks.cu != nullptr ? g.len : min(p.ks.L, p.ks.N - g.row0);
  const float* from = p.dS + ((size_t)g.seq * p.Hk + h) * E;
  load_matrix<D>(mat, mat_t, from);
  if (tid < D) dz[tid] = from[D * D + tid];
  for (int t = 0; t < rows; t += kBackRows) {
    const int n = min(kBackRows, max(g.len - t, 0)), m = min(kBackRows, rows - t);
    __syncthreads();
    load_rows<T, D, kBackRows>(fk, kp + (long long)t * p.k.sn, p.k.sn, n, p.k.feature, kr);
    load_rows<T, D, kBackRows>(v, vp + (long long)t * p.v.sn, p.v.sn, n, kFeatIdentity);
    __syncthreads();
    float gv[RN][S::CN] = {}, gk[RN][S::CN] = {};
    rows_times<D, RN>(gv, fk, mat, ty, tx);
    rows_times<D, RN>(gk, v, mat_t, ty, tx);
#pragma unroll
    for (int i = 0; i < RN; ++i) {
      const int r = ty + 16 * i;
      if (r >= m) continue;
#pragma unroll
      for (int j = 0; j < S::CN; ++j) {
        const int c = S::col(tx, j);
        gk[i][j] = r < n ? ret_dphi(kr[r * S::LD + c], p.k.feature) * (gk[i][j] + dz[c]) : 0.f;
        if (r >= n) gv[i][j] = 0.f;
      }
      store_cols<D>(dkp + (long long)(t + r) * p.dk.sn, tx, gk[i]);
      store_cols<D>(dvp + (long long)(t + r) * p.dv.sn, tx, gv[i]);
    }
  }
}

// ---- one query a row: a block a row and key head; its query heads share the read of S
template <int D>
struct Step {
  static constexpr int kThreads = D * D / 4 < 128 ? D * D / 4 : 128;
};
template <typename T, int D>
__global__ void __launch_bounds__(Step<D>::kThreads) cross_step_kernel(const __grid_constant__ CrossArgs p) {
  launch_dependents();
  grid_dependency_wait();
  constexpr int THREADS = Step<D>::kThreads, LANES = D / 4, ROWS = THREADS / LANES;  // threads of a row of S, rows at a time
  __shared__ float fq[D];
  __shared__ float red[THREADS / 32][D + 1];
  const int hk = blockIdx.x % p.Hk, b = blockIdx.x / p.Hk, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = p.slots != nullptr ? p.slots[b] : b;
  if (slot < 0 || slot >= p.n_slots) return;
  const int c0 = tid / LANES, e = tid % LANES * 4;
  const float* Sp = p.S + ((size_t)slot * p.Hk + hk) * D * D;
  const float* zp = p.z + ((size_t)slot * p.Hk + hk) * D;
  float4 s[D / ROWS];
#pragma unroll
  for (int i = 0; i < D / ROWS; ++i) s[i] = *reinterpret_cast<const float4*>(Sp + (c0 + i * ROWS) * D + e);
  const float zc = tid < D ? zp[tid] : 0.f;
  const int G = p.H / p.Hk;
  for (int m = 0; m < G; ++m) {
    const int h = hk * G + m;
    const T* q = static_cast<const T*>(p.q.p) + (long long)b * p.q.sb + (long long)h * p.q.sh;
    T* y = static_cast<T*>(const_cast<void*>(p.y.p)) + (long long)b * p.y.sb + (long long)h * p.y.sh;
    float den = 0.f;
    if (tid < D) {
      const float f = ret_phi(to_f(q[tid]), p.q.feature);
      fq[tid] = f;
      den = f * zc;
    }
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < D / ROWS; ++i) {
      const float f = fq[c0 + i * ROWS];
      a.x = fmaf(f, s[i].x, a.x);
      a.y = fmaf(f, s[i].y, a.y);
      a.z = fmaf(f, s[i].z, a.z);
      a.w = fmaf(f, s[i].w, a.w);
    }
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
      a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
      a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
      a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
      a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane < LANES) {
      red[warp][e] = a.x;
      red[warp][e + 1] = a.y;
      red[warp][e + 2] = a.z;
      red[warp][e + 3] = a.w;
    }
    if (lane == 0) red[warp][D] = den;
    __syncthreads();
    if (tid < D) {
      float num = 0.f, d = 0.f;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        num += red[w][tid];
        d += red[w][D];
      }
      y[tid] = from_f<T>(p.normalise ? num * cross_inverse(d + p.eps) : num);
    }
  }
}

// ---- host
cudaError_t launch(void (*kernel)(CrossArgs), SmemOptIn& opt, long long blocks, int smem, const CrossArgs& a, cudaStream_t st) {
  const cudaError_t e = opt.ensure((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)blocks), kThreads, (size_t)smem, st, true, a);
}

template <typename T, int D>
cudaError_t states_t(const CrossArgs& a, cudaStream_t st) {
  static SmemOptIn opt;
  return launch(cross_states_kernel<T, D>, opt, (long long)a.ks.segs * a.Hk, 2 * kSumRows * Simt<D>::LD * 4, a, st);
}
template <typename T, int D>
cudaError_t read_t(const CrossArgs& a, cudaStream_t st) {
  static SmemOptIn opt;
  return launch(cross_read_kernel<T, D>, opt, (long long)a.qs.segs * a.H, (D + kReadRows) * Simt<D>::LD * 4, a, st);
}
template <typename T, int D>
cudaError_t backward_t(const CrossArgs& a, cudaStream_t st) {
  static SmemOptIn opt_q, opt_k;
  cudaError_t e = cudaSuccess;
  if (a.qs.segs > 0)
    e = launch(cross_backward_query_kernel<T, D>, opt_q, (long long)a.qs.segs * a.H, (D + 4 * kBackRows) * Simt<D>::LD * 4, a, st);
  if (e != cudaSuccess || a.ks.segs == 0) return e;
  e = cross_join_launch(a, true, st);
  if (e != cudaSuccess) return e;
  return launch(cross_backward_key_kernel<T, D>, opt_k, (long long)a.ks.segs * a.Hk, (2 * D + 3 * kBackRows) * Simt<D>::LD * 4, a, st);
}
template <typename T, int D>
cudaError_t step_t(const CrossArgs& a, cudaStream_t st) {
  return launch_dependent(cross_step_kernel<T, D>, dim3((unsigned)((long long)a.qs.B * a.Hk)), Step<D>::kThreads, 0, st, true, a);
}

#define CROSS_DISPATCH(fn)                                                                        \
  switch (a.d) {                                                                                  \
    case 16: return dt == MHLA_BF16 ? fn<__nv_bfloat16, 16>(a, st) : fn<float, 16>(a, st);        \
    case 32: return dt == MHLA_BF16 ? fn<__nv_bfloat16, 32>(a, st) : fn<float, 32>(a, st);        \
    case 64: return dt == MHLA_BF16 ? fn<__nv_bfloat16, 64>(a, st) : fn<float, 64>(a, st);        \
    default: return dt == MHLA_BF16 ? fn<__nv_bfloat16, 128>(a, st) : fn<float, 128>(a, st);      \
  }

}  // namespace

cudaError_t cross_join_launch(const CrossArgs& a, bool backward, cudaStream_t st) {
  const int per = ((a.d * a.d + a.d) / 4 + kJoinRuns - 1) / kJoinRuns;
  const int B = backward ? a.qs.B : a.ks.B;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)((long long)B * a.Hk * per));
  c.blockDim = dim3(kJoinThreads);
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, cross_join_kernel, a, (int)backward);
  note_launch();
  return e;
}

cudaError_t simt_cross_states_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st) { CROSS_DISPATCH(states_t) }
cudaError_t simt_cross_read_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st) { CROSS_DISPATCH(read_t) }
cudaError_t simt_cross_backward_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st) { CROSS_DISPATCH(backward_t) }
cudaError_t cross_step_launch(const CrossArgs& a, mhla_dtype dt, cudaStream_t st) { CROSS_DISPATCH(step_t) }

}  // namespace mhla
