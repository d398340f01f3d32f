// Retention passes of fp32 tensors on the SIMT cores, the scan over segments, the single-token step
// and the copies between state slots.  The mathematics is in retention.h.
#include <algorithm>

#include "internal.h"
#include "retention.cuh"

namespace mhla {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 64;  // tokens of a chunk

// ================================================================ passes
// A block takes one segment of one head and ES columns of c: per chunk of 64 tokens
//   P = (A B^T) gamma^(t-s), masked;  out = P C + gamma^(i+1) A X;  X = gamma^len X + (B w)^T C,
// w_s = gamma^(len-1-s), with X [D][ES] and the chunk's A, B, C and P in shared memory and 4 x 4 (X: up
// to 8 x 4) register tiles.  With SUM only X is formed: the segment's own sum.
template <int D>
struct SimtTile {
  static constexpr int ES = D < 64 ? D : 64;
  static constexpr int LD = D + 4;           // row of A and B: lanes on neighbouring rows hit other banks
  static constexpr int LP = kTok + 4;
  static constexpr int NX = ES / 4, NY = kThreads / NX;
  static constexpr int RO = kTok / NY;       // rows of out a thread holds
  static constexpr int RS = D >= NY ? D / NY : 1;
  static constexpr int kFloats = 2 * kTok * LD + kTok * ES + D * ES + kTok * LP + kTok;
  static constexpr size_t kBytes = kFloats * sizeof(float);
};

template <typename T>
__device__ __forceinline__ void load_row_piece(const T* p, float* f);
template <>
__device__ __forceinline__ void load_row_piece<float>(const float* p, float* f) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
}
template <>
__device__ __forceinline__ void load_row_piece<__nv_bfloat16>(const __nv_bfloat16* p, float* f) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xffff0000u);
}

// Rows 0 .. len - 1, columns c0 .. c0 + W - 1 of a tensor from row `row`, widened, phi applied; zeros behind.
template <int W, int LDS>
__device__ __forceinline__ void load_tile(float* dst, const RetTensor& t, long long base, int row, int len, int c0) {
  const float* src = static_cast<const float*>(t.p) + base + (long long)row * t.sn + c0;
  for (int i = threadIdx.x; i < kTok * (W / 4); i += kThreads) {
    const int r = i / (W / 4), c = (i % (W / 4)) * 4;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < len) {
      load_row_piece<float>(src + (long long)r * t.sn + c, f);
      if (t.feature != kFeatIdentity)
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = ret_phi(f[x], t.feature);
    }
    *reinterpret_cast<float4*>(dst + r * LDS + c) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

template <int D, bool SUM>
__global__ void __launch_bounds__(kThreads) retention_simt_kernel(const __grid_constant__ RetArgs a) {
  using C = SimtTile<D>;
  extern __shared__ float4 smem4[];
  float* sA = reinterpret_cast<float*>(smem4);
  float* sB = sA + kTok * C::LD;
  float* sC = sB + kTok * C::LD;
  float* sX = sC + kTok * C::ES;
  float* sP = sX + D * C::ES;
  float* sW = sP + kTok * C::LP;
  __shared__ int scratch[2 * kOrdered];
  const int tid = threadIdx.x;
  launch_dependents();
  const int h = blockIdx.x % a.H, g = blockIdx.x / a.H;
  int z = blockIdx.z;
  if (SUM)  // the pass that makes set z
    for (int i = 0; i < a.npass; ++i)
      if (a.pass[i].sum == (int)blockIdx.z && !a.pass[i].sum_t) z = i;
  const RetPass& p = a.pass[z];
  Segment sg = find_segment(a, g, SUM ? SEG_INNER : SEG_ALL, scratch);
  if (sg.seq < 0) return;
  if (SUM) inner_segment(a, sg, p.reverse);
  const int e0 = blockIdx.y * C::ES;
  const float lg = decay_log2(a.gamma[h]);
  const int tx = tid % C::NX, ty = tid / C::NX;
  float* seg = a.seg == nullptr ? nullptr : a.seg + (((size_t)p.sum * a.G + sg.g0 + sg.seg) * a.H + h) * (D * D);
  if (SUM)
    for (int i = tid; i < D * C::ES; i += kThreads) sX[i] = 0.f;
  int slot = -1;
  if (!SUM) {
    if (a.states != nullptr) slot = ret_slot(a.slots, a.n_slots, sg.seq);
    const float* src = entering_state(a, p, sg, h, slot);
    const bool tr = sg.nseg > 1 && p.sum_t;
    grid_dependency_wait();
    for (int i = tid; i < D * C::ES; i += kThreads) {
      const int r = i / C::ES, e = e0 + i % C::ES;
      sX[i] = src == nullptr ? 0.f : __ldcg(src + (tr ? e * D + r : r * D + e));
    }
  }
  const long long ba = ret_base(a, p.a, sg.seq, h), bb = ret_base(a, p.b, sg.seq, h), bc = ret_base(a, p.c, sg.seq, h);
  const int nch = (sg.len + kTok - 1) / kTok;
  for (int it = 0; it < nch; ++it) {
    const int ch = p.reverse ? nch - 1 - it : it;
    const int row = sg.row0 + ch * kTok, len = min(kTok, sg.len - ch * kTok);
    __syncthreads();
    if (!SUM) load_tile<D, C::LD>(sA, p.a, ba, row, len, 0);
    load_tile<D, C::LD>(sB, p.b, bb, row, len, 0);
    load_tile<C::ES, C::ES>(sC, p.c, bc, row, len, e0);
    if (tid < kTok) sW[tid] = tid < len ? decay_pow(lg, p.reverse ? tid : len - 1 - tid) : 0.f;
    __syncthreads();
    if (!SUM) {
      // P: 4 rows t, 4 columns s = tp + 16 j
      const int tp = tid & 15, tr = tid >> 4;
      float acc[4][4] = {};
      for (int c = 0; c < D; c += 4) {
        float4 fa[4], fb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) fa[i] = *reinterpret_cast<const float4*>(sA + (4 * tr + i) * C::LD + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) fb[j] = *reinterpret_cast<const float4*>(sB + (tp + 16 * j) * C::LD + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j] = fmaf(fa[i].x, fb[j].x, acc[i][j]);
            acc[i][j] = fmaf(fa[i].y, fb[j].y, acc[i][j]);
            acc[i][j] = fmaf(fa[i].z, fb[j].z, acc[i][j]);
            acc[i][j] = fmaf(fa[i].w, fb[j].w, acc[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 4 * tr + i, s = tp + 16 * j, n = p.reverse ? s - t : t - s;
          sP[t * C::LP + s] = n >= 0 && s < len ? acc[i][j] * decay_pow(lg, n) : 0.f;
        }
      __syncthreads();
      // out = P C + gamma^(i+1) A X
      float in[C::RO][4] = {}, ac[C::RO][4] = {};
      for (int s = 0; s < kTok; s += 4) {
        float4 fp[C::RO];
#pragma unroll
        for (int i = 0; i < C::RO; ++i) fp[i] = *reinterpret_cast<const float4*>(sP + (C::RO * ty + i) * C::LP + s);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 v = *reinterpret_cast<const float4*>(sC + (s + u) * C::ES + 4 * tx);
#pragma unroll
          for (int i = 0; i < C::RO; ++i) {
            const float w = u == 0 ? fp[i].x : u == 1 ? fp[i].y : u == 2 ? fp[i].z : fp[i].w;
            in[i][0] = fmaf(w, v.x, in[i][0]);
            in[i][1] = fmaf(w, v.y, in[i][1]);
            in[i][2] = fmaf(w, v.z, in[i][2]);
            in[i][3] = fmaf(w, v.w, in[i][3]);
          }
        }
      }
      for (int c = 0; c < D; c += 4) {
        float4 fa[C::RO];
#pragma unroll
        for (int i = 0; i < C::RO; ++i) fa[i] = *reinterpret_cast<const float4*>(sA + (C::RO * ty + i) * C::LD + c);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 v = *reinterpret_cast<const float4*>(sX + (c + u) * C::ES + 4 * tx);
#pragma unroll
          for (int i = 0; i < C::RO; ++i) {
            const float w = u == 0 ? fa[i].x : u == 1 ? fa[i].y : u == 2 ? fa[i].z : fa[i].w;
            ac[i][0] = fmaf(w, v.x, ac[i][0]);
            ac[i][1] = fmaf(w, v.y, ac[i][1]);
            ac[i][2] = fmaf(w, v.z, ac[i][2]);
            ac[i][3] = fmaf(w, v.w, ac[i][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < C::RO; ++i) {
        const int t = C::RO * ty + i;
        if (t >= len) continue;
        const float w = decay_pow(lg, p.reverse ? len - t : t + 1);
        float o[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) o[x] = a.scale * fmaf(w, ac[i][x], in[i][x]);
        if (p.x.p != nullptr) {
          float fx[4];
          load_row_piece<float>(static_cast<const float*>(p.x.p) + ret_base(a, p.x, sg.seq, h) + (long long)(row + t) * p.x.sn +
                                e0 + 4 * tx, fx);
#pragma unroll
          for (int x = 0; x < 4; ++x) o[x] *= ret_dphi(fx[x], p.x.feature);
        }
        float* dst = static_cast<float*>(const_cast<void*>(p.out.p)) + ret_base(a, p.out, sg.seq, h) +
                     (long long)(row + t) * p.out.sn + e0 + 4 * tx;
        *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
      }
      __syncthreads();  // every A X has read X
    }
    // X = gamma^len X + (B w)^T C: rows RS ty .., columns 4 tx ..
    if (C::RS * ty < D) {
      float acc[C::RS][4];
      const float w0 = decay_pow(lg, len);
#pragma unroll
      for (int i = 0; i < C::RS; ++i) {
        const float4 u = *reinterpret_cast<const float4*>(sX + (C::RS * ty + i) * C::ES + 4 * tx);
        acc[i][0] = w0 * u.x;
        acc[i][1] = w0 * u.y;
        acc[i][2] = w0 * u.z;
        acc[i][3] = w0 * u.w;
      }
      for (int s = 0; s < len; ++s) {
        const float w = sW[s];
        float4 v = *reinterpret_cast<const float4*>(sC + s * C::ES + 4 * tx);
        v.x *= w;
        v.y *= w;
        v.z *= w;
        v.w *= w;
#pragma unroll
        for (int i = 0; i < C::RS; ++i) {
          const float b = sB[s * C::LD + C::RS * ty + i];
          acc[i][0] = fmaf(b, v.x, acc[i][0]);
          acc[i][1] = fmaf(b, v.y, acc[i][1]);
          acc[i][2] = fmaf(b, v.z, acc[i][2]);
          acc[i][3] = fmaf(b, v.w, acc[i][3]);
        }
      }
#pragma unroll
      for (int i = 0; i < C::RS; ++i)
        *reinterpret_cast<float4*>(sX + (C::RS * ty + i) * C::ES + 4 * tx) =
            make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    }
  }
  __syncthreads();
  float* dst = SUM ? seg : slot >= 0 && sg.seg == sg.nseg - 1 ? a.states + ((size_t)slot * a.H + h) * (D * D) : nullptr;
  if (dst != nullptr)
    for (int i = tid; i < D * C::ES; i += kThreads) dst[(i / C::ES) * D + e0 + i % C::ES] = sX[i];
}

template <int D>
cudaError_t launch_passes(const RetArgs& a, cudaStream_t st) {
  using C = SimtTile<D>;
  static SmemOptIn opt_sum, opt_out;
  cudaError_t e = opt_sum.ensure((const void*)retention_simt_kernel<D, true>, (int)C::kBytes);
  if (e == cudaSuccess) e = opt_out.ensure((const void*)retention_simt_kernel<D, false>, (int)C::kBytes);
  if (e != cudaSuccess) return e;
  dim3 grid((unsigned)((long long)a.inner * a.H), D / C::ES, a.nsum);
  if (a.seg != nullptr) {
    retention_simt_kernel<D, true><<<grid, kThreads, C::kBytes, st>>>(a);
    note_launch();
    e = retention_scan_launch(a, st);
    if (e != cudaSuccess) return e;
  }
  grid.x = (unsigned)((long long)a.G * a.H);
  grid.z = a.npass;
  return launch_dependent(retention_simt_kernel<D, false>, grid, kThreads, C::kBytes, st, a.seg != nullptr, a);
}

// ================================================================ scan
// A thread carries E groups of V elements of a head's state over its sequence's segments, in the pass's direction:
// the slot of a segment holds the segment's own sum before, the state entering it after.  V = E = 4 where there are
// many heads (most packed sequences have one segment, and their blocks end at once), single elements where few.
template <int V, int E>
__global__ void __launch_bounds__(kThreads) retention_scan_kernel(const __grid_constant__ RetArgs a) {
  __shared__ int scratch[2 * kOrdered];
  launch_dependents();
  const int h = blockIdx.x % a.H, set = blockIdx.z;
  int ps = 0;
  for (int i = 0; i < a.npass; ++i)
    if (a.pass[i].sum == set && !a.pass[i].sum_t) ps = i;
  const bool reverse = a.pass[ps].reverse != 0;
  const Segment sg = find_segment(a, blockIdx.x / a.H, SEG_SPLIT, scratch);
  const int slot = sg.seq >= 0 && a.load && a.states != nullptr ? ret_slot(a.slots, a.n_slots, sg.seq) : -1;
  grid_dependency_wait();  // the sums are there
  if (sg.seq < 0) return;
  const int nseg = sg.nseg, g0 = sg.g0, len = sg.all;
  const int n = a.d * a.d, e0 = (blockIdx.y * E * kThreads + threadIdx.x) * V;
  const float lg = decay_log2(a.gamma[h]);
  const float wfull = decay_pow(lg, a.L), wlast = decay_pow(lg, len - (nseg - 1) * a.L);
  const size_t step = (size_t)a.H * n;
  struct alignas(4 * V) Vec {
    float v[V];
  };
  Vec x[E] = {};
  if (slot >= 0)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (e0 + i * kThreads * V < n)
        x[i] = *reinterpret_cast<const Vec*>(a.states + ((size_t)slot * a.H + h) * n + e0 + i * kThreads * V);
  float* w = a.seg + (((size_t)set * a.G + g0) * a.H + h) * n + e0;
  constexpr int kAhead = E == 1 ? 16 : 2;  // segments loaded ahead
  for (int j0 = 0; j0 < nseg; j0 += kAhead) {
    Vec u[kAhead][E];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = j0 + j;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        u[j][i] = Vec{};
        if (k < nseg - 1 && e0 + i * kThreads * V < n)
          u[j][i] = *reinterpret_cast<const Vec*>(w + (size_t)(reverse ? nseg - 1 - k : k) * step + i * kThreads * V);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = j0 + j;
      if (k >= nseg) break;
      const int sgm = reverse ? nseg - 1 - k : k;
      const float wl = sgm == nseg - 1 ? wlast : wfull;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (e0 + i * kThreads * V < n) *reinterpret_cast<Vec*>(w + (size_t)sgm * step + i * kThreads * V) = x[i];
#pragma unroll
        for (int q = 0; q < V; ++q) x[i].v[q] = fmaf(wl, x[i].v[q], u[j][i].v[q]);
      }
    }
  }
}

// ================================================================ single-token step
// S = gamma S + phi(k) v^T, out = scale phi(q) S.  A block takes ES columns of a (row, head) state; a thread RPT
// neighbouring rows of four columns, all its loads issued before the first use; the columns' sums over c go through
// shuffles and shared memory.  Bound by the state's traffic (8 d^2 bytes a head).
template <typename T, int N>
__device__ __forceinline__ void load_values(const T* p, float* f) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) load_row_piece<T>(p + i, f + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f(p[i]);
  }
}

template <typename T, int D, int ES>
__global__ void __launch_bounds__(kThreads, 6) retention_step_kernel(int H, RetTensor q, RetTensor k, RetTensor v,
                                                                     RetTensor out, const float* gamma, float scale,
                                                                     float* states, const int* slots, int n_slots) {
  constexpr int NG = ES / 4, RT = kThreads / NG, RPT = D >= RT ? D / RT : 1;
  __shared__ float4 red[kThreads / 32][NG];
  const int tid = threadIdx.x, cg = tid % NG, r0 = (tid / NG) * RPT;
  const int h = blockIdx.x % H, b = blockIdx.x / H, e0 = blockIdx.y * ES + 4 * cg;
  const int s0 = slots == nullptr ? b : slots[b];
  const bool in = s0 >= 0 && s0 < n_slots;
  const bool act = r0 < D;
  float4* S = reinterpret_cast<float4*>(states + ((size_t)(in ? s0 : 0) * H + h) * (D * D) + (act ? r0 : 0) * D + e0);
  float4 x[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) x[i] = in && act ? __ldcs(S + i * (D / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
  float fv[4], fq[RPT], fk[RPT];
  load_row_piece<T>(static_cast<const T*>(v.p) + b * v.sb + h * v.sh + e0, fv);
  load_values<T, RPT>(static_cast<const T*>(q.p) + b * q.sb + h * q.sh + (act ? r0 : 0), fq);
  load_values<T, RPT>(static_cast<const T*>(k.p) + b * k.sb + h * k.sh + (act ? r0 : 0), fk);
  const float gm = gamma[h];
  if (ret_slot(slots, n_slots, b) < 0) return;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const float kk = ret_phi(fk[i], k.feature), qq = act ? ret_phi(fq[i], q.feature) : 0.f;
    x[i].x = fmaf(gm, x[i].x, kk * fv[0]);
    x[i].y = fmaf(gm, x[i].y, kk * fv[1]);
    x[i].z = fmaf(gm, x[i].z, kk * fv[2]);
    x[i].w = fmaf(gm, x[i].w, kk * fv[3]);
    if (act) __stcs(S + i * (D / 4), x[i]);
    if (act) {
      y.x = fmaf(qq, x[i].x, y.x);
      y.y = fmaf(qq, x[i].y, y.y);
      y.z = fmaf(qq, x[i].z, y.z);
      y.w = fmaf(qq, x[i].w, y.w);
    }
  }
#pragma unroll
  for (int o = NG; o < 32; o <<= 1) {
    y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
    y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
    y.z += __shfl_xor_sync(0xffffffffu, y.z, o);
    y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
  }
  if ((tid & 31) < NG) red[tid >> 5][cg] = y;
  __syncthreads();
  if (tid < ES) {  // a column a thread
    const float* f = reinterpret_cast<const float*>(red) + tid;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += f[w * ES];
    static_cast<T*>(const_cast<void*>(out.p))[b * out.sb + h * out.sh + blockIdx.y * ES + tid] = from_f<T>(scale * s);
  }
}

template <typename T, int D, int ES>
cudaError_t launch_step(int B, int H, const RetTensor& q, const RetTensor& k, const RetTensor& v, const RetTensor& out,
                        const float* gamma, float scale, float* states, const int* slots, int n_slots,
                        cudaStream_t st) {
  retention_step_kernel<T, D, ES><<<dim3((unsigned)(B * H), D / ES), kThreads, 0, st>>>(H, q, k, v, out, gamma, scale,
                                                                                       states, slots, n_slots);
  note_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_d(int B, int H, int d, const RetTensor& q, const RetTensor& k, const RetTensor& v,
                          const RetTensor& out, const float* gamma, float scale, float* states, const int* slots,
                          int n_slots, cudaStream_t st) {
  switch (d) {
    case 16: return launch_step<T, 16, 16>(B, H, q, k, v, out, gamma, scale, states, slots, n_slots, st);
    case 32: return launch_step<T, 32, 32>(B, H, q, k, v, out, gamma, scale, states, slots, n_slots, st);
    case 64: return launch_step<T, 64, 64>(B, H, q, k, v, out, gamma, scale, states, slots, n_slots, st);
    default: return launch_step<T, 128, 32>(B, H, q, k, v, out, gamma, scale, states, slots, n_slots, st);
  }
}

// ================================================================ state copies
// A block takes R floats of every slot: it reads them from all sources into shared memory, then writes all targets,
// so that a slot may be source and target of different pairs in any order.  A source of several pairs is read once.
// Bound by the traffic; asynchronous copies keep a block's whole part in flight.
constexpr int kCopyBytes = 100 * 1024;  // of shared memory a block, so that two are on an SM: one reads, one writes

__device__ __forceinline__ void copy_async16(void* smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
               : "memory");
}

__global__ void __launch_bounds__(kThreads) retention_copy_kernel(float* states, long long slot_elems, int n_slots,
                                                                  const int* src, const int* dst, int n, int log_r4) {
  extern __shared__ float4 buf[];
  const int r4 = 1 << log_r4;  // float4 of a part
  int* sdst = reinterpret_cast<int*>(buf + ((size_t)n << log_r4));
  int* ssrc = sdst + n;   // source; -1: zeros; n_slots: the pair does nothing
  int* lead = ssrc + n;   // the first pair of the same source, whose part of buf both use
  const long long e0 = (long long)blockIdx.x << (log_r4 + 2);
  const int w4 = (int)min((long long)r4, (slot_elems - e0) / 4);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int s = src[i], d = dst[i];
    sdst[i] = d;
    ssrc[i] = d < 0 || d >= n_slots || s >= n_slots ? n_slots : max(s, -1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int d = sdst[i], s = ssrc[i];
    int l = i, m = s == n_slots ? -1 : i;
    for (int j = 0; j < i; ++j)
      if (ssrc[j] == s) {
        l = j;
        break;
      }
    for (int j = i + 1; j < n && m >= 0; ++j)
      if (sdst[j] == d && ssrc[j] != n_slots) m = -1;  // of several pairs with one target the last counts
    lead[i] = m < 0 ? -1 - l : l;                      // negative: nothing to write (but others may use its part)
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n << log_r4; i += kThreads) {
    const int pr = i >> log_r4, c = i & (r4 - 1), s = ssrc[pr], l = lead[pr];
    if ((l == pr || l == -1 - pr) && s < n_slots && c < w4) {
      if (s < 0)
        buf[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      else
        copy_async16(buf + i, states + s * slot_elems + e0 + 4 * c);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  for (int i = threadIdx.x; i < n << log_r4; i += kThreads) {
    const int pr = i >> log_r4, c = i & (r4 - 1), l = lead[pr];
    if (l >= 0 && c < w4)
      __stcs(reinterpret_cast<float4*>(states + sdst[pr] * slot_elems + e0) + c, buf[((size_t)l << log_r4) + c]);
  }
}

}  // namespace

cudaError_t simt_retention_launch(const RetArgs& a, cudaStream_t st) {
  switch (a.d) {
    case 16: return launch_passes<16>(a, st);
    case 32: return launch_passes<32>(a, st);
    case 64: return launch_passes<64>(a, st);
    default: return launch_passes<128>(a, st);
  }
}

cudaError_t retention_scan_launch(const RetArgs& a, cudaStream_t st) {
  const int n = a.d * a.d, per = (long long)a.split * a.H * a.nsum >= 64 ? 16 : 1;  // elements of a thread
  const dim3 grid((unsigned)((long long)a.split * a.H), (n + per * kThreads - 1) / (per * kThreads), a.nsum);
  return per == 16 ? launch_dependent(retention_scan_kernel<4, 4>, grid, kThreads, 0, st, true, a)
                   : launch_dependent(retention_scan_kernel<1, 1>, grid, kThreads, 0, st, true, a);
}

cudaError_t retention_step_launch(int B, int H, int d, mhla_dtype dt, const RetTensor& q, const RetTensor& k,
                                  const RetTensor& v, const RetTensor& out, const float* gamma, float scale,
                                  float* states, const int* slots, int n_slots, cudaStream_t st) {
  return dt == MHLA_F32
             ? launch_step_d<float>(B, H, d, q, k, v, out, gamma, scale, states, slots, n_slots, st)
             : launch_step_d<__nv_bfloat16>(B, H, d, q, k, v, out, gamma, scale, states, slots, n_slots, st);
}

cudaError_t retention_copy_launch(float* states, long long slot_elems, int n_slots, const int* src, const int* dst,
                                  int n, cudaStream_t st) {
  // parts of 128 bytes to 4 KB: as much shared memory as two blocks an SM allow, but a few parts for every SM
  int log_r4 = 3;
  while (log_r4 < 8 && ((size_t)n << (log_r4 + 1)) * 16 <= (size_t)kCopyBytes && (slot_elems >> (log_r4 + 3)) >= 608)
    ++log_r4;
  const size_t bytes = ((size_t)n << log_r4) * 16 + (size_t)n * 3 * sizeof(int);
  static SmemOptIn opt;
  cudaError_t e = opt.ensure((const void*)retention_copy_kernel, 227 * 1024);
  if (e != cudaSuccess) return e;
  const long long r = 4ll << log_r4;
  retention_copy_kernel<<<(unsigned)((slot_elems + r - 1) / r), kThreads, bytes, st>>>(states, slot_elems, n_slots, src,
                                                                                       dst, n, log_r4);
  note_launch();
  return cudaGetLastError();
}

}  // namespace mhla
