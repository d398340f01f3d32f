// Retention passes of fp32 tensors on the SIMT cores, the scan over segments, the single-token step
// and the copies between state slots.  The mathematics is in retention.h.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "retention.cuh"

namespace mhla {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 64;  // tokens of a chunk

// ================================================================ passes
// A block takes one segment of one head and ES columns of c: per chunk of 64 tokens
//   P = (A B^T) gamma^(t-s), masked;  out = P C + gamma^(i+1) A X;  X = gamma^len X + (B w)^T C,
// w_s = gamma^(len-1-s), with X [D][ES] and the chunk's A, B, C and P in shared memory and 4 x 4 (X: up to 8 x 4)
// register tiles; the masked half of the first two products is left out by blocks of 4 rows.  With SUM only X is
// formed: the segment's own sum.  Bound by shared memory: 8 loads of 16 bytes a lane, four cycles each, for 32 multiply-adds of pairs (12 heads of 4096
// tokens, d = 64: 80 us; FMA units 30 % busy).  The multiply-adds go in pairs; the next chunk's rows are on their way in
// registers while X is computed.  (C and X transposed, so that pairs lie side by side, cost more in their stores and
// uneven loads than it saved: 124 us against 97.)
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
  static constexpr int kPerSm = D == 128 ? 1 : 2;
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

// A chunk's rows of one operand, W columns from c0, on their way to shared memory: fetched into registers (zeros
// behind the sequence), later stored with phi applied.
template <int W, int LDS>
struct Fetch {
  static constexpr int kN = kTok * (W / 4) / kThreads;
  float4 v[kN];
  __device__ __forceinline__ void load(const RetTensor& t, long long base, int row, int len, int c0) {
    const float* src = static_cast<const float*>(t.p) + base + (long long)row * t.sn + c0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = threadIdx.x + i * kThreads, r = at / (W / 4), c = (at % (W / 4)) * 4;
      v[i] = r < len ? *reinterpret_cast<const float4*>(src + (long long)r * t.sn + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(float* dst, int feature, int len) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = threadIdx.x + i * kThreads, r = at / (W / 4), c = (at % (W / 4)) * 4;
      if (feature != kFeatIdentity && r < len)
        v[i] = make_float4(ret_phi(v[i].x, feature), ret_phi(v[i].y, feature), ret_phi(v[i].z, feature),
                           ret_phi(v[i].w, feature));
      *reinterpret_cast<float4*>(dst + r * LDS + c) = v[i];
    }
  }
};

// acc[i][0 .. 3] += sum over k of a[i][k] b[k][0 .. 3], k = 0 .. n - 1 (n a multiple of 4): rows of a LDA apart, of b LDB.
template <int R, int LDA, int LDB>
__device__ __forceinline__ void outer_rows(float2 (&acc)[R][2], const float* a, const float* b, int k0, int n) {
#pragma unroll 4
  for (int k = k0; k < n; k += 4) {
    float4 fa[R];
#pragma unroll
    for (int i = 0; i < R; ++i) fa[i] = *reinterpret_cast<const float4*>(a + i * LDA + k);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4 v = *reinterpret_cast<const float4*>(b + (k + u) * LDB);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = u == 0 ? fa[i].x : u == 1 ? fa[i].y : u == 2 ? fa[i].z : fa[i].w;
        acc[i][0] = fma2(make_float2(w, w), make_float2(v.x, v.y), acc[i][0]);
        acc[i][1] = fma2(make_float2(w, w), make_float2(v.z, v.w), acc[i][1]);
      }
    }
  }
}

template <int D, bool SUM>
__global__ void __launch_bounds__(kThreads, SimtTile<D>::kPerSm) retention_simt_kernel(const __grid_constant__ RetArgs a) {
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
  if (sg.seq < 0) {
    grid_dependency_wait();  // (a kernel does not end before those it may overlap)
    return;
  }
  const int reverse = p.reverse;
  if (SUM) inner_segment(a, sg, reverse);
  const int e0 = blockIdx.y * C::ES;
  const long long ba = ret_base(a, p.a, sg.seq, h), bb = ret_base(a, p.b, sg.seq, h), bc = ret_base(a, p.c, sg.seq, h);
  const int nch = (sg.len + kTok - 1) / kTok;
  Fetch<D, C::LD> fA, fB;
  Fetch<C::ES, C::ES> fC;
  auto fetch = [&](int it) {
    const int ch = reverse ? nch - 1 - it : it;
    const int row = sg.row0 + ch * kTok, len = min(kTok, sg.len - ch * kTok);
    if (!SUM) fA.load(p.a, ba, row, len, 0);
    fB.load(p.b, bb, row, len, 0);
    fC.load(p.c, bc, row, len, e0);
  };
  fetch(0);
  const float lg = decay_log2(a.gamma[h]);
  const int tx = tid % C::NX, ty = tid / C::NX;
  float* seg = a.seg == nullptr ? nullptr : a.seg + (((size_t)p.sum * a.W + sg.w0 + sg.seg) * a.H + h) * (D * D);
  int slot = -1;
  if (!SUM && a.states != nullptr) slot = ret_slot(a.slots, a.n_slots, sg.seq);
  {
    const float* src = SUM ? nullptr : entering_state(a, p, sg, h, slot);
    const bool tr = !SUM && sg.nseg > 1 && p.sum_t;
    if (!SUM) grid_dependency_wait();
#pragma unroll 8
    for (int i = tid; i < D * C::ES; i += kThreads) {
      const int r = i / C::ES, e = e0 + i % C::ES;
      sX[i] = src == nullptr ? 0.f : __ldcg(src + (tr ? e * D + r : r * D + e));
    }
  }
  for (int it = 0; it < nch; ++it) {
    const int ch = reverse ? nch - 1 - it : it;
    const int row = sg.row0 + ch * kTok, len = min(kTok, sg.len - ch * kTok);
    __syncthreads();
    if (!SUM) fA.store(sA, p.a.feature, len);
    fB.store(sB, p.b.feature, len);
    fC.store(sC, p.c.feature, len);
    if (tid < kTok) sW[tid] = tid < len ? decay_pow(lg, reverse ? tid : len - 1 - tid) : 0.f;
    __syncthreads();
    if (!SUM) {
      // P: 4 rows t, 4 columns s = tp + 16 j; blocks wholly masked stay zero
      const int tp = tid & 15, t0 = 4 * (tid >> 4);
      float2 acc[4][4] = {};
      auto scores = [&](auto lo, auto hi) {  // columns j = lo .. hi - 1
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
          float4 fa[4], fb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) fa[i] = *reinterpret_cast<const float4*>(sA + (t0 + i) * C::LD + c);
#pragma unroll
          for (int j = lo(); j < hi(); ++j) fb[j] = *reinterpret_cast<const float4*>(sB + (tp + 16 * j) * C::LD + c);
#pragma unroll
          for (int j = lo(); j < hi(); ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[i][j] = fma2(make_float2(fa[i].x, fa[i].y), make_float2(fb[j].x, fb[j].y), acc[i][j]);
              acc[i][j] = fma2(make_float2(fa[i].z, fa[i].w), make_float2(fb[j].z, fb[j].w), acc[i][j]);
            }
        }
      };
      // a warp holds 8 rows, so these branches are its own: half of the columns, or all
      using I0 = std::integral_constant<int, 0>;
      using I2 = std::integral_constant<int, 2>;
      using I4 = std::integral_constant<int, 4>;
      if (t0 < kTok / 2) {
        if (reverse)
          scores(I0(), I4());
        else
          scores(I0(), I2());
      } else {
        if (reverse)
          scores(I2(), I4());
        else
          scores(I0(), I4());
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + i, s = tp + 16 * j, n = reverse ? s - t : t - s;
          sP[t * C::LP + s] = n >= 0 && s < len ? (acc[i][j].x + acc[i][j].y) * decay_pow(lg, n) : 0.f;
        }
      __syncthreads();
      // out = P C + gamma^(i+1) A X
      float2 in[C::RO][2] = {}, ac[C::RO][2] = {};
      const int r0 = C::RO * ty, first = r0 & ~3, last = (r0 + C::RO + 3) & ~3;  // columns of P that are not all masked
      outer_rows<C::RO, C::LP, C::ES>(in, sP + r0 * C::LP, sC + 4 * tx, reverse ? first : 0, reverse ? kTok : last);
      outer_rows<C::RO, C::LD, C::ES>(ac, sA + r0 * C::LD, sX + 4 * tx, 0, D);
#pragma unroll
      for (int i = 0; i < C::RO; ++i) {
        const int t = r0 + i;
        if (t >= len) continue;
        const float w = decay_pow(lg, reverse ? len - t : t + 1);
        float o[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[2 * x] = a.scale * fmaf(w, ac[i][x].x, in[i][x].x);
          o[2 * x + 1] = a.scale * fmaf(w, ac[i][x].y, in[i][x].y);
        }
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
    if (it + 1 < nch) fetch(it + 1);
    // X = gamma^len X + (B w)^T C: rows RS ty .., columns 4 tx ..
    if (C::RS * ty < D) {
      float2 acc[C::RS][2];
      const float w0 = decay_pow(lg, len);
#pragma unroll
      for (int i = 0; i < C::RS; ++i) {
        const float4 u = *reinterpret_cast<const float4*>(sX + (C::RS * ty + i) * C::ES + 4 * tx);
        acc[i][0] = make_float2(w0 * u.x, w0 * u.y);
        acc[i][1] = make_float2(w0 * u.z, w0 * u.w);
      }
#pragma unroll 8
      for (int s = 0; s < kTok; ++s) {  // (rows behind the sequence are zeros)
        const float w = sW[s];
        const float4 v = *reinterpret_cast<const float4*>(sC + s * C::ES + 4 * tx);
        const float2 v0 = mul2(make_float2(w, w), make_float2(v.x, v.y)), v1 = mul2(make_float2(w, w), make_float2(v.z, v.w));
        float b[C::RS];
        if constexpr (C::RS % 4 == 0) {
#pragma unroll
          for (int i = 0; i < C::RS; i += 4) load_row_piece<float>(sB + s * C::LD + C::RS * ty + i, b + i);
        } else {
#pragma unroll
          for (int i = 0; i < C::RS; ++i) b[i] = sB[s * C::LD + C::RS * ty + i];
        }
#pragma unroll
        for (int i = 0; i < C::RS; ++i) {
          acc[i][0] = fma2(make_float2(b[i], b[i]), v0, acc[i][0]);
          acc[i][1] = fma2(make_float2(b[i], b[i]), v1, acc[i][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < C::RS; ++i)
        *reinterpret_cast<float4*>(sX + (C::RS * ty + i) * C::ES + 4 * tx) =
            make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
    }
  }
  __syncthreads();
  float* dst = SUM ? seg : slot >= 0 && sg.seg == sg.nseg - 1 ? a.states + ((size_t)slot * a.H + h) * (D * D) : nullptr;
  if (dst != nullptr)
#pragma unroll 4
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
// many heads (most packed sequences have one segment, and their blocks end at once), single elements where few.  Whole
// calls, by fours and by ones: 24 packed sequences x 16 heads in segments of 2048 tokens 151 and 181 us, 64 heads of 8192
// tokens 101 and 100; 8 heads of 65,536 165 and 152, gradients of 8 heads of 500 tokens fp32 32.8 and 30.7.  Bound by the
// loads' latency: 8 us.
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
  const int nseg = sg.nseg, len = sg.all;
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
  float* w = a.seg + (((size_t)set * a.W + sg.w0) * a.H + h) * n + e0;
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
// shuffles and shared memory.  At most 16 elements a thread, so that six blocks fit on an SM: d = 128 takes its columns
// in four blocks.  Bound by the state's traffic (8 d^2 bytes a head): 256 x 16 heads, d = 64, 24.6 us = 5.5 TB/s, 82 %
// of a copy's rate; a few rows by the launch: 4 us for 3 x 16 heads, d = 128.
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
// A block takes a part of every slot at a time: it reads that part of all sources into shared memory, then writes all
// targets, so that a slot may be source and target of different pairs in any order.  A source of several pairs is read
// once.  Asynchronous copies keep a part in flight, and two blocks an SM take parts until none is left, one reading
// while the other writes; the pairs are compared once a block (with a block a part that was half of the time: 160
// moves of 1 MB took 121 us, now 64: 325 MB at 5.1 TB/s, 75 % of a copy's rate).
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
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int s = src[i], d = dst[i];
    sdst[i] = d;
    ssrc[i] = d < 0 || d >= n_slots || s >= n_slots ? n_slots : max(s, -1);
  }
  __syncthreads();
  for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) {  // a warp a pair
    const int d = sdst[i], s = ssrc[i];
    int l = i;
    bool later = s == n_slots;
    for (int j = threadIdx.x & 31; j < n; j += 32) {
      const int sj = ssrc[j];
      if (sj == s) l = min(l, j);
      later |= j > i && sdst[j] == d && sj != n_slots;  // of several pairs with one target the last counts
    }
    l = __reduce_min_sync(0xffffffffu, l);
    later = __any_sync(0xffffffffu, later);
    if ((threadIdx.x & 31) == 0) lead[i] = later ? -1 - l : l;  // negative: nothing to write, others may use its part
  }
  __syncthreads();
  const int parts = (int)((slot_elems + (4ll << log_r4) - 1) >> (log_r4 + 2));
  for (int part = blockIdx.x; part < parts; part += gridDim.x) {
    const long long e0 = (long long)part << (log_r4 + 2);
    const int w4 = (int)min((long long)r4, (slot_elems - e0) / 4);
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
    __syncthreads();
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
  while (log_r4 < 8 && ((size_t)n << (log_r4 + 1)) * 16 <= (size_t)kCopyBytes && (slot_elems >> (log_r4 + 3)) >= 4 * kRetSms)
    ++log_r4;
  const size_t bytes = ((size_t)n << log_r4) * 16 + (size_t)n * 3 * sizeof(int);
  static SmemOptIn opt;
  cudaError_t e = opt.ensure((const void*)retention_copy_kernel, 227 * 1024);
  if (e != cudaSuccess) return e;
  const long long r = 4ll << log_r4, parts = (slot_elems + r - 1) / r;
  const long long per_sm = std::max<long long>(2, std::min<long long>(8, (long long)(200 * 1024 / bytes)));
  retention_copy_kernel<<<(unsigned)std::min<long long>(parts, kRetSms * per_sm), kThreads, bytes, st>>>(
      states, slot_elems, n_slots, src, dst, n, log_r4);
  note_launch();
  return cudaGetLastError();
}

}  // namespace mhla
