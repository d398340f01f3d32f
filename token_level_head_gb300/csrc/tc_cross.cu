// Linear cross attention on the sm_103a tensor cores (bf16, d = 64 or 128): the same steps as the FP32 kernels'
// (cross_simt.cu), a tile of 128 tokens at a time.
//
//   states  D[e][c] += sum_t v[t][e] phi(k)[t][c]   (A = v, B = phi(k) as a sum of three bf16 numbers: S is an fp32
//           result), z in fp32 registers
//   read    y[t][e] = (sum_c phi(q)[t][c] S[c][e]) / den_t   (S as a sum of two bf16 numbers)
//   query   u[t][c] = sum_e dy[t][e] S[c][e], dS^T[e][c] += sum_t dy[t][e] w[t][c] with w = phi(q) / den; S (less a middle of
//           the values, `middle`) and w as sums of two bf16 numbers, as dq is a difference, dy as it is; dz in fp32
//   key     dv[t][e] = sum_c phi(k)[t][c] dS[c][e], dphi(k)[t][c] = sum_e v[t][e] dS[c][e] (dS as a sum of two)
//
// Bound: memory (2, 2, 3 and 4 tensors), next to it the instructions that take the features and turn tiles.  A block has a
// segment of a head and walks over its tiles: a warp of its own issues the copies (TMA, into the buffer that is free) and the
// MMAs, D / 8 warps take the features (a thread 32 columns of a row, in place in the 128-byte-swizzled tile), take the results
// from tensor memory and put them into the tile's buffer, whence TMA copies them out (a packed sequence's last tile: the warps,
// as its rows end within it).  Two blocks an SM for d = 64 (reads: three), one for d = 128, hide one another's waits.  Every
// wait is bounded (on time-out the block stops, sets the status word and drains what it has in flight).
// Measured in a graph: states and read of 8 x 6 heads, 4096 queries, 77 keys, d 64: 18 us; of 4 key heads of 65,536 keys, d 128,
// and 777 queries of 16 heads: 45 (3.1 TB/s); forward and gradients of 8 x 6 heads, 4096 queries, 2048 keys, d 64: 76 (2.7
// TB/s), of 8 x 8 heads, d 128: 227 (2.4 TB/s).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "cross.cuh"
#include "cross_ring.h"
#include "tc_common.cuh"
#include "tc_cross.h"

namespace mhla {
namespace {

using namespace tc;

constexpr int kT = 128;                       // tokens of a tile
constexpr int kAtom = kT * 128;               // bytes of 64 columns of a tile
constexpr uint64_t kWaitNs = 500000000ull;    // 0.5 s: a wait's default limit

template <int D>
struct Tc {
  static constexpr int kTile = kT * D * 2;    // bytes of a tile of tokens
  static constexpr int kMat = D * D * 2;      // of a d x d matrix
  static constexpr int kWork = 4 * D;         // threads that take features and results: a row 32 columns a thread
  static constexpr int kThreads = kWork + 32; // and a warp that issues the copies and the MMAs
  static constexpr int kCols = D / 32;        // threads of a row
};

struct Bars {
  uint64_t full[4];   // a tile's tensors landed (tx), by its buffer
  uint64_t ready[3];  // a tile's operands are written (the working warps)
  uint64_t mma[3];    // MMA commits
  uint64_t out[2];    // a tile's results lie in its place
  uint64_t ready2, mma2;
  unsigned long long wait_ns;
  unsigned* status;
  uint32_t tbase;
  int abort;
  int scratch;
  int issued, mmas, mmas2;  // by the issuing thread: tiles copied, commits (for the wind-down)
};

struct TcArgs {
  CrossArgs c;
  CUtensorMap a, b;            // the tile's tensors: states, key: k, v; read: q; query: q, dy
  CUtensorMap c_map, d_map;    // what is written: read: y; query: dq; key: dk, dv
  int a_h, a_b, b_h, b_b;      // whether the tensors have heads and batch entries (stride not 0)
  int c_h, c_b, d_h, d_b;
  unsigned long long wait_ns;
};

__device__ __forceinline__ bool aborted(const int* ab) { return *reinterpret_cast<const volatile int*>(ab) != 0; }
// (The global timer takes long to read, so the first tries, up to about 16 us, go without it; a diagnostic's short limit
// counts from the start.)
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Bars* b) {
  const unsigned long long limit = b->wait_ns;
  if (limit > 1000000ull)
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait_ns(bar, parity, 1000)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait_ns(bar, parity, 256)) return true;
    if (aborted(&b->abort)) return false;
    if (globaltimer_ns() - t0 > limit) break;
  }
  *reinterpret_cast<volatile int*>(&b->abort) = 1;
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars* b) {
  return mbar_test(bar, parity) || wait_slow(bar, parity, b);
}
// Short wait (10 ms at most), only while winding down.
__device__ __noinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_ns(bar, parity, 1000))
    if (globaltimer_ns() - t0 > 10000000ull) return;
}

// 16-byte piece j (columns 8 j ..) of row r of a tile of 64-column atoms of `rows` rows.
__device__ __forceinline__ uint4* piece(uint8_t* tile, int rows, int r, int j) {
  return reinterpret_cast<uint4*>(tile + (j >> 3) * (rows * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4));
}
// Eight columns as pairs.
__device__ __forceinline__ void unpack8(uint4 u, float2* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int m = 0; m < 4; ++m) f[m] = make_float2(__uint_as_float(w[m] << 16), __uint_as_float(w[m] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const float2* v) {
  return make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 r;
  asm("sub.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
// f - bf16(f) in place, given bf16(f) packed.
__device__ __forceinline__ void remainder8(float2* f, uint4 h) {
  float2 g[4];
  unpack8(h, g);
#pragma unroll
  for (int x = 0; x < 4; ++x) f[x] = sub2(f[x], g[x]);
}
// 16 columns of the thread's lane of tensor memory.
__device__ __forceinline__ void tmem_ld8(uint32_t at, float2* v) { tmem_ld16(at, reinterpret_cast<float*>(v)); }
// Eight fp32 values of shared memory.
__device__ __forceinline__ void load8(const float* p, float2* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(v + 2 * i) = *reinterpret_cast<const float4*>(p + 4 * i);
}

// phi and, from phi alone, phi'.
__device__ __forceinline__ float exp2_of(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
// cross_inverse by the hardware's reciprocal (within a step of 2^-23; not flushed: that of a den from 2^126 on is below the normal
// numbers, and y is not 0 there).
__device__ __forceinline__ float inverse(float den) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(den));
  return fabsf(den) < kLeastDen ? 0.f : r;
}
__device__ __forceinline__ float min_nan(float a, float b) {  // not-a-number stays
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
// exp(x), and x + 1 in its place where x > 0: a comparison and an addition under it.
__device__ __forceinline__ float elu1(float x) {
  float e = exp2_of(x * kLog2e);
  asm("{\n\t.reg .pred p;\n\tsetp.gt.f32 p, %1, 0f00000000;\n\t@p add.f32 %0, %1, 0f3F800000;\n\t}" : "+f"(e) : "f"(x));
  return e;
}
template <int F>
__device__ __forceinline__ float2 feature(float2 x) {
  if (F == MHLA_PHI_ELU1) return make_float2(elu1(x.x), elu1(x.y));
  if (F == MHLA_PHI_RELU) return make_float2(x.x != x.x ? x.x : fmaxf(x.x, 0.f), x.y != x.y ? x.y : fmaxf(x.y, 0.f));
  if (F == MHLA_PHI_EXP) return make_float2(exp2_of(x.x * kLog2e), exp2_of(x.y * kLog2e));
  return x;
}
template <int F>
__device__ __forceinline__ float2 slope(float2 phi) {
  if (F == MHLA_PHI_ELU1) return make_float2(min_nan(phi.x, 1.f), min_nan(phi.y, 1.f));
  if (F == MHLA_PHI_RELU) return make_float2(phi.x > 0.f ? 1.f : 0.f, phi.y > 0.f ? 1.f : 0.f);
  return F == MHLA_PHI_EXP ? phi : both(1.f);
}

// The start of a block: barriers, tensor memory, the maps; and then everything that the kernel before left.  Every kernel
// here is launched while the one before it in the stream drains (whichever that is), so nothing is read before.
__device__ __forceinline__ void setup(const TcArgs& p, Bars* b, uint32_t cols) {
  launch_dependents();
  if (threadIdx.x == 0) {
    for (uint64_t& f : b->full) mbar_init(&f, 1);
    for (uint64_t& m : b->mma) mbar_init(&m, 1);
    for (uint64_t& r : b->ready) mbar_init(&r, blockDim.x / 32 - 1);
    for (uint64_t& r : b->out) mbar_init(&r, blockDim.x / 32 - 1);
    mbar_init(&b->ready2, blockDim.x / 32 - 1);
    mbar_init(&b->mma2, 1);
    b->issued = b->mmas = b->mmas2 = 0;
    b->abort = 0;
    b->wait_ns = p.wait_ns;
    b->status = p.c.status;
    fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    tmem_alloc(&b->tbase, cols);
    tmem_relinquish();
  }
  if (threadIdx.x == 32) prefetch_tmap(&p.a);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
}
// A working warp has written its part of a tile's operands (and read what the next MMAs overwrite).
__device__ __forceinline__ void arrive(uint64_t* bar, int lane) {
  fence_proxy_async_smem();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// The end of a block: after an abort (one thread) short waits for the copies and MMAs in flight; then the columns are
// freed.  NB: buffers that the copies went to in turn, NM: barriers that the commits did.
template <int NB, int NM>
__device__ __forceinline__ void finish(Bars* b, uint32_t cols) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && aborted(&b->abort)) {
    for (int j = max(b->issued - NB, 0); j < b->issued; ++j) drain(&b->full[j % NB], (j / NB) & 1);
    for (int j = max(b->mmas - NM, 0); j < b->mmas; ++j) drain(&b->mma[j % NM], (j / NM) & 1);
    if (b->mmas2 > 0) drain(&b->mma2, (b->mmas2 - 1) & 1);
    atomicOr(b->status, 1u);
  }
  __syncthreads();
  if (threadIdx.x < 32) tmem_dealloc(b->tbase, cols);
}

// One thread: a tile of one tensor (its atoms of 64 columns one behind the other).
__device__ __forceinline__ void load_tile(uint8_t* to, const CUtensorMap* m, int row, int h, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %2, %4, %5}], [%6];" ::"r"(smem_u32(to)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(row), "r"(h), "r"(b), "r"(smem_u32(bar))
      : "memory");
}

// One thread: a tile's rows to memory (rows behind the tensor are not), and the wait until its place may be written again.
__device__ __forceinline__ void store_tile(const CUtensorMap* m, uint8_t* from, int row, int h, int b) {
  asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %1, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(0), "r"(row), "r"(h), "r"(b), "r"(smem_u32(from))
               : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A d x d fp32 matrix [r][c] as the working threads hold it: eight columns of a row, the same columns in every row of a thread.
template <int D>
struct Matrix {
  static constexpr int N = D * D / 8 / Tc<D>::kWork, P = D / 8;  // pieces of a thread, of a row
  float2 f[N][4];
  static __device__ __forceinline__ int row(int n) { return ((int)threadIdx.x + n * Tc<D>::kWork) / P; }
  static __device__ __forceinline__ int piece_of_row() { return (int)threadIdx.x % P; }
  __device__ __forceinline__ void load(const float* from) {
#pragma unroll
    for (int n = 0; n < N; ++n) load8(from + ((int)threadIdx.x + n * Tc<D>::kWork) * 8, f[n]);
  }
  // as bf16 tiles of D rows, the high part and, where lo is given, the low part
  __device__ __forceinline__ void put(uint8_t* hi, uint8_t* lo) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint4 u = pack8(f[n]);
      *piece(hi, D, row(n), piece_of_row()) = u;
      if (lo != nullptr) {
        remainder8(f[n], u);
        *piece(lo, D, row(n), piece_of_row()) = pack8(f[n]);
      }
    }
  }
};
// A vector m near the values (backward): the mean of v under the features' sums, m[e] = sum_c S[c][e] / sum_c z[c], rounded to
// bf16.  The gradients of q and k are small differences where the values of a sequence are alike (of one token they vanish), so
// they are taken of v - m:  u' = (S - z m^T) dy,  dden' = -(phi(q) . u') / den^2 + (m . dy) eps / den^2,
//   dq = phi'(q) (u' / den + dden' z),  dz' = sum phi(q) dden',  dk = phi'(k) (dS v + (dz' - dS m))
// where the roundings of S - z m^T and dS then meet v - m.  Any m is right; without a normaliser, and where it is no number, 0.
// (Working threads; id: a barrier of theirs; scratch: kWork / 32 rows of D floats; z is there after it.)
template <int D>
__device__ __forceinline__ void middle(const Matrix<D>& S, const float* z_from, bool on, float* z, float* scratch,
                                       __nv_bfloat16* m, int id) {
  constexpr int kWork = Tc<D>::kWork, P = Matrix<D>::P;
  const int tid = threadIdx.x, lane = tid & 31;
  float2 s[4] = {};
#pragma unroll
  for (int n = 0; n < Matrix<D>::N; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) s[x] = add2(s[x], S.f[n][x]);
#pragma unroll
  for (int o = P; o < 32; o <<= 1)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[x].x += __shfl_xor_sync(0xffffffffu, s[x].x, o);
      s[x].y += __shfl_xor_sync(0xffffffffu, s[x].y, o);
    }
  if (lane < P)
#pragma unroll
    for (int x = 0; x < 4; ++x) *reinterpret_cast<float2*>(scratch + (tid >> 5) * D + lane * 8 + 2 * x) = s[x];
  if (tid < D) z[tid] = z_from[tid];
  named_bar(id, kWork);
  if (tid < D) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < kWork / 32; ++w) a += scratch[w * D + tid];
#pragma unroll 4
    for (int i = 0; i < D; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(z + i);
      b += (v.x + v.y) + (v.z + v.w);
    }
    const float mean = a / b;
    m[tid] = __float2bfloat16_rn(on && fabsf(mean) < 1e38f ? mean : 0.f);
  }
  named_bar(id, kWork);
}

// A thread's places in every tile: its row's four pieces of 32 columns.
struct Places {
  uint32_t own[4];
  int row, col;
};
__device__ __forceinline__ Places places(int warp, int lane) {
  Places p;
  p.row = (warp & 3) * 32 + lane;
  p.col = (warp >> 2) * 32;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = p.col / 8 + i;
    p.own[i] = (j >> 3) * kAtom + p.row * 128 + (((j & 7) ^ (p.row & 7)) << 4);
  }
  return p;
}
__device__ __forceinline__ uint4& at_byte(uint8_t* tile, uint32_t offset) { return *reinterpret_cast<uint4*>(tile + offset); }
// The last tile of a packed sequence, whose rows end in it: the thread's 32 columns from their place to its row.
__device__ __forceinline__ void store_own(uint8_t* tile, const Places& p, __nv_bfloat16* to) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(to)[i] = at_byte(tile, p.own[i]);
}

// Descriptors.  Tokens' tile as A or B with the tokens along K ("MN-major"): K steps of 16 rows are 2048 bytes apart, 64
// columns an atom; with the columns along K ("K-major"): steps of 32 bytes, 4 to an atom.
__device__ __forceinline__ uint64_t along_rows(uint32_t tile, uint32_t atom) { return smem_desc(tile, atom, 1024); }
template <int D>
__device__ __forceinline__ uint64_t along_cols(uint32_t tile, uint32_t atom, int k) {
  return smem_desc(tile + (k >> 2) * atom, 16, 1024) + (k & 3) * 2;
}

// ================================================================ states
// 4 heads of 65,536 tokens, d = 128: 36 us from a cold cache (134 MB, 3.7 TB/s; issue slots 52 %, tensor pipe 33 %); 48 heads of
// 77 tokens, d = 64: 8.5.
// Tiles of 64 tokens: four buffers of K and V, so that three tiles are on their way at a time, and two of phi(k)'s three
// parts, so that the features of a tile are taken while the MMAs of the one before run.  (65,536 tokens of 4 heads, d = 128:
// with 128 tokens and one set of parts 44 us, with three buffers of 64 tokens that hold K, V and the parts together 40 us.)
constexpr int kSumT = 64, kSumBuffers = 4;
template <int D>
struct SumSmem {
  static constexpr int kPart = kSumT * D * 2;  // bytes of a tile of one tensor
  static constexpr int kV = 0, kK = kSumBuffers * kPart, kParts = 2 * kSumBuffers * kPart, kEnd = kParts + 6 * kPart;
  static constexpr int kSmall = (int)sizeof(Bars);
  static constexpr int kBytes = (kSmall + 1023) / 1024 * 1024 + kEnd;
  static_assert(kBytes <= (D == 64 ? 115712 : 232448), "two blocks of d = 64 an SM, one of d = 128");
};
template <int D, int F>
__global__ void __launch_bounds__(Tc<D>::kThreads, D == 64 ? 2 : 1) tc_cross_states_kernel(const __grid_constant__ TcArgs p) {
  using X = Tc<D>;
  using M = SumSmem<D>;
  constexpr bool kExact = F == MHLA_PHI_RELU || F == MHLA_PHI_IDENTITY;  // phi(k) is a bf16 number
  constexpr uint32_t kColumns = 4 * D;  // the tiles in turn into two sets: half as many additions, which are cut, one behind the other
  constexpr int kSumAtom = kSumT * 128;
  extern __shared__ __align__(16) uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + M::kSmall + 1023) & ~uintptr_t(1023));
  if (sm + M::kEnd > smraw + M::kBytes) {  // (shared memory starts at a multiple of 1024 bytes, or near enough)
    if (threadIdx.x == 0) atomicOr(p.c.status, 1u);
    return;
  }
  Bars* b = reinterpret_cast<Bars*>(smraw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.c.Hk, k = blockIdx.x / p.c.Hk;
  setup(p, b, kColumns);
  const CrossSegment g = cross_segment(p.c.ks, k, &b->scratch);
  if (g.seq < 0) return finish<kSumBuffers, 2>(b, kColumns);
  const uint32_t tmem = b->tbase;
  const int tiles = (g.len + kSumT - 1) / kSumT, bb = p.c.ks.cu == nullptr ? g.seq : 0;
  constexpr int P = D / 8, ROWS = X::kWork / P;  // pieces of a row, rows at a time
  const int pc = tid % P, r0 = tid / P;
  float2 z[4] = {};
  bool ok = true;
  if (tid >= X::kWork) {
    if (lane == 0) {
      const auto fetch = [&](int j) {
        uint64_t* bar = &b->full[j % kSumBuffers];
        uint8_t* to = sm + j % kSumBuffers * M::kPart;
        mbar_arrive_expect_tx(bar, 2 * M::kPart);
        load_tile(to + M::kK, &p.a, g.row0 + j * kSumT, p.a_h ? h : 0, p.a_b ? bb : 0, bar);
        load_tile(to + M::kV, &p.b, g.row0 + j * kSumT, p.b_h ? h : 0, p.b_b ? bb : 0, bar);
        b->issued = j + 1;
      };
      for (int j = 0; j < min(tiles, kSumBuffers); ++j) fetch(j);
      for (int j = 0; j < tiles; ++j) {
        if (!wait(&b->ready[j & 1], (j >> 1) & 1, b)) break;
        tc_fence_after();
        const uint32_t va = smem_u32(sm + M::kV + j % kSumBuffers * M::kPart), pa = smem_u32(sm + M::kParts + (j & 1) * 3 * M::kPart);
        // A = v.  d = 64: its rows 64 .. 127 are what lies behind the tile (another tile's columns), whose results are not
        // read.  B = the high and the middle part side by side, then the low part onto the middle one's columns.
        const uint64_t da = along_rows(va, kSumAtom), d1 = along_rows(pa, kSumAtom), d2 = along_rows(pa + 2 * M::kPart, kSumAtom);
#pragma unroll
        for (int s = 0; s < kSumT / 16; ++s) {
          const uint32_t acc = tmem + (j & 1) * 2 * D;
          mma_bf16(acc, da + s * 128, d1 + s * 128, idesc_bf16_f32(128, kExact ? D : 2 * D, 1, 1), j > 1 || s > 0);
          if (!kExact) mma_bf16(acc + D, da + s * 128, d2 + s * 128, idesc_bf16_f32(128, D, 1, 1), true);
        }
        mma_commit(&b->mma[j & 1]);
        b->mmas = j + 1;
        if (j > 0 && j + kSumBuffers - 1 < tiles) {  // the buffer of tile j - 1 takes the next one
          if (!wait(&b->mma[(j - 1) & 1], ((j - 1) >> 1) & 1, b)) break;
          fetch(j + kSumBuffers - 1);
        }
      }
    }
    __syncwarp();
  } else {
    for (int j = 0; ok && j < tiles; ++j) {
      uint8_t *kt = sm + M::kK + j % kSumBuffers * M::kPart, *vt = sm + M::kV + j % kSumBuffers * M::kPart;
      uint8_t* part = sm + M::kParts + (j & 1) * 3 * M::kPart;
      ok = wait(&b->full[j % kSumBuffers], (j / kSumBuffers) & 1, b);
      if (ok && j >= 2) ok = wait(&b->mma[j & 1], ((j - 2) >> 1) & 1, b);  // the parts have been read
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int n = g.len - j * kSumT;
#pragma unroll
      for (int i = 0; i < kSumT / ROWS; ++i) {
        const int r = r0 + i * ROWS;
        float2 f[4];
        unpack8(*piece(kt, kSumT, r, pc), f);
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = feature<F>(f[x]);
        if (r >= n) {  // behind the sequence: nothing of what lies there counts
#pragma unroll
          for (int x = 0; x < 4; ++x) f[x] = both(0.f);
          *piece(vt, kSumT, r, pc) = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) z[x] = add2(z[x], f[x]);
        const uint4 hi = pack8(f);
        *piece(part, kSumT, r, pc) = hi;
        if (!kExact) {
          remainder8(f, hi);
          const uint4 mid = pack8(f);
          *piece(part + M::kPart, kSumT, r, pc) = mid;
          remainder8(f, mid);
          *piece(part + 2 * M::kPart, kSumT, r, pc) = pack8(f);
        }
      }
      arrive(&b->ready[j & 1], lane);
    }
    if (ok && tiles > 0) ok = wait(&b->mma[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1, b);  // (and all MMAs before it)
  }
  float *so = nullptr, *zo = nullptr;
  if (cross_joined(p.c.ks) && g.nseg != 1) {
    so = p.c.part + ((size_t)k * p.c.Hk + h) * (D * D + D);
    zo = so + D * D;
  } else {
    const int slot = ret_slot(p.c.slots, p.c.n_slots, g.seq);
    if (slot >= 0) {
      so = p.c.S + ((size_t)slot * p.c.Hk + h) * D * D;
      zo = p.c.z + ((size_t)slot * p.c.Hk + h) * D;
    }
  }
  if (__syncthreads_and(ok && !aborted(&b->abort))) {
    tc_fence_after();
    float* zp = reinterpret_cast<float*>(sm);  // [ROWS][D]: the buffers have been read
    if (tid < X::kWork)
#pragma unroll
      for (int x = 0; x < 4; ++x) *reinterpret_cast<float2*>(zp + r0 * D + 8 * pc + 2 * x) = z[x];
    __syncthreads();
    if (zo != nullptr && tid < X::kWork) {
      if (tid < D) {
        float s = 0.f;
#pragma unroll 8
        for (int i = 0; i < ROWS; ++i) s += zp[i * D + tid];
        zo[tid] = s;
      }
      const int e = (warp & 3) * 32 + lane, c0 = (warp >> 2) * 32;
      if ((warp & 3) * 32 < D) {
        float v[32];
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        if (tiles > 0) {
          tmem_ld16(at, v);
          tmem_ld16(at + 16, v + 16);
          tmem_ld_wait();
          const auto add = [&](uint32_t at) {
            float w[32];
            tmem_ld16(at, w);
            tmem_ld16(at + 16, w + 16);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] += w[x];
          };
          if (!kExact) add(at + D);
          if (tiles > 1) {
            add(at + 2 * D);
            if (!kExact) add(at + 3 * D);
          }
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) so[(c0 + x) * D + e] = tiles > 0 ? v[x] : 0.f;
      }
    }
  }
  finish<kSumBuffers, 2>(b, kColumns);
}

// ================================================================ read
// 8 x 6 heads of 4096 queries, d = 64: 13 us (50 MB, 3.9 TB/s), 8 x 8 heads, d = 128: 36 (134 MB, 3.7 TB/s); issue slots 40 %,
// the rest the start and the chain of a tile (copy, features, MMA, results) that three blocks an SM share.  With S as one bf16
// number and den of the unrounded phi(q) 12 and 32, but y of one key off by up to 2e-4 of it; the same with the warps storing
// rows of 64 bytes, which occupies the shared memory's data path, and three buffers throughout: 13 and 50.
// Three buffers (d = 128: four) and two accumulators: while the MMA of a tile runs the warps put the results of the one before
// into its place, whence they are copied out, and take the next one's features.
// phi(q) is rounded to bf16 for den as for the product, so that the weights of the values add up to one whatever the rounding; with S
// as two bf16 numbers y is then as exact as its own rounding where the values are alike (one key: y is its value).
template <int D>
struct ReadSmem {
  static constexpr int kBuffers = read_buffers(D), kSums = read_sums(D);
  static constexpr int kQ = 0, kS = kBuffers * Tc<D>::kTile, kSLo = kS + Tc<D>::kMat, kZ = kSLo + Tc<D>::kMat, kDen = kZ + D * 4,
                       kBars = kDen + kSums * Tc<D>::kCols * kT * 4;
  static_assert(kSums == kBuffers, "a tile's sums lie beside its buffer");
  static constexpr int kBytes = 1024 + kBars + (int)sizeof(Bars);
  static_assert(kBytes <= (D == 64 ? 76800 : 232448), "three blocks of d = 64 an SM, one of d = 128");
};
template <int D, int F>
__global__ void __launch_bounds__(Tc<D>::kThreads, D == 64 ? 3 : 1) tc_cross_read_kernel(const __grid_constant__ TcArgs p) {
  using X = Tc<D>;
  using M = ReadSmem<D>;
  constexpr int NB = M::kBuffers;
  constexpr uint32_t kColumns = 2 * D;
  extern __shared__ __align__(16) uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  Bars* b = reinterpret_cast<Bars*>(sm + M::kBars);
  float *z = reinterpret_cast<float*>(sm + M::kZ), *den = reinterpret_cast<float*>(sm + M::kDen);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.c.H, k = blockIdx.x / p.c.H;
  setup(p, b, kColumns);
  const CrossSegment g = cross_segment(p.c.qs, k, &b->scratch);
  const int slot = g.seq < 0 ? -1 : p.c.slots != nullptr ? p.c.slots[g.seq] : g.seq;
  if (slot < 0 || slot >= p.c.n_slots) return finish<NB, 2>(b, kColumns);
  const uint32_t tmem = b->tbase;
  const int tiles = (g.len + kT - 1) / kT, bb = p.c.qs.cu == nullptr ? g.seq : 0;
  const auto whole = [&](int j) { return p.c.qs.cu == nullptr || (j + 1) * kT <= g.len; };  // (dense: the tensor ends there too)
  const size_t unit = (size_t)slot * p.c.Hk + h / (p.c.H / p.c.Hk);
  if (tid < X::kWork) {
    Matrix<D> S;
    S.load(p.c.S + unit * D * D);
    S.put(sm + M::kS, sm + M::kSLo);
  }
  if (tid < D) z[tid] = p.c.z[unit * D + tid];
  if (tid >= X::kWork) {
    if (lane == 0) {
      const auto fetch = [&](int j) {
        uint64_t* bar = &b->full[j % NB];
        mbar_arrive_expect_tx(bar, X::kTile);
        load_tile(sm + M::kQ + j % NB * X::kTile, &p.a, g.row0 + j * kT, p.a_h ? h : 0, p.a_b ? bb : 0, bar);
        b->issued = j + 1;
      };
      const uint32_t sa = smem_u32(sm + M::kS), sl = smem_u32(sm + M::kSLo);
      // the results of tile j, and another tile into its place
      const auto out = [&](int j) {
        if (!wait(&b->out[j & 1], (j >> 1) & 1, b)) return false;
        if (whole(j)) {
          store_tile(&p.c_map, sm + M::kQ + j % NB * X::kTile, g.row0 + j * kT, p.c_h ? h : 0, p.c_b ? bb : 0);
          stores_commit();
        }
        if (j + NB < tiles) {
          stores_read();
          fetch(j + NB);
        }
        return true;
      };
      for (int j = 0; j < min(tiles, NB); ++j) fetch(j);
      for (int j = 0; j < tiles; ++j) {
        // every warp has the features of tile j (the first time: S) written, and the results of tile j - 2 taken
        if (!wait(&b->ready[j % 3], (j / 3) & 1, b)) break;
        tc_fence_after();
        const uint32_t qa = smem_u32(sm + M::kQ + j % NB * X::kTile);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_bf16(tmem + (j & 1) * D, along_cols<D>(qa, kAtom, s), along_rows(part ? sl : sa, D * 128) + s * 128,
                     idesc_bf16_f32(128, D, 0, 1), s > 0 || part > 0);
        mma_commit(&b->mma[j & 1]);
        b->mmas = j + 1;
        if (j > 0 && !out(j - 1)) break;
        if (j == tiles - 1) out(j);
      }
      stores_done();
    }
    __syncwarp();
    __syncthreads();
    return finish<NB, 2>(b, kColumns);
  }
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(X::kWork) : "memory");  // z
  const Places pl = places(warp, lane);
  const int row = pl.row, cg = warp >> 2;  // the thread's row, and its 32 columns
  const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + cg * 32;
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(const_cast<void*>(p.c.y.p)) + cross_base(p.c.qs, p.c.y, g.seq, h) +
                     ((long long)g.row0 + row) * p.c.y.sn + pl.col;
  bool ok = true;
  int buf = 0, before = 0, phase = 0, slot3 = 0;  // of tiles j and j - 1: their buffers, with their sums (and phase); j % 3
  for (int j = 0; ok && j <= tiles; ++j) {
    if (j < tiles) {  // the features of tile j
      uint8_t* qt = sm + M::kQ + buf * X::kTile;
      ok = __all_sync(0xffffffffu, wait(&b->full[buf], phase, b));
      if (!ok) break;
      float2 d = both(0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4* q = &at_byte(qt, pl.own[i]);
        float2 f[4], zz[4];
        unpack8(*q, f);
        load8(z + cg * 32 + 8 * i, zz);
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = feature<F>(f[x]);
        if (F != MHLA_PHI_IDENTITY) {
          const uint4 u = pack8(f);
          *q = u;
          unpack8(u, f);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) d = fma2(f[x], zz[x], d);
      }
      den[(buf * X::kCols + cg) * kT + row] = d.x + d.y;
      arrive(&b->ready[slot3], lane);
    }
    if (j > 0) {  // tile j - 1 goes out
      const int t = j - 1;
      ok = __all_sync(0xffffffffu, wait(&b->mma[t & 1], (t >> 1) & 1, b));
      if (!ok) break;
      tc_fence_after();
      float2 v[16];
      tmem_ld8(at + (t & 1) * D, v);
      tmem_ld8(at + (t & 1) * D + 16, v + 8);
      float inv = 1.f;
      if (p.c.normalise) {
        float d = p.c.eps;
#pragma unroll
        for (int i = 0; i < X::kCols; ++i) d += den[(before * X::kCols + i) * kT + row];
        inv = inverse(d);
      }
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], both(inv));
      uint8_t* qt = sm + M::kQ + before * X::kTile;
#pragma unroll
      for (int i = 0; i < 4; ++i) at_byte(qt, pl.own[i]) = pack8(v + 4 * i);
      if (!whole(t) && row < g.len - t * kT) store_own(qt, pl, y + (long long)t * kT * p.c.y.sn);
      arrive(&b->out[t & 1], lane);
    }
    before = buf;
    buf = buf == NB - 1 ? 0 : buf + 1;
    phase ^= buf == 0;
    slot3 = slot3 == 2 ? 0 : slot3 + 1;
  }
  __syncthreads();
  finish<NB, 2>(b, kColumns);
}

// ================================================================ backward over the queries
// 8 x 6 heads of 4096 queries, d = 64: about 26 us (75 MB), 8 x 8 heads, d = 128: about 85 (201 MB); issue slots 40 %, tensor
// pipe 20 %.  Bound by the chain of a tile: u, its row sums, dq and the copy out; dS from w runs next to the sums.  With the next
// tile's u taken ahead, in a second place of tensor memory: 1 and 9 us more, as the tile after comes in later.
// The tiles of d = 128 leave 3 KB of a block's 227: what is small lies before them, up to the next 1024 bytes.
template <int D>
struct QuerySmem {
  static constexpr int kQ = 0, kY = 2 * Tc<D>::kTile, kLo = 4 * Tc<D>::kTile, kS = 5 * Tc<D>::kTile, kSLo = kS + Tc<D>::kMat,
                       kEnd = kSLo + Tc<D>::kMat;
  static constexpr int kZ = 0, kM = kZ + D * 4, kDen = kM + D * 2, kBars = kDen + Tc<D>::kCols * kT * 4,
                       kSmall = kBars + (int)sizeof(Bars);
  static constexpr int kBytes = (kSmall + 1023) / 1024 * 1024 + kEnd;
  static_assert(kBytes <= 232448 / (D == 64 ? 2 : 1), "two blocks of d = 64 an SM, one of d = 128");
};
// All of the n threads of the warps that share 32 rows, or none; what they wrote before is there.
__device__ __forceinline__ bool row_and(bool ok, int warp, int n) { return group_and(1 + (warp & 3), n, ok); }
// 32 values a lane: the sum of value i over the warp, for lane i.
__device__ __forceinline__ float sum_turned(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}
template <int D, int F>
__global__ void __launch_bounds__(Tc<D>::kThreads, D == 64 ? 2 : 1) tc_cross_query_kernel(const __grid_constant__ TcArgs p) {
  using X = Tc<D>;
  using M = QuerySmem<D>;
  constexpr uint32_t kColumns = 256;  // u, dS^T (d = 64: in two parts)
  extern __shared__ __align__(16) uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + M::kSmall + 1023) & ~uintptr_t(1023));
  if (sm + M::kEnd > smraw + M::kBytes) {  // (shared memory starts at a multiple of 1024 bytes, or near enough)
    if (threadIdx.x == 0) atomicOr(p.c.status, 1u);
    return;
  }
  Bars* b = reinterpret_cast<Bars*>(smraw + M::kBars);
  float *z = reinterpret_cast<float*>(smraw + M::kZ), *den = reinterpret_cast<float*>(smraw + M::kDen);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.c.H, k = blockIdx.x / p.c.H;
  setup(p, b, kColumns);
  const CrossSegment g = cross_segment(p.c.qs, k, &b->scratch);
  if (g.seq < 0) return finish<2, 1>(b, kColumns);
  const uint32_t tmem = b->tbase;
  const int tiles = (g.len + kT - 1) / kT, bb = p.c.qs.cu == nullptr ? g.seq : 0;
  const auto whole = [&](int j) { return p.c.qs.cu == nullptr || (j + 1) * kT <= g.len; };  // (dense: the tensor ends there too)
  const size_t unit = (size_t)g.seq * p.c.Hk + h / (p.c.H / p.c.Hk);
  __nv_bfloat16* mid = reinterpret_cast<__nv_bfloat16*>(smraw + M::kM);
  if (tid < X::kWork) {  // S - z m^T
    Matrix<D> S;
    S.load(p.c.S + unit * D * D);
    middle<D>(S, p.c.z + unit * D, p.c.normalise, z, reinterpret_cast<float*>(sm + M::kLo), mid, 5);
    float2 m[4];
    unpack8(*reinterpret_cast<const uint4*>(mid + 8 * S.piece_of_row()), m);
#pragma unroll
    for (int n = 0; n < S.N; ++n) {
      const float minus = -z[S.row(n)];
#pragma unroll
      for (int x = 0; x < 4; ++x) S.f[n][x] = fma2(both(minus), m[x], S.f[n][x]);
    }
    S.put(sm + M::kS, sm + M::kSLo);
  }
  if (tid >= X::kWork) {
    if (lane == 0) {
      const auto fetch = [&](int j) {
        uint64_t* bar = &b->full[j & 1];
        mbar_arrive_expect_tx(bar, 2 * X::kTile);
        load_tile(sm + M::kQ + (j & 1) * X::kTile, &p.a, g.row0 + j * kT, p.a_h ? h : 0, p.a_b ? bb : 0, bar);
        load_tile(sm + M::kY + (j & 1) * X::kTile, &p.b, g.row0 + j * kT, p.b_h ? h : 0, p.b_b ? bb : 0, bar);
        b->issued = j + 1;
      };
      const uint32_t sa = smem_u32(sm + M::kS), sl = smem_u32(sm + M::kSLo), wl = smem_u32(sm + M::kLo);
      const auto store = [&](int j) {  // dq of tile j, where the warps' arrival for the next turn has been seen
        if (!whole(j)) return;
        store_tile(&p.c_map, sm + M::kQ + (j & 1) * X::kTile, g.row0 + j * kT, p.c_h ? h : 0, p.c_b ? bb : 0);
        stores_commit();
      };
      if (tiles > 0) fetch(0);
      for (int j = 0; j < tiles; ++j) {
        const uint32_t qa = smem_u32(sm + M::kQ + (j & 1) * X::kTile), ya = smem_u32(sm + M::kY + (j & 1) * X::kTile);
        // every warp has the tile before stored (the first time: S written), and rows without a token cleared
        if (!wait(&b->ready[0], j & 1, b)) break;
        tc_fence_after();
        // u = dy S^T
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_bf16(tmem, along_cols<D>(ya, kAtom, s), along_cols<D>(part ? sl : sa, D * 128, s), idesc_bf16_f32(128, D, 0, 0),
                     s > 0 || part > 0);
        mma_commit(&b->mma[0]);
        b->mmas = j + 1;
        if (j > 0) store(j - 1);
        if (j + 1 < tiles) {
          stores_read();
          fetch(j + 1);
        }
        if (!wait(&b->ready2, j & 1, b)) break;
        tc_fence_after();
        // dS^T += dy^T w  (d = 64: A's rows 64 .. 127 are another tile's columns, whose results are not read)
        // d = 64: the high and the low part of w side by side, in columns of their own
        const uint64_t da = along_rows(ya, D == 64 ? wl - ya : kAtom);
#pragma unroll
        for (int part = 0; part < (D == 64 ? 1 : 2); ++part) {
          const uint64_t db = along_rows(part ? wl : qa, D == 64 ? wl - qa : kAtom);
#pragma unroll
          for (int s = 0; s < kT / 16; ++s)
            mma_bf16(tmem + D, da + s * 128, db + s * 128, idesc_bf16_f32(128, 128, 1, 1), j > 0 || s > 0 || part > 0);
        }
        mma_commit(&b->mma2);
        b->mmas2 = j + 1;
        if (j == tiles - 1 && wait(&b->out[0], 0, b)) store(j);
      }
      stores_done();
    }
    __syncwarp();
    __syncthreads_and(true);  // (the two barriers of the other warps' end)
    __syncthreads();
    return finish<2, 1>(b, kColumns);
  }
  __syncwarp();
  asm volatile("bar.sync 5, %0;" ::"n"(X::kWork) : "memory");  // z
  const Places pl = places(warp, lane);
  const int row = pl.row, cg = warp >> 2;
  const auto row_sync = [&] { named_bar(1 + (warp & 3), X::kWork / 4); };  // the warps that share 32 rows
  const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + cg * 32;
  __nv_bfloat16* dq = static_cast<__nv_bfloat16*>(const_cast<void*>(p.c.dq.p)) + cross_base(p.c.qs, p.c.dq, g.seq, h) +
                      ((long long)g.row0 + row) * p.c.dq.sn + pl.col;
  float2 dz[16] = {};  // of the thread's 32 columns, over its rows
  bool ok = true;
  for (int j = 0; j < tiles; ++j) {
    uint8_t *qt = sm + M::kQ + (j & 1) * X::kTile, *yt = sm + M::kY + (j & 1) * X::kTile;
    const int n = g.len - j * kT;
    const bool live = row < n;
    ok = wait(&b->full[j & 1], (j >> 1) & 1, b);
    if (!row_and(ok, warp, X::kWork / 4)) {
      ok = false;
      break;
    }
    if (!live)
#pragma unroll
      for (int i = 0; i < 4; ++i) at_byte(yt, pl.own[i]) = make_uint4(0, 0, 0, 0);
    arrive(&b->ready[0], lane);
    float2 f[16], d = both(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack8(at_byte(qt, pl.own[i]), f + 4 * i);
      float2 zz[4];
      load8(z + cg * 32 + 8 * i, zz);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        f[4 * i + x] = feature<F>(f[4 * i + x]);
        if (!live) f[4 * i + x] = both(0.f);
        d = fma2(f[4 * i + x], zz[x], d);
      }
    }
    den[cg * kT + row] = d.x + d.y;
    row_sync();
    float inv = 1.f;
    if (p.c.normalise) {
      float dd = p.c.eps;
#pragma unroll
      for (int i = 0; i < X::kCols; ++i) dd += den[i * kT + row];
      inv = inverse(dd);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // w over q's place (the low part's has been read: the tile before is stored)
      float2 w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) w[x] = mul2(f[4 * i + x], both(inv));
      const uint4 hi = pack8(w);
      at_byte(qt, pl.own[i]) = hi;
      remainder8(w, hi);
      at_byte(sm + M::kLo, pl.own[i]) = pack8(w);
    }
    arrive(&b->ready2, lane);
    ok = wait(&b->mma[0], j & 1, b);
    ok = __all_sync(0xffffffffu, ok);
    float s = 0.f;
    if (ok) {
      tc_fence_after();
      float2 s2 = both(0.f);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float2 u[8];
        tmem_ld8(at + 16 * c, u);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 8; ++x) s2 = fma2(f[8 * c + x], u[x], s2);
      }
      s = s2.x + s2.y;
    }
    row_sync();  // den has been read
    den[cg * kT + row] = s;
    if (!row_and(ok, warp, X::kWork / 4)) {
      ok = false;
      break;
    }
    float dd = 0.f;
    if (p.c.normalise && live) {
#pragma unroll
      for (int i = 0; i < X::kCols; ++i) dd += den[i * kT + row];
      dd = -(dd * inv) * inv;  // (inv^2 alone is 0 for a den of 2^75 and above, inf for one of 2^-64)
      if (p.c.eps * inv > 0x1p-26f) {  // (m . dy) eps / den^2, no less than a rounding of u' / den
        float s1 = 0.f;
        for (int i = 0; i < D / 8; ++i) {
          float2 a[4], e[4];
          unpack8(*piece(yt, kT, row, i), a);
          unpack8(*reinterpret_cast<const uint4*>(mid + 8 * i), e);
#pragma unroll
          for (int x = 0; x < 4; ++x) s1 = fmaf(a[x].x, e[x].x, fmaf(a[x].y, e[x].y, s1));
        }
        dd = fmaf(s1 * (p.c.eps * inv), inv, dd);
      }
    }
    ok = row_and(wait(&b->mma2, j & 1, b), warp, X::kWork / 4);  // w has been read; and the row's sums
    if (!ok) break;
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 u[8];
      tmem_ld8(at + 16 * c, u);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 zz[4];
        load8(z + cg * 32 + 16 * c + 8 * i, zz);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int at_f = 8 * c + 4 * i + x;
          dz[at_f] = fma2(f[at_f], both(dd), dz[at_f]);
          u[4 * i + x] = mul2(slope<F>(f[at_f]), fma2(u[4 * i + x], both(inv), mul2(zz[x], both(dd))));
        }
        at_byte(qt, pl.own[2 * c + i]) = pack8(u + 4 * i);
      }
    }
    if (!whole(j) && live) store_own(qt, pl, dq + (long long)j * kT * p.c.dq.sn);
    if (j == tiles - 1) arrive(&b->out[0], lane);
  }
  if (__syncthreads_and(ok && !aborted(&b->abort))) {
    tc_fence_after();
    float* out = p.c.part + ((size_t)k * p.c.H + h) * (D * D + D);
    float v[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[2 * i] = dz[i].x;
      v[2 * i + 1] = dz[i].y;
    }
    den[(warp & 3) * D + cg * 32 + lane] = sum_turned(v, lane);  // (4 D floats are there: kCols * kT)
    const int e = (warp & 3) * 32 + lane, c0 = cg * 32;
    if ((warp & 3) * 32 < D) {
      if (tiles > 0) {
        tmem_ld16(at + D, v);
        tmem_ld16(at + D + 16, v + 16);
        tmem_ld_wait();
        if (D == 64) {
          float w[32];
          tmem_ld16(at + 2 * D, w);
          tmem_ld16(at + 2 * D + 16, w + 16);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] += w[x];
        }
      }
#pragma unroll
      for (int x = 0; x < 32; ++x) out[(c0 + x) * D + e] = tiles > 0 ? v[x] : 0.f;
    }
    __syncthreads();
    if (tid < D) out[D * D + tid] = den[tid] + den[D + tid] + den[2 * D + tid] + den[3 * D + tid];
  } else {
    __syncthreads();
  }
  finish<2, 1>(b, kColumns);
}

// ================================================================ backward over the keys
// 8 x 6 heads of 2048 keys, d = 64: about 14 us (50 MB); 8 x 8 heads, d = 128: about 48 (134 MB), where two buffers wait for
// one another's copies in and out.  phi(k) is one bf16 number for dv (off by 2^-9 of each term in the mean, of 64 or 128 of them;
// dv by 1.69e-3 where its own rounding makes 1.66e-3), as a second part would take the third buffer's room; dS is two.
// Two accumulators: while the MMAs of a tile run the warps put the results of the one before into its place, whence they are
// copied out; three buffers, two for d = 128.
template <int D>
struct KeySmem {
  static constexpr int kBuffers = D == 64 ? 3 : 2;
  static constexpr int kK = 0, kV = kBuffers * Tc<D>::kTile, kS = 2 * kBuffers * Tc<D>::kTile, kSLo = kS + Tc<D>::kMat,
                       kEnd = kSLo + Tc<D>::kMat;
  static constexpr int kZ = 0, kM = kZ + D * 4, kBars = kM + D * 2, kSmall = kBars + (int)sizeof(Bars);
  static constexpr int kBytes = (kSmall + 1023) / 1024 * 1024 + kEnd;
  static_assert(kBytes <= (D == 64 ? 115712 : 232448), "two blocks of d = 64 an SM, one of d = 128");
};
template <int D, int F>
__global__ void __launch_bounds__(Tc<D>::kThreads, D == 64 ? 2 : 1) tc_cross_key_kernel(const __grid_constant__ TcArgs p) {
  using X = Tc<D>;
  using M = KeySmem<D>;
  constexpr bool kExpSlope = F == MHLA_PHI_EXP || F == MHLA_PHI_ELU1;
  constexpr int NB = M::kBuffers;
  constexpr uint32_t kColumns = 4 * D;  // dv and dphi(k), twice
  extern __shared__ __align__(16) uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + M::kSmall + 1023) & ~uintptr_t(1023));
  if (sm + M::kEnd > smraw + M::kBytes) {  // (shared memory starts at a multiple of 1024 bytes, or near enough)
    if (threadIdx.x == 0) atomicOr(p.c.status, 1u);
    return;
  }
  Bars* b = reinterpret_cast<Bars*>(smraw + M::kBars);
  float* z = reinterpret_cast<float*>(smraw + M::kZ);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.c.Hk, k = blockIdx.x / p.c.Hk;
  setup(p, b, kColumns);
  const CrossSegment g = cross_segment(p.c.ks, k, &b->scratch);
  if (g.seq < 0) return finish<NB, 2>(b, kColumns);
  const int rows = p.c.ks.cu != nullptr ? g.len : min(p.c.ks.L, p.c.ks.N - g.row0);  // dense: zeros behind the tokens
  const uint32_t tmem = b->tbase;
  const int tiles = (rows + kT - 1) / kT, bb = p.c.ks.cu == nullptr ? g.seq : 0;
  const auto whole = [&](int j) { return p.c.ks.cu == nullptr || (j + 1) * kT <= g.len; };  // (dense: the tensor ends there too)
  const float* from = p.c.dS + ((size_t)g.seq * p.c.Hk + h) * (D * D + D);
  if (tid < X::kWork) {
    const size_t unit = (size_t)g.seq * p.c.Hk + h;
    __nv_bfloat16* mid = reinterpret_cast<__nv_bfloat16*>(smraw + M::kM);
    Matrix<D> S, dS;
    S.load(p.c.S + unit * D * D);
    dS.load(from);
    middle<D>(S, p.c.z + unit * D, p.c.normalise, z, reinterpret_cast<float*>(sm + M::kS), mid, 1);
    float2 m[4];
    unpack8(*reinterpret_cast<const uint4*>(mid + 8 * S.piece_of_row()), m);
    dS.put(sm + M::kS, sm + M::kSLo);
    // z: dz' - dS m, of dS as it lies there
#pragma unroll
    for (int n = 0; n < S.N; ++n) {
      const int r = S.row(n);
      float2 a[4], e[4], s2 = both(0.f);
      unpack8(*piece(sm + M::kS, D, r, S.piece_of_row()), a);
      unpack8(*piece(sm + M::kSLo, D, r, S.piece_of_row()), e);
#pragma unroll
      for (int x = 0; x < 4; ++x) s2 = fma2(add2(a[x], e[x]), m[x], s2);
      float s1 = s2.x + s2.y;
#pragma unroll
      for (int o = 1; o < S.P; o <<= 1) s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      if (S.piece_of_row() == 0) z[r] = from[D * D + r] - s1;
    }
  }
  if (tid >= X::kWork) {
    if (lane == 0) {
      const auto fetch = [&](int j) {
        uint64_t* bar = &b->full[j % NB];
        mbar_arrive_expect_tx(bar, 2 * X::kTile);
        load_tile(sm + M::kK + j % NB * X::kTile, &p.a, g.row0 + j * kT, p.a_h ? h : 0, p.a_b ? bb : 0, bar);
        load_tile(sm + M::kV + j % NB * X::kTile, &p.b, g.row0 + j * kT, p.b_h ? h : 0, p.b_b ? bb : 0, bar);
        b->issued = j + 1;
      };
      const uint32_t sa = smem_u32(sm + M::kS), sl = smem_u32(sm + M::kSLo);
      // the results of tile j, and another tile into its place
      const auto out = [&](int j) {
        if (!wait(&b->out[j & 1], (j >> 1) & 1, b)) return false;
        if (whole(j)) {
          store_tile(&p.c_map, sm + M::kK + j % NB * X::kTile, g.row0 + j * kT, p.c_h ? h : 0, p.c_b ? bb : 0);
          store_tile(&p.d_map, sm + M::kV + j % NB * X::kTile, g.row0 + j * kT, p.d_h ? h : 0, p.d_b ? bb : 0);
          stores_commit();
        }
        if (j + NB < tiles) {
          stores_read();
          fetch(j + NB);
        }
        return true;
      };
      for (int j = 0; j < min(tiles, NB); ++j) fetch(j);
      for (int j = 0; j < tiles; ++j) {
        // every warp has the features of tile j (the first time: dS) written, and the results of tile j - 2 taken
        if (!wait(&b->ready[j % 3], (j / 3) & 1, b)) break;
        tc_fence_after();
        const uint32_t ka = smem_u32(sm + M::kK + j % NB * X::kTile), va = smem_u32(sm + M::kV + j % NB * X::kTile);
        const uint32_t acc = tmem + (j & 1) * 2 * D;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            mma_bf16(acc, along_cols<D>(ka, kAtom, s), along_rows(part ? sl : sa, D * 128) + s * 128, idesc_bf16_f32(128, D, 0, 1),
                     s > 0 || part > 0);
            mma_bf16(acc + D, along_cols<D>(va, kAtom, s), along_cols<D>(part ? sl : sa, D * 128, s),
                     idesc_bf16_f32(128, D, 0, 0), s > 0 || part > 0);
          }
        mma_commit(&b->mma[j & 1]);
        b->mmas = j + 1;
        if (j > 0 && !out(j - 1)) break;
        if (j == tiles - 1) out(j);
      }
      stores_done();
    }
    __syncwarp();
    __syncthreads();
    return finish<NB, 2>(b, kColumns);
  }
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(X::kWork) : "memory");  // z
  const Places pl = places(warp, lane);
  const int row = pl.row, cg = warp >> 2;
  const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + cg * 32;
  __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(const_cast<void*>(p.c.dk.p)) + cross_base(p.c.ks, p.c.dk, g.seq, h) +
                      ((long long)g.row0 + row) * p.c.dk.sn + pl.col;
  __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(const_cast<void*>(p.c.dv.p)) + cross_base(p.c.ks, p.c.dv, g.seq, h) +
                      ((long long)g.row0 + row) * p.c.dv.sn + pl.col;
  const __nv_bfloat16* keys = static_cast<const __nv_bfloat16*>(p.c.k.p) + cross_base(p.c.ks, p.c.k, g.seq, h) +
                              ((long long)g.row0 + row) * p.c.k.sn + pl.col;
  // phi(k) of tile j over its keys
  const auto features = [&](int j) {
    uint8_t* kt = sm + M::kK + j % NB * X::kTile;
    if (!__all_sync(0xffffffffu, wait(&b->full[j % NB], (j / NB) & 1, b))) return false;
    if (F != MHLA_PHI_IDENTITY)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f[4];
        unpack8(at_byte(kt, pl.own[i]), f);
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = feature<F>(f[x]);
        at_byte(kt, pl.own[i]) = pack8(f);
      }
    arrive(&b->ready[j % 3], lane);
    return true;
  };
  bool ok = tiles == 0 || features(0);
  for (int j = 0; ok && j < tiles; ++j) {
    if (j + 1 < tiles && !features(j + 1)) break;
    const bool live = row < g.len - j * kT;  // (dense: zeros behind the tokens)
    // k once more, where phi' is an exponential: by phi as it lies there, rounded to bf16, dk would be off by a second rounding
    // (ELU + 1, 8 x 6 heads of 2048 keys: by 1.83e-3 in the mean, so by 1.66e-3, its own; 3 us, 8 x 8 heads of d 128 12 us)
    uint4 own[4];
    if (kExpSlope && live)
#pragma unroll
      for (int i = 0; i < 4; ++i) own[i] = reinterpret_cast<const uint4*>(keys + (long long)j * kT * p.c.k.sn)[i];
    ok = __all_sync(0xffffffffu, wait(&b->mma[j & 1], (j >> 1) & 1, b));
    if (!ok) break;
    tc_fence_after();
    uint8_t *kt = sm + M::kK + j % NB * X::kTile, *vt = sm + M::kV + j % NB * X::kTile;
    const uint32_t acc = at + (j & 1) * 2 * D;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 u[8], v[8];
      tmem_ld8(acc + D + 16 * c, u);
      tmem_ld8(acc + 16 * c, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 f[4], zz[4];
        if (kExpSlope) {
          unpack8(own[2 * c + i], f);
#pragma unroll
          for (int x = 0; x < 4; ++x) f[x] = feature<F>(f[x]);
        } else if (F != MHLA_PHI_IDENTITY) {
          unpack8(at_byte(kt, pl.own[2 * c + i]), f);
        }
        load8(z + cg * 32 + 16 * c + 8 * i, zz);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          u[4 * i + x] = add2(u[4 * i + x], zz[x]);
          if (F != MHLA_PHI_IDENTITY) u[4 * i + x] = mul2(slope<F>(f[x]), u[4 * i + x]);
          if (!live) u[4 * i + x] = v[4 * i + x] = both(0.f);
        }
        at_byte(kt, pl.own[2 * c + i]) = pack8(u + 4 * i);
        at_byte(vt, pl.own[2 * c + i]) = pack8(v + 4 * i);
      }
    }
    if (!whole(j) && live) {
      store_own(kt, pl, dk + (long long)j * kT * p.c.dk.sn);
      store_own(vt, pl, dv + (long long)j * kT * p.c.dv.sn);
    }
    arrive(&b->out[j & 1], lane);
  }
  __syncthreads();
  finish<NB, 2>(b, kColumns);
}

// ================================================================ host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// A token tensor as [batch][head][64 columns][row][column]; a dimension of stride 0 has one entry.  Rows behind the tensor read as zeros.
bool make_map(CUtensorMap* m, const RetTensor& t, const CrossSide& s, int heads, int d, int box_rows) {
  auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t row_bytes = t.sn ? (cuuint64_t)t.sn * 2 : (cuuint64_t)d * 2;
  const cuuint64_t dims[5] = {64, (cuuint64_t)s.N, (cuuint64_t)d / 64, t.sh ? (cuuint64_t)heads : 1,
                              t.sb && s.cu == nullptr ? (cuuint64_t)s.B : 1};
  const cuuint64_t strides[4] = {row_bytes, 128, t.sh ? (cuuint64_t)t.sh * 2 : row_bytes, t.sb ? (cuuint64_t)t.sb * 2 : row_bytes};
  const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)d / 64, 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(t.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

unsigned long long g_wait_ns = kWaitNs;

// The launch's arguments, with the maps of the tile's one or two tensors and of what is written.
bool make_args(TcArgs* t, const CrossArgs& a, const CrossSide& s, int heads, const RetTensor& x, const RetTensor* y,
               const RetTensor* out, const RetTensor* out2, int box_rows = kT) {
  t->c = a;
  t->wait_ns = g_wait_ns;
  const auto map = [&](CUtensorMap* m, int* has_h, int* has_b, const RetTensor* x) {
    if (x == nullptr) return true;
    *has_h = x->sh != 0;
    *has_b = x->sb != 0 && s.cu == nullptr;
    return make_map(m, *x, s, heads, a.d, box_rows);
  };
  return map(&t->a, &t->a_h, &t->a_b, &x) && map(&t->b, &t->b_h, &t->b_b, y) && map(&t->c_map, &t->c_h, &t->c_b, out) &&
         map(&t->d_map, &t->d_h, &t->d_b, out2);
}

cudaError_t launch(void (*kernel)(TcArgs), SmemOptIn& opt, long long blocks, int threads, int smem, const TcArgs& t,
                   cudaStream_t st) {
  const cudaError_t e = opt.ensure((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)blocks), (unsigned)threads, (size_t)smem, st, true, t);
}

template <int D, int F>
cudaError_t states_t(const CrossArgs& a, cudaStream_t st) {
  TcArgs t;
  if (!make_args(&t, a, a.ks, a.Hk, a.k, &a.v, nullptr, nullptr, kSumT)) return cudaErrorInvalidValue;
  static SmemOptIn opt;
  return launch(tc_cross_states_kernel<D, F>, opt, (long long)a.ks.segs * a.Hk, Tc<D>::kThreads, SumSmem<D>::kBytes, t, st);
}
template <int D, int F>
cudaError_t read_t(const CrossArgs& a, cudaStream_t st) {
  TcArgs t;
  if (!make_args(&t, a, a.qs, a.H, a.q, nullptr, &a.y, nullptr)) return cudaErrorInvalidValue;
  static SmemOptIn opt;
  return launch(tc_cross_read_kernel<D, F>, opt, (long long)a.qs.segs * a.H, Tc<D>::kThreads, ReadSmem<D>::kBytes, t, st);
}
template <int D, int F>
cudaError_t backward_t(const CrossArgs& a, cudaStream_t st) {
  TcArgs t;
  static SmemOptIn opt_q, opt_k;
  cudaError_t e = cudaSuccess;
  if (a.qs.segs > 0) {
    if (!make_args(&t, a, a.qs, a.H, a.q, &a.dy, &a.dq, nullptr)) return cudaErrorInvalidValue;
    e = launch(tc_cross_query_kernel<D, F>, opt_q, (long long)a.qs.segs * a.H, Tc<D>::kThreads, QuerySmem<D>::kBytes, t, st);
  }
  if (e != cudaSuccess || a.ks.segs == 0) return e;
  e = cross_join_launch(a, true, st);
  if (e != cudaSuccess) return e;
  if (!make_args(&t, a, a.ks, a.Hk, a.k, &a.v, &a.dk, &a.dv)) return cudaErrorInvalidValue;
  return launch(tc_cross_key_kernel<D, F>, opt_k, (long long)a.ks.segs * a.Hk, Tc<D>::kThreads, KeySmem<D>::kBytes, t, st);
}

#define CROSS_FEATURES(fn, D)                                                   \
  switch (f) {                                                                  \
    case MHLA_PHI_ELU1: return fn<D, MHLA_PHI_ELU1>(a, st);                     \
    case MHLA_PHI_RELU: return fn<D, MHLA_PHI_RELU>(a, st);                     \
    case MHLA_PHI_EXP: return fn<D, MHLA_PHI_EXP>(a, st);                       \
    default: return fn<D, MHLA_PHI_IDENTITY>(a, st);                            \
  }
#define CROSS_WIDTHS(fn)          \
  if (a.d == 64) {                \
    CROSS_FEATURES(fn, 64)        \
  }                               \
  CROSS_FEATURES(fn, 128)

}  // namespace

void tc_cross_set_wait_limit(unsigned long long ns) { g_wait_ns = ns == 0 ? kWaitNs : ns; }
bool tc_cross_supported(int d, mhla_dtype dt) { return dt == MHLA_BF16 && (d == 64 || d == 128); }
cudaError_t tc_cross_states_launch(const CrossArgs& a, cudaStream_t st) {
  const int f = a.k.feature;
  CROSS_WIDTHS(states_t)
}
cudaError_t tc_cross_read_launch(const CrossArgs& a, cudaStream_t st) {
  const int f = a.q.feature;
  CROSS_WIDTHS(read_t)
}
cudaError_t tc_cross_backward_launch(const CrossArgs& a, cudaStream_t st) {
  const int f = a.q.feature;
  CROSS_WIDTHS(backward_t)
}

}  // namespace mhla
