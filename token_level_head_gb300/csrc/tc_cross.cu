// Linear cross attention on the sm_103a tensor cores (bf16, d = 64 or 128): the same steps as the FP32 kernels'
// (cross_simt.cu), a tile of 128 tokens at a time.
//
//   states  D[e][c] += sum_t v[t][e] phi(k)[t][c]   (A = v, B = phi(k) as a sum of three bf16 numbers: S is an fp32
//           result), z in fp32 registers
//   read    y[t][e] = (sum_c phi(q)[t][c] S[c][e]) / den_t
//   query   u[t][c] = sum_e dy[t][e] S[c][e], dS^T[e][c] += sum_t dy[t][e] w[t][c] with w = phi(q) / den; S and w as sums of
//           two bf16 numbers (dq is a difference of two nearly equal terms: u / den and dden z), dy as it is; dz in fp32
//   key     dv[t][e] = sum_c phi(k)[t][c] dS[c][e], dphi(k)[t][c] = sum_e v[t][e] dS[c][e] (dS as a sum of two)
//
// Bound: memory (2, 2, 3 and 4 tensors), next to it the instructions that take the features and turn tiles.  A block has a
// segment of a head and walks over its tiles: a warp of its own issues the copies (TMA, into the buffer that is free) and the
// MMAs, D / 8 warps take the features (a thread 32 columns of a row, in place in the 128-byte-swizzled tile), take the results
// from tensor memory, put them into the tile's buffer and store 64 bytes of a row together.  Two blocks an SM for d = 64
// (reads: three), one for d = 128, hide one another's waits.  Every wait is bounded (on time-out the block stops, sets the
// status word and drains what it has in flight).
// Measured, whole calls: 8 x 6 heads, 4096 queries, 77 keys, d 64: 22 us; 4 key heads of 65,536 keys, d 128, and 777 queries
// of 16 heads: 41 (3.5 TB/s); forward and gradients of 8 x 6 heads, 4096 queries, 2048 keys, d 64: 80 (2.5 TB/s).  Next to
// them the start of a kernel (barriers, tensor memory, S: 2 us) and, of the small ones, the launches.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "cross.cuh"
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
  int a_h, a_b, b_h, b_b;      // whether the tensors have heads and batch entries (stride not 0)
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
// cross_inverse by the hardware's reciprocal (within a step of 2^-23).
__device__ __forceinline__ float inverse(float den) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(den));
  return den == 0.f ? 0.f : r;
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

// A d x d fp32 matrix [r][c] as bf16 tiles of D rows, the high part and, where lo is given, the low part.
template <int D>
__device__ __forceinline__ void load_matrix(uint8_t* hi, uint8_t* lo, const float* from) {
#pragma unroll
  for (int i = threadIdx.x; i < D * D / 8; i += Tc<D>::kWork) {
    const int r = i / (D / 8), j = i % (D / 8);
    float2 f[4];
    load8(from + r * D + 8 * j, f);
    const uint4 u = pack8(f);
    *piece(hi, D, r, j) = u;
    if (lo != nullptr) {
      remainder8(f, u);
      *piece(lo, D, r, j) = pack8(f);
    }
  }
}

// A thread's places in every tile: its row's four pieces of 32 columns, and what it stores, four times a piece of eight rows
// of 64 bytes (a warp's 32 rows x 32 columns).
struct Places {
  uint32_t own[4], out[4];
  int row, out_row, out_col;  // out_row: of the first of the four, eight apart
};
__device__ __forceinline__ Places places(int warp, int lane) {
  Places p;
  p.row = (warp & 3) * 32 + lane;
  p.out_row = (warp & 3) * 32 + lane / 4;
  const int j0 = (warp >> 2) * 4;
  p.out_col = 8 * (j0 + lane % 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + i, o = j0 + lane % 4, r = p.out_row + 8 * i;
    p.own[i] = (j >> 3) * kAtom + p.row * 128 + (((j & 7) ^ (p.row & 7)) << 4);
    p.out[i] = (o >> 3) * kAtom + r * 128 + (((o & 7) ^ (r & 7)) << 4);
  }
  return p;
}
__device__ __forceinline__ uint4& at_byte(uint8_t* tile, uint32_t offset) { return *reinterpret_cast<uint4*>(tile + offset); }
// The warp's part of a tile to memory; out: the tile's first row and the thread's columns; n rows of the tile are written.
__device__ __forceinline__ void store_rows(uint8_t* tile, const Places& p, __nv_bfloat16* out, long long sn, int n) {
  __nv_bfloat16* to = out + p.out_row * sn;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.out_row + 8 * i < n) *reinterpret_cast<uint4*>(to) = at_byte(tile, p.out[i]);
    to += 8 * sn;
  }
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
  constexpr uint32_t kColumns = 2 * D;
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
          mma_bf16(tmem, da + s * 128, d1 + s * 128, idesc_bf16_f32(128, kExact ? D : 2 * D, 1, 1), j > 0 || s > 0);
          if (!kExact) mma_bf16(tmem + D, da + s * 128, d2 + s * 128, idesc_bf16_f32(128, D, 1, 1), true);
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
          if (!kExact) {
            float w[32];
            tmem_ld16(at + D, w);
            tmem_ld16(at + D + 16, w + 16);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] += w[x];
          }
          tmem_ld_wait();
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) so[(c0 + x) * D + e] = tiles > 0 ? v[x] : 0.f;
      }
    }
  }
  finish<kSumBuffers, 2>(b, kColumns);
}

// ================================================================ read
// 8 x 6 heads of 4096 queries, d = 64: 19 us from a cold cache (50 MB); issue slots 40 %, the rest the start and the chain of a
// tile (copy, features, MMA, results) that three blocks an SM share.
// Three buffers and two accumulators: while the MMA of a tile runs the warps store the tile before and take the next one's
// features; one barrier of the block a tile, so what a tile leaves for the next turn lies in one of three places.
template <int D>
struct ReadSmem {
  static constexpr int kQ = 0, kS = 3 * Tc<D>::kTile, kZ = kS + Tc<D>::kMat, kDen = kZ + D * 4, kBars = kDen + 3 * Tc<D>::kCols * kT * 4;
  static constexpr int kBytes = 1024 + kBars + (int)sizeof(Bars);
};
template <int D, int F>
__global__ void __launch_bounds__(Tc<D>::kThreads, D == 64 ? 3 : 1) tc_cross_read_kernel(const __grid_constant__ TcArgs p) {
  using X = Tc<D>;
  using M = ReadSmem<D>;
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
  if (slot < 0 || slot >= p.c.n_slots) return finish<3, 2>(b, kColumns);
  const uint32_t tmem = b->tbase;
  const int tiles = (g.len + kT - 1) / kT, bb = p.c.qs.cu == nullptr ? g.seq : 0;
  const size_t unit = (size_t)slot * p.c.Hk + h / (p.c.H / p.c.Hk);
  if (tid < X::kWork) load_matrix<D>(sm + M::kS, nullptr, p.c.S + unit * D * D);
  if (tid < D) z[tid] = p.c.z[unit * D + tid];
  if (tid >= X::kWork) {
    if (lane == 0) {
      const auto fetch = [&](int j) {
        uint64_t* bar = &b->full[j % 3];
        mbar_arrive_expect_tx(bar, X::kTile);
        load_tile(sm + M::kQ + j % 3 * X::kTile, &p.a, g.row0 + j * kT, p.a_h ? h : 0, p.a_b ? bb : 0, bar);
        b->issued = j + 1;
      };
      const uint32_t sa = smem_u32(sm + M::kS);
      for (int j = 0; j < min(tiles, 3); ++j) fetch(j);
      for (int j = 0; j < tiles; ++j) {
        // every warp has the features of tile j (the first time: S) written, and tile j - 2 stored
        if (!wait(&b->ready[j % 3], (j / 3) & 1, b)) break;
        tc_fence_after();
        const uint32_t qa = smem_u32(sm + M::kQ + j % 3 * X::kTile);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_bf16(tmem + (j & 1) * D, along_cols<D>(qa, kAtom, s), along_rows(sa, D * 128) + s * 128, idesc_bf16_f32(128, D, 0, 1),
                   s > 0);
        mma_commit(&b->mma[j & 1]);
        b->mmas = j + 1;
        if (j >= 2 && j + 1 < tiles) fetch(j + 1);
      }
    }
    __syncwarp();
    __syncthreads();
    return finish<3, 2>(b, kColumns);
  }
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(X::kWork) : "memory");  // z
  const Places pl = places(warp, lane);
  const int row = pl.row, cg = warp >> 2;  // the thread's row, and its 32 columns
  const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + cg * 32;
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(const_cast<void*>(p.c.y.p)) + cross_base(p.c.qs, p.c.y, g.seq, h) +
                     (long long)g.row0 * p.c.y.sn + pl.out_col;
  bool ok = true;
  int buf = 0, before = 2, phase = 0;  // j % 3, (j - 1) % 3, j / 3 & 1
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
        for (int x = 0; x < 4; ++x) {
          f[x] = feature<F>(f[x]);
          d = fma2(f[x], zz[x], d);
        }
        if (F != MHLA_PHI_IDENTITY) *q = pack8(f);
      }
      den[(buf * X::kCols + cg) * kT + row] = d.x + d.y;
      arrive(&b->ready[buf], lane);
    }
    if (j > 0) {  // tile j - 1 goes out
      const int t = j - 1;
      uint8_t* qt = sm + M::kQ + before * X::kTile;
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
#pragma unroll
      for (int i = 0; i < 4; ++i) at_byte(qt, pl.own[i]) = pack8(v + 4 * i);
      __syncwarp();
      store_rows(qt, pl, y + (long long)t * kT * p.c.y.sn, p.c.y.sn, g.len - t * kT);
    }
    before = buf;
    buf = buf == 2 ? 0 : buf + 1;
    phase ^= buf == 0;
  }
  __syncthreads();
  finish<3, 2>(b, kColumns);
}

// ================================================================ backward over the queries
// 8 x 6 heads of 4096 queries, d = 64: 30 us from a cold cache (75 MB); issue slots 42 %, tensor pipe 17 %.  Bound by the chain
// of a tile: u, its row sums, dq and the stores; dS from w runs next to the sums.
// The tiles of d = 128 leave 3 KB of a block's 227: what is small lies before them, up to the next 1024 bytes.
template <int D>
struct QuerySmem {
  static constexpr int kQ = 0, kY = 2 * Tc<D>::kTile, kLo = 4 * Tc<D>::kTile, kS = 5 * Tc<D>::kTile, kSLo = kS + Tc<D>::kMat,
                       kEnd = kSLo + Tc<D>::kMat;
  static constexpr int kZ = 0, kDen = kZ + D * 4, kBars = kDen + Tc<D>::kCols * kT * 4, kSmall = kBars + (int)sizeof(Bars);
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
  const size_t unit = (size_t)g.seq * p.c.Hk + h / (p.c.H / p.c.Hk);
  if (tid < X::kWork) load_matrix<D>(sm + M::kS, sm + M::kSLo, p.c.S + unit * D * D);
  if (tid < D) z[tid] = p.c.z[unit * D + tid];
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
        if (j + 1 < tiles) fetch(j + 1);
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
      }
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
                      (long long)g.row0 * p.c.dq.sn + pl.out_col;
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
      dd *= -inv * inv;
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
    __syncwarp();
    store_rows(qt, pl, dq + (long long)j * kT * p.c.dq.sn, p.c.dq.sn, n);
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
// 8 x 6 heads of 2048 keys, d = 64: 19 us from a cold cache (50 MB), the matrices' parts and the chain of a tile.
// d = 64: three buffers and two accumulators, as the read; d = 128: two buffers and one accumulator.
template <int D>
struct KeySmem {
  static constexpr int kBuffers = D == 64 ? 3 : 2, kAcc = D == 64 ? 2 : 1;
  static constexpr int kK = 0, kV = kBuffers * Tc<D>::kTile, kS = 2 * kBuffers * Tc<D>::kTile, kSLo = kS + Tc<D>::kMat,
                       kEnd = kSLo + Tc<D>::kMat;
  static constexpr int kZ = 0, kBars = kZ + D * 4, kSmall = kBars + (int)sizeof(Bars);
  static constexpr int kBytes = (kSmall + 1023) / 1024 * 1024 + kEnd;
  static_assert(kBytes <= (D == 64 ? 115712 : 232448), "two blocks of d = 64 an SM, one of d = 128");
};
template <int D, int F>
__global__ void __launch_bounds__(Tc<D>::kThreads, D == 64 ? 2 : 1) tc_cross_key_kernel(const __grid_constant__ TcArgs p) {
  using X = Tc<D>;
  using M = KeySmem<D>;
  constexpr int NB = M::kBuffers, NA = M::kAcc;
  constexpr uint32_t kColumns = 2 * D * NA;  // dv, dphi(k), an accumulator each
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
  if (g.seq < 0) return finish<NB, NA>(b, kColumns);
  const int rows = p.c.ks.cu != nullptr ? g.len : min(p.c.ks.L, p.c.ks.N - g.row0);  // dense: zeros behind the tokens
  const uint32_t tmem = b->tbase;
  const int tiles = (rows + kT - 1) / kT, bb = p.c.ks.cu == nullptr ? g.seq : 0;
  const float* from = p.c.dS + ((size_t)g.seq * p.c.Hk + h) * (D * D + D);
  if (tid < X::kWork) load_matrix<D>(sm + M::kS, sm + M::kSLo, from);
  if (tid < D) z[tid] = from[D * D + tid];
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
      // so many tiles that the warps may be at: tile j's features wait for the tile j - LAG stored
      constexpr int LAG = NA;
      for (int j = 0; j < min(tiles, NB == 3 ? 3 : 1); ++j) fetch(j);
      for (int j = 0; j < tiles; ++j) {
        // every warp has the features of tile j (the first time: dS) written, and tile j - LAG stored
        if (!wait(&b->ready[j % NB], (j / NB) & 1, b)) break;
        tc_fence_after();
        const uint32_t ka = smem_u32(sm + M::kK + j % NB * X::kTile), va = smem_u32(sm + M::kV + j % NB * X::kTile);
        const uint32_t acc = tmem + j % NA * 2 * D;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            mma_bf16(acc, along_cols<D>(ka, kAtom, s), along_rows(part ? sl : sa, D * 128) + s * 128, idesc_bf16_f32(128, D, 0, 1),
                     s > 0 || part > 0);
            mma_bf16(acc + D, along_cols<D>(va, kAtom, s), along_cols<D>(part ? sl : sa, D * 128, s),
                     idesc_bf16_f32(128, D, 0, 0), s > 0 || part > 0);
          }
        mma_commit(&b->mma[j % NA]);
        b->mmas = j + 1;
        if (j >= LAG && j + 1 < tiles && NB == 3) fetch(j + 1);
        if (NB == 2 && j + 1 < tiles) fetch(j + 1);
      }
    }
    __syncwarp();
    __syncthreads();
    return finish<NB, NA>(b, kColumns);
  }
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(X::kWork) : "memory");  // z
  const Places pl = places(warp, lane);
  const int row = pl.row, cg = warp >> 2;
  const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + cg * 32;
  __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(const_cast<void*>(p.c.dk.p)) + cross_base(p.c.ks, p.c.dk, g.seq, h) +
                      (long long)g.row0 * p.c.dk.sn + pl.out_col;
  __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(const_cast<void*>(p.c.dv.p)) + cross_base(p.c.ks, p.c.dv, g.seq, h) +
                      (long long)g.row0 * p.c.dv.sn + pl.out_col;
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
    arrive(&b->ready[j % NB], lane);
    return true;
  };
  bool ok = tiles == 0 || features(0);
  for (int j = 0; ok && j < tiles; ++j) {
    uint8_t *kt = sm + M::kK + j % NB * X::kTile, *vt = sm + M::kV + j % NB * X::kTile;
    if (NA == 2 && j + 1 < tiles && !features(j + 1)) break;
    ok = __all_sync(0xffffffffu, wait(&b->mma[j % NA], (j / NA) & 1, b));
    if (!ok) break;
    tc_fence_after();
    const bool live = row < g.len - j * kT;
    const uint32_t acc = at + j % NA * 2 * D;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 u[8], v[8];
      tmem_ld8(acc + D + 16 * c, u);
      tmem_ld8(acc + 16 * c, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 f[4], zz[4];
        unpack8(at_byte(kt, pl.own[2 * c + i]), f);  // (phi rounded to bf16: phi' goes by it, and its rounding by dk's)
        load8(z + cg * 32 + 16 * c + 8 * i, zz);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          u[4 * i + x] = mul2(slope<F>(f[x]), add2(u[4 * i + x], zz[x]));
          if (!live) u[4 * i + x] = v[4 * i + x] = both(0.f);
        }
        at_byte(kt, pl.own[2 * c + i]) = pack8(u + 4 * i);
        at_byte(vt, pl.own[2 * c + i]) = pack8(v + 4 * i);
      }
    }
    __syncwarp();
    const int m = rows - j * kT;
    store_rows(kt, pl, dk + (long long)j * kT * p.c.dk.sn, p.c.dk.sn, m);
    store_rows(vt, pl, dv + (long long)j * kT * p.c.dv.sn, p.c.dv.sn, m);
    if (NA == 1 && j + 1 < tiles) ok = features(j + 1);
  }
  __syncthreads();
  finish<NB, NA>(b, kColumns);
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

// The launch's arguments, with the maps of the tile's one or two tensors.
bool make_args(TcArgs* t, const CrossArgs& a, const CrossSide& s, int heads, const RetTensor& x, const RetTensor* y,
               int box_rows = kT) {
  t->c = a;
  t->wait_ns = g_wait_ns;
  t->a_h = x.sh != 0;
  t->a_b = x.sb != 0 && s.cu == nullptr;
  t->b_h = y != nullptr && y->sh != 0;
  t->b_b = y != nullptr && y->sb != 0 && s.cu == nullptr;
  return make_map(&t->a, x, s, heads, a.d, box_rows) && (y == nullptr || make_map(&t->b, *y, s, heads, a.d, box_rows));
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
  if (!make_args(&t, a, a.ks, a.Hk, a.k, &a.v, kSumT)) return cudaErrorInvalidValue;
  static SmemOptIn opt;
  return launch(tc_cross_states_kernel<D, F>, opt, (long long)a.ks.segs * a.Hk, Tc<D>::kThreads, SumSmem<D>::kBytes, t, st);
}
template <int D, int F>
cudaError_t read_t(const CrossArgs& a, cudaStream_t st) {
  TcArgs t;
  if (!make_args(&t, a, a.qs, a.H, a.q, nullptr)) return cudaErrorInvalidValue;
  static SmemOptIn opt;
  return launch(tc_cross_read_kernel<D, F>, opt, (long long)a.qs.segs * a.H, Tc<D>::kThreads, ReadSmem<D>::kBytes, t, st);
}
template <int D, int F>
cudaError_t backward_t(const CrossArgs& a, cudaStream_t st) {
  TcArgs t;
  static SmemOptIn opt_q, opt_k;
  cudaError_t e = cudaSuccess;
  if (a.qs.segs > 0) {
    if (!make_args(&t, a, a.qs, a.H, a.q, &a.dy)) return cudaErrorInvalidValue;
    e = launch(tc_cross_query_kernel<D, F>, opt_q, (long long)a.qs.segs * a.H, Tc<D>::kThreads, QuerySmem<D>::kBytes, t, st);
  }
  if (e != cudaSuccess || a.ks.segs == 0) return e;
  e = cross_join_launch(a, true, st);
  if (e != cudaSuccess) return e;
  if (!make_args(&t, a, a.ks, a.Hk, a.k, &a.v)) return cudaErrorInvalidValue;
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
