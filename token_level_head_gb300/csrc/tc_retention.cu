// Retention passes on the sm_103a tensor cores (bf16).  The mathematics is in retention.h; a pass cuts
// a segment into chunks of 128 tokens (len of them in the sequence) and carries X, the state entering
// the chunk ([D][D], fp32 in tensor memory):
//   scores = A B^T                               M 128, N 128, K D
//   P      = scores * gamma^(t-s), masked        bf16, written over the scores in TMEM
//   inter  = A bf16(X)                           M 128, N D, K D
//   intra  = P C                                 M 128, N D, K 128 (A from TMEM)
//   dX     = (B w)^T C, w_s = gamma^(len-1-s)    M D, N D, K 128
//   out    = scale (intra + gamma^(i+1) inter),  X = gamma^len X + dX
// A reverse pass is the same with the order of the tokens turned round: P takes s >= t, w_s = gamma^s,
// inter is weighted by gamma^(len-i).
//
// What is rounded to bf16: the masked scores, the copy of X that the product reads (X itself stays
// fp32) and phi of operands with a feature map.  B w is carried as a sum of bf16 numbers: of two (over
// the B tile and in a tile of its own: 2^-16 of a term) where only bf16 outputs come of it or the decay
// leaves less than 1/8 of it, of three (the last over the tile of X: 2^-24) in the chunks that make up a
// state which is returned in fp32.
//
// Roles (D = 128: 22 warps and one CTA an SM, D = 64: 14 warps and two):
//   warp 0       TMA producer: the tiles of a chunk, B and C two chunks deep, A one
//   warp 1       MMA issuer
//   8 out warps  scores -> P, then out = scale (intra + gamma^(i+1) inter) to global memory: two for each
//                quarter of the rows, with half of the scores and of the columns each
//   4 W warps    feature maps in place, B w
//   X warps      X and its bf16 tile for the next chunk: eight (D = 128), or the W warps themselves (D = 64)
// What bounds it: chains of short steps, not a pipe.  With D = 128 a chunk takes about 6 thousand cycles an SM; its
// products need 2.6 of the tensor cores (128 x 128 x 16: 64 cycles) and about 4.4 thousand of shared memory's bandwidth
// (128 bytes a cycle: the products' operands 2.3, TMA 0.8, B w 0.8, X and the scores' weights 0.6).  Two chains run
// beside each other: scores, P, intra, out (the out warps are busy nearly all of it), and dX, X, inter.  With D = 64
// a chunk takes 4.5 thousand cycles in one CTA, 6 thousand in each of two on an SM; the instruction issue is at 34 %,
// the tensor cores at 25 %, HBM at 45 %.  Measured for prompts: 8 heads of 65,536 tokens, d = 128, 97 us of the call's
// 152 (537 MB at 5.5 TB/s); 4 x 16 heads of 8192 tokens, d = 64, 65 us of 101 (268 MB at 4.1 TB/s).  A block by itself, 16
// heads, d = 64: a call of one whole chunk takes 5.5 us on the device without a state, 7.9 with one taken and left, 0.5 more
// with slot numbers, and every further chunk 2.4 or 3.2; a chunk that is not whole 1.3 to 2 us more at the start (rows behind it are
// cleared before the scores, behind the state's load).
// Feature maps are far dearer: they are applied in the operands' tiles between the loads and the scores of every chunk, and
// where a state is returned every chunk's B w has three parts, of phi taken again from global memory.  ELU + 1 against the
// identity: 4 x 16 heads of 8192 tokens 344 us and 102, 8 heads of 65,536, d = 128, 659 and 154, gradients of 64 heads of 4096
// tokens 412 and 103, of 12 packed sequences of 16,384 tokens, d = 128, 650 and 162.  Widths below 64 run as 64 with zero
// columns: 91 us with d = 16, 93 with 32, 102 with 64.
//
// The roles' loops are kept short and free of branches: with whole rows unrolled the instruction fetch,
// not the arithmetic, set the pace (23,000 cycles a chunk), and stores of one row a thread held up the
// loads and stores of shared memory beside them (67 cycles each).
// All waits are bounded: on time-out the kernel sets the status word and winds down.
//
// A sequence of several segments needs the states that enter them: retention_sum_kernel forms each
// segment's own sum of gamma^(distance to its end) b c^T (the decays go into B w, so the accumulator
// stays in TMEM over the whole segment), the scan of retention_simt.cu chains them.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "internal.h"
#include "retention.cuh"
#include "tc_common.cuh"

namespace mhla {
namespace {

using namespace tc;

constexpr int kTok = 128;                    // tokens of a chunk
constexpr int kAtom = kTok * 128;            // 16 KB: 128 rows x 64 bf16, 128-byte swizzle
constexpr int kWarpProd = 0, kWarpMma = 1, kWarpOut = 2;
constexpr int kStages = 2;
constexpr uint64_t kWaitLimitNs = 500000000ull;
unsigned long long g_wait_ns = kWaitLimitNs;

struct TcArgs {
  CUtensorMap tm[4];                         // q, k, v, dy as [B][H][N][d], box 64 x 128
  int by_b[4], by_h[4];                      // 0: shared by the batch / the heads
  int ia[kRetMaxPasses], ib[kRetMaxPasses], ic[kRetMaxPasses];  // tensor maps of a pass's operands
  unsigned long long wait_ns;
  RetArgs r;
};

// ---------------------------------------------------------------- bounded waits
struct Guard {
  int* abort;
  unsigned long long limit;
};
__device__ __forceinline__ Guard make_guard(int* abort, unsigned long long limit) { return {abort, limit}; }
__device__ __forceinline__ bool aborted(const Guard& g) { return *reinterpret_cast<volatile int*>(g.abort) != 0; }
constexpr uint32_t kNapNs = 1000;
// The thread sleeps in the barrier's own wait; the clock is read only after about a microsecond of that, and a limit
// below one sleep gives up at once.  (Inline: a call would save the caller's registers, and most waits do wait.)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Guard& g) {
  if (mbar_test(bar, parity)) return true;
  uint64_t t0 = 0;
#pragma unroll 1
  while (g.limit >= kNapNs) {
    if (mbar_try_wait_ns(bar, parity, kNapNs)) return true;
    if (aborted(g)) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0)
      t0 = now;
    else if (now - t0 > g.limit)
      break;
  }
  *reinterpret_cast<volatile int*>(g.abort) = 1;
  return false;
}
// The whole warp: all lanes go on, or none.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Guard& g) {
  return __all_sync(0xffffffffu, wait(bar, parity, g)) != 0;
}
// Short wait (10 ms at most), only while winding down.
__device__ __noinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_ns(bar, parity, 1000))
    if (globaltimer_ns() - t0 > 10000000ull) return;
}

// ---------------------------------------------------------------- tiles
// 16-byte piece j (columns 8 j ..) of row r of a tile of 64-column atoms of `rows` rows each.
__device__ __forceinline__ uint4* piece(uint8_t* tile, int rows, int r, int j) {
  return reinterpret_cast<uint4*>(tile + (j >> 3) * (rows * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void unpack8(uint4 u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    f[2 * m] = __uint_as_float(w[m] << 16);
    f[2 * m + 1] = __uint_as_float(w[m] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// phi over the d columns of row r of a tile in place, zeros for a row behind the sequence.
template <int D>
__device__ __noinline__ void map_row(uint8_t* tile, int r, int len, int d, int feature) {
#pragma unroll 2
  for (int j = 0; j < D / 8; ++j) {
    uint4* p = piece(tile, kTok, r, j);
    if (r >= len) {
      *p = make_uint4(0, 0, 0, 0);
    } else if (feature != kFeatIdentity && 8 * j < d) {
      float f[8];
      unpack8(*p, f);
#pragma unroll
      for (int x = 0; x < 8; ++x) f[x] = ret_phi(f[x], feature);
      *p = pack8(f);
    }
  }
}

// f - bf16(f) in place, given bf16(f) packed.
__device__ __forceinline__ void remainder8(float* f, uint4 h) {
  float g[8];
  unpack8(h, g);
#pragma unroll
  for (int x = 0; x < 8; ++x) f[x] -= g[x];
}

// f[0..8) as a sum of three bf16 numbers at piece j of row r: over the B tile, the remainder in lo, the
// remainder of that in lo2.
__device__ __forceinline__ void split8(float* f, uint8_t* hi, uint8_t* lo, uint8_t* lo2, int r, int j) {
  const uint4 h = pack8(f);
  *piece(hi, kTok, r, j) = h;
  remainder8(f, h);
  const uint4 l = pack8(f);
  *piece(lo, kTok, r, j) = l;
  remainder8(f, l);
  *piece(lo2, kTok, r, j) = pack8(f);
}

// D columns, from 8 jb, of row r of B times w as a sum of three bf16 numbers.
template <int D>
__device__ __forceinline__ void weigh_row3(uint8_t* hi, uint8_t* lo, uint8_t* lo2, int r, int jb, float w) {
#pragma unroll 1
  for (int j0 = jb; j0 < jb + D / 8; j0 += 2) {
    uint4 u[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) u[j] = *piece(hi, kTok, r, j0 + j);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float f[8];
      unpack8(u[j], f);
#pragma unroll
      for (int x = 0; x < 8; ++x) f[x] *= w;
      split8(f, hi, lo, lo2, r, j0 + j);
    }
  }
}

// D columns, from 8 jb, of row r of B times w as a sum of two bf16 numbers, in packed bf16 arithmetic: with w = wh + wl in
// bf16, hi = round(b wh), b wh - hi is exact (16 bits less the first 8), lo = round(b wl + that).  A quarter of
// the instructions of the same in fp32.
template <int D>
__device__ __forceinline__ void weigh_row2(uint8_t* hi, uint8_t* lo, int r, int jb, float w) {
  const __nv_bfloat16 wh1 = __float2bfloat16_rn(w);
  const __nv_bfloat162 wh = __bfloat162bfloat162(wh1);
  const __nv_bfloat162 wl = __bfloat162bfloat162(__float2bfloat16_rn(w - __bfloat162float(wh1)));
#pragma unroll 1
  for (int j0 = jb; j0 < jb + D / 8; j0 += 4) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = *piece(hi, kTok, r, j0 + j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t x[4] = {u[j].x, u[j].y, u[j].z, u[j].w}, h[4], l[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&x[m]);
        const __nv_bfloat162 hv = __hmul2_rn(v, wh);
        const __nv_bfloat162 lv = __hfma2(v, wl, __hfma2(v, wh, __hneg2(hv)));
        h[m] = *reinterpret_cast<const uint32_t*>(&hv);
        l[m] = *reinterpret_cast<const uint32_t*>(&lv);
      }
      *piece(hi, kTok, r, j0 + j) = make_uint4(h[0], h[1], h[2], h[3]);
      *piece(lo, kTok, r, j0 + j) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

// weigh_row3 of phi of the row, in fp32, over its d columns: of the row in global memory (raw), the tile holds
// the rounded phi already.
template <int D>
__device__ __noinline__ void weigh_phi_row3(uint8_t* hi, uint8_t* lo, uint8_t* lo2, int r, int jb, float w,
                                            const __nv_bfloat16* raw, int d, int feature) {
#pragma unroll 1
  for (int j = jb; j < jb + D / 8; ++j) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (w != 0.f && 8 * j < d) {
      unpack8(*reinterpret_cast<const uint4*>(raw + 8 * j), f);
#pragma unroll
      for (int x = 0; x < 8; ++x) f[x] = w * ret_phi(f[x], feature);
    }
    split8(f, hi, lo, lo2, r, j);
  }
}

// D columns, from 8 jb, of phi of row r of B times w as a sum of two bf16 numbers; w = 0: zeros.
template <int D>
__device__ __noinline__ void weigh_phi_row2(uint8_t* hi, uint8_t* lo, int r, int jb, float w, int d, int feature) {
#pragma unroll 1
  for (int j = jb; j < jb + D / 8; ++j) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (w != 0.f && 8 * j < d) {
      unpack8(*piece(hi, kTok, r, j), f);
#pragma unroll
      for (int x = 0; x < 8; ++x) f[x] = w * ret_phi(f[x], feature);
    }
    const uint4 h = pack8(f);
    *piece(hi, kTok, r, j) = h;
    remainder8(f, h);
    *piece(lo, kTok, r, j) = pack8(f);
  }
}

// ---------------------------------------------------------------- products
// Shared-memory descriptors are kept as their two words: only the start address, in the low one, changes.
struct Desc {
  uint32_t lo, hi;
};
__device__ __forceinline__ Desc make_desc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  const uint64_t d = smem_desc(saddr, lbo_bytes, sbo_bytes);
  return {(uint32_t)d, (uint32_t)(d >> 32)};
}

// One MMA, K = 16: A at `bytes_a` behind its descriptor's start, B at `bytes_b`; the constants are immediates, so
// that the issuing thread spends a few instructions on each.
template <uint32_t IDESC, bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, Desc a, uint32_t bytes_a, Desc b, uint32_t bytes_b) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a.lo + (bytes_a >> 4)), "r"(a.hi), "r"(b.lo + (bytes_b >> 4)), "r"(b.hi), "r"(IDESC), "n"(ACC ? 1 : 0)
      : "memory");
}
template <uint32_t IDESC, bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, Desc b, uint32_t bytes_b) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b.lo + (bytes_b >> 4)), "r"(b.hi), "r"(IDESC), "n"(ACC ? 1 : 0)
      : "memory");
}

// D[tmem] (+)= A^T B, both operands MN-major: A [128 rows][M], B [128 rows][N columns from `col`].
template <int M, int N, bool ACC>
__device__ __forceinline__ void mma_outer(uint32_t d, Desc a, Desc b, uint32_t col = 0) {
  constexpr uint32_t kId = idesc_bf16_f32(M, N, 1, 1);
  mma_ss<kId, ACC>(d, a, 0, b, 2 * col);
#pragma unroll
  for (int k = 1; k < kTok / 16; ++k) mma_ss<kId, true>(d, a, k * 2048, b, k * 2048 + 2 * col);
}

// Prefetch of one operand's chunk into L2.
template <int D>
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int row, int h, int seq) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(64 * c), "r"(row), "r"(h), "r"(seq)
                 : "memory");
}

// TMA of one operand's chunk: D / 64 atoms.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int row, int h, int seq,
                                          uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * kAtom, map, 64 * c, row, h, seq, bar);
}

// ================================================================ pass
template <int D>
struct PassTile {
  static constexpr int kOp = (D / 64) * kAtom;          // an operand's tile
  static constexpr int kOffA = 0, kOffBC = kOp;         // A; kStages x (B, C)
  static constexpr int kOffLo = kOffBC + kStages * 2 * kOp;  // second part of B w
  static constexpr int kOffX = kOffLo + kOp;            // bf16 X: D rows c, D columns e (third part of B w)
  static constexpr int kOffBars = kOffX + kOp;
  static constexpr uint32_t kCols = D == 128 ? 512 : 256;
  // scores; P of tokens 0 .. 63 over their columns 0 .. 31, of tokens 64 .. 127 over 64 .. 95: each over scores
  // that its own warp has read
  static constexpr uint32_t kColS = 0;
  // intra: D = 128 in columns of its own, D = 64 over the scores that P leaves free, 32 columns in two places
  static constexpr uint32_t intra(uint32_t c) { return D == 128 ? 256 + c : 32 + c + (c & 32); }
  static constexpr uint32_t kColInter = 128;
  static constexpr uint32_t kColX = D == 128 ? 384 : 192;     // X gamma^len, dX is added to it
  // dX by itself, where the state is returned: over P (D = 64: in its two places)
  static constexpr uint32_t apart(uint32_t c) { return D == 128 ? c : c + (c & 32); }
  static constexpr int kPerSm = D == 128 ? 1 : 2;
  static constexpr int kWarpW = kWarpOut + 8, kWarpX = D == 128 ? kWarpW + 4 : kWarpW;
  static constexpr int kXWarps = D == 128 ? 8 : 4;
  static constexpr int kThreads = 32 * (kWarpX + kXWarps);
};

// What the roles share.  It is kept in shared memory and the roles are functions of their own, so that none
// holds registers for another.
struct PassCtx {
  const CUtensorMap *ma, *mb, *mc;
  int ha, hb, hc, ba, bb, bc;    // head and batch coordinates in the maps
  int row0, len, n;              // first row, tokens, chunks
  int nx;                        // chunks whose dX is needed
  int reverse;                   // direction
  int exact;                     // first chunk whose B w is a sum of three bf16 numbers and whose dX is apart
  int fa, fb, fc, fx;            // feature maps of A, B, C and x
  int d;
  float lg;
  __nv_bfloat16* out;            // of the head; rows out_n apart
  const __nv_bfloat16 *x, *b;    // of the head: x (null: none), B
  long long out_n, x_n, b_n;
  const float* from;             // state entering the segment, null: zero
  int from_t, from_ws;           // it is transposed; it is in the workspace
  float* to;                     // where the state after it goes, null: nowhere
  unsigned long long wait_ns;
  __device__ __forceinline__ bool mapped() const {
    return fa != kFeatIdentity || fb != kFeatIdentity || fc != kFeatIdentity;
  }
};
__device__ __forceinline__ int chunk_of(int i, int n, int reverse) { return reverse ? n - 1 - i : i; }
__device__ __forceinline__ int chunk_len(int ch, int len) { return min(kTok, len - ch * kTok); }

struct PassBars {
  uint64_t a_full;    // A (read for the last time by inter: in_full)
  uint64_t full[kStages], empty[kStages];  // B, C
  uint64_t mapped;    // feature maps applied / rows behind the sequence cleared (W warps)
  uint64_t s_full;    // scores
  uint64_t in_full;   // inter
  uint64_t p_full;    // P in TMEM (out warps)
  uint64_t w_full;    // B w (W warps)
  uint64_t w2_full;   // D = 128, three parts: the X warps' columns of it
  uint64_t dx_full;   // dX
  uint64_t x_full;    // the bf16 tile of X (X warps)
  uint64_t o_full;    // intra
  uint64_t o_free;    // inter and intra read (out warps)
  uint64_t fin;       // every MMA of the CTA has completed
  uint32_t tbase;
  int abort;
  int issued, issued_a;  // chunks whose B and C, whose A the producer asked for
  // scale gamma^n, 32 zeros beside it: forward [32 + n], reverse [kTok - 1 - n] (first the segment search's scratch)
  float decay[kTok + 32];
  PassCtx ctx;
};

template <int D>
constexpr size_t pass_smem() {  // (the kernels' shared memory starts on 1024 bytes: no room to align it)
  return PassTile<D>::kOffBars + sizeof(PassBars);
}
static_assert(pass_smem<128>() <= 232448 && 2 * (pass_smem<64>() + 1024) <= 233472, "shared memory budget");

// The loads of chunk i's B and C, and of its A (one thread).
template <int D>
__device__ __forceinline__ void load_bc(uint8_t* sm, PassBars* b, const PassCtx& c, int i) {
  using P = PassTile<D>;
  const int s = i % kStages, row = c.row0 + chunk_of(i, c.n, c.reverse) * kTok;
  uint8_t* st = sm + P::kOffBC + s * 2 * P::kOp;
  mbar_arrive_expect_tx(&b->full[s], 2 * P::kOp);
  load_tile<D>(st, c.mb, row, c.hb, c.bb, &b->full[s]);
  load_tile<D>(st + P::kOp, c.mc, row, c.hc, c.bc, &b->full[s]);
  b->issued = i + 1;
}
template <int D>
__device__ __forceinline__ void load_a(uint8_t* sm, PassBars* b, const PassCtx& c, int i) {
  mbar_arrive_expect_tx(&b->a_full, PassTile<D>::kOp);
  load_tile<D>(sm + PassTile<D>::kOffA, c.ma, c.row0 + chunk_of(i, c.n, c.reverse) * kTok, c.ha, c.ba, &b->a_full);
  b->issued_a = i + 1;
}

// (The block's start has loaded chunk 0 and B and C of chunk 1.)  A has one tile: it is asked for when the last one
// has been read, and brought to L2 before.
template <int D>
__device__ __noinline__ void pass_producer(uint8_t* sm, PassBars* b) {
  const PassCtx c = b->ctx;
  const Guard gd = make_guard(&b->abort, c.wait_ns);
  for (int i = 1; i < c.n; ++i) {
    prefetch_tile<D>(c.ma, c.row0 + chunk_of(i, c.n, c.reverse) * kTok, c.ha, c.ba);
    if (!wait(&b->in_full, (i - 1) & 1, gd)) return;
    load_a<D>(sm, b, c, i);
    if (i + 1 < c.n) {
      if (!wait(&b->empty[(i + 1) % kStages], ((i + 1) / kStages - 1) & 1, gd)) return;
      load_bc<D>(sm, b, c, i + 1);
    }
  }
}

// The whole warp waits, one lane issues (the same one each time: elect.sync is deterministic).  With the issue
// under an election the operands stay in uniform registers: an MMA costs the issuing lane 14 cycles, not 45.
template <int D>
__device__ __noinline__ void pass_mma(uint8_t* sm, PassBars* b) {
  using P = PassTile<D>;
  const int n = b->ctx.n, nx = b->ctx.nx, len = b->ctx.len, reverse = b->ctx.reverse, exact = b->ctx.exact;
  const bool mapped = b->ctx.mapped();
  const uint32_t tmem = b->tbase;
  const Guard gd = make_guard(&b->abort, b->ctx.wait_ns);
  // K-major A and B for the scores; MN-major: X (rows c), B w, its other parts and C (rows = tokens)
  const Desc qa = make_desc(smem_u32(sm + P::kOffA), 16, 1024), x = make_desc(smem_u32(sm + P::kOffX), D * 128, 1024);
  const Desc bk0 = make_desc(smem_u32(sm + P::kOffBC), 16, 1024);
  const Desc bm0 = make_desc(smem_u32(sm + P::kOffBC), kAtom, 1024);
  const Desc lo = make_desc(smem_u32(sm + P::kOffLo), kAtom, 1024), lo2 = make_desc(smem_u32(sm + P::kOffX), kAtom, 1024);
  auto stage = [&](Desc d, int i) {  // of chunk i
    d.lo += (i % kStages) * (2 * P::kOp >> 4);
    return d;
  };
  const Desc cm0{bm0.lo + (P::kOp >> 4), bm0.hi};
  int maps = 0;  // chunks whose operands the W warps have changed
  auto scores = [&](int i) {
    if (!wait_warp(&b->full[i % kStages], (i / kStages) & 1, gd) || !wait_warp(&b->a_full, i & 1, gd)) return false;
    if (mapped || chunk_len(chunk_of(i, n, reverse), len) < kTok) {
      if (!wait_warp(&b->mapped, maps & 1, gd)) return false;
      ++maps;
    }
    tc_fence_after();
    __syncwarp();
    if (elect_one()) {
      constexpr uint32_t kId = idesc_bf16_f32(128, 128, 0, 0);
      const Desc bk = stage(bk0, i);
      mma_ss<kId, false>(tmem + P::kColS, qa, 0, bk, 0);
#pragma unroll
      for (int k = 1; k < D / 16; ++k) {
        const uint32_t off = (k / 4) * kAtom + (k % 4) * 32;
        mma_ss<kId, true>(tmem + P::kColS, qa, off, bk, off);
      }
      mma_commit(&b->s_full);
    }
    return true;
  };
  if (!scores(0)) return;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int s = i % kStages;
    const Desc cm = stage(cm0, i);
    if (!wait_warp(&b->x_full, i & 1, gd)) return;
    if (D != 64 && i > 0 && !wait_warp(&b->o_free, (i - 1) & 1, gd)) return;
    tc_fence_after();
    __syncwarp();
    if (elect_one()) {
      constexpr uint32_t kId = idesc_bf16_f32(128, D, 0, 1);
      mma_ss<kId, false>(tmem + P::kColInter, qa, 0, x, 0);
#pragma unroll
      for (int k = 1; k < D / 16; ++k)
        mma_ss<kId, true>(tmem + P::kColInter, qa, (k / 4) * kAtom + (k % 4) * 32, x, k * 2048);
      mma_commit(&b->in_full);
    }
    if (!wait_warp(&b->p_full, i & 1, gd)) return;
    tc_fence_after();
    __syncwarp();
    if (elect_one()) {
      constexpr int kN = D == 128 ? 128 : 32;  // columns of intra in one place
      constexpr uint32_t kId = idesc_bf16_f32(128, kN, 0, 1);
#pragma unroll
      for (int e = 0; e < D; e += kN) {
        mma_ts<kId, false>(tmem + P::intra(e), tmem + P::kColS, cm, 2 * e);
#pragma unroll
        for (int k = 1; k < kTok / 16; ++k)
          mma_ts<kId, true>(tmem + P::intra(e), tmem + P::kColS + 8 * k + (k >= 4 ? 32 : 0), cm, k * 2048 + 2 * e);
      }
      mma_commit(&b->o_full);
      if (i >= nx) mma_commit(&b->empty[s]);
    }
    const bool more = i + 1 < n, apart = i >= exact && i < nx;
    // The next chunk's scores go over P, with D = 64 over intra too, so behind the intra (the out warps) of this one.
    // D = 64: the longest chain is scores, P, intra, out; this chunk's dX comes behind the scores (gradients of 64 heads
    // of 4096 tokens: 104 us, 107 the other way).  D = 128: it is dX, X, inter; dX comes first (8 heads of 65,536
    // tokens: 156 us, 169 the other way).
    // (w_full: the W warps have passed s_full, which may go on.)
    if (i < nx && !wait_warp(&b->w_full, i & 1, gd)) return;
    if (D == 64 && more && !apart && (!wait_warp(&b->o_free, i & 1, gd) || !scores(i + 1))) return;
    if (i < nx) {
      if (apart && (!wait_warp(&b->o_full, i & 1, gd) || (D == 128 && !wait_warp(&b->w2_full, (i - exact) & 1, gd)))) return;
      const Desc bm = stage(bm0, i);
      tc_fence_after();
      __syncwarp();
      if (elect_one()) {
        if (apart) {
          // The accumulator rounds towards zero at each of these: dX is added up by itself, over P, and then, in fp32,
          // to X.  (On top of X the state of 4,000 tokens was off by 2^-19, so by 2^-21.)
          constexpr int kN = D == 128 ? 128 : 32;
#pragma unroll
          for (int e = 0; e < D; e += kN) {
            mma_outer<D, kN, false>(tmem + P::kColS + P::apart(e), bm, cm, e);
            mma_outer<D, kN, true>(tmem + P::kColS + P::apart(e), lo, cm, e);
            mma_outer<D, kN, true>(tmem + P::kColS + P::apart(e), lo2, cm, e);
          }
        } else {
          mma_outer<D, D, true>(tmem + P::kColX, bm, cm);
          mma_outer<D, D, true>(tmem + P::kColX, lo, cm);
        }
        mma_commit(&b->dx_full);
        mma_commit(&b->empty[s]);
      }
    }
    if (more && (D == 128 || apart)) {
      if (!wait_warp(&b->o_full, i & 1, gd) || (D == 64 && !wait_warp(&b->o_free, i & 1, gd))) return;
      if (apart && !wait_warp(&b->x_full, (i + 1) & 1, gd)) return;  // (dX has been read)
      if (!scores(i + 1)) return;
    }
  }
}

// 16 lanes x 32 columns: registers 4 g + {0, 1} are columns 8 g + 2 (l % 4) + {0, 1} of row l / 4, 4 g + {2, 3}
// those of row l / 4 + 8.
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// The reverse of tmem_ld16x32.
__device__ __forceinline__ void tmem_st16x32(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}

// The four lanes of a group of four hold e[0 .. 3]: lane q gets element q of lane k as its element k.
__device__ __forceinline__ void turn4(uint32_t* e, int lane) {
#pragma unroll
  for (int s = 1; s <= 2; s <<= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & s) continue;
      uint32_t &a = e[k], &b = e[k | s];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, s);
      if (up)
        a = got;
      else
        b = got;
    }
  }
}

// Out warps, TMEM lane quadrant = warp % 4, token row t = a lane.  The two warps of a quadrant take half of the scores
// and of the output columns each.  What does not change is kept out of the loop: with D = 128 three instructions more
// for each store cost 7 % of a call of 8 heads of 65,536 tokens (156 -> 167 us).
template <int D, bool DERIV>
__device__ __noinline__ void pass_out(PassBars* b, int warp, int lane) {
  using P = PassTile<D>;
  const int qd = warp & 3, row = 32 * qd + lane, half = (warp - kWarpOut) >> 2;
  const int n = b->ctx.n, all = b->ctx.len, reverse = b->ctx.reverse;
  const int d0 = half * (D / 2);
  const uint32_t tl = b->tbase + ((uint32_t)(32 * qd) << 16);
  const Guard gd = make_guard(&b->abort, b->ctx.wait_ns);
  const float* decay = b->decay + (reverse ? kTok - 1 : 32);  // [t - s]: its weight, 0 on the masked side
  // out: this lane's rows rw, rw + 8, .. of a chunk, and the first of its columns once they are turned round
  const int rw = 32 * qd + (lane >> 2);
  long long sn8 = 8 * b->ctx.out_n;
  __nv_bfloat16* out = b->ctx.out + (long long)(b->ctx.row0 + chunk_of(0, n, reverse) * kTok + rw) * b->ctx.out_n + d0 + 8 * (lane & 3);
  const int room = min(b->ctx.d, d0 + D / 2) - d0 - 8 * (lane & 3);  // columns from there on
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int ch = chunk_of(i, n, reverse), len = chunk_len(ch, all);
    if (!wait_warp(&b->s_full, i & 1, gd)) return;
    tc_fence_after();
#pragma unroll 1
    for (int j = 2 * half; j < 2 * half + 2; ++j) {  // 32 scores -> 16 columns of P
      const uint32_t dst = tl + P::kColS + 16 * j + half * 32;
      if (reverse ? j < qd : j > qd) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = 0;
        tmem_st16u(dst, w);
        continue;
      }
      const float* f = decay + (row - 32 * j);
      float v[32];
      tmem_ld16(tl + P::kColS + 32 * j, v);
      tmem_ld16(tl + P::kColS + 32 * j + 16, v + 16);
      tmem_ld_wait();
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float2 p = mul2(make_float2(v[2 * x], v[2 * x + 1]), make_float2(f[-2 * x], f[-2 * x - 1]));
        w[x] = pack_bf16(p.x, p.y);
      }
      tmem_st16u(dst, w);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->p_full);

    if (!wait_warp(&b->o_full, i & 1, gd)) return;
    tc_fence_after();
    // 16 rows and 32 columns at a time: lane l holds columns 8 g + 2 (l % 4) + {0, 1} of rows l / 4 and l / 4 + 8
    // D = 64: the next scores go over intra, so everything is read before anything is stored (gradients of 64 heads of
    // 4096 tokens 115 -> 107 us); D = 128 has columns for both, and no registers to hold the rows (8 heads of 65,536
    // tokens 165 -> 190 us)
    constexpr bool kHold = D == 64 && !DERIV;
    uint32_t e[kHold ? 2 : 1][2][4];
    // the four lanes of a row turn their pairs round, so that each has 8 columns in a row and they store 64 bytes
    auto store = [&](int hh, int cc, int k) {
      uint32_t* p = e[kHold ? hh : 0][k];
      turn4(p, lane);
      if (rw + 16 * hh + 8 * k < len && (kHold ? d0 + 8 * (lane & 3) < b->ctx.d : cc < room))
        *reinterpret_cast<uint4*>(out + (2 * hh + k) * sn8 + cc) = make_uint4(p[0], p[1], p[2], p[3]);
    };
    const float gamma = decay_pow(b->ctx.lg, 1);
    const float* wt = b->decay + (reverse ? kTok - len + rw : 32 + rw);
#pragma unroll(kHold ? 2 : 1)
    for (int hh = 0; hh < 2; ++hh) {
      float wi[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) wi[k] = rw + 16 * hh + 8 * k < len ? gamma * wt[16 * hh + 8 * k] : 0.f;
#pragma unroll
      for (int cc = 0; cc < D / 2; cc += 32) {
        float u[16], v[16];
        const uint32_t tr = tl + ((uint32_t)(16 * hh) << 16);
        tmem_ld16x32(tr + P::kColInter + d0 + cc, u);
        tmem_ld16x32(tr + P::intra(d0 + cc), v);
        uint32_t xx[2][4];
        if (DERIV) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = rw + 16 * hh + 8 * k;
            const __nv_bfloat16* xp = b->ctx.x + (long long)(b->ctx.row0 + ch * kTok + t) * b->ctx.x_n + d0 + cc + 2 * (lane & 3);
#pragma unroll
            for (int g = 0; g < 4; ++g)
              xx[k][g] = t < len && d0 + cc + 8 * g < b->ctx.d ? *reinterpret_cast<const uint32_t*>(xp + 8 * g) : 0u;
          }
        }
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float2 o = fma2(make_float2(wi[k], wi[k]), make_float2(u[4 * g + 2 * k], u[4 * g + 2 * k + 1]),
                            make_float2(v[4 * g + 2 * k], v[4 * g + 2 * k + 1]));
            if (DERIV) {
              o.x *= ret_dphi(__uint_as_float(xx[k][g] << 16), b->ctx.fx);
              o.y *= ret_dphi(__uint_as_float(xx[k][g] & 0xffff0000u), b->ctx.fx);
            }
            e[kHold ? hh : 0][k][g] = pack_bf16(o.x, o.y);
          }
          if (!kHold) store(hh, cc, k);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->o_free);
    if (kHold) {
      sn8 = 8 * b->ctx.out_n;
      out = b->ctx.out + (long long)(b->ctx.row0 + ch * kTok + rw) * b->ctx.out_n + d0 + 8 * (lane & 3);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int k = 0; k < 2; ++k) store(hh, 0, k);
    }
    if (!kHold) out += reverse ? -16 * sn8 : 16 * sn8;
  }
}

// W warps, token row = 32 (warp % 4) + lane: the feature maps of chunk i and zeros behind the sequence, before its
// scores.  (Functions of their own where they are rare: their registers would spill those of the loops.)
template <int D>
__device__ __noinline__ bool map_chunk(uint8_t* sm, PassBars* b, int row, int i, int len) {
  using P = PassTile<D>;
  const int s = i % kStages, d = b->ctx.d, fa = b->ctx.fa, fb = b->ctx.fb, fc = b->ctx.fc;
  const Guard gd = make_guard(&b->abort, b->ctx.wait_ns);
  if (!wait_warp(&b->full[s], (i / kStages) & 1, gd) || !wait_warp(&b->a_full, i & 1, gd)) return false;
  uint8_t *at = sm + P::kOffA, *bt = sm + P::kOffBC + s * 2 * P::kOp;
  if (fa != kFeatIdentity) map_row<D>(at, row, kTok, d, fa);
  if (fb != kFeatIdentity || len < kTok) map_row<D>(bt, row, len, d, fb);
  if (fc != kFeatIdentity || len < kTok) map_row<D>(bt + P::kOp, row, len, d, fc);
  fence_proxy_async_smem();
  __syncwarp();
  if ((row & 31) == 0) mbar_arrive(&b->mapped);
  return true;
}

// C columns, from 8 jb, of row `row` of B w of chunk i in three parts, the third one over X's tile, once inter has
// read it.  D = 128: the W warps take 64 columns, the X warps, which have nothing else to do then, the others.
template <int D, int C>
__device__ __noinline__ bool weigh_chunk3(uint8_t* sm, PassBars* b, int row, int jb, int i) {
  using P = PassTile<D>;
  const Guard gd = make_guard(&b->abort, b->ctx.wait_ns);
  if (!wait_warp(&b->s_full, i & 1, gd) || !wait_warp(&b->in_full, i & 1, gd)) return false;
  const int ch = chunk_of(i, b->ctx.n, b->ctx.reverse), len = chunk_len(ch, b->ctx.len);
  const float w = row < len ? decay_pow(b->ctx.lg, b->ctx.reverse ? row : len - 1 - row) : 0.f;
  uint8_t *bt = sm + P::kOffBC + (i % kStages) * 2 * P::kOp, *lo = sm + P::kOffLo, *lo2 = sm + P::kOffX;
  if (b->ctx.fb != kFeatIdentity) {  // phi(b) in fp32 for the state
    const __nv_bfloat16* raw = b->ctx.b + (long long)(b->ctx.row0 + ch * kTok + row) * b->ctx.b_n;
    weigh_phi_row3<C>(bt, lo, lo2, row, jb, w, raw, b->ctx.d, b->ctx.fb);
  } else {
    weigh_row3<C>(bt, lo, lo2, row, jb, w);
  }
  fence_proxy_async_smem();
  __syncwarp();
  return true;
}

// One W warp: what precedes a chunk's scores (map), then B w (weigh).
template <int D>
struct Weigh {
  using P = PassTile<D>;
  uint8_t* sm;
  PassBars* b;
  int row, n, all, reverse;
  bool mapped;
  float lg;
  Guard gd;
  __device__ __forceinline__ Weigh(uint8_t* sm_, PassBars* b_, int warp, int lane)
      : sm(sm_), b(b_), row(32 * (warp & 3) + lane), n(b_->ctx.n), all(b_->ctx.len), reverse(b_->ctx.reverse),
        mapped(b_->ctx.mapped()), lg(b_->ctx.lg), gd(make_guard(&b_->abort, b_->ctx.wait_ns)) {}

  __device__ __forceinline__ bool map(int i) {
    const int len = chunk_len(chunk_of(i, n, reverse), all);
    return (!mapped && len == kTok) || map_chunk<D>(sm, b, row, i, len);
  }
  __device__ __forceinline__ bool weigh(int i) {
    // B has been read by the scores, the second part's tile by the last dX
    if (!wait_warp(&b->s_full, i & 1, gd) || (i > 0 && !wait_warp(&b->dx_full, (i - 1) & 1, gd))) return false;
    if (i >= b->ctx.exact) {
      if (!weigh_chunk3<D, 64>(sm, b, row, 0, i)) return false;
    } else {  // no fp32 state comes of it: the tile's rounded phi is good enough
      const int len = chunk_len(chunk_of(i, n, reverse), all);
      const float w = row < len ? decay_pow(lg, reverse ? row : len - 1 - row) : 0.f;
      weigh_row2<D>(sm + P::kOffBC + (i % kStages) * 2 * P::kOp, sm + P::kOffLo, row, 0, w);
      fence_proxy_async_smem();
      __syncwarp();
    }
    if ((row & 31) == 0) mbar_arrive(&b->w_full);
    return true;
  }
};

// One X warp.  TMEM lane quadrant = warp % 4: rows 32 quadrant .. of X, or with D = 64 (M = 64) 16 quadrant .. in
// its first 16 lanes; 16 rows and 32 columns at a time, a lane's elements as in tmem_ld16x32.  D = 128: the two
// warps of a quadrant take half of the columns each.
template <int D>
struct Carry {
  using P = PassTile<D>;
  static constexpr int kBlocks = D == 128 ? 4 : 2;          // of 16 x 32 elements
  uint8_t* xt;
  PassBars* b;
  int lane, r0, c0, d, n, all, reverse;
  uint32_t tl;
  float lg;
  Guard gd;
  __device__ __forceinline__ Carry(uint8_t* sm, PassBars* b_, int warp, int lane_)
      : xt(sm + P::kOffX), b(b_), lane(lane_), r0((D == 128 ? 32 : 16) * (warp & 3) + (lane_ >> 2)),
        c0(64 * ((warp - P::kWarpX) >> 2)), d(b_->ctx.d), n(b_->ctx.n), all(b_->ctx.len), reverse(b_->ctx.reverse),
        tl(b_->tbase + ((uint32_t)(32 * (warp & 3)) << 16) + P::kColX), lg(b_->ctx.lg),
        gd(make_guard(&b_->abort, b_->ctx.wait_ns)) {}

  // block k: rows r, r + 8, columns c + 8 g + {0, 1}
  __device__ __forceinline__ int row_of(int k) const { return r0 + 16 * (k >> 1); }
  __device__ __forceinline__ int col_of(int k) const { return c0 + 32 * (k & 1); }
  __device__ __forceinline__ uint32_t tmem_of(int k) const {
    return tl + ((uint32_t)(16 * (k >> 1)) << 16) + (uint32_t)col_of(k);
  }
  // decay of X over chunk i
  __device__ __forceinline__ float over(int i) const { return decay_pow(lg, chunk_len(chunk_of(i, n, reverse), all)); }
  // the tile for the next chunk, and X times its decay over that chunk for dX to be added to
  __device__ __forceinline__ void keep(int k, float* v, float wl) {
    const int r = row_of(k);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t* p = reinterpret_cast<uint32_t*>(piece(xt, D, r, col_of(k) / 8 + g)) + (lane & 3);
      p[0] = pack_bf16(v[4 * g], v[4 * g + 1]);
      p[256] = pack_bf16(v[4 * g + 2], v[4 * g + 3]);  // 8 rows of 128 bytes on: the same swizzle
    }
#pragma unroll
    for (int x = 0; x < 8; ++x)
      reinterpret_cast<float2*>(v)[x] = mul2(reinterpret_cast<float2*>(v)[x], make_float2(wl, wl));
    tmem_st16x32(tmem_of(k), v);
  }
  __device__ __forceinline__ void publish() {
    tmem_st_wait();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->x_full);
  }
  __device__ __forceinline__ bool update(int i) {
    const bool more = i + 1 < n;
    const float wl = more ? over(i + 1) : 1.f;
    float* to = more ? nullptr : b->ctx.to;
    // (inter has read the last tile)
    if (!wait_warp(&b->in_full, i & 1, gd) || !wait_warp(&b->dx_full, i & 1, gd)) return false;
    tc_fence_after();
#pragma unroll 2
    for (int k = 0; k < kBlocks; ++k) {
      float v[16];
      tmem_ld16x32(tmem_of(k), v);
      if (i >= b->ctx.exact) {
        float u[16];
        tmem_ld16x32(tl - P::kColX + P::kColS + ((uint32_t)(16 * (k >> 1)) << 16) + P::apart(col_of(k)), u);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] += u[x];
      } else {
        tmem_ld_wait();
      }
      if (more) {
        keep(k, v, wl);
      } else if (to != nullptr) {
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int r = row_of(k) + 8 * (m & 1), c = col_of(k) + 8 * (m >> 1) + 2 * (lane & 3);
          if (r < d && c < d)
            *reinterpret_cast<float2*>(to + r * d + c) =
                make_float2(v[4 * (m >> 1) + 2 * (m & 1)], v[4 * (m >> 1) + 2 * (m & 1) + 1]);
        }
        __syncwarp();
      }
    }
    if (more) publish();
    return true;
  }
};

// The state entering the segment: into X and its tile.  (A function of its own, once a block: its registers would
// spill those of the loops.)
template <int D>
__device__ __noinline__ void carry_start(uint8_t* sm, PassBars* b, int warp, int lane) {
  Carry<D> x(sm, b, warp, lane);
  const int d = b->ctx.d;
  const float* from = b->ctx.from;
  const bool from_t = b->ctx.from_t != 0;
  const float wl = x.over(0);
#pragma unroll 2
  for (int k = 0; k < Carry<D>::kBlocks; ++k) {
    float2 v[8];  // (loads without branches between them)
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const int r = x.row_of(k) + 8 * (m & 1), c = x.col_of(k) + 8 * (m >> 1) + 2 * (lane & 3);
      const bool in = from != nullptr && r < d && c < d;
      v[m] = make_float2(0.f, 0.f);
      if (in && !from_t) v[m] = __ldcg(reinterpret_cast<const float2*>(from + r * d + c));
      if (in && from_t) v[m].x = __ldcg(from + c * d + r);
      if (in && from_t) v[m].y = __ldcg(from + (c + 1) * d + r);
    }
    __syncwarp();
    x.keep(k, reinterpret_cast<float*>(v), wl);
  }
  x.publish();
}

template <int D>
__device__ __noinline__ void pass_weigh(uint8_t* sm, PassBars* b, int warp, int lane) {
  Weigh<D> w(sm, b, warp, lane);
  const int n = b->ctx.n, nx = b->ctx.nx;
#pragma unroll 1
  for (int i = 0; i < n; ++i)
    if (!w.map(i) || i >= nx || !w.weigh(i)) return;
}

template <int D>
__device__ __noinline__ void pass_x(uint8_t* sm, PassBars* b, int warp, int lane) {
  carry_start<D>(sm, b, warp, lane);
  Carry<D> x(sm, b, warp, lane);
  const int nx = b->ctx.nx;
  const int exact = b->ctx.exact;
#pragma unroll 1
  for (int i = 0; i < nx; ++i) {
    if (i >= exact) {
      if (!weigh_chunk3<D, 32>(sm, b, 32 * (warp & 3) + lane, 8 + 4 * ((warp - PassTile<D>::kWarpX) >> 2), i)) return;
      if (lane == 0) mbar_arrive(&b->w2_full);
    }
    if (!x.update(i)) return;
  }
}

// Both in the same warps.
template <int D>
__device__ __noinline__ void pass_weigh_x(uint8_t* sm, PassBars* b, int warp, int lane) {
  Weigh<D> w(sm, b, warp, lane);
  const int n = b->ctx.n, nx = b->ctx.nx;
  carry_start<D>(sm, b, warp, lane);
  if (!w.map(0)) return;
  Carry<D> x(sm, b, warp, lane);
#pragma unroll 1
  for (int i = 0; i < nx; ++i)
    if (!w.weigh(i) || (i + 1 < n && !w.map(i + 1)) || !x.update(i)) return;
}

template <int D>
__global__ void __launch_bounds__(PassTile<D>::kThreads, PassTile<D>::kPerSm) retention_pass_kernel(const __grid_constant__ TcArgs t) {
  using P = PassTile<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  PassBars* b = reinterpret_cast<PassBars*>(sm + P::kOffBars);
  const RetArgs& r = t.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int z = blockIdx.x % r.npass;  // a head's passes side by side: they read the same tensors
  const int unit = blockIdx.x / r.npass, g = unit / r.H, h = unit % r.H;
  const Segment sg = find_segment(r, g, SEG_ALL, reinterpret_cast<int*>(b->decay));
  if (sg.seq < 0) {
    grid_dependency_wait();  // (a kernel does not end before those it may overlap)
    return;
  }
  const RetPass& p = r.pass[z];
  if (threadIdx.x == 0) {  // the barriers, what the producer needs, and the first loads
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&b->full[s], 1);
      mbar_init(&b->empty[s], 1);
    }
    for (uint64_t* m : {&b->a_full, &b->s_full, &b->in_full, &b->dx_full, &b->o_full, &b->fin}) mbar_init(m, 1);
    for (uint64_t* m : {&b->mapped, &b->w_full}) mbar_init(m, 4);
    for (uint64_t* m : {&b->p_full, &b->o_free}) mbar_init(m, 8);
    mbar_init(&b->x_full, P::kXWarps);
    mbar_init(&b->w2_full, 8);
    b->abort = 0;
    b->issued = b->issued_a = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    const int ia = t.ia[z], ib = t.ib[z], ic = t.ic[z];
    PassCtx& c = b->ctx;
    c.ma = &t.tm[ia];
    c.mb = &t.tm[ib];
    c.mc = &t.tm[ic];
    c.ha = t.by_h[ia] ? h : 0;
    c.hb = t.by_h[ib] ? h : 0;
    c.hc = t.by_h[ic] ? h : 0;
    c.ba = t.by_b[ia] ? sg.seq : 0;
    c.bb = t.by_b[ib] ? sg.seq : 0;
    c.bc = t.by_b[ic] ? sg.seq : 0;
    c.row0 = sg.row0;
    c.n = (sg.len + kTok - 1) / kTok;
    c.reverse = p.reverse;
    c.wait_ns = t.wait_ns;
    load_bc<D>(sm, b, c, 0);
    load_a<D>(sm, b, c, 0);
    if (c.n > 1) load_bc<D>(sm, b, c, 1);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&b->tbase, P::kCols);
    tmem_relinquish();
  }
  const int slot = r.states != nullptr ? ret_slot(r.slots, r.n_slots, sg.seq) : -1;
  const float lg = decay_log2(r.gamma[h]);
  if (threadIdx.x == 64) {
    const size_t dd = (size_t)r.d * r.d;
    PassCtx& c = b->ctx;
    const int n = (sg.len + kTok - 1) / kTok;
    c.len = sg.len;
    c.to = slot >= 0 && sg.seg == sg.nseg - 1 ? r.states + ((size_t)slot * r.H + h) * dd : nullptr;
    c.nx = c.to != nullptr ? n : n - 1;
    c.fa = p.a.feature;
    c.fb = p.b.feature;
    c.fc = p.c.feature;
    c.fx = p.x.feature;
    // the last chunks, whose terms the decay leaves more than 1/8 of (the last may be short); all, where the others
    // would take the rounded phi
    const float reach = lg == 0.f || c.fb != kFeatIdentity ? (float)n : fminf((float)n, 2.f + 3.f / (kTok * fabsf(lg)));
    c.exact = c.to == nullptr ? n : n - (int)reach;
    c.d = r.d;
    c.lg = lg;
    c.out = static_cast<__nv_bfloat16*>(const_cast<void*>(p.out.p)) + ret_base(r, p.out, sg.seq, h);
    c.x = p.x.p == nullptr ? nullptr : static_cast<const __nv_bfloat16*>(p.x.p) + ret_base(r, p.x, sg.seq, h);
    c.b = static_cast<const __nv_bfloat16*>(p.b.p) + ret_base(r, p.b, sg.seq, h);
    c.out_n = p.out.sn;
    c.x_n = p.x.sn;
    c.b_n = p.b.sn;
    c.from = entering_state(r, p, sg, h, slot);
    c.from_t = sg.nseg > 1 && p.sum_t;
    c.from_ws = sg.nseg > 1;
  }
  if (threadIdx.x >= P::kThreads - kTok - 32) {
    const int i = threadIdx.x - (P::kThreads - kTok - 32), n = p.reverse ? kTok - 1 - i : i - 32;
    b->decay[i] = n >= 0 ? r.scale * decay_pow(lg, n) : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (b->ctx.from_ws) grid_dependency_wait();  // the state entering the segment; no wait with a limit before it

  if (warp == kWarpProd) {
    if (lane == 0) pass_producer<D>(sm, b);
    __syncwarp();
  } else if (warp == kWarpMma) {
    pass_mma<D>(sm, b);
    __syncwarp();
    if (elect_one()) mma_commit(&b->fin);
    __syncwarp();
  } else if (warp < P::kWarpW) {
    if (b->ctx.x == nullptr)
      pass_out<D, false>(b, warp, lane);
    else
      pass_out<D, true>(b, warp, lane);
  } else if constexpr (D == 128) {
    if (warp < P::kWarpX)
      pass_weigh<D>(sm, b, warp, lane);
    else
      pass_x<D>(sm, b, warp, lane);
  } else {
    pass_weigh_x<D>(sm, b, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) {
    drain(&b->fin, 0);
    if (b->abort) {
      if (b->issued_a > 0) drain(&b->a_full, (b->issued_a - 1) & 1);
      for (int q = b->issued > kStages ? b->issued - kStages : 0; q < b->issued; ++q)
        drain(&b->full[q % kStages], (q / kStages) & 1);
      atomicOr(r.status, 1u);
    }
  }
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(b->tbase, P::kCols);
  grid_dependency_wait();  // (a kernel does not end before those it may overlap)
}

// ================================================================ segment sums
// A segment's own sum of gamma^(distance to its end) b c^T: B w, with the distance counted to the segment's
// end, is added up by the tensor cores over all its chunks.  B w is a sum of two bf16 numbers; in a call that returns
// states, of three where the decay up to the sequence's end leaves more than 2^-2.75, and those chunks' sums are added up in
// fp32 (as in the pass; with two parts throughout, states of 2000 to 4000 tokens were off by 2e-6 to 3e-6).  Bound by HBM where the segments fill the SMs (8
// heads of 65,536 tokens, d = 128: 43 us, 91 % of a copy's rate), else by a block's chain load, B w, products: 1.4 us
// a chunk (64 heads of 8192 tokens, d = 64: 192 blocks, 25 us, 60 % of that rate; where states are
// returned the chunks of three parts add 5 us).  A row of B is shared by D / 32
// threads and the second part's product goes first, so that the next chunk's B w runs beside the first part's: 53
// -> 43 us and 28 -> 25 us together.
template <int D>
struct SumTile {
  static constexpr int kStages = 3;                     // chunks of B and C in flight
  static constexpr int kOp = (D / 64) * kAtom;
  static constexpr int kOffLo = kStages * 2 * kOp;      // the second part of B w
  static constexpr int kOffBars = kOffLo + kOp;
  static constexpr int kSplit = D / 32;                 // threads that share a row of B
  static constexpr int kThreads = 32 * (kWarpOut + 4 * kSplit);
  // blocks an SM by registers (shared memory allows one less): room for the next kernels' blocks
  static constexpr int kPerSm = D == 128 ? 2 : 3;
};

template <int D>
struct SumBars {
  uint64_t full[SumTile<D>::kStages], empty[SumTile<D>::kStages], ready[SumTile<D>::kStages];
  uint64_t lo_free;  // the second part's tile has been read
  uint64_t fin;
  uint32_t tbase;
  int abort;
  int issued;
  int scratch[2 * kOrdered];
};

template <int D>
constexpr size_t sum_smem() {
  return SumTile<D>::kOffBars + sizeof(SumBars<D>);
}
static_assert(sum_smem<128>() <= 232448 && 2 * (sum_smem<64>() + 1024) <= 233472, "shared memory budget");

// 32 columns, from 8 jb, of row r of B w in three parts.  (Chunks of three parts are whole: states are returned by the
// forward direction alone, whose inner segments have exactly L tokens, a multiple of a chunk's.)  (This and the next
// are functions of their own, for the few chunks that need them: with their registers no block of the scan fits beside
// this kernel's, which cost 6 to 11 us.)
__device__ __noinline__ void sum_weigh3(uint8_t* hi, uint8_t* lo, uint8_t* lo2, int r, int jb, float w,
                                        const RetTensor& b, long long at, int d) {
  if (b.feature != kFeatIdentity)
    weigh_phi_row3<32>(hi, lo, lo2, r, jb, w, static_cast<const __nv_bfloat16*>(b.p) + at, d, b.feature);
  else
    weigh_row3<32>(hi, lo, lo2, r, jb, w);
}
// Adds chunk i's own sum of three parts, in the columns D behind, to the segment's: a warp's 32 columns.
template <int D>
__device__ __noinline__ void sum_add(uint32_t at, int i) {
  tc_fence_after();
#pragma unroll 1
  for (int hh = 0; hh < D / 64; ++hh, at += 16u << 16) {
    float u[16], v[16];
    tmem_ld16x32(at + D, v);
    if (i > 0) {
      tmem_ld16x32(at, u);
      tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 16; ++x) v[x] += u[x];
    }
    tmem_ld_wait();
    tmem_st16x32(at, v);
  }
  tmem_st_wait();
}

template <int D>
__global__ void __launch_bounds__(SumTile<D>::kThreads, SumTile<D>::kPerSm)
    retention_sum_kernel(const __grid_constant__ TcArgs t) {
  using P = SumTile<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  SumBars<D>* b = reinterpret_cast<SumBars<D>*>(sm + P::kOffBars);
  launch_dependents();
  const RetArgs& r = t.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int set = blockIdx.x % r.nsum, unit = blockIdx.x / r.nsum, h = unit % r.H;
  int z = 0;
  for (int i = 0; i < r.npass; ++i)
    if (r.pass[i].sum == set && !r.pass[i].sum_t) z = i;
  const RetPass& p = r.pass[z];
  Segment sg = find_segment(r, unit / r.H, SEG_INNER, b->scratch);
  if (sg.seq < 0) return;
  inner_segment(r, sg, p.reverse);
  if (threadIdx.x == 0) {
    for (int s = 0; s < P::kStages; ++s) {
      mbar_init(&b->full[s], 1);
      mbar_init(&b->empty[s], 1);
      mbar_init(&b->ready[s], 4 * P::kSplit);
    }
    mbar_init(&b->lo_free, 1);
    mbar_init(&b->fin, 1);
    b->abort = 0;
    b->issued = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&b->tbase, 2 * D);
    tmem_relinquish();
  }
  if (warp == kWarpProd && lane == 0) {
    prefetch_tmap(&t.tm[t.ib[z]]);
    prefetch_tmap(&t.tm[t.ic[z]]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Guard gd = make_guard(&b->abort, t.wait_ns);
  const uint32_t tmem = b->tbase;
  const int n = (sg.len + kTok - 1) / kTok;
  uint8_t* lo = sm + P::kOffLo;
  const float lg = decay_log2(r.gamma[h]);
  // the first chunk of three parts; the third part's tile takes the place of a stage
  int three = n;
  if (r.states != nullptr) {
    const int rest = sg.all - sg.seg * r.L - sg.len;  // tokens behind the segment
    const float reach = lg == 0.f ? 1e9f : fminf(1e9f, 2.75f / fabsf(lg));
    three = n - min(n, (max(0, (int)reach - rest) + kTok - 1) / kTok);
  }
  const int stages = three < n ? P::kStages - 1 : P::kStages;
  uint8_t* lo2 = sm + (P::kStages - 1) * 2 * P::kOp;

  if (warp == kWarpProd) {
    if (lane == 0) {
      const int ib = t.ib[z], ic = t.ic[z];
      const int hb = t.by_h[ib] ? h : 0, sb = t.by_b[ib] ? sg.seq : 0, hc = t.by_h[ic] ? h : 0,
                sc = t.by_b[ic] ? sg.seq : 0;
      int i = 0;
      for (; i < n; ++i) {
        const int s = i % stages;
        if (i >= stages && !wait(&b->empty[s], ((i / stages) - 1) & 1, gd)) break;
        uint8_t* st = sm + s * 2 * P::kOp;
        mbar_arrive_expect_tx(&b->full[s], 2 * P::kOp);
        load_tile<D>(st, &t.tm[ib], sg.row0 + i * kTok, hb, sb, &b->full[s]);
        load_tile<D>(st + P::kOp, &t.tm[ic], sg.row0 + i * kTok, hc, sc, &b->full[s]);
      }
      b->issued = i;
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    const Desc b0 = make_desc(smem_u32(sm), kAtom, 1024), dlo = make_desc(smem_u32(lo), kAtom, 1024);
    const Desc dlo2 = make_desc(smem_u32(lo2), kAtom, 1024);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int s = i % stages;
      if (!wait_warp(&b->ready[s], (i / stages) & 1, gd)) break;
      tc_fence_after();
      const Desc bm{b0.lo + s * (2 * P::kOp >> 4), b0.hi}, cm{bm.lo + (P::kOp >> 4), b0.hi};
      __syncwarp();
      if (elect_one()) {
        if (i >= three) {
          mma_outer<D, D, false>(tmem + D, bm, cm);
          mma_outer<D, D, true>(tmem + D, dlo, cm);
          mma_outer<D, D, true>(tmem + D, dlo2, cm);
          mma_commit(&b->lo_free);
        } else {
          // the second part first: its tile has to be free for the next chunk
          if (i == 0)
            mma_outer<D, D, false>(tmem, dlo, cm);
          else
            mma_outer<D, D, true>(tmem, dlo, cm);
          mma_commit(&b->lo_free);
          mma_outer<D, D, true>(tmem, bm, cm);
        }
        mma_commit(&b->empty[s]);
      }
      __syncwarp();
    }
    __syncwarp();
    if (elect_one()) mma_commit(&b->fin);
    __syncwarp();
  } else {
    const int qd = warp & 3, row = 32 * qd + lane, half = (warp - kWarpOut) >> 2;
    const int reverse = p.reverse, all = sg.len, d = r.d, fb = p.b.feature, fc = p.c.feature;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int s = i % stages, at = i * kTok + row, len = min(kTok, all - i * kTok);
      ok = wait_warp(&b->full[s], (i / stages) & 1, gd);
      if (ok && i > 0) ok = wait_warp(&b->lo_free, (i - 1) & 1, gd);
      if (!ok) break;
      if (i > three) sum_add<D>(tmem + ((uint32_t)(32 * qd) << 16) + 32 * half, i - 1);
      uint8_t* st = sm + s * 2 * P::kOp;
      if (half == 0) {  // (the operands of a whole row: rarely)
        if (fc != kFeatIdentity || len < kTok) map_row<D>(st + P::kOp, row, len, d, fc);
      }
      const float w = row < len ? decay_pow(lg, reverse ? at : all - 1 - at) : 0.f;
      if (i >= three)
        sum_weigh3(st, lo, lo2, row, 4 * half, w, p.b, ret_base(r, p.b, sg.seq, h) + (long long)(sg.row0 + at) * p.b.sn, d);
      else if (fb != kFeatIdentity || len < kTok)
        weigh_phi_row2<32>(st, lo, row, 4 * half, w, d, fb);
      else
        weigh_row2<32>(st, lo, row, 4 * half, w);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->ready[s]);
    }
    if (ok && wait_warp(&b->fin, 0, gd) && !aborted(gd)) {
      tc_fence_after();
      if (three < n) sum_add<D>(tmem + ((uint32_t)(32 * qd) << 16) + 32 * half, n - 1);
      float* dst = r.seg + (((size_t)set * r.W + sg.w0 + sg.seg) * r.H + h) * d * d;
#pragma unroll 1
      for (int hh = 0; hh < D / 64; ++hh) {  // 16 rows x 32 columns
        const int c0 = 32 * half;
        const int r0 = (D == 128 ? 32 * qd + 16 * hh : 16 * qd) + (lane >> 2);
        float v[16];
        tmem_ld16x32(tmem + ((uint32_t)(32 * qd + 16 * hh) << 16) + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int rr = r0 + 8 * (m & 1), cc = c0 + 8 * (m >> 1) + 2 * (lane & 3);
          if (rr < d && cc < d)
            *reinterpret_cast<float2*>(dst + rr * d + cc) =
                make_float2(v[4 * (m >> 1) + 2 * (m & 1)], v[4 * (m >> 1) + 2 * (m & 1) + 1]);
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) {
    drain(&b->fin, 0);
    if (aborted(gd)) {
      for (int q = b->issued > stages ? b->issued - stages : 0; q < b->issued; ++q)
        drain(&b->full[q % stages], (q / stages) & 1);
      atomicOr(r.status, 1u);
    }
  }
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tmem, 2 * D);
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

// A token tensor as [batch][head][row][d]; a dimension of stride 0 has one entry.  Rows behind the tensor
// and columns behind d read as zeros.
bool make_map(CUtensorMap* m, const RetTensor& t, const RetArgs& a) {
  auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t rows = a.N, row_bytes = t.sn ? (cuuint64_t)t.sn * 2 : (cuuint64_t)a.d * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)a.d, rows, t.sh ? (cuuint64_t)a.H : 1,
                              t.sb && a.cu == nullptr ? (cuuint64_t)a.B : 1};
  const cuuint64_t strides[3] = {row_bytes, t.sh ? (cuuint64_t)t.sh * 2 : row_bytes,
                                 t.sb ? (cuuint64_t)t.sb * 2 : row_bytes};
  const cuuint32_t box[4] = {64, (cuuint32_t)kTok, 1, 1}, es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor map of an operand, made when it is new.
int map_of(TcArgs* t, int* used, const RetTensor** seen, const RetTensor& x, bool* ok) {
  for (int i = 0; i < *used; ++i)
    if (seen[i]->p == x.p && seen[i]->sb == x.sb && seen[i]->sh == x.sh && seen[i]->sn == x.sn) return i;
  if (*used == 4) {
    *ok = false;
    return 0;
  }
  const int i = (*used)++;
  seen[i] = &x;
  t->by_b[i] = x.sb != 0 && t->r.cu == nullptr;
  t->by_h[i] = x.sh != 0;
  *ok = *ok && make_map(&t->tm[i], x, t->r);
  return i;
}

template <int D>
cudaError_t launch(const TcArgs& t, cudaStream_t st) {
  static SmemOptIn opt_pass, opt_sum;
  cudaError_t e = opt_pass.ensure((const void*)retention_pass_kernel<D>, (int)pass_smem<D>());
  if (e == cudaSuccess) e = opt_sum.ensure((const void*)retention_sum_kernel<D>, (int)sum_smem<D>());
  if (e != cudaSuccess) return e;
  if (t.r.seg != nullptr) {
    retention_sum_kernel<D><<<(unsigned)(t.r.inner * t.r.H * t.r.nsum), SumTile<D>::kThreads, sum_smem<D>(), st>>>(t);
    note_launch();
    e = retention_scan_launch(t.r, st);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(retention_pass_kernel<D>, dim3((unsigned)(t.r.G * t.r.H * t.r.npass)), PassTile<D>::kThreads, pass_smem<D>(), st,
                          t.r.seg != nullptr, t);
}

}  // namespace

void tc_retention_set_wait_limit(unsigned long long ns) { g_wait_ns = ns == 0 ? kWaitLimitNs : ns; }

cudaError_t tc_retention_launch(const RetArgs& a, cudaStream_t st) {
  TcArgs t;
  t.r = a;
  t.wait_ns = g_wait_ns;
  int used = 0;
  const RetTensor* seen[4];
  bool ok = true;
  for (int i = 0; i < a.npass; ++i) {
    t.ia[i] = map_of(&t, &used, seen, a.pass[i].a, &ok);
    t.ib[i] = map_of(&t, &used, seen, a.pass[i].b, &ok);
    t.ic[i] = map_of(&t, &used, seen, a.pass[i].c, &ok);
  }
  if (!ok) return cudaErrorInvalidValue;
  return a.d == 128 ? launch<128>(t, st) : launch<64>(t, st);
}

}  // namespace mhla
