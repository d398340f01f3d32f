// Retention passes on the sm_103a tensor cores (bf16).  The mathematics is in retention.h; a pass cuts
// a segment into chunks of 128 tokens (len of them in the sequence) and carries X, the state entering
// the chunk ([D][D], fp32 in registers):
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
// the B tile, the remainder over the A tile: 2^-16 of a term) where only bf16 outputs come of it, of
// three (the last over the tile of X: 2^-24) where the call returns the final state in fp32.
//
// The roles' loops are kept short rather than unrolled: one warp a scheduler runs each of them, and with
// whole rows unrolled the instruction fetch, not the arithmetic, set the pace (a chunk took 23,000 cycles).
//
// Roles (10 warps; D = 128: one CTA an SM, D = 64: two):
//   warp 0     TMA producer: the A, B and C tiles of a chunk (2-stage ring)
//   warp 1     MMA issuer
//   warps 2-5  scores -> P, then out = scale (intra + gamma^(i+1) inter) to global memory
//   warps 6-9  feature maps in place, B w over B, and X: registers, and its bf16 tile for the next chunk
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
constexpr int kThreads = 320;
constexpr int kWarpProd = 0, kWarpMma = 1, kWarpX = 6;
constexpr int kStages = 2;
constexpr uint64_t kWaitLimitNs = 500000000ull;
unsigned long long g_wait_ns = kWaitLimitNs;

struct TcArgs {
  CUtensorMap tm[4];                         // q, k, v, dy as [B][H][N][d], box 64 x 128
  int by_b[4], by_h[4];                      // 0: shared by the batch / the heads
  int ia[kRetMaxPasses], ib[kRetMaxPasses], ic[kRetMaxPasses];  // tensor maps of a pass's operands
  int wide_out[kRetMaxPasses];               // rows of out (and x) start on 32 bytes
  unsigned long long wait_ns;
  RetArgs r;
};

// ---------------------------------------------------------------- bounded waits
struct Guard {
  int* abort;
  unsigned long long limit;
};
__device__ __forceinline__ bool aborted(const Guard& g) { return *reinterpret_cast<volatile int*>(g.abort) != 0; }
// The thread sleeps in the barrier's own wait; the clock is read only after about a microsecond of that.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* ab, unsigned long long limit) {
  const uint32_t nap = limit < 1000 ? (uint32_t)limit : 1000u;
  uint64_t t0 = 0;
  for (;;) {
    if (mbar_try_wait_ns(bar, parity, nap)) return true;
    if (*reinterpret_cast<volatile int*>(ab) != 0) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0)
      t0 = now;
    else if (now - t0 > limit)
      break;
  }
  *reinterpret_cast<volatile int*>(ab) = 1;
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Guard& g) {
  return mbar_test(bar, parity) || wait_slow(bar, parity, g.abort, g.limit);
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

// Row r of B times w as a sum of bf16 numbers: over the B tile, the remainder in lo, with lo2 the
// remainder of that.  The row is read from raw (global memory, d columns) where given, else from the
// tile; a feature map, if any, is applied to it in fp32.
template <int D>
__device__ __forceinline__ void weigh_row(uint8_t* hi, uint8_t* lo, uint8_t* lo2, int r, float w,
                                          const __nv_bfloat16* raw, int d, int feature) {
#pragma unroll 1
  for (int j0 = 0; j0 < D / 8; j0 += 4) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = *piece(hi, kTok, r, j0 + j);
      if (raw != nullptr && 8 * (j0 + j) < d) u[j] = *reinterpret_cast<const uint4*>(raw + 8 * (j0 + j));
      if (w == 0.f) u[j] = make_uint4(0, 0, 0, 0);  // rows behind the sequence, whatever they hold
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
      unpack8(u[j], f);
      if (feature != kFeatIdentity && 8 * (j0 + j) < d) {
#pragma unroll
        for (int x = 0; x < 8; ++x) f[x] = ret_phi(f[x], feature);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) f[x] *= w;
      const uint4 h = pack8(f);
      *piece(hi, kTok, r, j0 + j) = h;
      remainder8(f, h);
      const uint4 l = pack8(f);
      *piece(lo, kTok, r, j0 + j) = l;
      if (lo2 != nullptr) {
        remainder8(f, l);
        *piece(lo2, kTok, r, j0 + j) = pack8(f);
      }
    }
  }
}

// MMAs of one product D[tmem] (+)= A^T-like operands, MN-major in both: A [K rows][M], B [K rows][N], K = 128.
template <int M, int N>
__device__ __forceinline__ void mma_outer(uint32_t d, uint32_t a, uint32_t b, bool acc) {
  const uint64_t da = smem_desc(a, kAtom, 1024), db = smem_desc(b, kAtom, 1024);
#pragma unroll
  for (int k = 0; k < kTok / 16; ++k)
    mma_bf16(d, da + k * (2048 >> 4), db + k * (2048 >> 4), idesc_bf16_f32(M, N, 1, 1), acc || k > 0);
}

// TMA of one operand's chunk: D / 64 atoms.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const TcArgs& t, int map, int row, int h, int seq,
                                          uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    tma_load_4d(dst + c * kAtom, &t.tm[map], 64 * c, row, t.by_h[map] ? h : 0, t.by_b[map] ? seq : 0, bar);
}

// ================================================================ pass
template <int D>
struct PassTile {
  static constexpr int kOp = (D / 64) * kAtom;          // an operand's tile
  static constexpr int kStage = 3 * kOp;
  static constexpr int kOffX = kStages * kStage;        // bf16 X: D rows c, D columns e
  static constexpr int kOffBars = kOffX + kOp;          // (a tile's room: also the third part of B w)
  static constexpr uint32_t kCols = D == 128 ? 512 : 256;
  static constexpr uint32_t kColS = 0;                  // scores, P over their first half
  static constexpr uint32_t kColInter = 128, kColIntra = 128 + D;
  static constexpr uint32_t kColDX = D == 128 ? 384 : 64;  // D = 64: over the scores that P leaves free
  static constexpr int kPerSm = D == 128 ? 1 : 2;
};

struct PassBars {
  uint64_t full[kStages], empty[kStages];
  uint64_t mapped;    // feature maps applied / rows behind the sequence cleared (4 X warps)
  uint64_t s_full;    // scores
  uint64_t in_full;   // inter
  uint64_t p_full;    // P in TMEM (4 out warps)
  uint64_t w_full;    // B w (4 X warps)
  uint64_t dx_full;   // dX
  uint64_t x_full;    // the bf16 tile of X (4 X warps)
  uint64_t o_full;    // intra
  uint64_t o_free;    // inter and intra read (4 out warps)
  uint64_t fin;       // every MMA of the CTA has completed
  uint32_t tbase;
  int abort;
  int issued;         // chunks whose loads the producer issued
  int scratch[34];
  float decay[kTok];  // gamma^n
};

template <int D>
constexpr size_t pass_smem() {  // (the kernels' shared memory starts on 1024 bytes: no room to align it)
  return PassTile<D>::kOffBars + sizeof(PassBars);
}
static_assert(pass_smem<128>() <= 232448 && 2 * (pass_smem<64>() + 1024) <= 233472, "shared memory budget");

// What the roles share.
struct PassCtx {
  uint8_t* sm;
  PassBars* b;
  Guard g;
  uint32_t tmem;
  int z, h, seq, row0, len, n;   // pass, head, sequence, first row, tokens, chunks
  int nx;                        // chunks whose dX is needed
  int reverse, terms;            // direction; bf16 numbers that B w is the sum of
  bool mapped;                   // some operand has a feature map
  float lg;
  __device__ __forceinline__ int chunk(int i) const { return reverse ? n - 1 - i : i; }
  __device__ __forceinline__ int chunk_len(int ch) const { return min(kTok, len - ch * kTok); }
};

template <int D>
__device__ __forceinline__ void pass_producer(const TcArgs& t, const PassCtx& c) {
  using P = PassTile<D>;
  int i = 0;
  for (; i < c.n; ++i) {
    const int s = i % kStages, row = c.row0 + c.chunk(i) * kTok;
    if (i >= kStages && !wait(&c.b->empty[s], ((i / kStages) - 1) & 1, c.g)) break;
    uint8_t* st = c.sm + s * P::kStage;
    mbar_arrive_expect_tx(&c.b->full[s], P::kStage);
    load_tile<D>(st, t, t.ia[c.z], row, c.h, c.seq, &c.b->full[s]);
    load_tile<D>(st + P::kOp, t, t.ib[c.z], row, c.h, c.seq, &c.b->full[s]);
    load_tile<D>(st + 2 * P::kOp, t, t.ic[c.z], row, c.h, c.seq, &c.b->full[s]);
  }
  c.b->issued = i;
}

template <int D>
__device__ __forceinline__ void pass_mma(const PassCtx& c) {
  using P = PassTile<D>;
  PassBars* b = c.b;
  int maps = 0;
  for (int i = 0; i < c.n; ++i) {
    const int s = i % kStages;
    const uint32_t a0 = smem_u32(c.sm + s * P::kStage), b0 = a0 + P::kOp, c0 = b0 + P::kOp;
    if (!wait(&b->full[s], (i / kStages) & 1, c.g)) return;
    if (i > 0 && !wait(&b->o_full, (i - 1) & 1, c.g)) return;  // the scores go over P of the last chunk
    if (c.mapped || c.chunk_len(c.chunk(i)) < kTok) {
      if (!wait(&b->mapped, maps & 1, c.g)) return;
      ++maps;
    }
    // D = 64: dX lies over the scores; X of this chunk is there once it has been read
    if (D == 64 && !wait(&b->x_full, i & 1, c.g)) return;
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (k / 4) * kAtom + (k % 4) * 32;
      mma_bf16(c.tmem + P::kColS, smem_desc(a0 + off, 16, 1024), smem_desc(b0 + off, 16, 1024),
               idesc_bf16_f32(128, 128, 0, 0), k > 0);
    }
    mma_commit(&b->s_full);
    if (D != 64 && !wait(&b->x_full, i & 1, c.g)) return;
    if (i > 0 && !wait(&b->o_free, (i - 1) & 1, c.g)) return;
    tc_fence_after();
    {
      const uint64_t dx = smem_desc(smem_u32(c.sm + P::kOffX), D * 128, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_bf16(c.tmem + P::kColInter, smem_desc(a0 + (k / 4) * kAtom + (k % 4) * 32, 16, 1024),
                 dx + k * (2048 >> 4), idesc_bf16_f32(128, D, 0, 1), k > 0);
    }
    mma_commit(&b->in_full);
    if (!wait(&b->p_full, i & 1, c.g)) return;
    tc_fence_after();
    {
      const uint64_t dc = smem_desc(c0, kAtom, 1024);
#pragma unroll
      for (int k = 0; k < kTok / 16; ++k)
        mma_bf16_ts(c.tmem + P::kColIntra, c.tmem + P::kColS + 8 * k, dc + k * (2048 >> 4),
                    idesc_bf16_f32(128, D, 0, 1), k > 0);
    }
    mma_commit(&b->o_full);
    if (i < c.nx) {
      if (!wait(&b->w_full, i & 1, c.g)) return;
      tc_fence_after();
      mma_outer<D, D>(c.tmem + P::kColDX, b0, c0, false);
      mma_outer<D, D>(c.tmem + P::kColDX, a0, c0, true);
      if (c.terms > 2) mma_outer<D, D>(c.tmem + P::kColDX, smem_u32(c.sm + P::kOffX), c0, true);
      mma_commit(&b->dx_full);
    }
    mma_commit(&b->empty[s]);
  }
}

// Warps 2-5, TMEM lane quadrant = warp % 4, one token row t a thread.
template <int D>
__device__ __forceinline__ void pass_out(const TcArgs& t, const PassCtx& c, int warp, int lane) {
  using P = PassTile<D>;
  PassBars* b = c.b;
  const RetPass& p = t.r.pass[c.z];
  const int qd = warp & 3, row = 32 * qd + lane, d = t.r.d;
  const uint32_t tl = c.tmem + ((uint32_t)(32 * qd) << 16);
  const float scale = t.r.scale;
  const bool wide = t.wide_out[c.z] != 0;
  const long long sn = p.out.sn, xsn = p.x.sn;
  const int xf = p.x.feature;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(const_cast<void*>(p.out.p)) + ret_base(t.r, p.out, c.seq, c.h);
  const __nv_bfloat16* xin = static_cast<const __nv_bfloat16*>(p.x.p);
  if (xin != nullptr) xin += ret_base(t.r, p.x, c.seq, c.h);
#pragma unroll 1
  for (int i = 0; i < c.n; ++i) {
    const int ch = c.chunk(i), len = c.chunk_len(ch);
    if (!wait_warp(&b->s_full, i & 1, c.g)) return;
    tc_fence_after();
    // block j of scores lies in columns 32 j .., its P in 16 j ..: never over scores still to be read
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      uint32_t w[16];
      if (c.reverse ? j < qd : j > qd) {
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = 0;
      } else {
        float v[32];
        tmem_ld16(tl + P::kColS + 32 * j, v);
        tmem_ld16(tl + P::kColS + 32 * j + 16, v + 16);
        // gamma^|t-s|; on the diagonal block the entries of the wrong sign are read beside the table and dropped
        const int n = row - 32 * j;
        float f[32];
        if (c.reverse) {
#pragma unroll
          for (int x = 0; x < 32; ++x) f[x] = b->decay[x - n];
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) f[x] = b->decay[n - x];
        }
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; ++x) v[x] *= f[x];
        if (j == qd) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (c.reverse ? x < lane : x > lane) v[x] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = pack_bf16(v[2 * x], v[2 * x + 1]);
      }
      tmem_st16u(tl + P::kColS + 16 * j, w);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->p_full);

    const bool live = row < len;
    const long long at = (long long)(c.row0 + ch * kTok + row);
    __nv_bfloat16* dst = out + at * sn;
    const __nv_bfloat16* xp = xin == nullptr ? nullptr : xin + at * xsn;
    const float wi = scale * decay_pow(c.lg, c.reverse ? max(len - row, 0) : row + 1);
    if (!wait_warp(&b->o_full, i & 1, c.g)) return;
    tc_fence_after();
#pragma unroll 1
    for (int g = 0; g < d; g += 16) {
      float u[16], v[16];
      tmem_ld16(tl + P::kColInter + g, u);
      tmem_ld16(tl + P::kColIntra + g, v);
      tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 16; ++x) v[x] = fmaf(wi, u[x], scale * v[x]);
      if (live) {
        if (xp != nullptr) {
          unpack8(*reinterpret_cast<const uint4*>(xp + g), u);
          unpack8(*reinterpret_cast<const uint4*>(xp + g + 8), u + 8);
#pragma unroll
          for (int x = 0; x < 16; ++x) v[x] *= ret_dphi(u[x], xf);
        }
        const uint4 lo8 = pack8(v), hi8 = pack8(v + 8);
        if (wide) {  // one whole 32-byte sector a store
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + g), "r"(lo8.x), "r"(lo8.y),
                       "r"(lo8.z), "r"(lo8.w), "r"(hi8.x), "r"(hi8.y), "r"(hi8.z), "r"(hi8.w)
                       : "memory");
        } else {
          *reinterpret_cast<uint4*>(dst + g) = lo8;
          *reinterpret_cast<uint4*>(dst + g + 8) = hi8;
        }
      }
      __syncwarp();  // the TMEM loads are the whole warp's
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->o_free);
  }
}

// Warps 6-9.  B w and the feature maps: one token row a thread.  X: TMEM lane quadrant = warp % 4, row c
// of X a lane (D = 64: M = 64 puts 16 rows into the first lanes of each quadrant).
template <int D>
__device__ __forceinline__ void pass_state(const TcArgs& t, const PassCtx& c, int warp, int lane, const float* from,
                                           bool from_t, float* to) {
  using P = PassTile<D>;
  PassBars* b = c.b;
  const RetPass& p = t.r.pass[c.z];
  const int qd = warp & 3, row = 32 * qd + lane, d = t.r.d;
  const int xr = D == 128 ? row : 16 * qd + lane;           // row of X
  const bool has = (D == 128 || lane < 16) && xr < d;
  const uint32_t tl = c.tmem + ((uint32_t)(32 * qd) << 16);
  const int fa = p.a.feature, fb = p.b.feature, fc = p.c.feature;
  const bool anew = c.terms > 2 && fb != kFeatIdentity;  // phi(b) in fp32 for the state
  uint8_t* xt = c.sm + P::kOffX;
  float X[D];
#pragma unroll
  for (int e = 0; e < D; e += 4) {
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
    if (from != nullptr && has && e < d) {
      if (from_t)
        u = make_float4(__ldcg(from + e * d + xr), __ldcg(from + (e + 1) * d + xr), __ldcg(from + (e + 2) * d + xr),
                        __ldcg(from + (e + 3) * d + xr));
      else
        u = __ldcg(reinterpret_cast<const float4*>(from + xr * d + e));
    }
    X[e] = u.x;
    X[e + 1] = u.y;
    X[e + 2] = u.z;
    X[e + 3] = u.w;
  }
  auto publish = [&] {
    if (D == 128 || lane < 16) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) *piece(xt, D, xr, j) = pack8(X + 8 * j);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->x_full);
  };
  auto map = [&](int i) -> bool {  // feature maps of chunk i, rows behind the sequence cleared in B and C
    const int len = c.chunk_len(c.chunk(i));
    if (!c.mapped && len == kTok) return true;
    if (!wait_warp(&b->full[i % kStages], (i / kStages) & 1, c.g)) return false;
    uint8_t* st = c.sm + (i % kStages) * P::kStage;
    if (fa != kFeatIdentity) map_row<D>(st, row, kTok, d, fa);
    if (fb != kFeatIdentity || len < kTok) map_row<D>(st + P::kOp, row, len, d, fb);
    if (fc != kFeatIdentity || len < kTok) map_row<D>(st + 2 * P::kOp, row, len, d, fc);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->mapped);
    return true;
  };
  if (!map(0)) return;
  publish();
#pragma unroll 1
  for (int i = 0; i < c.nx; ++i) {
    const int ch = c.chunk(i), len = c.chunk_len(ch);
    uint8_t* st = c.sm + (i % kStages) * P::kStage;
    // B has been read by the scores, A (and the old X) by inter
    if (!wait_warp(&b->s_full, i & 1, c.g) || !wait_warp(&b->in_full, i & 1, c.g)) return;
    const float w = row < len ? b->decay[c.reverse ? row : len - 1 - row] : 0.f;
    const __nv_bfloat16* raw = nullptr;
    if (anew && row < len)
      raw = static_cast<const __nv_bfloat16*>(p.b.p) + ret_base(t.r, p.b, c.seq, c.h) +
            (long long)(c.row0 + ch * kTok + row) * p.b.sn;
    // (without fp32 states the tile's rounded phi is good enough)
    weigh_row<D>(st + P::kOp, st, c.terms > 2 ? xt : nullptr, row, w, raw, d, anew ? fb : kFeatIdentity);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b->w_full);
    if (i + 1 < c.n && !map(i + 1)) return;
    const float wl = decay_pow(c.lg, len);
    if (!wait_warp(&b->dx_full, i & 1, c.g)) return;
    tc_fence_after();
#pragma unroll
    for (int g = 0; g < D / 16; ++g) {
      float u[16];
      tmem_ld16(tl + P::kColDX + 16 * g, u);
      tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 16; ++x) X[16 * g + x] = fmaf(wl, X[16 * g + x], u[x]);
    }
    if (i + 1 < c.n) publish();
  }
  if (to != nullptr && has) {
#pragma unroll
    for (int e = 0; e < D; e += 4)
      if (e < d) *reinterpret_cast<float4*>(to + xr * d + e) = make_float4(X[e], X[e + 1], X[e + 2], X[e + 3]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, PassTile<D>::kPerSm) retention_pass_kernel(const __grid_constant__ TcArgs t) {
  using P = PassTile<D>;
  extern __shared__ __align__(1024) uint8_t smraw[];
  PassCtx c;
  c.sm = smraw;
  c.b = reinterpret_cast<PassBars*>(c.sm + P::kOffBars);
  PassBars* b = c.b;
  const RetArgs& r = t.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  c.z = blockIdx.x % r.npass;  // a head's passes side by side: they read the same tensors
  const int unit = blockIdx.x / r.npass, g = unit / r.H;
  c.h = unit % r.H;
  const Segment sg = find_segment(r, g, b->scratch);
  if (sg.seq < 0) return;
  const int slot = r.states != nullptr ? ret_slot(r.slots, r.n_slots, sg.seq) : -1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&b->full[s], 1);
      mbar_init(&b->empty[s], 1);
    }
    for (uint64_t* m : {&b->s_full, &b->in_full, &b->dx_full, &b->o_full, &b->fin}) mbar_init(m, 1);
    for (uint64_t* m : {&b->mapped, &b->p_full, &b->w_full, &b->x_full, &b->o_free}) mbar_init(m, 4);
    b->abort = 0;
    b->issued = 0;
    fence_mbar_init();
  }
  c.lg = decay_log2(r.gamma[c.h]);
  if (threadIdx.x >= kThreads - kTok) {
    const int n = threadIdx.x - (kThreads - kTok);
    b->decay[n] = decay_pow(c.lg, n);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&b->tbase, P::kCols);
    tmem_relinquish();
  }
  if (warp == kWarpProd && lane == 0) {
    prefetch_tmap(&t.tm[t.ia[c.z]]);
    prefetch_tmap(&t.tm[t.ib[c.z]]);
    prefetch_tmap(&t.tm[t.ic[c.z]]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const RetPass& p = r.pass[c.z];
  c.g = {&b->abort, t.wait_ns};
  c.tmem = b->tbase;
  c.seq = sg.seq;
  c.row0 = sg.row0;
  c.len = sg.len;
  c.n = (sg.len + kTok - 1) / kTok;
  const size_t dd = (size_t)r.d * r.d;
  float* to = slot >= 0 && sg.seg == sg.nseg - 1 ? r.states + ((size_t)slot * r.H + c.h) * dd : nullptr;
  c.nx = to != nullptr ? c.n : c.n - 1;
  c.reverse = p.reverse;
  c.terms = r.states != nullptr ? 3 : 2;
  c.mapped = p.a.feature != kFeatIdentity || p.b.feature != kFeatIdentity || p.c.feature != kFeatIdentity;
  const float* from = nullptr;
  if (sg.nseg > 1)
    from = r.seg + (((size_t)p.sum * r.G + g) * r.H + c.h) * dd;
  else if (r.load && slot >= 0)
    from = r.states + ((size_t)slot * r.H + c.h) * dd;

  if (warp == kWarpProd) {
    if (lane == 0) pass_producer<D>(t, c);
    __syncwarp();
  } else if (warp == kWarpMma) {
    if (lane == 0) {
      pass_mma<D>(c);
      mma_commit(&b->fin);
    }
    __syncwarp();
  } else if (warp < kWarpX) {
    pass_out<D>(t, c, warp, lane);
  } else {
    pass_state<D>(t, c, warp, lane, from, sg.nseg > 1 && p.sum_t, to);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) {
    drain(&b->fin, 0);
    if (aborted(c.g)) {
      for (int q = b->issued > kStages ? b->issued - kStages : 0; q < b->issued; ++q)
        drain(&b->full[q % kStages], (q / kStages) & 1);
      atomicOr(r.status, 1u);
    }
  }
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(c.tmem, P::kCols);
}

// ================================================================ segment sums
template <int D>
struct SumTile {
  static constexpr int kOp = (D / 64) * kAtom;
  static constexpr int kStage = 2 * kOp;                // B, C
  static constexpr int kOffLo = kStages * kStage;       // the second and third part of B w
  static constexpr int kOffBars = kOffLo + 2 * kOp;
};

constexpr int kSumThreads = 192;                         // producer, MMA issuer, 4 warps for the rest

struct SumBars {
  uint64_t full[kStages], empty[kStages], ready[kStages];
  uint64_t fin;
  uint32_t tbase;
  int abort;
  int issued;
  int scratch[34];
};

template <int D>
constexpr size_t sum_smem() {
  return SumTile<D>::kOffBars + sizeof(SumBars);
}
static_assert(sum_smem<128>() <= 232448 && 2 * (sum_smem<64>() + 1024) <= 233472, "shared memory budget");

template <int D>
__global__ void __launch_bounds__(kSumThreads) retention_sum_kernel(const __grid_constant__ TcArgs t) {
  using P = SumTile<D>;
  extern __shared__ __align__(1024) uint8_t smraw[];
  uint8_t* sm = smraw;
  SumBars* b = reinterpret_cast<SumBars*>(sm + P::kOffBars);
  const RetArgs& r = t.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int set = blockIdx.x % r.nsum, unit = blockIdx.x / r.nsum, h = unit % r.H, g = unit / r.H;
  int z = 0;
  for (int i = 0; i < r.npass; ++i)
    if (r.pass[i].sum == set && !r.pass[i].sum_t) z = i;
  const RetPass& p = r.pass[z];
  const Segment sg = find_segment(r, g, b->scratch);
  if (sg.seq < 0 || (p.reverse ? sg.seg == 0 : sg.seg == sg.nseg - 1)) return;  // enters no other segment
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&b->full[s], 1);
      mbar_init(&b->empty[s], 1);
      mbar_init(&b->ready[s], 4);
    }
    mbar_init(&b->fin, 1);
    b->abort = 0;
    b->issued = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&b->tbase, D);
    tmem_relinquish();
  }
  if (warp == kWarpProd && lane == 0) {
    prefetch_tmap(&t.tm[t.ib[z]]);
    prefetch_tmap(&t.tm[t.ic[z]]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Guard gd{&b->abort, t.wait_ns};
  const uint32_t tmem = b->tbase;
  const int n = (sg.len + kTok - 1) / kTok;
  const int terms = r.states != nullptr ? 3 : 2;
  uint8_t* lo = sm + P::kOffLo;

  if (warp == kWarpProd) {
    if (lane == 0) {
      int i = 0;
      for (; i < n; ++i) {
        const int s = i % kStages;
        if (i >= kStages && !wait(&b->empty[s], ((i / kStages) - 1) & 1, gd)) break;
        uint8_t* st = sm + s * P::kStage;
        mbar_arrive_expect_tx(&b->full[s], 2 * P::kOp);
        load_tile<D>(st, t, t.ib[z], sg.row0 + i * kTok, h, sg.seq, &b->full[s]);
        load_tile<D>(st + P::kOp, t, t.ic[z], sg.row0 + i * kTok, h, sg.seq, &b->full[s]);
      }
      b->issued = i;
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    if (lane == 0) {
      for (int i = 0; i < n; ++i) {
        const int s = i % kStages;
        if (!wait(&b->ready[s], (i / kStages) & 1, gd)) break;
        tc_fence_after();
        const uint32_t b0 = smem_u32(sm + s * P::kStage);
        mma_outer<D, D>(tmem, b0, b0 + P::kOp, i > 0);
        mma_outer<D, D>(tmem, smem_u32(lo), b0 + P::kOp, true);
        if (terms > 2) mma_outer<D, D>(tmem, smem_u32(lo) + P::kOp, b0 + P::kOp, true);
        mma_commit(&b->empty[s]);
      }
      mma_commit(&b->fin);
    }
    __syncwarp();
  } else {
    const int qd = warp & 3, row = 32 * qd + lane;
    const float lg = decay_log2(r.gamma[h]);
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int s = i % kStages, at = i * kTok + row, len = min(kTok, sg.len - i * kTok);
      ok = wait_warp(&b->full[s], (i / kStages) & 1, gd);
      if (!ok) break;
      uint8_t* st = sm + s * P::kStage;
      // the remainders' tiles have been read by the MMAs of the chunk before
      if (i > 0) ok = wait_warp(&b->empty[(i - 1) % kStages], ((i - 1) / kStages) & 1, gd);
      if (!ok) break;
      if (p.c.feature != kFeatIdentity || len < kTok) map_row<D>(st + P::kOp, row, len, r.d, p.c.feature);
      const float w = row < len ? decay_pow(lg, p.reverse ? at : sg.len - 1 - at) : 0.f;
      weigh_row<D>(st, lo, terms > 2 ? lo + P::kOp : nullptr, row, w, nullptr, r.d, p.b.feature);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->ready[s]);
    }
    if (ok && wait_warp(&b->fin, 0, gd) && !aborted(gd)) {
      tc_fence_after();
      const int xr = D == 128 ? row : 16 * qd + lane;
      const bool has = (D == 128 || lane < 16) && xr < r.d;
      float* dst = r.seg + (((size_t)set * r.G + g) * r.H + h) * r.d * r.d + (size_t)xr * r.d;
#pragma unroll
      for (int q = 0; q < D / 16; ++q) {
        float u[16];
        tmem_ld16(tmem + ((uint32_t)(32 * qd) << 16) + 16 * q, u);
        tmem_ld_wait();
        if (has && 16 * q < r.d) {
#pragma unroll
          for (int x = 0; x < 16; x += 4)
            *reinterpret_cast<float4*>(dst + 16 * q + x) = make_float4(u[x], u[x + 1], u[x + 2], u[x + 3]);
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
      for (int q = b->issued > kStages ? b->issued - kStages : 0; q < b->issued; ++q)
        drain(&b->full[q % kStages], (q / kStages) & 1);
      atomicOr(r.status, 1u);
    }
  }
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tmem, D);
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

bool wide_rows(const RetTensor& x) {
  return (reinterpret_cast<uintptr_t>(x.p) & 31) == 0 && x.sb % 16 == 0 && x.sh % 16 == 0 && x.sn % 16 == 0;
}

template <int D>
cudaError_t launch(const TcArgs& t, cudaStream_t st) {
  static SmemOptIn opt_pass, opt_sum;
  cudaError_t e = opt_pass.ensure((const void*)retention_pass_kernel<D>, (int)pass_smem<D>());
  if (e == cudaSuccess) e = opt_sum.ensure((const void*)retention_sum_kernel<D>, (int)sum_smem<D>());
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)(t.r.G * t.r.H);
  if (t.r.seg != nullptr) {
    retention_sum_kernel<D><<<units * t.r.nsum, kSumThreads, sum_smem<D>(), st>>>(t);
    note_launch();
    e = retention_scan_launch(t.r, st);
    if (e != cudaSuccess) return e;
  }
  retention_pass_kernel<D><<<units * t.r.npass, kThreads, pass_smem<D>(), st>>>(t);
  note_launch();
  return cudaGetLastError();
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
    t.wide_out[i] = wide_rows(a.pass[i].out);
  }
  if (!ok) return cudaErrorInvalidValue;
  return a.d == 128 ? launch<128>(t, st) : launch<64>(t, st);
}

}  // namespace mhla
