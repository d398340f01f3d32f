/*
 * mhla.h — C ABI of the GB300 (sm_103a) token-level multi-head linear
 * attention (MHLA) forward library.
 *
 * Sources of the operations (cited by page title and section):
 *   [MHLA]  "MHLA: Restoring Expressivity of Linear Attention via Token-Level
 *           Multi-Head" — §4.1 (local KV summaries, multi-head mixing,
 *           output), §4.2 (token-level form, chunkwise-parallel causal form),
 *           App. C (causal chunked linear attention and causal inference).
 *   [LA]    "Linear Attention（线性注意力）笔记" — §二 (phi = ELU + 1),
 *           §四 (recurrent form, eps in the denominator), §五 (parallel form),
 *           §七 (RetNet decay), §八 (the constant-size state).
 *   [MASK]  "4. Attention" tutorial — "Mask": the causal mask removes only
 *           the future (strict upper triangle).
 *   [RALA]  "Breaking the Low-Rank Dilemma of Linear Attention" notes — key
 *           designs 1 (KV buffer rank augmentation) and 2 (output rank
 *           augmentation).
 *
 * Conventions shared by every entry point
 *   - phi(x) = ELU(x) + 1 = (x > 0 ? x + 1 : exp(x))            [LA §二]
 *   - Q, K, V, Y are dense row-major [B, H, N, d] (d innermost); the (b, h)
 *     slices are independent problems.  d must be 16, 32, 64 or 128.
 *   - dtype: MHLA_F32 (fp32 in/out, fp32 arithmetic) or MHLA_BF16 (bf16
 *     in/out, fp32 accumulation; summaries, normalisers and decode state are
 *     fp32).  Outputs have the input dtype.
 *   - Every pointer is a DEVICE pointer unless stated otherwise, 16-byte
 *     aligned; the caller owns all memory, including the workspace.  No call
 *     allocates memory (the one device-resident buffer of the library is the
 *     fixed scratch array of mhla_forward_noalloc, below) and no call keeps
 *     per-call state outside the workspace; calls are asynchronous on `stream`
 *     (a cudaStream_t, 0 = the legacy default stream) and do not synchronise
 *     the host.
 *   - Argument errors are detected on the host before any launch and return
 *     MHLA_ERR_INVALID_ARG (or MHLA_ERR_UNSUPPORTED for valid but
 *     unimplemented combinations) without touching device memory.  Launch
 *     failures return MHLA_ERR_CUDA.  Sizes with B*H*N == 0 are a no-op.
 *   - Workspace: at least the size returned by the matching *_workspace_bytes
 *     query, 256-byte aligned.  Before its FIRST use a workspace must be
 *     zero-filled (e.g. cudaMemsetAsync); the library leaves it ready for the
 *     next call.  Calls that share a workspace must not overlap on the GPU.
 *     A workspace may be reused across shapes as long as it is big enough.
 *   - Device-side waits (between the summary, mixing and output stages of
 *     one launch) are bounded; if one gives up, the output is incomplete and
 *     MHLA_ERR_TIMEOUT is latched in the workspace; mhla_query_status()
 *     reports it.
 */
#ifndef MHLA_GB300_H
#define MHLA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MHLA_OK = 0,
  MHLA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, bad size, aliasing, small workspace */
  MHLA_ERR_UNSUPPORTED = 2,  /* valid request this build does not implement */
  MHLA_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed */
  MHLA_ERR_TIMEOUT = 4       /* a bounded device-side wait gave up (latched in the workspace) */
} mhla_status;

typedef enum { MHLA_F32 = 0, MHLA_BF16 = 1 } mhla_dtype;

/* Which kernel family mhla_forward / mhla_forward_causal would run:
 * TCGEN05 the three-pass tensor-core kernel (summaries, grid-wide mixing,
 * output), TCGEN05_STREAM the tensor-core kernel that runs them as one stream
 * of work items with per-head readiness (bf16, d = 64, N / 128 not a multiple
 * of 16). */
typedef enum {
  MHLA_PATH_NONE = 0,
  MHLA_PATH_SIMT = 1,
  MHLA_PATH_TCGEN05 = 2,
  MHLA_PATH_TCGEN05_STREAM = 3
} mhla_path;

/* Workspace bytes for mhla_forward (causal = 0) or mhla_forward_causal
 * (causal = 1, block_size = chunk) with these sizes; 0 if the sizes are
 * invalid.  Valid for both dtypes. */
size_t mhla_workspace_bytes(int B, int H, int N, int d, int block_size, int causal);

/* MHLA forward, non-causal ([MHLA] §4.1; eps as in [LA] §五).
 *   Blocks are the M = N / block_size contiguous token ranges of block_size
 *   tokens.  For each (b, h) and block j:
 *     S_j = sum_{t in j} phi(K_t) V_t^T  (d x d, S_j[c][e]),  z_j = sum_{t in j} phi(K_t)
 *   for each query block i:  S~_i = sum_j m[h][i][j] S_j,   z~_i = sum_j m[h][i][j] z_j
 *   for token t in block i:  Y_t = phi(Q_t) S~_i / (phi(Q_t) . z~_i + eps)
 *   q, k, v : [B, H, N, d] (dtype dt)            — inputs
 *   mixing  : [H, M, M] fp32, row i = query block — input; not inspected
 *             (non-negative rows are the caller's contract, [MHLA] §4.2)
 *   y       : [B, H, N, d] (dtype dt)            — output, must not overlap q, k, v
 *   den_out : [B, H, N] fp32 or NULL             — optional output of the denominator
 *   block_size divides N; M = 1 is global linear attention ([LA] §五).
 *   causal  : 0 for the form above; 1 computes causal MHLA exactly as
 *             mhla_forward_causal(..., mixing, ..., chunk = block_size).
 *   eps     : finite, >= 0 (1e-6 in [LA]). */
mhla_status mhla_forward(const void* q, const void* k, const void* v, const float* mixing,
                         void* y, float* den_out, int B, int H, int N, int d, int block_size,
                         int causal, mhla_dtype dt, float eps, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Causal chunked forward ([MHLA] App. C with the [MASK] convention and the
 * [LA] §四 normaliser).  Chunks are contiguous ranges of `chunk` tokens
 * (chunk divides N).  For token t in chunk i:
 *   mixing == NULL (plain causal linear attention):
 *     Y_t = [phi(Q_t) P_i + sum_{s in i, s<=t} (phi(Q_t).phi(K_s)) V_s]
 *         / [phi(Q_t) . zeta_i + sum_{s in i, s<=t} phi(Q_t).phi(K_s) + eps]
 *     with P_i = sum_{j<i} S_j, zeta_i = sum_{j<i} z_j (exclusive prefixes);
 *     equal to the recurrence S_t = S_{t-1} + phi(k_t) v_t^T of [LA] §四.
 *   mixing != NULL ([H, M, M] fp32, M = N / chunk; causal MHLA, [MHLA] §4.2
 *     chunkwise form): P_i = sum_{j<i} m[h][i][j] S_j, zeta_i likewise, and
 *     the intra-chunk sums are scaled by m[h][i][i]; entries above the
 *     diagonal are ignored.
 *   Other arguments as in mhla_forward. */
mhla_status mhla_forward_causal(const void* q, const void* k, const void* v, const float* mixing,
                                void* y, float* den_out, int B, int H, int N, int d, int chunk,
                                mhla_dtype dt, float eps, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Variants of the forward (mhla_forward_ex). */
typedef enum {
  MHLA_PHI_ELU1 = 0, /* phi(x) = ELU(x) + 1 (the default everywhere)   [LA §二] */
  MHLA_PHI_RELU = 1, /* phi(x) = max(x, 0)                              [LA §二] */
  MHLA_PHI_EXP = 2,  /* phi(x) = exp(x)                                 [LA §二] */
  MHLA_PHI_IDENTITY = 3 /* phi(x) = x: the retention_* and linattn_cross_* entries only [LA §七] */
} mhla_feature;

typedef struct {
  int feature;   /* an mhla_feature */
  int normalise; /* 1: Y = numerator / (phi(q) . z~ + eps) (default);
                    0: Y = numerator alone ([MHLA] §4.1: the normalisation may be
                    omitted for long sequences); den_out, if given, still receives
                    the denominator */
  float gamma;   /* RetNet decay of plain causal linear attention ([LA] §七), in
                    [0, 1]; 1 = none.  Y_t = sum_{s<=t} gamma^(t-s) (phi(q_t).phi(k_s)) v_s
                    / (sum_{s<=t} gamma^(t-s) phi(q_t).phi(k_s) + eps) */
} mhla_options;

/* mhla_forward with variants (opt NULL = the defaults {ELU1, 1, 1.0}, exactly
 * mhla_forward).  gamma != 1 needs causal = 1 and mixing = NULL (plain causal
 * linear attention), else MHLA_ERR_INVALID_ARG; a feature outside the enum,
 * normalise not 0 / 1 or gamma outside [0, 1] are MHLA_ERR_INVALID_ARG.  The
 * tensor-core kernels take ELU + 1 without decay (normalise 0 or 1); the other
 * variants run on the SIMT kernels.  Same workspace as mhla_forward. */
mhla_status mhla_forward_ex(const void* q, const void* k, const void* v, const float* mixing,
                            void* y, float* den_out, int B, int H, int N, int d, int block_size,
                            int causal, mhla_dtype dt, float eps, const mhla_options* opt,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Kernel family mhla_forward_ex would use for these arguments (no launch);
 * `with_mixing` says whether a mixing matrix is passed (it selects causal MHLA
 * or plain causal linear attention when causal = 1). */
mhla_path mhla_forward_ex_path(int B, int H, int N, int d, int block_size, int causal, int with_mixing,
                               mhla_dtype dt, const mhla_options* opt);

/* Non-causal MHLA with 2-D blocks ([MHLA] §4.1: for images the blocks lie on
 * a 2-D grid, Fig. 4b).  The N = grid_h * grid_w tokens of each (b, h) slice
 * are a grid_h x grid_w grid in row-major order (token t = row * grid_w + col,
 * the layout of the [B, H, N, d] tensors is unchanged); the blocks are the
 * tile_h x tile_w tiles of the grid, numbered row-major over the
 * (grid_h / tile_h) x (grid_w / tile_w) tile grid, M = their count; b(t) is
 * the tile holding token t.  Then, as in mhla_forward:
 *   S_b = sum_{t: b(t)=b} phi(K_t) V_t^T,  z_b likewise,
 *   S~_i = sum_b m[h][i][b] S_b,  Y_t = phi(Q_t) S~_{b(t)} / (phi(Q_t) . z~_{b(t)} + eps).
 *   mixing : [H, M, M] fp32 (mhla_locality_mixing gives the paper's initial value).
 *   tile_h must divide grid_h and tile_w grid_w, else MHLA_ERR_INVALID_ARG.
 *   workspace: mhla_workspace_bytes(B, H, grid_h * grid_w, d, tile_h * tile_w, 0).
 *   On a one-row grid (grid_h = tile_h = 1) the blocks are contiguous ranges
 *   of tile_w tokens and the result is that of mhla_forward.
 *   Other arguments as in mhla_forward. */
mhla_status mhla_forward_grid(const void* q, const void* k, const void* v, const float* mixing,
                              void* y, float* den_out, int B, int H, int grid_h, int grid_w,
                              int tile_h, int tile_w, int d, mhla_dtype dt, float eps,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Kernel family mhla_forward_grid would use (no launch): the tensor-core
 * kernels take bf16, d = 64, tiles of a multiple of 128 tokens with tile_w
 * dividing 128 or a multiple of 128, M <= 64; else the SIMT kernels. */
mhla_path mhla_forward_grid_path(int B, int H, int grid_h, int grid_w, int tile_h, int tile_w, int d,
                                 mhla_dtype dt);

/* The locality-based initial mixing matrix of [MHLA] §4.2 for blocks on a
 * blocks_h x blocks_w grid (M = blocks_h * blocks_w, numbered row-major):
 * m[i][j] proportional to 1 - dist(i, j) / max_k dist(i, k), dist the
 * Euclidean distance between the blocks' grid positions, each row normalised
 * to sum to 1 (a single block: [[1]]).  `m` is a HOST array [M][M] fp32 that
 * the caller owns; computed on the host (a one-off initialisation, not part
 * of the forward).  M above 65536 returns MHLA_ERR_INVALID_ARG. */
mhla_status mhla_locality_mixing(float* m, int blocks_h, int blocks_w);

/* One recurrent decode step for B*H independent (batch, head) states
 * ([LA] §四; the fixed-size state of [LA] §八; [MHLA] App. C inference).
 *   q, k, v : [B, H, d] (dtype dt)       — this step's token
 *   S       : [B, H, d, d] fp32, in/out — S[c][e] = sum over past tokens of phi(k)_c v_e
 *   z       : [B, H, d] fp32, in/out    — sum over past tokens of phi(k)
 *   out     : [B, H, d] (dtype dt)      — output; must not overlap the inputs or the state
 *   den_out : [B, H] fp32 or NULL
 *   Order: S += phi(k) v^T; z += phi(k); out = phi(q) S / (phi(q) . z + eps),
 *   i.e. the token attends to itself.  No workspace. */
mhla_status linattn_decode_step(const void* q, const void* k, const void* v, float* S, float* z,
                                void* out, float* den_out, int B, int H, int d, mhla_dtype dt,
                                float eps, void* stream);

/* T consecutive recurrent decode steps in one call, for B*H independent
 * (batch, head) states ([LA] §四 recurrence; [LA] §七 RetNet decay; the
 * fixed-size state of [LA] §八).
 *   q, k, v : [T, B, H, d] (dtype dt)    — step t's tokens at [t]
 *   S       : [B, H, d, d] fp32, in/out — as in linattn_decode_step
 *   z       : [B, H, d] fp32, in/out
 *   out     : [T, B, H, d] (dtype dt)    — must not overlap the inputs or the state
 *   den_out : [T, B, H] fp32 or NULL     — each step's phi(q) . z + eps
 *   gamma   : decay in [0, 1]; 1 gives exactly the steps of linattn_decode_step.
 *   Per step: S <- gamma S + phi(k) v^T; z <- gamma z + phi(k);
 *   out = phi(q) S / (phi(q) . z + eps).  (The notes decay S; z decays with
 *   it so that the output stays a weighted mean of the values.)
 *   Equal, up to fp32 rounding, to T calls of linattn_decode_step when
 *   gamma = 1; the state is read once and written once per call.
 *   T = 0 or B*H = 0 returns MHLA_OK without a launch.  B*H above 2^29
 *   returns MHLA_ERR_UNSUPPORTED.  No workspace. */
mhla_status linattn_decode_steps(const void* q, const void* k, const void* v, float* S, float* z,
                                 void* out, float* den_out, int T, int B, int H, int d, mhla_dtype dt,
                                 float eps, float gamma, void* stream);

/* Causal MHLA inference, token by token ([MHLA] App. C, causal inference):
 * tokens t0 .. t0 + T - 1 of each (b, h) sequence, whose blocks are the
 * contiguous ranges of `block` tokens (block i holds tokens i*block ..).
 *   q, k, v : [T, B, H, d] (dtype dt) — token t0 + n at [n]
 *   mixing  : [H, M, M] fp32, read at and below the diagonal (m[h][i][b], b <= i)
 *   S       : [B, H, M, d, d] fp32, in/out — slot b: the summary sum phi(k) v^T of
 *             block b (S[c][e] = sum phi(k)_c v_e); slots of finished blocks are
 *             frozen, the slot of the block holding token t0 holds its running
 *             summary of the tokens before t0 (ignored, taken as zero, when t0
 *             starts the block)
 *   z       : [B, H, M, d] fp32, in/out — the same for sum phi(k)
 *   out     : [T, B, H, d] (dtype dt);  den_out : [T, B, H] fp32 or NULL
 *   Per token t in block i: S_i += phi(k) v^T; z_i += phi(k);
 *     out = phi(q) (sum_{b<i} m_ib S_b + m_ii S_i)
 *         / (phi(q) . (sum_{b<i} m_ib z_b + m_ii z_i) + eps);
 *   on return the slots of the blocks the call touched hold their summaries
 *   (running for the last one).  Token by token this equals
 *   mhla_forward_causal with this mixing and chunk = block.
 *   t0 + T must not pass M * block (MHLA_ERR_INVALID_ARG).  No workspace. */
mhla_status mhla_causal_stream(const void* q, const void* k, const void* v, const float* mixing, float* S,
                               float* z, void* out, float* den_out, int t0, int T, int B, int H, int d,
                               int block, int M, mhla_dtype dt, float eps, void* stream);

/* Workspace bytes for mhla_backward; 0 if the sizes are invalid or unsupported
 * (N / block_size above 64). */
size_t mhla_backward_workspace_bytes(int B, int H, int N, int d, int block_size);

/* Backward of the non-causal MHLA forward (mhla_forward with causal = 0:
 * contiguous blocks, phi = ELU + 1, with the normaliser) for training the
 * mixing end to end ([MHLA] §4.2; the pages give no backward formulas, these
 * are the chain rule through the steps of [MHLA] §4.1):
 *   dnum_t = dY_t / den_t,  dden_t = -(dY_t . Y_t) / den_t
 *   dS~_i = sum_{t in i} phi(q_t) dnum_t^T,  dz~_i = sum_{t in i} phi(q_t) dden_t
 *   dq_t = phi'(q_t) * (S~_i dnum_t + dden_t z~_i)
 *   dS_b = sum_i m_ib dS~_i,  dz_b = sum_i m_ib dz~_i
 *   dm[h][i][b] = sum over the samples of <dS~_i, S_b> + dz~_i . z_b
 *   dk_j = phi'(k_j) * (dS_b v_j + dz_b),  dv_j = dS_b^T phi(k_j)
 * with phi'(x) = 1 for x > 0 and exp(x) otherwise.  S, z, S~, z~, Y and den
 * are recomputed from q, k, v and the mixing (the forward saves nothing).
 *   q, k, v, dy     : [B, H, N, d] (dtype dt), as given to the forward; dy = dL/dY
 *   mixing          : [H, M, M] fp32, M = N / block_size <= 64
 *   dq, dk, dv      : [B, H, N, d] (dtype dt), written (not accumulated)
 *   dmixing         : [H, M, M] fp32, written (not accumulated); sums over the B samples
 *   workspace       : >= mhla_backward_workspace_bytes(...) device bytes,
 *                     256-byte aligned; must not overlap any argument
 *   workspace       : zero-filled before its first use (a status word at its
 *                     start, as for mhla_forward; the library leaves it zero
 *                     unless a device wait gave up, which mhla_query_status
 *                     reports as MHLA_ERR_TIMEOUT and clears)
 * Paths (mhla_backward_path): bf16 with d = 64 and block_size a multiple of
 * 128 runs the token passes on the tensor cores (bf16 operands: phi(Q),
 * phi(K), V, dY, dnum, dden and the bf16-rounded S~ and dS; fp32
 * accumulation); everything else, and the summaries, mixing and dM, run on
 * the SIMT cores in fp32 (bf16 values widened at the loads, gradients rounded
 * at the stores).  Outputs must not overlap the inputs or each other
 * (MHLA_ERR_INVALID_ARG).  M above 64 returns MHLA_ERR_UNSUPPORTED.
 * B*H*N = 0 returns MHLA_OK without a launch.  Deterministic: every sum has a
 * fixed order. */
mhla_status mhla_backward(const void* q, const void* k, const void* v, const float* mixing, const void* dy,
                          void* dq, void* dk, void* dv, float* dmixing, int B, int H, int N, int d, int block_size,
                          mhla_dtype dt, float eps, void* workspace, size_t workspace_bytes, void* stream);

/* Kernel family mhla_backward would use for these arguments (no launch):
 * MHLA_PATH_TCGEN05 for the tensor-core token passes, MHLA_PATH_SIMT
 * otherwise, MHLA_PATH_NONE for invalid or unsupported sizes. */
mhla_path mhla_backward_path(int B, int H, int N, int d, int block_size, mhla_dtype dt);

/* ---------------------------------------------------------------- retention
 * Linear attention with a decay for each head ([LA] §七, RetNet):
 *   S_t = gamma_h S_{t-1} + phi(k_t) v_t^T,   y_t = scale * phi(q_t) S_t
 * (update, then read, as everywhere in this library; no normaliser and no eps).
 * Prompts and training run in chunks, single tokens recurrently; the state S
 * [d][d] fp32 (S[c][e] = sum gamma^(t-s) phi(k_s)_c v_se) carries a sequence
 * from one call to the next.
 *
 * Conventions of the retention_* entries:
 *   - Token tensors are [B, H, N, d], d = 16, 32, 64 or 128 for keys and
 *     values alike, with any strides: an mhla_strides holds
 *     the element strides of b, h and n (d contiguous); NULL means dense
 *     row-major.  Strides are >= 0 and, like the pointers, multiples of 16
 *     bytes; an input may have stride 0 in b and h (keys shared by several
 *     heads), an output may not overlap itself.  So token-major tensors and slices of a fused
 *     projection are taken as they are.
 *   - cu_seqlens: NULL, or device int32 [B + 1]: then the tensors are
 *     [1, H, N, d] (the b strides are not used) and sequence i is the rows
 *     cu_seqlens[i] .. cu_seqlens[i + 1] - 1, of any lengths, empty ones among
 *     them.  Rows of no sequence are not written.  The offsets are not
 *     inspected by the host: non-decreasing values in [0, N] are the caller's
 *     contract, anything else is clamped to it and touches no other memory.
 *   - A call takes up to 2^31 - 128 tokens (dense: B N); more:
 *     MHLA_ERR_UNSUPPORTED, and no workspace size.
 *   - gamma: device fp32 [H], each in [0, 1] (the caller's contract).
 *   - states: [n_slots, H, d, d] fp32.  slots: device int32 [B], the slot of
 *     each sequence or row, or NULL (sequence i uses slot i).  A sequence whose
 *     slot is outside [0, n_slots), or is the slot of a sequence before it, has
 *     none: see the entries.
 *   - Not-a-number or infinite values of a token reach its own sequence only;
 *     in retention_forward and retention_backward they, and products
 *     phi(q_t) . phi(k_s) that overflow, may reach all 128 tokens of the chunk
 *     that they are in, also those before them. */

/* Element strides of a [B, H, N, d] tensor. */
typedef struct {
  long long b, h, n;
} mhla_strides;

typedef struct {
  int feature; /* an mhla_feature, applied to q and k (default MHLA_PHI_IDENTITY) */
  float scale; /* finite (default 1) */
} retention_options;

/* Workspace bytes of retention_forward (backward = 0) or retention_backward
 * (backward = 1) for B sequences of `tokens` tokens in all (dense: B N); 0 if
 * the sizes are invalid or more than a call takes.  Valid for both dtypes, dense and packed. */
size_t retention_workspace_bytes(int B, int H, int tokens, int d, int backward);

/* The outputs of whole prompts.
 *   q, k, v : inputs;  y : output, overlapping no input
 *   states  : NULL, or read (load_state = 1: a sequence starts from its slot's
 *             state; 0: from zero) and written (the state after its last token).
 *             A sequence without a slot starts from zero and its state is not
 *             kept; one without tokens leaves its slot as it is.
 *   opt     : NULL = the defaults
 *   B*H*N = 0 returns MHLA_OK without a launch. */
mhla_status retention_forward(const void* q, const mhla_strides* q_strides, const void* k,
                              const mhla_strides* k_strides, const void* v, const mhla_strides* v_strides,
                              const float* gamma, void* y, const mhla_strides* y_strides, int B, int H, int N, int d,
                              const int* cu_seqlens, float* states, const int* slots, int n_slots, int load_state,
                              mhla_dtype dt, const retention_options* opt, void* workspace, size_t workspace_bytes,
                              void* stream);

/* The gradients of q, k and v of retention_forward without states, for training:
 *   G_t = gamma_h G_{t+1} + scale phi(q_t) dy_t^T
 *   dq_t = phi'(q_t) * (scale S_t dy_t),  dk_t = phi'(k_t) * (G_t v_t),  dv_t = G_t^T phi(k_t)
 * from a zero state before the first token and with none asked for behind the last,
 * with phi' = 1 (identity), phi'(x) = 1 for x > 0 and exp(x) otherwise (ELU + 1),
 * 1 for x > 0 and 0 otherwise (ReLU), exp(x) (exp).  gamma is a constant.
 *   dy : input, dL/dY;  dq, dk, dv : outputs, written (not accumulated), of the
 *   full shape also where an input is shared by stride 0; overlapping neither
 *   an input nor each other.  Deterministic: every sum has a fixed order. */
mhla_status retention_backward(const void* q, const mhla_strides* q_strides, const void* k,
                               const mhla_strides* k_strides, const void* v, const mhla_strides* v_strides,
                               const float* gamma, const void* dy, const mhla_strides* dy_strides, void* dq,
                               const mhla_strides* dq_strides, void* dk, const mhla_strides* dk_strides, void* dv,
                               const mhla_strides* dv_strides, int B, int H, int N, int d, const int* cu_seqlens,
                               mhla_dtype dt, const retention_options* opt, void* workspace, size_t workspace_bytes,
                               void* stream);

/* One token for each of B rows: updates the rows' states and writes out.
 *   q, k, v, out : [B, H, d]; of the strides b and h are used
 *   A row without a slot is left out: neither its output nor a state is touched.
 *   No workspace. */
mhla_status retention_step(const void* q, const mhla_strides* q_strides, const void* k, const mhla_strides* k_strides,
                           const void* v, const mhla_strides* v_strides, const float* gamma, float* states,
                           const int* slots, int n_slots, void* out, const mhla_strides* out_strides, int B, int H,
                           int d, mhla_dtype dt, const retention_options* opt, void* stream);

/* states[dst[i]] = states[src[i]] for the n pairs, src[i] < 0: zeros.  Forks one
 * state to many, moves states together, clears slots.  As if every source were
 * read before any target is written, so slots may be sources and targets in
 * any combination.  src, dst: device int32 [n], n <= 1024 (more:
 * MHLA_ERR_UNSUPPORTED).  A pair whose src is >= n_slots or whose dst is outside
 * [0, n_slots) does nothing; of several pairs with one target the last counts.
 * No workspace. */
mhla_status retention_copy_states(float* states, int n_slots, int H, int d, const int* src, const int* dst, int n,
                                  void* stream);

/* --------------------------------------------------------------- gated scan
 * A recurrence with a gate of its own for every token and channel ([LA] §七, the
 * gated update S_t = G_t * S_{t-1} + ..., for a state of one vector):
 *   h_t = a_t h_{t-1} + b_t,   y_t = h_t      (elementwise over the D channels)
 *   GATED_SCAN_SIGMOID: a = sigmoid(g),  b = (1 - a) x
 *   GATED_SCAN_LOG    : a = exp(g),      b = x     (g <= 0 is the caller's contract)
 *   GATED_SCAN_DECAY  : a = g,           b = x     (g in [0, 1] is the caller's contract)
 * Conventions of the gated_scan_* entries:
 *   - Token tensors are [B, N, D] (the step: [B, D]), D a multiple of 8 (bf16) or
 *     4 (fp32), with any strides (the members b and n of mhla_strides; h is not
 *     used) under the rules of the retention_* entries; an input may have stride
 *     0 in b.  Outputs overlap neither inputs nor each other nor themselves.
 *   - cu_seqlens as there: NULL, or device int32 [B + 1] with tensors [1, N, D].
 *     Rows of no sequence are not written.
 *   - At most 2^31 - 1024 tokens a sequence (packed: a call) and as many channels:
 *     MHLA_ERR_UNSUPPORTED.
 *   - states: [n_slots, D] fp32, slots as there: a sequence whose slot is outside
 *     [0, n_slots), or is the slot of a sequence before it, has none.
 *   - h, the gradients and every sum are fp32.  Sums have a fixed order: equal
 *     calls give equal bits.  No workspace and no device-side wait.  Gates are fp32
 *     numbers; sigmoid(g), 1 - sigmoid(g) and exp(g) are each within 2^-21 of themselves
 *     (bf16 tensors: and 2^-23 |g|).
 *   - Not-a-number or infinite values of a token reach later tokens (backward:
 *     earlier ones too) of its own sequence and channel only. */
typedef enum { GATED_SCAN_SIGMOID = 0, GATED_SCAN_LOG = 1, GATED_SCAN_DECAY = 2 } gated_scan_gate;

/* Rows of D floats that gated_scan_forward keeps for gated_scan_backward: the
 * state before every 64th token of the tensors' rows.  B, N: the first two sizes
 * of the token tensors (packed: 1 and all tokens); 0 if they are invalid. */
long long gated_scan_checkpoint_rows(int B, int N);

/* The outputs of whole prompts.
 *   states      : NULL, or read (load_state = 1: a sequence starts from its slot's
 *                 state; 0: from zero) and written (the state after its last
 *                 token).  A sequence without a slot starts from zero and its
 *                 state is not kept; one without tokens leaves its slot as it is.
 *   checkpoints : NULL, or [gated_scan_checkpoint_rows][D] fp32, written, for
 *                 gated_scan_backward.
 *   B*N*D = 0 returns MHLA_OK without a launch. */
mhla_status gated_scan_forward(const void* x, const mhla_strides* x_strides, const void* g, const mhla_strides* g_strides,
                               void* y, const mhla_strides* y_strides, int B, int N, int D, const int* cu_seqlens,
                               float* states, const int* slots, int n_slots, int load_state, float* checkpoints,
                               mhla_dtype dt, int gate, void* stream);

/* The gradients of gated_scan_forward:
 *   G_t = dy_t + a_{t+1} G_{t+1}  (the last token: dy_t + dh_last),  da_t = G_t h_{t-1}
 *   SIGMOID: dx = (1 - a) G, dg = a (1 - a) G (h_{t-1} - x);  LOG: dx = G, dg = a da;
 *   DECAY: dx = G, dg = da;   dh0 = a_1 G_1
 *   checkpoints : those of the forward call with the same x, g and starts
 *   h0          : [B, D] fp32, the states that the forward call started from, NULL: zero
 *   dh_last     : [B, D] fp32, dL/d(last state), NULL: zero
 *   dh0         : [B, D] fp32 or NULL: written, a sequence without tokens: dh_last
 *   dx, dg      : written (not accumulated), of the full shape also where an input
 *                 is shared by stride 0.
 *   Rows of h0, dh_last and dh0 are the sequences in their order. */
mhla_status gated_scan_backward(const void* x, const mhla_strides* x_strides, const void* g,
                                const mhla_strides* g_strides, const void* dy, const mhla_strides* dy_strides,
                                const float* checkpoints, void* dx, const mhla_strides* dx_strides, void* dg,
                                const mhla_strides* dg_strides, int B, int N, int D, const int* cu_seqlens,
                                const float* h0, const float* dh_last, float* dh0, mhla_dtype dt, int gate, void* stream);

/* One token for each of B rows: updates the rows' states and writes out.  x, g,
 * out: [B, D]; of the strides b is used.  A row without a slot is left out:
 * neither its output nor a state is touched. */
mhla_status gated_scan_step(const void* x, const mhla_strides* x_strides, const void* g, const mhla_strides* g_strides,
                            float* states, const int* slots, int n_slots, void* out, const mhla_strides* out_strides,
                            int B, int D, mhla_dtype dt, int gate, void* stream);

/* ---------------------------------------------------- linear cross attention
 * Queries of one sequence that read another one, an encoder's tokens, of another
 * length ([LA] §三 with the keys and values of the encoder; its sums are the
 * constant-size state of [LA] §八):
 *   S = sum_j phi(k_j) v_j^T  (d x d, S[c][e]),  z = sum_j phi(k_j)
 *   y_t = phi(q_t) S / (phi(q_t) . z + eps)       (normalise = 0: y_t = phi(q_t) S)
 * The encoder is summed up once (linattn_cross_states) and read by any number of
 * calls, of prompts and of single queries (linattn_cross_read).
 * Conventions of the linattn_cross_* entries:
 *   - Queries [B, H, Nq, d], keys and values [B, Hk, Nk, d], H a multiple of Hk:
 *     query head h reads key head h / (H / Hk).  d = 16, 32, 64 or 128.  Strides as
 *     in the retention_* entries.
 *   - cu_seqlens as there (packed, one side or both), at most 2^31 - 128 tokens a
 *     side.  lens: NULL, or device int32 [B], the tokens of each encoder row of a
 *     padded batch (not with cu_seqlens of the keys), clamped to [0, Nk]: what lies
 *     behind them is not read, not-a-number among it.
 *   - An encoder without tokens gives S = 0, z = 0.  Where phi(q) . z + eps is 0
 *     (eps = 0 and nothing summed) or below 2^-120 the output is 0, and so are the
 *     gradients through it.
 *   - S: [n_slots, Hk, d, d] fp32, z: [n_slots, Hk, d] fp32.
 *   - mhla_options: feature and normalise (gamma = 1); NULL: ELU + 1 with the
 *     normaliser.  MHLA_PHI_IDENTITY goes without one (normalise = 0).
 *   - Not-a-number or infinite values reach what is computed from their own
 *     sequence only (a query's: its own outputs, and backward dk and dv of its sequence).
 *   - Every sum has a fixed order: equal calls give equal bits.
 *   - bf16 with d = 64 or 128 runs on the tensor cores, everything else on the FP32
 *     units.  There bf16 operands stand for 32-bit ones: phi(q) of a read (numerator
 *     and denominator alike) and phi(k) of dv are rounded once (2^-8 at most; ReLU
 *     and the identity not at all), S, dS and phi(q) / den are sums of two bf16
 *     numbers (2^-17), phi(k) of S one of three (2^-24); exponentials and 1 / den are
 *     within 2^-22.  All sums are fp32, of which the tensor cores cut each by at most
 *     2^-23 (S of 65,536 tokens is off by 8e-7 of its terms).  Everything else is fp32
 *     arithmetic. */

/* Workspace bytes of linattn_cross_states and linattn_cross_read (backward = 0) or
 * of linattn_cross_backward (backward = 1; enough for the others too) for B
 * sequences of tokens_q queries and tokens_k encoder tokens in all (dense: B Nq,
 * B Nk); 0 if the sizes are invalid or more than a call takes.  Valid for both
 * dtypes, dense and packed. */
size_t linattn_cross_workspace_bytes(int B, int H, int Hk, int tokens_q, int tokens_k, int d, int backward);

/* The sums of B encoder sequences.
 *   slots : NULL (sequence i writes slot i), or device int32 [B]: a sequence whose
 *           slot is outside [0, n_slots), or is the slot of a sequence before it, is
 *           not kept.
 *   S, z  : written (not accumulated), zeros for a sequence without tokens; slots
 *           of no sequence stay as they are. */
mhla_status linattn_cross_states(const void* k, const mhla_strides* k_strides, const void* v, const mhla_strides* v_strides,
                                 float* S, float* z, int B, int Hk, int N, int d, const int* cu_seqlens, const int* lens,
                                 const int* slots, int n_slots, mhla_dtype dt, const mhla_options* opt, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Queries of B sequences read their sums.  N = 1 without cu_seqlens is the step of
 * a decoder: every key head's S is read once for its query heads, and the workspace
 * may be NULL.
 *   slots : NULL (sequence i reads slot i), or device int32 [B]; several sequences
 *           may read one slot.  A sequence whose slot is outside [0, n_slots) is left
 *           out: its rows of y are not written. */
mhla_status linattn_cross_read(const void* q, const mhla_strides* q_strides, const float* S, const float* z, void* y,
                               const mhla_strides* y_strides, int B, int H, int Hk, int N, int d, const int* cu_seqlens,
                               const int* slots, int n_slots, mhla_dtype dt, const mhla_options* opt, float eps,
                               void* workspace, size_t workspace_bytes, void* stream);

/* The gradients of q, k and v through both, with den_t = phi(q_t) . z + eps:
 *   u_t = S dy_t,  dden_t = -(phi(q_t) . u_t) / den_t^2
 *   dq_t = phi'(q_t) * (u_t / den_t + dden_t z)
 *   dS = sum_t (phi(q_t) / den_t) dy_t^T,  dz = sum_t phi(q_t) dden_t   (over a key head's query heads)
 *   dk_j = phi'(k_j) * (dS v_j + dz),  dv_j = dS^T phi(k_j)
 * (normalise = 0: den = 1, dden = 0); phi' as in retention_backward.
 *   S, z       : those of linattn_cross_states for these k and v: slot i is sequence i
 *   dq, dk, dv : written (not accumulated); rows of a padded encoder batch behind
 *                lens become zeros, rows of no packed sequence stay as they are;
 *                without a query (H or Nq = 0) dk and dv are zeros. */
mhla_status linattn_cross_backward(const void* q, const mhla_strides* q_strides, const void* k, const mhla_strides* k_strides,
                                   const void* v, const mhla_strides* v_strides, const float* S, const float* z,
                                   const void* dy, const mhla_strides* dy_strides, void* dq, const mhla_strides* dq_strides,
                                   void* dk, const mhla_strides* dk_strides, void* dv, const mhla_strides* dv_strides, int B,
                                   int H, int Hk, int Nq, int Nk, int d, const int* cu_seqlens_q, const int* cu_seqlens_k,
                                   const int* lens, mhla_dtype dt, const mhla_options* opt, float eps, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Workspace bytes for rala_forward; 0 if the sizes are invalid. */
size_t rala_workspace_bytes(int B, int H, int N, int d, int cx);

/* Rank-augmented linear attention forward ([RALA] key designs 1 and 2).
 * For each (b, h):
 *   Q_g = (1/N) sum_t Q_t (raw queries);  l_j = Q_g . phi(K_j);
 *   alpha = softmax_j(l);  Bkv = sum_j alpha_j phi(K_j) V_j^T  (d x d);
 *   G = X_b W  ([N, d], shared by the heads of sample b);
 *   Y_t = G_t * (phi(Q_t) Bkv)   (elementwise product; no normaliser).
 *   q, k, v : [B, H, N, d] (dtype dt);  x : [B, N, cx] (dtype dt);
 *   w : [cx, d] (dtype dt);  y : [B, H, N, d] (dtype dt).
 *   cx must be a multiple of 16 and at most 256. */
mhla_status rala_forward(const void* q, const void* k, const void* v, const void* x,
                         const void* w, void* y, int B, int H, int N, int d, int cx,
                         mhla_dtype dt, void* workspace, size_t workspace_bytes, void* stream);

/* Kernel family rala_forward would use for these arguments (no launch):
 * the tensor-core kernels take bf16 with d = 32, cx = 64, H <= 2 and N a
 * multiple of 64 (at most 8192); everything else runs the SIMT kernels. */
mhla_path rala_forward_path(int B, int H, int N, int d, int cx, mhla_dtype dt);

/* Scratch held by mhla_forward_noalloc on every GPU that loads the library. */
#define MHLA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20) /* 32 MiB */

/* Non-causal MHLA forward that allocates nothing and takes no workspace.
 * The paper has no counterpart: this exists for callers that cannot obtain
 * device memory for a workspace (no allocator is available to them, or they
 * must not allocate after start-up, e.g. inside a host framework that owns a
 * fixed memory pool).  The result is that of mhla_forward(..., causal = 0,
 * ...) computed by the SIMT kernels; all arguments mean the same.
 *   Scratch: a file-scope device array of MHLA_NOALLOC_SCRATCH_BYTES per GPU,
 *   held until the process exits.  The CUDA runtime reserves it when it loads
 *   the library's device code on that GPU: with the default lazy module
 *   loading (CUDA_MODULE_LOADING=LAZY) that is the first call of this entry
 *   point on the device, which can therefore still fail for lack of device
 *   memory; make one warm-up call at start-up, while memory is known to be
 *   free (with CUDA_MODULE_LOADING=EAGER it happens at context creation).
 *   Sizes whose scratch need exceeds it return MHLA_ERR_UNSUPPORTED before
 *   any launch (the DiT-like B8 H6 N4096 d64 M16 case needs 25.2 MB).
 *   Set-up: the first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   outside any stream capture.
 *   Every call uses the same array; nothing in it needs to start at zero,
 *   but calls whose kernels overlap on the GPU (other streams, other host
 *   threads) race on it and must be serialised by the caller.
 *   Errors as for mhla_forward; no cudaMalloc/cudaFree is ever called. */
mhla_status mhla_forward_noalloc(const void* q, const void* k, const void* v, const float* mixing,
                                 void* y, float* den_out, int B, int H, int N, int d,
                                 int block_size, mhla_dtype dt, float eps, void* stream);

/* Kernel family mhla_forward would use for these arguments (no launch).
 * With causal = 1 the answer is for plain causal linear attention (mixing
 * NULL); mhla_forward_ex_path answers for causal MHLA with a mixing matrix,
 * which runs on the tensor cores for bf16, d = 64, chunk = 128 and
 * N / 128 <= 64 (the MHLA kernel's summary and mixing passes with the weights
 * below the diagonal, then the causal output kernel), else on the SIMT kernels. */
mhla_path mhla_forward_path(int B, int H, int N, int d, int block_size, int causal,
                            mhla_dtype dt);

/* Synchronises `stream`, then returns MHLA_ERR_TIMEOUT if a device-side wait
 * in a call that used this workspace gave up (and clears the flag), MHLA_OK
 * otherwise, or MHLA_ERR_CUDA if the synchronisation or read failed. */
mhla_status mhla_query_status(void* workspace, void* stream);

/* Static description of a status code (never NULL). */
const char* mhla_status_string(mhla_status s);

/* Number of kernels this library has launched (or captured into a graph) in
 * this process since it was loaded; a diagnostic counter. */
unsigned long long mhla_launch_count(void);

/* Diagnostic: sets the limit, in nanoseconds, of the bounded device-side
 * waits of the non-causal bf16 tensor-core kernels (every wait of the stream
 * path; the waits for the mixed summaries of the three-pass path), of the
 * tensor-core passes of mhla_backward and of those of retention_forward,
 * retention_backward and the linattn_cross_* entries (every wait) for calls launched
 * after it (process wide; 0 restores the default of 0.5 s).  With a limit too short for the
 * work in flight a call gives up: its output is incomplete, the kernel lets
 * its copies and MMAs in flight finish, leaves the workspace counters at
 * zero, and mhla_query_status() then reports MHLA_ERR_TIMEOUT.  The pages
 * describe no such control; it exists to exercise that failure path. */
void mhla_debug_set_wait_limit_ns(unsigned long long ns);

#ifdef __cplusplus
}
#endif

#endif /* MHLA_GB300_H */
