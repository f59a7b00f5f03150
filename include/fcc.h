/*
 * fcc.h -- libfcc: GEMMs fused with the collective that consumes their output,
 * for one GB300 (sm_103a), across R tensor-parallel ranks whose buffers are
 * disjoint allocations in the one GPU's HBM.
 *
 * "Communication" between ranks is a kernel storing into (or loading from)
 * another rank's buffer.  The operators are the fused kernels named in
 * "GPU-vezerelt kommunikacioval gyorsitjak az AI-betanitast a kutatok"
 * (mKernel article, section on the five fused kernels: AllGather + GEMM,
 * GEMM + AllReduce, MoE Dispatch + GEMM, GEMM + ReduceScatter) and in
 * "Optimizing Distributed ML Communication with Fused Computation-Collective
 * Operations" (SC24, abstract: GEMV + AllReduce, GEMM + All-to-All, with
 * workgroups that ship their results as soon as they finish).
 *
 * Conventions for every call
 *  - Matrices are row-major and contiguous.  A_r is [M,K], B_r is [K,N]; the
 *    product is A_r @ B_r as in torch.  Shard j of an M-row result is the
 *    contiguous row block [j*M/R, (j+1)*M/R).
 *  - Pointer arrays (A, B, out, ...) are HOST arrays of DEVICE pointers, one
 *    per rank; they are read during the call and not retained.  Device
 *    pointers must be 16-byte aligned.  The caller owns every buffer.
 *  - Inputs are bf16; accumulation is f32; f32 results are stored as f32 and
 *    bf16 results are rounded to nearest even.
 *  - Calls are asynchronous on `stream` and return after enqueueing.
 *    Argument errors are reported synchronously and nothing is launched.
 *    Errors found on the device (a wait that timed out, a receive buffer too
 *    small) are recorded in a per-device status word that fcc_stream_status()
 *    reads and clears.
 *  - opts may be NULL for the defaults (fused, deterministic, library-owned
 *    workspace, 1 s wait limit).
 *  - Workspace: calls that need scratch memory take it from opts->workspace
 *    (size from fcc_workspace_size / fcc_moe_workspace_size); with no
 *    workspace given, the library keeps an internal per-device pool that it
 *    grows with cudaMalloc on first use (and when a larger call comes), which
 *    synchronises the device at that moment.
 *  - Not thread-safe for concurrent calls on the same stream; calls on
 *    different streams share the internal pool and must not overlap unless
 *    each passes its own workspace.
 *  - Environment defaults, read once when the library first needs one:
 *    FCC_ALGO=fused|unfused|interdecom|ce replaces FCC_ALGO_AUTO (also in
 *    fcc_choose_algo) for the operators with several forms (a form an
 *    operator lacks gives FCC_ERR_UNSUPPORTED; the attentions, the cache,
 *    the MoE combine and the losses have one form and ignore it); FCC_DETERMINISTIC=0|1 is the
 *    summation mode of calls with opts == NULL; FCC_CHUNKS=n (1..64) the
 *    InterDecom chunk count where opts->chunks is 0; FCC_TIMEOUT_MS=n the
 *    device wait limit where opts->timeout_ns is 0.  Unset or unparsable
 *    values leave the built-in defaults.
 */
#ifndef FCC_H_
#define FCC_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without pulling in the CUDA headers. */
typedef struct CUstream_st *fcc_stream_t;

#define FCC_MAX_RANKS 8
#define FCC_MAX_EXPERTS 64
#define FCC_MAX_TABLES 256  /* embedding tables per call */
#define FCC_MAX_TEACHER 256 /* teacher entries per token (distillation) */

/* FCC_E4M3 (one sign, four exponent and three mantissa bits, no infinities) is a
 * type of the paged cache's contents only. */
typedef enum { FCC_BF16 = 0, FCC_F16 = 1, FCC_F32 = 2, FCC_E4M3 = 3 } fcc_dtype;

typedef enum {
  FCC_OK = 0,
  FCC_ERR_INVALID = 1,     /* bad argument: null or misaligned pointer, bad size */
  FCC_ERR_UNSUPPORTED = 2, /* valid but not implemented (dtype, algorithm) */
  FCC_ERR_CUDA = 3,        /* a CUDA runtime call failed */
  FCC_ERR_CAPACITY = 4,    /* a receive buffer is too small (MoE cap) */
  FCC_ERR_TIMEOUT = 5,     /* a device-side wait ran out of time */
  FCC_ERR_WORKSPACE = 6    /* caller workspace too small */
} fcc_status;

typedef enum {
  FCC_ALGO_AUTO = 0,       /* chosen per operator and shape (fcc_choose_algo) */
  FCC_ALGO_FUSED = 1,      /* fused GEMM + collective in one persistent kernel */
  FCC_ALGO_UNFUSED = 2,    /* per-rank GEMM to f32 partials, then a reduce/copy kernel */
  FCC_ALGO_INTERDECOM = 3, /* chunks: the GEMM of one chunk overlaps the data movement of
                              another (row chunks; MoE: expert ranges) */
  FCC_ALGO_CE = 4          /* the data between ranks moved by the copy engines
                              (cudaMemcpyAsync), no SMs */
} fcc_algo;

typedef struct {
  fcc_algo algo;
  /* Fused GEMM+ReduceScatter/AllReduce: 1 = ordered tile-owner accumulation
   * (each output tile sums ranks 0..R-1 in order in one accumulator; bitwise
   * repeatable), 0 = push mode (each rank's tile is added into the owner's f32
   * shard with red.global.add.v4.f32; order-free). */
  int deterministic;
  int chunks;              /* InterDecom chunk count; 0 = the cost model */
  int max_ctas;            /* persistent grid size cap; 0 = one CTA per SM */
  int64_t timeout_ns;      /* device wait limit; 0 = 1 s */
  void *workspace;         /* device scratch, or NULL for the internal pool */
  size_t workspace_bytes;
  /* Tensor-core tile shape of the GEMMs: 0 = automatic (a CTA pair when the
   * rows exceed 128 and the 128 x 256 tiles outnumber the CTAs, else 1; the
   * MoE expert GEMM: a CTA pair), 1 = one CTA per 128 x 256 tile, 2 = a CTA pair
   * (cluster of 2, tcgen05 cta_group::2) per 256 x 256 tile.  Any other value
   * is FCC_ERR_INVALID.  Every TMA load lands in the issuing CTA's own shared
   * memory (no multicast loads), so the library may run in processes that
   * drive several GPUs. */
  int cta_pair;
  /* Phase timing, for profiling: NULL (the default), or a device array of
   * 4 uint64 per CTA of the grid (at most the SM count) that the tensor-core
   * GEMM kernels (RS, AR, AG, their unfused GEMMs and the MoE expert GEMM)
   * fill from %globaltimer, for the call's last GEMM launch: [0] ns from the
   * CTA's start to its end, [1] ns its epilogue warps spent on tiles (from an
   * accumulator becoming ready to its last store issued), [2] ns its MMA
   * warp waited for an accumulator the epilogue had not yet handed back (the
   * part of the epilogue not hidden behind the next tile's MMAs; 0 on the
   * second CTA of a pair, which issues no MMAs), [3] tiles it stored. */
  uint64_t *phase_ns;
} fcc_opts;

/* Operator identifiers for fcc_workspace_size. */
typedef enum {
  FCC_OP_GEMM_RS = 0,
  FCC_OP_GEMM_AR = 1,
  FCC_OP_GEMV_AR = 2,
  FCC_OP_AG_GEMM = 3,
  FCC_OP_EMBEDDING_A2A = 4
} fcc_op;

/*
 * GEMM + ReduceScatter (mKernel article, fused kernel list; SC24 abstract).
 *   out_shard[j][i][n] = sum_{r<R} sum_{k<K} A[r][j*M/R + i][k] * B[r][k][n]
 * R in 1..8; A[r]: [M,K] bf16; B[r]: [K,N] bf16; out_shard[j]: [M/R, N] of
 * dtype `out` (FCC_BF16 or FCC_F32).  M % R == 0, K % 8 == 0, N % 8 == 0.
 * Deterministic mode: each output tile sums its k terms (rank after rank)
 * in a fixed order, so results repeat bit for bit and equal fcc_gemm_ar's
 * rows.  When a launch of several rounds of tiles ends with a round of at
 * most half the tiles it could hold, each of those tiles runs as two halves
 * of its k range on two CTA pairs, whose f32 partial sums are then added
 * (still a fixed order); the partials take workspace (fcc_workspace_size).
 * A caller workspace too small for them makes those tiles run as column
 * halves instead, with the tile's whole k range (no error).
 */
fcc_status fcc_gemm_rs(int R, const void *const *A, const void *const *B,
                       void *const *out_shard, int64_t M, int64_t N, int64_t K,
                       fcc_dtype in, fcc_dtype out, const fcc_opts *opts,
                       fcc_stream_t stream);

/*
 * GEMM + AllReduce (mKernel article, fused kernel list).
 *   out[r'] = sum_{r<R} A[r] @ B[r]  for every rank r' (M x N each).
 * Shapes as fcc_gemm_rs (no divisibility of M needed); the same tiling,
 * summation order and workspace use as fcc_gemm_rs.
 */
fcc_status fcc_gemm_ar(int R, const void *const *A, const void *const *B, void *const *out,
                       int64_t M, int64_t N, int64_t K, fcc_dtype in, fcc_dtype out_dtype,
                       const fcc_opts *opts, fcc_stream_t stream);

/*
 * GEMV + AllReduce, the decode shape (SC24 abstract, Transformer operator).
 *   out[r'] = sum_{r<R} A[r] @ B[r] for every rank r'; A[r]: [M,K] with
 *   1 <= M <= 16 tokens; B[r]: [K,N]; out[r']: [M,N] f32 (or bf16).
 * The cross-rank sum is deterministic (fixed order).  Uses workspace.
 */
fcc_status fcc_gemv_ar(int R, const void *const *A, const void *const *B, void *const *out,
                       int64_t M, int64_t N, int64_t K, fcc_dtype in, fcc_dtype out_dtype,
                       const fcc_opts *opts, fcc_stream_t stream);

/*
 * GEMV + AllReduce that allocates nothing.  The pages have no counterpart:
 * this is an addition for callers that cannot call cudaMalloc -- a process
 * whose device memory is already reserved by its own allocator, or a
 * latency-critical path that cannot take cudaMalloc/cudaFree's implicit
 * device synchronisation.  Same arguments and results as fcc_gemv_ar; the
 * caller passes inputs and outputs, and the kernel's scratch (partial sums
 * and arrival tickets) is a 4 MiB static device array inside the library,
 * held on every GPU that loads the library until the process exits.
 *  - Limit: each CTA keeps an M x 512 f32 partial (M x 2 KiB) per group of
 *    512 columns, in the array's 4 MiB less 4 KiB of tickets, so
 *    ceil(N/512) * M <= 2046 (N <= 130,560 for 8 tokens,
 *    65,024 for 16); within that the call uses as many CTAs per column group
 *    as fit in the array (possibly fewer than fcc_gemv_ar uses, which changes
 *    only the f32 summation order).  Beyond it the call returns
 *    FCC_ERR_WORKSPACE and launches nothing.  opts->workspace is ignored;
 *    algo must be AUTO or FUSED (UNFUSED, INTERDECOM and CE give
 *    FCC_ERR_UNSUPPORTED, values outside the enum FCC_ERR_INVALID, as in
 *    fcc_gemv_ar).
 *  - The first call on a device looks up the array's device address and the
 *    SM count (cudaGetSymbolAddress, cudaDeviceGetAttribute) with that device
 *    current; make that first call before any stream capture.
 *  - Every call uses the same array and clears its tickets (cudaMemsetAsync)
 *    first.  Calls that overlap on the GPU (other streams, other threads)
 *    race on the array: serialise them.
 */
fcc_status fcc_gemv_ar_static(int R, const void *const *A, const void *const *B,
                              void *const *out, int64_t M, int64_t N, int64_t K, fcc_dtype in,
                              fcc_dtype out_dtype, const fcc_opts *opts, fcc_stream_t stream);

/*
 * AllGather + GEMM (mKernel article, fused kernel list).
 *   X = [X_shard[0]; ...; X_shard[R-1]]   (each [M/R, K], X is [M, K])
 *   out[r] = X @ B[r]                      ([M, N] per rank, dtype `out_dtype`)
 *   gathered[r] (nullable array, or NULL entries): receives X ([M, K] bf16).
 * opts->algo: FUSED (AUTO) = one kernel whose tiles read their A rows from
 * the owning shard; UNFUSED = a gather kernel into gathered[0] (or
 * workspace), then the per-rank GEMMs; INTERDECOM = the same in row chunks
 * of 256-row tiles, each chunk's gather on a side stream ahead of that
 * chunk's GEMMs (chunk count opts->chunks, else the fcc_interdecom_chunks
 * model with G = the GEMMs, X = the gather); CE = the gather by one
 * cudaMemcpyAsync per shard.  The non-fused forms use workspace of M*K*2
 * bytes when gathered[0] is NULL (fcc_workspace_size).
 */
fcc_status fcc_ag_gemm(int R, const void *const *X_shard, const void *const *B,
                       void *const *out, void *const *gathered, int64_t M, int64_t N,
                       int64_t K, fcc_dtype in, fcc_dtype out_dtype, const fcc_opts *opts,
                       fcc_stream_t stream);

/*
 * MoE Dispatch + GEMM (mKernel article, fused kernel list; SC24 abstract,
 * GEMM + All-to-All for MoE).  R source ranks with T tokens each; E experts,
 * E/R per rank, expert e on rank e/(E/R).
 *   route:    topk_idx[s][t][0..topk) = experts with the largest logits
 *             (ties: lower index first); topk_gate = their softmax probability
 *             over all E experts (not renormalised, not applied below).
 *   dispatch: assignments (s, t, slot) sorted stably by expert; rank d
 *             receives its experts' rows in (expert, s, t, slot) order:
 *             recv_src[d][row] = s*T + t, recv_x[d][row] = X[s][t],
 *             expert_counts[e], send_counts[s*R + d].
 *   GEMM:     recv_y[d][row] = X[s][t] @ W[e]  ([F] per row, dtype out_dtype).
 * X[s]: [T,H] bf16; logits[s]: [T,E] f32, finite; W[e]: [H,F] bf16 (E
 * pointers); recv_x: NULL, or per rank [cap,H] bf16 to receive the
 * dispatched rows.  By default (AUTO) the expert GEMM kernel moves the rows
 * itself, into recv_x or into workspace when it is NULL, one (expert,
 * m tile) unit after another, and its tensor cores read each unit as soon as
 * it is moved.  FCC_ALGO_UNFUSED (the unfused baseline) moves all rows with a
 * separate copy kernel before the GEMM.  FCC_ALGO_INTERDECOM (the chunked
 * baseline) splits the experts into c contiguous ranges (c = opts->chunks,
 * else the fcc_interdecom_chunks model with G = the expert GEMMs, X = the
 * row copy; at most E); each range's rows are copied on a side stream ahead
 * of that range's grouped GEMM, so copy i+1 overlaps GEMM i.  FCC_ALGO_CE
 * (the copy-engine baseline) packs each source rank's kept rows into a send
 * buffer in (expert, token, slot) order (a copy within the rank), reads the
 * (source, expert) run table back to the host (so this form synchronises
 * `stream` before it returns), and moves each run, contiguous on both sides,
 * with one cudaMemcpyAsync on the copy engines, then runs the GEMM.  With
 * opts->algo == FCC_ALGO_FUSED and the sources one [R*T,H] array (X[s] =
 * X[0] + s*T*H elements), the GEMM instead reads each row straight from its
 * source token (TMA gather) and a non-NULL recv_x is filled beside it (slower
 * on sm_103a: the gather is bound by its TMA request rate); FUSED with other
 * sources moves the rows as the default does.  recv_y[d]: [cap,F];
 * recv_src[d]: [cap] int32; topk_idx[s]: [T,topk] int32; topk_gate[s]:
 * [T,topk] f32; expert_counts: [E] int32 device; send_counts: [R*R] int32
 * device.  Rows of a receive buffer past the received count are left
 * untouched.  topk in {1, 2}; R <= E <= 64, E % R == 0; H % 8 == 0;
 * F % 8 == 0.  A rank receiving more than cap rows sets FCC_ERR_CAPACITY in
 * the status word; its rows past cap are dropped (not copied, not multiplied).
 * Index outputs are bit-exact and repeatable (no atomics decide a position).
 * Uses workspace (fcc_moe_workspace_size; with FCC_ALGO_CE in opts it
 * includes the R*T*topk*H*2 bytes of send buffers).
 */
fcc_status fcc_moe_dispatch_gemm(int R, const void *const *X, const float *const *logits,
                                 const void *const *W, int64_t T, int64_t H, int64_t F, int E,
                                 int topk, void *const *recv_x, void *const *recv_y,
                                 int64_t cap, int32_t *const *topk_idx,
                                 float *const *topk_gate, int32_t *expert_counts,
                                 int32_t *send_counts, int32_t *const *recv_src, fcc_dtype in,
                                 fcc_dtype out_dtype, const fcc_opts *opts,
                                 fcc_stream_t stream);

/*
 * MoE combine: the return all-to-all and the gate-weighted top-k sum (SC24
 * abstract, GEMM + All-to-All for MoE: the direction back to the token
 * owners).  For every source rank s and token t:
 *   y[s][t][f] = sum over slots j < topk of topk_gate[s][t][j] * recv_y[d][i][f]
 * where row i of receiving rank d is the row that assignment (s, t, j) was
 * given by the dispatch that produced recv_y (d = topk_idx[s][t][j] / (E/R)),
 * the slots added in order in f32 (so the result is repeatable).  A slot
 * whose row was dropped for capacity adds nothing.  The receive rows are
 * found from recv_src and expert_counts as fcc_moe_dispatch_gemm wrote them:
 * rank d holds its E/R experts' rows in expert order, min(cap, their total)
 * rows in all.
 * recv_y[d]: [cap,F] (in: bf16 or f32); topk_idx[s]: [T,topk] int32;
 * topk_gate[s]: [T,topk] f32; recv_src[d]: [cap] int32; expert_counts: [E]
 * int32 (device); y[s]: [T,F] (out_dtype: bf16 or f32).  topk in {1, 2};
 * R <= E <= 64, E % R == 0; F % 8 == 0.  Uses workspace
 * (fcc_moe_combine_workspace_size).
 */
fcc_status fcc_moe_combine(int R, const void *const *recv_y, int64_t cap, int64_t T, int64_t F,
                           int E, int topk, const int32_t *const *topk_idx,
                           const float *const *topk_gate, const int32_t *const *recv_src,
                           const int32_t *expert_counts, void *const *y, fcc_dtype in,
                           fcc_dtype out_dtype, const fcc_opts *opts, fcc_stream_t stream);

/*
 * Embedding + All-to-All (SC24 abstract: the embedding + All-to-All operator
 * for DLRM).  ntables embedding tables [V, D] (table t owned by rank
 * t / (ntables / R)); R ranks with Bl samples each (global sample g lives on
 * rank g / Bl).  Bag (t, g) is the index list
 * indices[t][offsets[t][g] .. offsets[t][g + 1]) into table t; its pooled
 * vector is the sum of those rows (f32, then stored in out_dtype; an empty
 * bag gives zeros).  The all-to-all delivers it to the sample's rank:
 *   out[g / Bl][g % Bl][t][:] = pooled vector of bag (t, g)
 * tables[t]: [V, D] bf16; offsets[t]: [R*Bl + 1] int32, non-decreasing;
 * indices[t]: [offsets[t][R*Bl]] int32 in [0, V); out[r]: [Bl, ntables, D]
 * (bf16 or f32).  R <= 8, ntables % R == 0, ntables <= FCC_MAX_TABLES,
 * D % 8 == 0.  opts->algo: FUSED (AUTO) = one kernel pools each bag and
 * stores it straight into its sample's rank buffer; UNFUSED = each table's
 * pooled vectors into a [ntables, R*Bl, D] workspace, then a kernel moves
 * them to the sample ranks; CE = the same workspace moved by copy-engine 2-D
 * copies (one per table and rank).  A negative offset step or an index
 * outside [0, V) is not read: the bag skips it and FCC_ERR_INVALID is
 * recorded in the status word.  Within a call the result is repeatable (a
 * fixed summation order).  Uses workspace for UNFUSED / CE
 * (fcc_embedding_workspace_size).
 */
fcc_status fcc_embedding_a2a(int R, int ntables, const void *const *tables, int64_t V,
                             int64_t D, int64_t Bl, const int32_t *const *offsets,
                             const int32_t *const *indices, void *const *out, fcc_dtype in,
                             fcc_dtype out_dtype, const fcc_opts *opts, fcc_stream_t stream);
size_t fcc_embedding_workspace_size(int R, int ntables, int64_t D, int64_t Bl,
                                    fcc_dtype out_dtype, const fcc_opts *opts);

/*
 * Ring attention (the mKernel article's fused kernel list: Ring Attention).
 * The sequence is split over R ranks, S positions each (rank r's row t is
 * global position r*S + t); every rank's queries attend to the keys and
 * values of all shards, which the ring brings round (here: each CTA reads
 * the blocks of every shard in ring order, its own shard first):
 *   O_r[t][h] = sum_j softmax_j(Q_r[t][h] . K[j][h] / sqrt(d)) V[j][h]
 * over all global positions j (causal != 0: only j <= r*S + t).
 * Q[r], K[r], V[r]: [S, H, d] bf16; O[r]: [S, H, d] (bf16 or f32).  d = 128
 * (others: FCC_ERR_UNSUPPORTED).  Scores, softmax and sums in f32; the
 * probabilities (relative to a running row maximum) enter the P V product as
 * bf16.  Repeatable (a fixed order).  No workspace.
 */
fcc_status fcc_ring_attention(int R, const void *const *Q, const void *const *K,
                              const void *const *V, void *const *O, int64_t S, int H, int64_t d,
                              int causal, fcc_dtype in, fcc_dtype out_dtype,
                              const fcc_opts *opts, fcc_stream_t stream);

/*
 * Linear cross entropy: the loss of a vocabulary-parallel head, forward.  The
 * head's rows are split over the ranks (rank r holds rows [r*V/R, (r+1)*V/R)),
 * every rank holds a copy of the tokens' hidden states, and the softmax
 * statistics are all-reduced:
 *   x_v = X[r][t] . W[r][v - r*V/R]   (f32)
 *   l_v = x_v, or softcap * tanh(x_v / softcap) when softcap > 0 (the cap's own
 *         error is below 2^-20 of l_v, whatever softcap)
 *   lse[t]  = log sum_v exp(l_v)
 *   loss[t] = lse - (1 - smoothing) l_y - smoothing / V * sum_v l_v
 *             + z_weight * lse^2,                     y = labels[t]
 * written to every rank's loss[r], lse[r].  A label equal to ignore_index
 * gives loss 0 (lse is still its row's).  Any other label outside [0, V) does
 * the same and records FCC_ERR_INVALID in the status word.  The logits are
 * never stored.
 * X[r]: [T,D] bf16 (the same values in every rank; entries may be one
 * buffer); W[r]: [V/R,D] bf16; labels: [T] int32 (device); loss[r], lse[r]:
 * [T] f32.  T, V >= 1 (any, odd ones too), V % R == 0, D % 8 == 0,
 * 0 <= smoothing < 1, z_weight >= 0, softcap 0 or from 2^-126 to 2^126.
 * Logits that are not finite give a loss that is not.  The label's logit is
 * summed in f32 by itself; the others come from the tensor cores, whose sums
 * lose a little of themselves: they are scaled by what sums of random products
 * lose (1.6e-8 for every 16 of D, up to D = 131072), and are off by as much where
 * nothing was lost, by up to 8e-8 for every 16 of D where all of a logit's
 * products are positive and 1.5e-7 where the first outweighs the rest (measured
 * on a GB300).  Repeatable (a fixed order of summation).  Uses workspace
 * (fcc_linear_loss_workspace_size with topk 0, grad 0).  opts->algo: AUTO or
 * FUSED; the environment's FCC_ALGO and FCC_CHUNKS do not apply.
 */
fcc_status fcc_linear_xent(int R, const void *const *X, const void *const *W,
                           const int32_t *labels, int64_t T, int64_t V, int64_t D,
                           float *const *loss, float *const *lse, int32_t ignore_index,
                           float smoothing, float z_weight, float softcap, fcc_dtype in,
                           const fcc_opts *opts, fcc_stream_t stream);

/*
 * Its gradient, from the forward pass's lse and the losses' upstream
 * gradients dloss ([T] f32, device; a mean over n tokens passes 1/n):
 *   dl_v = dloss ((1 + 2 z_weight lse) exp(l_v - lse) - smoothing / V
 *                 - (1 - smoothing) [v = y])
 *   dx_v = dl_v, times 1 - (l_v / softcap)^2 when softcap > 0
 *   dX[r]  = sum over all ranks s of dx_s @ W[s]   ([T,D] bf16, to every rank)
 *   dW[r]  = dx_r^T @ X[r]                         ([V/R,D] bf16)
 * Ignored rows have no gradient, whatever their dloss holds; their rows of X
 * must be finite all the same, for dx's zeros multiply them in dW.  dX or dW may
 * be NULL (not wanted).  The logits are computed again, a piece of every rank's
 * vocabulary at a time (opts->chunks pieces; 0 = as few as hold 512 MiB of dx),
 * scaled as in the forward pass and the label's summed by itself; dx is rounded
 * to bf16 (for up to 64 tokens, to a sum of two bf16 numbers); products
 * accumulate in f32.  out_dtype is FCC_BF16: gradients that are added up over
 * several calls are rounded in each.  Uses workspace
 * (fcc_linear_loss_workspace_size with topk 0, grad 1).
 */
fcc_status fcc_linear_xent_grad(int R, const void *const *X, const void *const *W,
                                const int32_t *labels, const float *const *lse,
                                const float *dloss, int64_t T, int64_t V, int64_t D,
                                void *const *dX, void *const *dW, int32_t ignore_index,
                                float smoothing, float z_weight, float softcap, fcc_dtype in,
                                fcc_dtype out_dtype, const fcc_opts *opts, fcc_stream_t stream);

/*
 * Distillation from a teacher's top logits on the same head:
 *   q       = softmax of teacher_logits[t][k] / temperature over the row's entries
 *   lse[t]  = log sum_v exp(l_v / temperature)       (l as above)
 *   loss[t] = temperature^2 (sum_k q_k (log q_k - l_{i_k} / temperature) + lse)
 * with i_k = teacher_idx[t][k]; an index < 0, or a logit of -inf, is no
 * entry, and a row without entries gives loss 0.  An index >= V is no entry
 * either and records FCC_ERR_INVALID.  An index given twice counts twice.
 * The gradient is dl_v = dloss temperature (exp(l_v / temperature - lse)
 * - sum_k q_k [v = i_k]).  teacher_idx, teacher_logits: [T,topk] int32 / f32
 * (device), 1 <= topk <= FCC_MAX_TEACHER, in any order; temperature from 2^-63
 * to 2^63.  All else as in fcc_linear_xent and fcc_linear_xent_grad, with the
 * entries of probability 1/8 or more in the label's place.
 */
fcc_status fcc_linear_distill(int R, const void *const *X, const void *const *W,
                              const int32_t *teacher_idx, const float *teacher_logits, int64_t T,
                              int64_t V, int64_t D, int topk, float *const *loss,
                              float *const *lse, float temperature, float softcap, fcc_dtype in,
                              const fcc_opts *opts, fcc_stream_t stream);
fcc_status fcc_linear_distill_grad(int R, const void *const *X, const void *const *W,
                                   const int32_t *teacher_idx, const float *teacher_logits,
                                   const float *const *lse, const float *dloss, int64_t T,
                                   int64_t V, int64_t D, int topk, void *const *dX,
                                   void *const *dW, float temperature, float softcap,
                                   fcc_dtype in, fcc_dtype out_dtype, const fcc_opts *opts,
                                   fcc_stream_t stream);

/* Scratch bytes of the four calls above (topk 0: cross entropy). */
size_t fcc_linear_loss_workspace_size(int R, int64_t T, int64_t V, int64_t D, int topk, int grad,
                                      const fcc_opts *opts);

/*
 * A paged cache of keys and values, and the sequences of one step that use it.
 * Heads are split over the ranks: rank r holds H key/value heads of every
 * sequence in its own two pools.  The sequences, their lengths and their page
 * tables are the same for every rank.  Position j of sequence b lies in row
 * j % page_size of page table[b][j / page_size].
 *
 * Pools of dtype FCC_BF16 hold the values themselves.  Pools of dtype FCC_E4M3
 * hold x / 2^k rounded to e4m3 (nearest, ties to even), with one k for each
 * position and head, kept as the byte k + 127 in K_exp / V_exp: the least power
 * of two (k >= -64) for which the row's largest finite |x| is at most 448 * 2^k.
 * A power of two costs a floating-point code no digits and makes reading back
 * exact.  A value that is not finite becomes NaN.  A row of zeros has k = -64;
 * values below about 2^-73 become zero.
 */
typedef struct {
  void *const *K;        /* R pools [pages, H, page_size, d] of `dtype` */
  void *const *V;
  uint8_t *const *K_exp; /* FCC_E4M3: R arrays [pages, H, page_size]; else ignored */
  uint8_t *const *V_exp;
  int64_t pages;         /* 1 .. 2^31 - 1 */
  int page_size;         /* a power of two, 1 .. 65536 */
  int H;                 /* key/value heads of one rank, 1 .. 1024 */
  int d;                 /* 64 or 128 (others: FCC_ERR_UNSUPPORTED) */
  fcc_dtype dtype;       /* FCC_BF16 or FCC_E4M3 */
} fcc_cache;

/*
 * Rows start[b] .. start[b+1] - 1 of the step's token arrays belong to sequence
 * b and are its newest positions: row start[b] + i is position
 * len[b] - n + i, n = start[b+1] - start[b].  Rows behind start[B] belong to
 * nobody and are left alone.  The three arrays lie on the device (4-byte
 * aligned) and are read by the kernels only, so a captured call can be replayed
 * with other contents.  What they say is checked there: a step with
 * start[b+1] < start[b], start[b] < 0 or start[b+1] > T, with len[b] < n, with
 * more positions than max_pages pages hold or with a page outside [0, pages)
 * among those it needs records FCC_ERR_INVALID in the status word, and nothing
 * is read or written there (fcc_paged_attention says what its results are then).
 * fcc_cache_append and fcc_cache_gather find a row's sequence by the starts: where
 * those are not in order, rows of other sequences may be left out too.
 */
typedef struct {
  const int32_t *start;  /* [B + 1] */
  const int32_t *len;    /* [B]: positions of each sequence, this step's included */
  const int32_t *table;  /* [B, max_pages]; entries past a sequence's last page are not read */
  int64_t max_pages;     /* 1 .. 2^31 - 1 */
  int64_t T;             /* rows of the step's token arrays, 1 .. 2^31 - 1 */
  int B;                 /* sequences, 1 .. 65536 */
} fcc_batch;

/*
 * Writes the keys and values of a step's rows into the cache.  K[r], V[r]:
 * [T, H, d] bf16, rows ld elements apart (0: H * d; ld % 8 == 0), so that they
 * may be parts of one fused projection's output.  Two rows of a call must not
 * have the same place in the pools (sequences that share a page write to
 * different rows of it, or to copies).  No workspace.
 */
fcc_status fcc_cache_append(int R, const void *const *K, const void *const *V, int64_t ld,
                            const fcc_cache *cache, const fcc_batch *batch, fcc_dtype in,
                            const fcc_opts *opts, fcc_stream_t stream);

/*
 * The reverse: reads the rows' positions back into K[r], V[r] ([T, H, d] bf16,
 * rows ld elements apart), as code * 2^k where the cache is e4m3 (exact down to
 * bf16's subnormal numbers, rounded there).  With start[b+1] - start[b] = len[b] whole
 * sequences come back.  Rows of a sequence that is not valid are left alone, and so
 * are rows whose page is not.  No workspace.
 */
fcc_status fcc_cache_gather(int R, const fcc_cache *cache, const fcc_batch *batch, void *const *K,
                            void *const *V, int64_t ld, fcc_dtype out, const fcc_opts *opts,
                            fcc_stream_t stream);

/*
 * Attention of a step's rows over the cache, whose pages already hold the
 * rows' own keys and values (fcc_cache_append first).  Every rank has Hq query
 * heads; head h reads key/value head h / (Hq / H).  For the row at position p:
 *   s_j = scale * Q[r][t][h] . K[j],  j <= p, and j > p - window if window > 0
 *   O[r][t][h] = sum_j softmax_j(s) V[j],   lse[r][t][h] = log sum_j exp(s_j)
 * Positions that a row does not see do not touch it, whatever their keys and
 * values hold.  Q[r], O[r]: [T, Hq, d] bf16, rows ldq / ldo elements apart (0:
 * Hq * d; multiples of 8): O[r] is the A of fcc_gemv_ar or fcc_gemm_ar for
 * the output projection.  lse: NULL, or R arrays [T, Hq] f32.  scale: 0 means
 * 1 / sqrt(d), otherwise positive and, times log2(e), finite.  Hq % H == 0, Hq <= 1024.
 * Scores, maxima, sums and O's accumulators are f32; the probabilities enter the
 * product with V in 16 bits (bf16; f16 where the cache is e4m3), relative to a running
 * maximum (f16: weights below 2^-33 of a row's largest may vanish, each 2^-33 of the
 * largest value that the row sees at most).  Repeatable (a fixed order of summation).
 * Powers of an e4m3 cache are read as append writes them (bytes 63 to 247); those of the
 * values that a row sees are at most 2^120 apart (beyond, the weights of the smaller ones
 * may be missing from the sum).  O[r] must not overlap Q[r].
 * A sequence with len[b] < n has no visible positions; a row with none has
 * O = 0, lse = -inf.  Where a needed page is not valid, or lies past
 * max_pages, its positions are left out.  Both record FCC_ERR_INVALID.
 * One token or many: a step with up to 16 query rows (e4m3: 32) to a sequence and
 * key/value head on average (T * Hq / H <= 16 B) is read as few rows over many
 * positions, any other one in tiles of 128 rows.  Both give every step's results, but
 * the average is all that decides: 84 sequences of one row and a chunk of 256, 4 heads
 * to a group, take 1030 us (e4m3 918) where the two parts take 440 (347).  Such a step is
 * two calls: sequences of one row first in the arrays, a call with their B and T, then
 * one with start, len and table advanced to the others.  T * Hq / H is below 2^31 - 256.
 * What tiles cannot give (sums that are not finite: infinities or NaN in keys or values,
 * scores that jump by more than 88; e4m3 powers more than 2^22 apart within 32
 * positions) is computed again behind them, row by row of those that met it: the same
 * results, 10 (bf16) to 40 times as slow.
 * Uses workspace (fcc_paged_attention_workspace_size).  A call made while its
 * stream is being captured must bring its own (FCC_ERR_WORKSPACE): the pool may
 * move before the graph is replayed.  Graphs and streams that run at the same time
 * need one each.
 */
fcc_status fcc_paged_attention(int R, const void *const *Q, int64_t ldq, const fcc_cache *cache,
                               const fcc_batch *batch, int Hq, void *const *O, int64_t ldo,
                               float *const *lse, float scale, int64_t window, fcc_dtype in,
                               fcc_dtype out, const fcc_opts *opts, fcc_stream_t stream);
size_t fcc_paged_attention_workspace_size(int R, int64_t T, int B, int Hq, int H, int64_t d,
                                          const fcc_opts *opts);

/* Scratch bytes a call needs (for opts->workspace); 0 if none. */
size_t fcc_workspace_size(fcc_op op, int R, int64_t M, int64_t N, int64_t K,
                          const fcc_opts *opts);
size_t fcc_moe_workspace_size(int R, int64_t T, int64_t H, int64_t F, int E, int topk,
                              int64_t cap, const fcc_opts *opts);
size_t fcc_moe_combine_workspace_size(int R, int64_t T, int topk);

/*
 * Synchronises `stream`, then returns and clears the device status word of
 * the current device (FCC_OK if no device-side error was recorded).
 */
fcc_status fcc_stream_status(fcc_stream_t stream);

/* Static description of a status code. */
const char *fcc_status_string(fcc_status s);

/*
 * The algorithm FCC_ALGO_AUTO runs for a call (the strategy selector, after
 * Compass's unified framework of operator variants: "Compass: Dissecting
 * Communication and Computation Operators for Efficient LLM Training",
 * abstract), from measurements on GB300: FCC_ALGO_FUSED for the GEMM +
 * ReduceScatter / AllReduce and AllGather + GEMM (fastest at every shape
 * measured); for the GEMV + AllReduce, FCC_ALGO_UNFUSED when the fused grid
 * would split the rank-and-K range 16 or more ways (few 512-column groups:
 * its final serial sum of the splits then costs more than the plain GEMM +
 * reduce), else FCC_ALGO_FUSED; for the embedding + All-to-All,
 * FCC_ALGO_FUSED (1133-1140 us on 8 ranks x 64 tables of 65536 x 128, 2048
 * samples a rank, bags of 32, against 1304-1308 us for pooling table by table
 * into a staging buffer and then the exchange).  sms: SMs to plan for (0 =
 * the current device's, 152 without one); max_ctas as in fcc_opts.
 * Host-only.
 */
fcc_algo fcc_choose_algo(fcc_op op, int R, int64_t M, int64_t N, int64_t K, int sms,
                         int max_ctas);

/*
 * InterDecom chunk-count model ("Compass: Dissecting Communication and
 * Computation Operators for Efficient LLM Training", abstract: a model that
 * derives the optimal decomposition degree; its formula is not given there).
 * Two-stage pipeline, c chunks, per-chunk overhead alpha:
 *   T(c) = max(G, X) + min(G, X) / c + c * alpha
 * minimised at c* = sqrt(min(G, X) / alpha), rounded to the better integer
 * neighbour and clamped to [1, max_chunks].  G = one-shot GEMM time, X =
 * one-shot collective time (any consistent unit).
 */
int fcc_interdecom_chunks(double G, double X, double alpha, int max_chunks);
double fcc_interdecom_time(double G, double X, double alpha, int chunks);

/*
 * Test support: launches one kernel whose bounded wait on a barrier that
 * nothing completes runs out after timeout_ns; the kernel then records
 * FCC_ERR_TIMEOUT in the status word and returns, leaving the context usable.
 * fcc_stream_status() afterwards returns FCC_ERR_TIMEOUT.
 */
fcc_status fcc_test_wait_timeout(int64_t timeout_ns, fcc_stream_t stream);

/* Test support: the same with the suspended form of the wait that the losses' kernels use. */
fcc_status fcc_test_suspended_wait_timeout(int64_t timeout_ns, fcc_stream_t stream);

/*
 * Test support: launches the MoE grouped expert GEMM kernel (the in-kernel
 * staging form of fcc_moe_dispatch_gemm) on a one-tile table whose unit row
 * counter nothing raises, so its TMA producers' bounded wait for the unit's
 * rows runs out after timeout_ns; the kernel records FCC_ERR_TIMEOUT and
 * returns, leaving the context usable.  Uses the internal workspace pool.
 */
fcc_status fcc_test_grouped_wait_timeout(int64_t timeout_ns, fcc_stream_t stream);

/*
 * Test support: launches the fused GEMM + ReduceScatter kernel on a small
 * problem (1 rank, 384 x 256 x 128, on two single CTAs) whose short last
 * round runs as two K halves, with the second half waiting for a flag value
 * the first never writes, so that bounded wait runs out after timeout_ns;
 * the kernel records FCC_ERR_TIMEOUT, stores nothing for that tile and
 * returns, leaving the context usable.  Uses the internal workspace pool.
 */
fcc_status fcc_test_ksplit_wait_timeout(int64_t timeout_ns, fcc_stream_t stream);

/* Number of kernels this library has launched in this process (all devices). */
uint64_t fcc_launch_count(void);

/* Library version, "major.minor.patch". */
const char *fcc_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FCC_H_ */
