/*
 * moe_route.h -- C ABI of the single-GPU MoE token-routing path for AMD
 * Instinct MI355X (gfx950): router top-k with gate weights, the expert demand
 * vector, METRO-style greedy replica assignment, the rank-grouped dispatch
 * layout with single-send dedup counts, the row dispatch, an expert stand-in,
 * and the weighted combine; around them, single-send dispatch (one row per
 * token and destination rank) with its receiver fan-out, the backward of the
 * combine and the dispatch, routing statistics, and token-balanced replica
 * routing as the greedy's baseline; and the layer around the routing: the
 * norm that makes its rows with its gradient, the experts' products in
 * block-scaled 8-bit floating point, and the whole layer for a few tokens.
 *
 * Sources (web pages on MoE dispatch and combine):
 *   [METRO]  "METRO AllGather vs AllToAll for MoE decode".
 *   [CORR]   News summary of "correlated expert placement and token
 *            shuffling" for MoE pretraining.
 *   [DODOCO] "Diagnosing Overhead in Dispatch Operations: Cross-architecture
 *            Observatory".
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every array argument is a DEVICE pointer allocated and owned by the
 *    caller. The library never allocates or frees device memory, never
 *    synchronises, and only enqueues kernels on `stream` (a hipStream_t;
 *    NULL means the null stream). Results are valid once the stream has
 *    reached that point. Calls are stateless and may run concurrently on
 *    different streams with different buffers.
 *  - Every call returns a moe_status and never aborts. Host-side argument
 *    checks happen before anything is enqueued: MOE_ERR_INVALID_ARG for a bad
 *    shape, dtype, flag, a NULL pointer where data is needed, or a
 *    misaligned pointer; MOE_ERR_WORKSPACE for a workspace smaller than
 *    moe_workspace_bytes(). A failed kernel launch returns MOE_ERR_HIP.
 *    moe_last_error() gives a one-line description of the last failure on
 *    the calling thread.
 *  - Data-dependent faults are not detected: expert ids in `idx` outside
 *    [0, E), replica entries outside [-1, R), or `pos` / `src` values that
 *    are not the permutation moe_layout wrote give an unspecified result,
 *    but every kernel keeps its memory accesses inside the buffers the shape
 *    describes (out-of-range entries are clamped or skipped).
 *  - T = 0 is valid: per-token outputs are empty, per-expert and per-rank
 *    outputs are written (zero counts, no active experts, zero offsets).
 *  - Token activations are 16-bit floats (fp16 or bf16) in row-major [rows, H]
 *    with H a multiple of 8, so each row is a whole number of 16-byte chunks;
 *    activation pointers must be 16-byte aligned.
 */
#ifndef MOE_ROUTE_H
#define MOE_ROUTE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,
  MOE_ERR_UNSUPPORTED = 2,
  MOE_ERR_WORKSPACE = 3,
  MOE_ERR_HIP = 4
} moe_status;

/* Activation formats. */
enum { MOE_F16 = 1, MOE_BF16 = 2 };

/* Flags (bit set). */
enum {
  /* Greedy replica assignment visits active experts in ascending id instead
   * of the default most-constrained-first order (fewest replicas, then id). */
  MOE_FLAG_GREEDY_ID_ORDER = 1u << 0,
  /* moe_combine writes fp32 rows instead of the activation format. */
  MOE_FLAG_OUT_F32 = 1u << 1,
  /* moe_expert_gemm sums exact products in fp32 for bf16 rows too. Other calls
   * take the flag and do the same with and without it. */
  MOE_FLAG_EXACT_SUMS = 1u << 2
};

/* Limits checked on the host. */
/* MOE_MAX_ROWS bounds T*k: kernels that give each send row a 256-thread
 * block launch up to T*k blocks, and one launch holds fewer than 2^32
 * work-items. */
enum { MOE_MAX_E = 1024, MOE_MAX_K = 16, MOE_MAX_R = 1024, MOE_MAX_REP = 16,
       MOE_MAX_ROWS = (1 << 24) - 1 };

/* 8-bit rows: the columns one scale covers, the widest row of the norm, and
 * the most tokens of moe_layer_few_tokens. */
enum { MOE_SCALE_BLOCK = 128, MOE_MAX_NORM_H = 16384, MOE_MAX_FEW_TOKENS = 64 };

/* One routing problem.
 *   T  tokens, T >= 0, T*k <= MOE_MAX_ROWS (2^24 - 1)
 *   E  experts, 1 <= E <= 1024
 *   k  experts selected per token, 1 <= k <= min(E, 16)
 *   H  hidden width (elements per activation row), H > 0, H % 8 == 0
 *   R  virtual expert-parallel ranks (= virtual GPUs), 1 <= R <= 1024; a
 *      layout inside this GPU's memory, nothing is communicated
 *   act_dtype  MOE_F16 or MOE_BF16
 *   flags      MOE_FLAG_* bits                                               */
typedef struct {
  int32_t T, E, k, H, R;
  int32_t act_dtype;
  uint32_t flags;
} moe_problem;

/* Version of this ABI (major * 10000 + minor * 100 + patch). */
int32_t moe_version(void);

/* Identity of the build: 16 hex digits of a SHA-256 over the compile flags
 * and the bytes of every source and header the library was compiled from
 * ("unknown" when built without the package's build script). A loader
 * compares it with the digest of the sources beside it to refuse a stale
 * library. Static string; host only. */
const char* moe_build_id(void);

/* Static text for a status code ("unknown status" for other values). */
const char* moe_status_string(int32_t status);

/* Description of the last non-OK status returned on this thread ("" if none). */
const char* moe_last_error(void);

/* Bytes of device workspace moe_route, moe_layout, moe_layout_single_send and
 * the one-call plans need for this problem (one buffer of this size serves
 * all of them; its contents need no initialisation and are not meaningful
 * between calls).
 * Host only; enqueues nothing. */
moe_status moe_workspace_bytes(const moe_problem* p, size_t* bytes);

/* Router top-k, gate weights and the global expert demand vector.
 * [METRO] section "METRO AllGather vs AllToAll changes the routing
 * information": top-k over every token, then one count per expert.
 *   logits  f32 [T, E] row-major (read)
 *   idx     i32 [T, k] (write): the k selected experts of each token, slot 0
 *           the largest logit; ties go to the lower expert id, -0.0 ties
 *           +0.0, a NaN logit ranks below every number
 *   w       f32 [T, k] (write): softmax over the k selected logits, evaluated
 *           in fp64 and rounded once to fp32 (the pages give no gate rule;
 *           this is the reading taken)
 *   counts  i32 [E] (write): number of (token, slot) pairs that chose e;
 *           sums to T*k
 *   ws      workspace of at least moe_workspace_bytes() bytes             */
moe_status moe_route(const moe_problem* p, const float* logits, int32_t* idx, float* w,
                     int32_t* counts, void* ws, size_t ws_bytes, void* stream);

/* Greedy replica assignment: every active expert (counts[e] > 0) goes to one
 * of its replicas, on the virtual GPU with the fewest experts activated so
 * far; ties go to the lower GPU index. [METRO] sections "METRO AllGather vs
 * AllToAll changes the routing information" and "Add the expert-weight
 * traffic term" (greedy, not the optimal min-max assignment).
 * Visiting order: most-constrained first (ascending number of replicas, then
 * id) unless MOE_FLAG_GREEDY_ID_ORDER is set.
 *   counts  i32 [E] (read)
 *   rep     i32 [E, maxrep] (read) virtual GPU ids in [0, R) holding a copy of
 *           each expert, -1 padded; rep[e][0] is the primary copy and must be
 *           valid. NULL means no replicas: expert e lives on GPU e / (E / R)
 *           (needs R | E).
 *   maxrep  columns of rep, 1..16 (ignored when rep is NULL)
 *   assign  i32 [E] (write): chosen GPU, or -1 for an inactive expert
 *   active  i32 [R] (write): activated experts per virtual GPU              */
moe_status moe_assign_replicas(const moe_problem* p, const int32_t* counts, const int32_t* rep,
                               int32_t maxrep, int32_t* assign, int32_t* active, void* stream);

/* Dispatch layout and single-send dedup counts.
 * [METRO] section "Work the 8-GPU payload example" (an all-to-all sends one
 * chunk per destination rank) and section "Distinguish METRO from backend
 * names" (variable-size all-to-all driven by destination counts); [CORR]
 * section "Two locality techniques" (a token is sent to a GPU at most once).
 * The send buffer has exactly T*k rows, grouped by destination rank, inside a
 * rank by expert id, inside an expert by token (stable).
 *   idx      i32 [T, k] (read), as written by moe_route; an id outside
 *            [0, E) is clamped into it
 *   assign   i32 [E] or NULL (read): destination of active experts; inactive
 *            experts (-1) and the NULL case use the primary copy
 *   rep, maxrep  as in moe_assign_replicas (NULL: contiguous partition)
 *   rank_of         i32 [E]   (write) destination rank of each expert
 *   expert_offsets  i32 [E]   (write) first send row of expert e's segment
 *   rank_offsets    i32 [R+1] (write) first send row of each rank; [R] = T*k
 *   pos   i32 [T*k] (write) send row of pair (t, j) at index t*k + j
 *   src   i32 [T*k] (write) inverse of pos: flat (t, j) index of each row
 *   dedup i32 [R]   (write) tokens with at least one expert on rank r: the
 *                   rows a single-send dispatcher sends to r               */
moe_status moe_layout(const moe_problem* p, const int32_t* idx, const int32_t* assign,
                      const int32_t* rep, int32_t maxrep, int32_t* rank_of,
                      int32_t* expert_offsets, int32_t* rank_offsets, int32_t* pos,
                      int32_t* src, int32_t* dedup, void* ws, size_t ws_bytes, void* stream);

/* Everything moe_layout computes, plus the single-send rows: one send row
 * per (token, destination rank) instead of one per (token, slot), so a token
 * goes to each virtual GPU once. [CORR] section "Two locality techniques"
 * (a dispatcher that sends each token to a GPU once; with correlated expert
 * placement it removes dispatched rows).
 * Single-send rows are grouped by destination rank, inside a rank by token.
 *   ss_rank_offsets i32 [R+1] (write) first single-send row of each rank;
 *                   [R] = n_ss = sum(dedup), the number of rows
 *   ss_row          i32 [T*k] (write) the single-send row carrying pair
 *                   (t, j) at index t*k + j; the pairs of one token whose
 *                   experts sit on the same rank share one row
 *   ss_token        i32 [T*k] (write) token of each single-send row; entries
 *                   from n_ss on are left untouched
 * The other arguments are those of moe_layout. The workspace is the same
 * size (moe_workspace_bytes).                                              */
moe_status moe_layout_single_send(const moe_problem* p, const int32_t* idx, const int32_t* assign,
                                  const int32_t* rep, int32_t maxrep, int32_t* rank_of,
                                  int32_t* expert_offsets, int32_t* rank_offsets, int32_t* pos,
                                  int32_t* src, int32_t* dedup, int32_t* ss_rank_offsets,
                                  int32_t* ss_row, int32_t* ss_token, void* ws, size_t ws_bytes,
                                  void* stream);

/* moe_route, moe_assign_replicas and moe_layout in one call, with the same
 * arguments and outputs as those three calls made in that order (assign is
 * both an output and the layout's input). For a decode batch fixed latency
 * rather than bytes sets the time ([METRO] section "Find the crossover
 * instead of copying 2 MB": below the crossover payload a fixed overhead
 * dominates), so the steps share launches:
 *   - a batch with T*k <= 8192 whose tables fit in 64 KiB of LDS: two
 *     launches, the top-k kernel, then one workgroup that sums the demand
 *     vector, runs the greedy and lays out the batch;
 *   - a larger batch without a replica table (rep NULL): three launches,
 *     the top-k kernel (which also counts each block's tokens per rank), a
 *     column scan, and the permutation;
 *   - a larger batch with a replica table: the kernels of the three calls.
 * ws is one workspace of moe_workspace_bytes().                             */
moe_status moe_route_assign_layout(const moe_problem* p, const float* logits, const int32_t* rep,
                                   int32_t maxrep, int32_t* idx, float* w, int32_t* counts,
                                   int32_t* assign, int32_t* active, int32_t* rank_of,
                                   int32_t* expert_offsets, int32_t* rank_offsets, int32_t* pos,
                                   int32_t* src, int32_t* dedup, void* ws, size_t ws_bytes,
                                   void* stream);

/* moe_route, moe_assign_replicas and moe_layout_single_send in one call, with
 * the same arguments and outputs as those three calls made in that order:
 * the routing and the plain layout, plus the single-send rows of a
 * dispatcher that sends each token to a GPU once (news summary of correlated
 * expert placement and token shuffling, section "Two locality techniques").
 *   - a batch with T <= 1024, T*k <= 8192 and R <= 64 whose tables fit in
 *     64 KiB of LDS: two launches, the top-k kernel, then one workgroup that
 *     sums the demand vector, runs the greedy and lays out the batch and its
 *     single-send rows;
 *   - a larger batch without a replica table (rep NULL): three launches, the
 *     top-k kernel (which also counts each block's tokens per rank and
 *     records each token's first slot on each of its ranks), a column scan,
 *     and one launch for the permutation and the single-send rows;
 *   - otherwise (a larger batch with a replica table, or T = 0): the kernels
 *     of the three calls.
 *   ss_rank_offsets, ss_row, ss_token as for moe_layout_single_send (ss_row
 *   and ss_token i32 [T*k], unused when T = 0).
 * ws is one workspace of moe_workspace_bytes().                             */
moe_status moe_route_assign_layout_single_send(
    const moe_problem* p, const float* logits, const int32_t* rep, int32_t maxrep, int32_t* idx,
    float* w, int32_t* counts, int32_t* assign, int32_t* active, int32_t* rank_of,
    int32_t* expert_offsets, int32_t* rank_offsets, int32_t* pos, int32_t* src, int32_t* dedup,
    int32_t* ss_rank_offsets, int32_t* ss_row, int32_t* ss_token, void* ws, size_t ws_bytes,
    void* stream);

/* Bytes of the static device scratch behind moe_route_assign_layout_noalloc
 * (2 MiB per GPU). */
#define MOE_NOALLOC_SCRATCH_BYTES (2u << 20)

/* moe_route_assign_layout without a workspace argument, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc). The scratch is a static device
 * array of MOE_NOALLOC_SCRATCH_BYTES that each GPU holds from the first call
 * on it until the process ends; the call itself allocates nothing.
 * Arguments and outputs are those of moe_route_assign_layout (the caller
 * still allocates every input and output), and so are the results.
 *   - A problem whose route and layout tables need more scratch than the
 *     array holds (E + R above 1024, with enough tokens; every
 *     problem with E + R <= 1024 fits) returns MOE_ERR_WORKSPACE before
 *     anything is enqueued.
 *   - The first call on a device looks up that device's copy of the array
 *     (a failure returns MOE_ERR_HIP).
 *   - The scratch needs no initialisation, and its contents are not
 *     meaningful between calls.
 *   - Every call on one GPU uses that GPU's one array: calls that overlap on
 *     one GPU (different streams, or host threads enqueueing concurrently)
 *     race on it and give unspecified results. Order them on one stream.   */
moe_status moe_route_assign_layout_noalloc(const moe_problem* p, const float* logits,
                                           const int32_t* rep, int32_t maxrep, int32_t* idx,
                                           float* w, int32_t* counts, int32_t* assign,
                                           int32_t* active, int32_t* rank_of,
                                           int32_t* expert_offsets, int32_t* rank_offsets,
                                           int32_t* pos, int32_t* src, int32_t* dedup,
                                           void* stream);

/* Single-send dispatch: each token row x[t] is copied once to each distinct
 * single-send row among ss_row[t*k .. t*k+k). [CORR] section "Two locality
 * techniques".
 *   x        16-bit [T, H] (read)   ss_row i32 [T*k] (read), from
 *            moe_layout_single_send
 *   send_ss  16-bit [ss_capacity, H] (write); ss_capacity >= n_ss rows
 *            (rows at or beyond ss_capacity are skipped)                   */
moe_status moe_single_send_dispatch(const moe_problem* p, const void* x, const int32_t* ss_row,
                                    void* send_ss, int32_t ss_capacity, void* stream);

/* Receiver-side fan-out of single-send rows to the expert-grouped layout:
 * send[pos[i]] = send_ss[ss_row[i]] for every pair i < T*k, which equals what
 * moe_dispatch writes. [CORR] section "Two locality techniques" (each GPU
 * receives a token once and serves every selected expert it holds). Each
 * single-send row is read once and written to the expert rows of all the
 * slots it carries.
 *   send_ss          16-bit [ss_capacity, H] (read)
 *   ss_rank_offsets  i32 [R+1] (read; [R] = n_ss)   ss_token i32 [n_ss] (read)
 *   ss_row, pos      i32 [T*k] (read), from moe_layout_single_send
 *   send             16-bit [T*k, H] (write)
 * Single-send rows at or beyond min(n_ss, ss_capacity), and out-of-range
 * tokens or positions, are skipped: their destination rows are left
 * untouched.                                                               */
moe_status moe_single_send_expand(const moe_problem* p, const void* send_ss,
                                  const int32_t* ss_rank_offsets, const int32_t* ss_token,
                                  const int32_t* ss_row, const int32_t* pos, int32_t ss_capacity,
                                  void* send, void* stream);

/* Row dispatch: send[pos[i]] = x[i / k] for every i < T*k, a bit copy.
 * [METRO] section "Work the 8-GPU payload example" (the dispatch payload is
 * token activation rows).
 *   x     16-bit [T, H] (read)    pos  i32 [T*k] (read)
 *   send  16-bit [T*k, H] (write); must not overlap x
 * A slot whose pos is outside [0, T*k) is skipped: no row is written for
 * it.                                                                      */
moe_status moe_dispatch(const moe_problem* p, const void* x, const int32_t* pos, void* send,
                        void* stream);

/* Expert stand-in (the pages' expert GEMMs need trained weights): for send
 * row r routed to expert e = idx[src[r]], y[r] = round16(fp32(send[r]) * s)
 * with s = 1 + e/E, s and the product each rounded to fp32, round16 to
 * nearest-even in the activation format.
 *   send 16-bit [T*k, H] (read)  src i32 [T*k]  idx i32 [T, k]
 *   y    16-bit [T*k, H] (write); may alias send
 * A row whose src is outside [0, T*k) is scaled as expert 0 (s = 1).      */
moe_status moe_expert_standin(const moe_problem* p, const void* send, const int32_t* src,
                              const int32_t* idx, void* y, void* stream);

/* Weighted combine back to token order:
 * out[t] = sum over j = 0..k-1 (ascending) of w[t, j] * y[pos[t*k + j]],
 * accumulated in fp32, written in the activation format (round to
 * nearest-even) or as fp32 with MOE_FLAG_OUT_F32.
 * [METRO] section "METRO AllGather vs AllToAll changes the routing
 * information" (expert outputs return through a combine); [CORR] section
 * "Why communication is the target".
 *   y    16-bit [T*k, H] (read)  pos i32 [T*k]  w f32 [T, k]
 *   out  [T, H] in the activation format or fp32 (write); must not overlap y
 * A slot whose pos is outside [0, T*k) takes weight 0 on row 0: it adds
 * nothing while row 0 is finite.                                           */
moe_status moe_combine(const moe_problem* p, const void* y, const int32_t* pos, const float* w,
                       void* out, void* stream);

/* Backward of the combine. With dout [T, H] the gradient of out:
 *   dy[pos[t*k + j]] = round16(fp32(w[t, j] * dout[t]))   (one rounding
 *                      of the fp32 product to the activation format)
 *   dw[t, j]         = <y[pos[t*k + j]], dout[t]>, summed in fp32
 * Derived from the forward definition of moe_combine; [CORR] section "Why
 * communication is the target" (the combine also runs in the backward
 * pass). One kernel reads each dout row once and, per slot, writes the dy
 * row and reads the y row for the dot product.
 *   dout 16-bit [T, H] (read)   pos i32 [T*k] (read)
 *   w    f32 [T, k] (read; may be NULL when dy is NULL)
 *   y    16-bit [T*k, H] (read; may be NULL when dw is NULL)
 *   dy   16-bit [T*k, H] (write, or NULL to skip); may alias y, must not
 *        overlap dout
 *   dw   f32 [T, k] (write, or NULL to skip)
 * With T > 0 at least one of dy, dw must be non-NULL (else
 * MOE_ERR_INVALID_ARG). A slot whose pos is out of range
 * writes no dy row and a dw of 0.                                          */
moe_status moe_combine_backward(const moe_problem* p, const void* dout, const void* y,
                                const int32_t* pos, const float* w, void* dy, float* dw,
                                void* stream);

/* Backward of the dispatch: dx[t] = sum over j = 0..k-1 (ascending) of
 * dsend[pos[t*k + j]], accumulated in fp32, written in the activation format
 * (round to nearest-even) or as fp32 with MOE_FLAG_OUT_F32. Derived from the
 * forward definition of moe_dispatch; [CORR] section "Why communication is
 * the target".
 *   dsend 16-bit [T*k, H] (read)   pos i32 [T*k] (read)
 *   dx    [T, H] in the activation format or fp32 (write); must not overlap
 *         dsend. A slot whose pos is out of range adds nothing.           */
moe_status moe_dispatch_backward(const moe_problem* p, const void* dsend, const int32_t* pos,
                                 void* dx, void* stream);

/* Routing statistics of one batch. [DODOCO] section "Methodology" (three
 * scalar summaries of the send-counts matrix: per-expert max/mean, Gini of
 * the per-rank load, a fitted symmetric Dirichlet alpha); [CORR] sections
 * "Correlations in router choices" (experts chosen together) and "Two
 * locality techniques" (share of assignments served on the token's own GPU).
 * Token t comes from virtual rank floor(t R / T).
 *   idx         i32 [T, k] (read)   counts i32 [E] (read, from moe_route)
 *   rank_of     i32 [E] (read, from moe_layout)
 *   send_counts i32 [R, R] (write): [s][d] = (token, slot) pairs from
 *               source rank s whose expert sits on rank d
 *   coselect    i32 [E, E] (write, or NULL to skip): [a][b] for a < b = the
 *               tokens that chose both a and b; 0 elsewhere
 *   stats       f64 [4] (write): with N = T k and L[d] = sum_s S[s][d],
 *               [0] max_e counts[e] / (N / E)
 *               [1] Gini of L: sum_i sum_j |L_i - L_j| / (2 R N)
 *               [2] symmetric Dirichlet alpha fitted by moments to the
 *                   shares L / N: ((R - 1) / (R D) - 1) / R with
 *                   D = sum_i (L_i / N - 1/R)^2; +inf when D = 0
 *               [3] locality: sum_r S[r][r] / N
 *               all four NaN when T = 0.
 * Every count is exact (integer adds); the ratios are a few fp64 operations
 * on exact integers.                                                        */
moe_status moe_routing_stats(const moe_problem* p, const int32_t* idx, const int32_t* counts,
                             const int32_t* rank_of, int32_t* send_counts, int32_t* coselect,
                             double* stats, void* stream);

/* Token-balanced (EPLB-style) replica routing, the baseline the greedy of
 * moe_assign_replicas is compared against. [METRO] section "Add the
 * expert-weight traffic term" (balancing tokens over an expert's replicas
 * activates more replicas per GPU than grouping them; the greedy is
 * reported against EPLB's token routing).
 * The n pairs routed to expert e, in the order of e's send segment (token
 * order), are cut into contiguous shares over e's valid replicas (entries
 * of rep[e] in [0, R), in table order): with m of them, replica j takes
 * n / m pairs, plus one when j < n mod m. rep = NULL: one copy per expert,
 * on rank e / (E / R).
 *   idx            i32 [T, k] (read)   counts i32 [E] (read, from moe_route)
 *   pos            i32 [T*k] (read)    expert_offsets i32 [E] (read), both
 *                  from moe_layout (any rank order: only the place of a
 *                  pair inside its expert's segment is used)
 *   rep, maxrep    as for moe_assign_replicas
 *   gpu_of_pair    i32 [T*k] (write, or NULL to skip): the GPU serving each
 *                  pair; -1 for an expert without a valid replica
 *   active         i32 [R] (write): replicas with a non-empty share per GPU
 *   tokens         i32 [R] (write): pairs served per GPU                    */
moe_status moe_token_balanced_split(const moe_problem* p, const int32_t* idx,
                                    const int32_t* counts, const int32_t* pos,
                                    const int32_t* expert_offsets, const int32_t* rep,
                                    int32_t maxrep, int32_t* gpu_of_pair, int32_t* active,
                                    int32_t* tokens, void* stream);

/* ---- the layer around the routing ------------------------------------------
 *
 * 8-bit rows hold e4m3 codes (the OCP format: largest value 448, no
 * infinities) with one fp32 scale for each block of 128 columns (the last
 * block may be shorter): a value is its code times its block's scale. For a
 * block of values v with the largest magnitude amax,
 *   scale = max(amax, 2^-100) / 448,  code = v / scale rounded to nearest even
 * (v times the scale's reciprocal: where that, within 1.5 steps of fp32 of v /
 * scale, lies on the other side of the middle, the neighbouring code).
 * A block that holds an infinity or a NaN takes a NaN scale: all its values
 * are NaN. Rows of C columns have ceil(C / 128) scales.
 * Weight matrices in 8 bits are [rows, C] codes with one scale for each block
 * of 128 x 128, [ceil(rows / 128), ceil(C / 128)]; which scales they hold is
 * the caller's choice. The experts' products multiply a row's scale by a weight
 * block's in fp32 before they apply them to the block's sum: where that product
 * overflows, an infinity comes out, or NaN for a sum of 0, and below 2^-126 it
 * loses bits. With weight scales of at most 256 no scale that this library
 * writes for a row can overflow it.                                          */

/* Root-mean-square norm of the activation rows, with the residual's addition
 * and 8-bit output: what makes the rows that the router scores and the
 * dispatch sends ([METRO] section "METRO AllGather vs AllToAll changes the
 * routing information" starts from them).
 *   h[t]    = round16(x[t] + residual[t])           (x[t] without residual)
 *   rstd[t] = 1 / sqrt(mean over H of h[t]^2 + eps)
 *   v       = h[t] * rstd[t] * gamma, in fp32
 *   y[t]    = round16(v),  (q[t], q_scale[t]) = 8-bit row of v
 * H is at most MOE_MAX_NORM_H (MOE_ERR_UNSUPPORTED); eps finite and >= 0.
 *   x         16-bit [T, H] (read)
 *   residual  16-bit [T, H] (read) or NULL
 *   gamma     16-bit [H] (read)
 *   h         16-bit [T, H] (write) with a residual, NULL without; may be x
 *             or residual itself
 *   y         16-bit [T, H] (write), or NULL to skip; may be x or residual
 *             itself (and then not h)
 *   q, q_scale  codes [T, H], 8-byte aligned, and f32 [T, ceil(H/128)]
 *             (write), or both NULL to skip
 *   rstd      f32 [T] (write), or NULL to skip
 * q, q_scale and rstd must not overlap any other buffer.
 * At least one of y and q must be given when T > 0.                          */
moe_status moe_rms_norm(const moe_problem* p, const void* x, const void* residual,
                        const void* gamma, float eps, void* h, void* y, void* q, float* q_scale,
                        float* rstd, void* stream);

/* Bytes of device workspace that moe_rms_norm_backward needs (0 for T = 0).
 * Host only.                                                                 */
moe_status moe_rms_norm_workspace_bytes(const moe_problem* p, size_t* bytes);

/* Backward of the norm. With dy the gradient of y (or of the values of q, the
 * rounding passed through) and dh the one that reaches h along the residual
 * stream, n = h[t] * rstd[t], u = dy[t] * gamma:
 *   dx[t]  = round16(rstd[t] * (u - n * mean over H of (u * n)) + dh[t])
 *   dgamma = sum over t of dy[t] * n, in fp32
 * dx is the gradient of x and of the residual alike. The sums' order depends
 * on the sizes alone, so results repeat bit for bit.
 *   dy, h   16-bit [T, H] (read); h from the forward (x without residual)
 *   dh      16-bit [T, H] (read) or NULL (no gradient along the residual)
 *   gamma   16-bit [H] (read)      rstd  f32 [T] (read), from the forward
 *   dx      16-bit [T, H] (write); may be dy or dh itself
 *   dgamma  f32 [H] (write; zeros for T = 0)
 *   ws      workspace of at least moe_rms_norm_workspace_bytes() bytes, 256-byte
 *           aligned (may be NULL for T = 0)                                  */
moe_status moe_rms_norm_backward(const moe_problem* p, const void* dy, const void* dh,
                                 const void* h, const void* gamma, const float* rstd, void* dx,
                                 float* dgamma, void* ws, size_t ws_bytes, void* stream);

/* Experts' products over the routed rows, in 8 bits:
 *   y[r, n] = sum over k of a[r', k] * w[e, n, k]
 * for every row r of expert e's segment [expert_offsets[e], + counts[e]), a
 * and w being the values that the codes and scales stand for; y is rounded
 * once to the activation format, or written as fp32 with MOE_FLAG_OUT_F32.
 * Each block of 128 products is summed by the matrix cores, the blocks with
 * their scales in fp32. An fp16 or fp32 y comes from 16-bit matrix instructions
 * on the codes: exact products, summed in fp32. A bf16 y comes from 8-bit ones,
 * at up to twice the rate, which cut a product off at 2^-13 of a power of two
 * that the largest of its eight neighbours reaches: at most 7 * 2^-13 of the
 * largest product of each eight is lost. Of a sum of one sign that is 0.22 of
 * half a bf16 step at worst (about 1.2e-5 of the sum for normal values); where
 * terms cancel it can be any part of the result. MOE_FLAG_EXACT_SUMS makes a
 * bf16 y from exact products as well.
 *   src NULL:  r' = r, a has T*k rows in send order
 *   src given: r' = src[r] / k, a has T rows in token order (the row dispatch
 *              happens in the product's loads)
 * Takes the place of moe_expert_standin where weights are at hand ([METRO]
 * section "Add the expert-weight traffic term": the weights of the activated
 * experts are what a decode batch reads). The gradient of a is the same
 * product with the weights and their scales transposed.
 *   K   columns of a and w, a multiple of 16     N  rows of w, a multiple of 8
 *   a, a_scale      codes [rows, K], f32 [rows, ceil(K/128)] (read)
 *   src             i32 [T*k] (read) from moe_layout, or NULL
 *   w, w_scale      codes [E, N, K], f32 [E, ceil(N/128), ceil(K/128)] (read)
 *   counts          i32 [E] (read) from moe_route
 *   expert_offsets  i32 [E] (read) from moe_layout
 *   y               [T*k, N] in the activation format or fp32 (write)
 * Codes are 16-byte aligned. Rows in no segment are left untouched; a src
 * outside [0, T*k) is clamped into it. H of the problem is not used. Sizes
 * that the kernel's 32-bit offsets do not hold return MOE_ERR_UNSUPPORTED: an
 * expert's N * K codes, and with src the T * K codes of a, are fewer than 2^32
 * (without src a may be of any size), K is at most 2^24 - 16 then, and there are
 * fewer than 2^30 tiles of 64 rows by 256 columns.                          */
moe_status moe_expert_gemm(const moe_problem* p, int32_t K, int32_t N, const void* a,
                           const float* a_scale, const int32_t* src, const void* w,
                           const float* w_scale, const int32_t* counts,
                           const int32_t* expert_offsets, void* y, void* stream);

/* The gate and up products of the experts with SwiGLU and 8-bit output, in
 * one pass: with z = the product above for weights of N = 2 I rows (gate
 * rows 0 .. I-1, up rows I .. 2I-1),
 *   v[r, i] = z[r, i] / (1 + exp(-z[r, i])) * z[r, I + i], in fp32
 *   (q[r], q_scale[r]) = 8-bit row of v[r]
 *   I   a multiple of 16; w [E, 2I, K], w_scale [E, ceil(2I/128), ceil(K/128)]
 *   q, q_scale  codes [T*k, I], 16-byte aligned, f32 [T*k, ceil(I/128)] (write)
 * The products are exact and summed in fp32 (see moe_expert_gemm on an fp32
 * y). The other arguments are those of moe_expert_gemm; act_dtype and the output
 * flag are not used.                                                         */
moe_status moe_expert_gemm_swiglu(const moe_problem* p, int32_t K, int32_t I, const void* a,
                                  const float* a_scale, const int32_t* src, const void* w,
                                  const float* w_scale, const int32_t* counts,
                                  const int32_t* expert_offsets, void* q, float* q_scale,
                                  void* stream);

/* Bytes of device workspace that moe_layer_few_tokens needs. Host only.      */
moe_status moe_layer_workspace_bytes(const moe_problem* p, int32_t I, size_t* bytes);

/* A whole mixture-of-experts layer for a few tokens (T <= 64) in two
 * launches, or up to four for hundreds of pairs and large weights: top-k and
 * gate weights as moe_route gives them, then
 *   h[t, j] = round16(silu(g) * u),  (g; u) = w_up[e] x[t], e = idx[t, j]
 *   out[t]  = sum over j of w[t, j] * (w_down[e] h[t, j]), in fp32, rounded
 *             once to the activation format (fp32 with MOE_FLAG_OUT_F32)
 * Nothing is dispatched: a decode step reads the chosen experts' weights and
 * little else ([METRO] section "Add the expert-weight traffic term").
 * Activations stay in 16 bits. With e4m3 weights the 128 products of a block are
 * summed in fp32 before its scale is applied, so these sums have to be finite
 * themselves (they are for values of x and h up to 2^112, so for any in fp16).
 *   H and I are multiples of 16 and at most 2^24; more, and T >
 *   MOE_MAX_FEW_TOKENS, return MOE_ERR_UNSUPPORTED. R is not used.
 *   logits  f32 [T, E] (read)       x  16-bit [T, H] (read)
 *   w_up    [E, 2I, H] (read), gate rows 0 .. I-1, up rows I .. 2I-1
 *   w_down  [E, H, I] (read)
 *   s_up, s_down  f32 [E, ceil(2I/128), ceil(H/128)] and
 *           [E, ceil(H/128), ceil(I/128)] (read) with e4m3 weights; both NULL
 *           with weights in the activation format
 *   idx, w  i32, f32 [T, k] (write)
 *   out     [T, H] in the activation format or fp32 (write); must not overlap x
 *   ws      workspace of at least moe_layer_workspace_bytes() bytes, 256-byte
 *           aligned                                                          */
moe_status moe_layer_few_tokens(const moe_problem* p, int32_t I, const float* logits, const void* x,
                                const void* w_up, const float* s_up, const void* w_down,
                                const float* s_down, int32_t* idx, float* w, void* out, void* ws,
                                size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTE_H */
