/*
 * ar.h -- ring / tree collectives over N rank buffers held in ONE GPU's HBM.
 *
 * C ABI of libar.so (HIP kernels for gfx950 / MI355X).  N logical ranks are N
 * separate device buffers of `count` elements each; a "send" from rank r to
 * rank d is a read of r's buffer and a write (or read-modify-write) of d's.
 *
 * Sources, cited by page title and section:
 *   [L09] "第09讲：网络通信基础与集合通信 Collective 原语直觉" (Lecture 09,
 *         collective primitives): 3.1 Broadcast, 3.4 reduction operators,
 *         3.5 AllReduce, 3.6 ReduceScatter, 3.7 AllGather, 3.9 AllReduce =
 *         ReduceScatter + AllGather, 4.2-4.4 ring, 5.2 double binary tree.
 *   [CH4] "4. 通信模式：集合通信（AllReduce、AllGather等）原理与实现"
 *         (Chapter 4, communication patterns): 4.3.1 ring, 4.3.2 tree.
 *   [SCR] "从零实现集合通信" (Collectives from scratch): section "two-pass
 *         ring allreduce" (两趟实现 ring allreduce) and its cost table.
 *
 * Conventions shared by every collective below
 * --------------------------------------------
 * bufs    HOST array of `nranks` DEVICE pointers; bufs[r] is rank r's buffer
 *         of `count` contiguous elements of `dtype`.  Every buffer must be
 *         aligned to the element size, and no two buffers may overlap.  When
 *         every buffer is 16-byte aligned the kernels move 16-byte packs;
 *         otherwise they move one element at a time, with the same
 *         arithmetic in the same order (identical results, lower speed).  The
 *         caller allocates and owns every buffer; the library never
 *         allocates user memory and keeps no pointer after returning (the
 *         pointers travel inside kernel arguments).
 * nranks  N, 1 <= N <= AR_MAX_RANKS.
 * count   T, elements per rank.  Chunk layout: C = ceil(T/N), chunk c =
 *         [c*C, min(T, (c+1)*C)); only trailing chunks are short, and a chunk
 *         is empty when c*C >= T.  Rank c owns chunk c.
 * stream  a hipStream_t (NULL = the null stream of the
 *         calling thread's current device, which must then be the device
 *         that holds the buffers; a non-null stream carries its device).  Calls are
 *         asynchronous and stream-ordered: they enqueue kernels and return;
 *         the library never synchronises.  Completion is observed through
 *         the stream.  All buffers are updated IN PLACE.
 * Arithmetic (the receiver stores `local (+) incoming`, as in the pages'
 *         per-hop in-place add [L09 7.1][CH4 4.3.1]):
 *           AR_INT32    two's-complement wrap-around for SUM and PROD;
 *           AR_FLOAT32  one IEEE binary32 operation, round to nearest even,
 *                       subnormals kept, never fused or reassociated;
 *           AR_BFLOAT16 widen both to binary32, apply the op, round back to
 *                       bfloat16 to nearest even after EVERY hop (a NaN
 *                       stays a NaN; its payload bits are unspecified);
 *           MAX / MIN   keep the local value unless the incoming one compares
 *                       strictly greater / smaller.
 *         The ring calls reproduce the ring's order per element exactly
 *         (chunk c folds ranks c+1, c+2, ..., c); the tree call reproduces the
 *         binomial double tree's pairing.  Results are therefore bit-exact
 *         and independent of the implementation chosen by ar_set_impl().
 * Errors  argument errors are reported synchronously BEFORE anything is
 *         enqueued, so such a call has no effect:
 *           AR_ERROR_INVALID_ARGUMENT  bufs or an entry NULL; nranks out of
 *               range; a pointer not aligned to the element size; two buffer
 *               ranges overlapping; count * element size overflowing; root
 *               out of range; unknown dtype or op;
 *           AR_ERROR_UNSUPPORTED       a valid request this build lacks;
 *           AR_ERROR_HIP               a kernel launch failed; the hipError_t
 *               is kept for ar_last_hip_error().  With the step
 *               implementation (or a fused ring or tree AllReduce that runs
 *               as two launches) the launches before the failing one may
 *               already be enqueued, so the buffers are then unspecified.  (Faults
 *               during execution surface at the caller's next
 *               synchronisation.)
 *         count == 0 or nranks == 1 is a valid no-op (AR_SUCCESS, nothing
 *         enqueued); with count == 0 the entries of bufs are not inspected
 *         (an empty tensor may have a NULL data pointer).
 * Counters every successful call adds the logical inter-rank bytes of its
 *         schedule (each transfer of k elements adds k * element size to the
 *         sender's `sent` and the receiver's `recv`) and its schedule steps
 *         to process-wide counters, whatever implementation runs.
 * Debug   with the environment variable AR_DEBUG set (and not "0") when the
 *         library loads, every call with work to do first builds the logical
 *         schedule it follows and checks it: every transfer inside the
 *         buffers and between two distinct ranks, no transfer of a step
 *         writing what another one of the step reads or writes [the ring's
 *         within-step disjointness, L09 4.3], the documented step count, and
 *         per-rank bytes equal to what the counters add.  A violation, which
 *         would be a defect of this library, is printed to stderr and aborts
 *         the process; nothing of that call is enqueued.
 */
#ifndef AR_H
#define AR_H

#include <stddef.h>
#include <stdint.h>

/* The HIP stream handle, declared as HIP's runtime API declares it (an
 * opaque pointer), so that this header needs no HIP include; including
 * <hip/hip_runtime_api.h> before or after it is fine. */
typedef struct ihipStream_t* hipStream_t;

#ifdef __cplusplus
extern "C" {
#endif

#define AR_MAX_RANKS 64
#define AR_VERSION 1

typedef enum {
  AR_SUCCESS = 0,
  AR_ERROR_INVALID_ARGUMENT = 1,
  AR_ERROR_UNSUPPORTED = 2,
  AR_ERROR_HIP = 3
} ar_status_t;

/* AR_BFLOAT16_ACC32: bfloat16 buffers ("bf16 with fp32 accumulation").  The
 * reductions (ring AllReduce and ReduceScatter, tree AllReduce, Reduce)
 * carry float32 partials from hop to hop in the schedule's own order and
 * round to bfloat16 once, at the end; a partial cannot live in a bfloat16
 * buffer between kernel launches, so these reductions run fused under either
 * implementation.  Copies (AllGather, Broadcast, Scatter, Gather, AllToAll)
 * are bfloat16 copies.  Elements count 2 bytes in every byte counter. */
typedef enum {
  AR_INT32 = 0,
  AR_FLOAT32 = 1,
  AR_BFLOAT16 = 2,
  AR_BFLOAT16_ACC32 = 3
} ar_dtype_t;

/* The reduction operators listed in [L09 3.4]. */
typedef enum { AR_SUM = 0, AR_PROD = 1, AR_MAX = 2, AR_MIN = 3 } ar_op_t;

typedef enum {
  AR_RING_ALLREDUCE = 0,
  AR_REDUCE_SCATTER = 1,
  AR_ALLGATHER = 2,
  AR_BROADCAST = 3,
  AR_TREE_ALLREDUCE = 4,
  AR_REDUCE = 5,
  AR_SCATTER = 6,
  AR_GATHER = 7,
  AR_ALLTOALL = 8
} ar_collective_t;

/* How a collective is executed; results are bit-identical either way.
 *   AR_IMPL_FUSED  one pass: every element's N inputs are read once, folded
 *                  in the schedule's order (tiles staged through LDS, the
 *                  partials in registers), and the result is written once
 *                  per destination rank; the copies (AllGather, Broadcast)
 *                  read each element once and write it into every other
 *                  rank, one destination rank per pass.  The AllReduces of
 *                  12 or more ranks and 384 MiB or more of inputs run as two
 *                  such launches (see ar_ring_allreduce, ar_tree_allreduce).
 *   AR_IMPL_STEP   the schedule literally: one kernel launch per ring step or
 *                  tree round, each applying all of that step's transfers. */
typedef enum { AR_IMPL_FUSED = 0, AR_IMPL_STEP = 1 } ar_impl_t;

/* Ring AllReduce [L09 3.5, 3.9, 4.3][CH4 4.3.1][SCR two-pass ring]:
 * ReduceScatter then AllGather.  Afterwards every bufs[r] holds, at element
 * i of chunk c, the fold x[c+1][i] (+) ... (+) x[c][i] taken in ring order
 * (each hop: the receiving rank's own value (+) the incoming partial).
 * AR_IMPL_FUSED: one fold storing into every rank; from 12 ranks and 384 MiB
 * of inputs (nranks * count * element size) up, the fused ReduceScatter and
 * then the fused AllGather (two launches, the same bits, faster there). */
ar_status_t ar_ring_allreduce(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype,
                              ar_op_t op, hipStream_t stream);

/* Ring ReduceScatter [L09 3.6][SCR two-pass ring, first pass]: N-1 steps; at
 * step t rank r forwards chunk (r-t-1) mod N to rank r+1, which stores
 * own (+) incoming.  Afterwards chunk r of bufs[r] holds the full reduction of
 * chunk r (same fold as ar_ring_allreduce).  The contents of the other chunks
 * of every buffer are UNSPECIFIED afterwards (partials or inputs, depending
 * on the implementation). */
ar_status_t ar_reduce_scatter(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype,
                              ar_op_t op, hipStream_t stream);

/* Ring AllGather [L09 3.7][SCR two-pass ring, second pass]: the input of
 * rank r is chunk r of bufs[r] (its other chunks are ignored and
 * overwritten); N-1 steps, at step t rank r forwards chunk (r-t) mod N to
 * rank r+1, which overwrites.  Afterwards every buffer holds every rank's
 * chunk. */
ar_status_t ar_allgather(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype,
                         hipStream_t stream);

/* Broadcast [L09 3.1][SCR cost table: T bytes over a log2 N tree]: every
 * bufs[r] ends equal to bufs[root].  Schedule (and counters): a binomial tree
 * on roles (r - root) mod N, ceil(log2 N) rounds. */
ar_status_t ar_broadcast(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype, int root,
                         hipStream_t stream);

/* Double-binary-tree AllReduce [L09 5.2][CH4 4.3.2][SCR cost table:
 * 2 log2 N steps].  Two binomial trees reduce toward role 0 and broadcast
 * back, each over half the data: tree 0 handles elements [0, ceil(T/2)) with
 * role == rank, tree 1 handles [ceil(T/2), T) with role == N-1-rank.  Reduce
 * round k: role q (q mod 2^(k+1) == 0, q + 2^k < N) stores
 * own (+) value of role q + 2^k.  Every bufs[r] ends with role 0's result.
 * AR_IMPL_FUSED: one fold storing into every rank; from 12 ranks and 384 MiB
 * of inputs up, the two trees' folds stored into their roots (rank 0, rank
 * N-1) and then both halves fanned out from there (two launches, the same
 * bits, faster there). */
ar_status_t ar_tree_allreduce(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype,
                              ar_op_t op, hipStream_t stream);

/* ---- rooted primitives ------------------------------------------------------ */

/* Reduce to `root` [L09 3.4]: bufs[root] ends with the reduction of every
 * rank's buffer; every other buffer keeps its data.  Order: the reduce
 * rounds of a binomial tree on roles (rank - root) mod N over the whole
 * buffer (the rounds of ar_tree_allreduce [L09 5.2]): round k, role q
 * (q mod 2^(k+1) == 0, q + 2^k < N) stores own (+) value of role q + 2^k;
 * the partials live in registers, never in a rank buffer.  One fused kernel
 * runs under either implementation.  Counters: each non-root rank sends its
 * buffer once to its parent; ceil(log2 N) steps.  root out of range ->
 * AR_ERROR_INVALID_ARGUMENT. */
ar_status_t ar_reduce(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype, ar_op_t op,
                      int root, hipStream_t stream);

/* Scatter from `root` [L09 3.2]: chunk c of bufs[root] (the ring chunk
 * layout above) is copied into chunk c of bufs[c] for every c != root; every
 * other element of every buffer is unchanged.  One step of N-1 direct
 * transfers. */
ar_status_t ar_scatter(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype, int root,
                       hipStream_t stream);

/* Gather to `root` [L09 3.3]: chunk c of bufs[c] is copied into chunk c of
 * bufs[root] for every c != root, so the root holds every rank's shard in
 * rank order; the other buffers are unchanged.  One step of N-1 direct
 * transfers. */
ar_status_t ar_gather(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype, int root,
                      hipStream_t stream);

/* AllToAll [L09 3.8, lab 4 in 7.4]: every buffer is N equal blocks of
 * count/N elements; block j of bufs[i] is meant for rank j, which receives
 * it in block i (recv[j][i] = send[i][j], a transpose across ranks).  Block
 * i of bufs[i] stays in place.  count must be a multiple of nranks
 * (otherwise AR_ERROR_INVALID_ARGUMENT).  One step: each rank sends and
 * receives (N-1) blocks.  One kernel swaps block j of rank i with block i of
 * rank j for every pair i < j, under either implementation. */
ar_status_t ar_alltoall(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype,
                        hipStream_t stream);

/* ---- size-based choice between ring and tree ----------------------------- */

/* AllReduce that picks the ring or the double tree by message size [L09 5.3:
 * NCCL runs the tree for small messages and the ring for large ones][SCR
 * exercises: ring vs tree at 1 KB, 1 MB and 16 MB].  It predicts the time of
 * both under the current implementation (ar_set_impl) with the cost model
 * below and runs ar_ring_allreduce or ar_tree_allreduce, whichever is lower
 * (the ring on a tie).  Arguments, errors and counters are those of the call
 * it runs; its result is that call's result bit for bit. */
ar_status_t ar_allreduce(void* const* bufs, int nranks, size_t count, ar_dtype_t dtype,
                         ar_op_t op, hipStream_t stream);

/* The collective ar_allreduce would run (AR_RING_ALLREDUCE or
 * AR_TREE_ALLREDUCE) for these arguments under the current implementation.
 * Host only. */
ar_status_t ar_allreduce_choice(int nranks, size_t count, ar_dtype_t dtype,
                                ar_collective_t* choice);

/* Kernel launches and HBM bytes of one call of `coll` under `impl` with these
 * arguments, as the library will run it: AR_IMPL_FUSED is one launch moving
 * every input once and every output once (2 N T s for an AllReduce), except
 * the AllReduces from 12 ranks and 384 MiB of inputs, which are two launches
 * moving (2 N + 1) T s; AR_IMPL_STEP is one launch per schedule step moving
 * 3 bytes per element of every reduce transfer (read both sides, write one)
 * and 2 per element of every copy transfer.  Reduce and AllToAll run their
 * one kernel, Scatter and Gather their one step (root 0), under either;
 * bfloat16 with float32 partials runs its reductions fused.  0 launches and
 * 0 bytes when nranks == 1.  AR_ERROR_INVALID_ARGUMENT for an out-of-range
 * argument or a NULL output pointer.  Host only. */
ar_status_t ar_launch_plan(ar_collective_t coll, ar_impl_t impl, int nranks, size_t count,
                           ar_dtype_t dtype, int* launches, uint64_t* hbm_bytes);

/* Cost model, the single-GPU form of the pages' alpha-beta model [L09 1.3,
 * 7.3]: predicted microseconds of one call
 *     = launches * alpha_us + hbm_bytes / (gbps * 1e3)
 * with launches and hbm_bytes those of ar_launch_plan.  One (alpha_us, gbps)
 * pair is kept per (collective, implementation); the defaults are fitted to
 * the message-size sweep measured on MI355X.  Host only. */
ar_status_t ar_predict_time(ar_collective_t coll, ar_impl_t impl, int nranks, size_t count,
                            ar_dtype_t dtype, double* microseconds);
ar_status_t ar_set_cost_model(ar_collective_t coll, ar_impl_t impl, double alpha_us,
                              double gbps);
ar_status_t ar_get_cost_model(ar_collective_t coll, ar_impl_t impl, double* alpha_us,
                              double* gbps);

/* ---- host-only helpers: no GPU work, usable without a GPU ---------------- */

/* C = ceil(count / nranks); 0 if nranks < 1. */
size_t ar_chunk_size(int nranks, size_t count);

/* Bounds [*begin, *end) of chunk `chunk`; AR_ERROR_INVALID_ARGUMENT if nranks
 * or chunk is out of range or an output pointer is NULL. */
ar_status_t ar_chunk_range(int nranks, size_t count, int chunk, size_t* begin, size_t* end);

/* Logical bytes each rank sends and receives in one call of `coll` with these
 * arguments ([SCR cost table]; e.g. 2T(N-1)/N per rank for the ring when N
 * divides T).  sent and recv are caller arrays of nranks uint64_t.  `root`
 * is used for AR_BROADCAST, AR_REDUCE, AR_SCATTER and AR_GATHER only;
 * AR_ALLTOALL needs count to be a multiple of nranks. */
ar_status_t ar_expected_bytes(ar_collective_t coll, int nranks, size_t count, ar_dtype_t dtype,
                              int root, uint64_t* sent, uint64_t* recv);

/* Schedule steps of one call: 2(N-1) ring AllReduce, N-1 ReduceScatter and
 * AllGather, ceil(log2 N) Broadcast and Reduce, 2 ceil(log2 N) tree
 * AllReduce, 1 Scatter, Gather and AllToAll (0 for every collective when
 * N == 1); -1 on a bad argument. */
int ar_expected_steps(ar_collective_t coll, int nranks);

/* Process-wide cumulative counters since load or the last reset [SCR
 * exercises: per-rank byte counter].  Copies the first nranks entries
 * (0 <= nranks <= AR_MAX_RANKS) of the logical bytes each rank sent and
 * received into sent / recv (either may be NULL).  Thread-safe. */
ar_status_t ar_counters_read(int nranks, uint64_t* sent, uint64_t* recv);
/* Total schedule steps counted since load or the last reset. */
uint64_t ar_counters_steps(void);
void ar_counters_reset(void);

/* Process-wide choice of implementation for subsequent calls (initially
 * AR_IMPL_FUSED, or AR_IMPL_STEP when the environment variable AR_IMPL is
 * "step" at load).  Thread-safe. */
ar_status_t ar_set_impl(ar_impl_t impl);
ar_impl_t ar_get_impl(void);

/* Static description of a status code. */
const char* ar_status_string(ar_status_t status);

/* hipError_t of this thread's most recent AR_ERROR_HIP (0 if none). */
int ar_last_hip_error(void);

/* AR_VERSION of the loaded library. */
int ar_version(void);

/* ---- the training step next to the collectives --------------------------------
 *
 * AdamW over many tensors at once (the update of the shards that a
 * ReduceScatter leaves with their owners, before the AllGather of the result)
 * and the router of a mixture of experts (which experts a token goes to, and
 * how many tokens go to each; no call here exchanges tokens by such counts,
 * ar_alltoall swaps equal blocks).  As above: device pointers, the caller's stream, argument errors
 * reported before anything is enqueued, no allocation, no synchronisation;
 * ar_debug_fail_launch counts these launches too.  None of these calls
 * touches the byte counters or the choice of implementation.
 */

/* Elements that share one scale of an 8-bit state. */
#define AR_ADAMW_BLOCK 256

/* One tensor of an AdamW plan: `count` contiguous elements of each.
 *   param       AR_FLOAT32 or AR_BFLOAT16, updated in place
 *   grad        AR_FLOAT32 or AR_BFLOAT16, only read
 *   copy        bfloat16 working copy of a float32 param, rewritten by every
 *               step; NULL for none (all tensors of a plan or none)
 *   exp_avg, exp_avg_sq    m and v: float32 (state_bits 32), or one code a
 *               element (state_bits 8): int8 for m, uint8 for v
 *   exp_avg_scale, exp_avg_sq_scale   state_bits 8: ceil(count / 256) float32
 *               scales each; NULL for 32
 * An 8-bit state holds m = a q |q| with q in [-127, 127] and v = (r u^2)^2
 * with u in [0, 255], a and r the scales of the element's block of 256:
 * a = max |m| / 127^2 and r = sqrt(max v) / 255^2 over the block.  A value
 * is held as the code nearest to it (for v: nearest in sqrt(v)), a tie as
 * the smaller code, a positive v never as 0.  The rounding of m and v to
 * codes is decided in 64 bits and comes after the parameter's update, which
 * uses their unrounded values.  A block whose m (or v) is not finite gets the
 * scale NaN, so that all of it reads as NaN. */
typedef struct {
  void* param;
  const void* grad;
  void* copy;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  size_t count;
} ar_adamw_tensor_t;

/* Hyperparameters of one step.  `step` counts from 1. */
typedef struct {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  double grad_scale;   /* the gradients' factor, e.g. 1/N for a mean over N ranks */
  int64_t step;
  int clip;            /* nonzero: use the factor of the last ar_adamw_grad_norm */
} ar_adamw_step_t;

/* Bytes of a plan for these tensors; 0 for what ar_adamw_plan refuses or when
 * the host runs out of memory. */
size_t ar_adamw_plan_bytes(const ar_adamw_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                           ar_dtype_t grad_dtype, int state_bits);

/* Writes the plan of these tensors into `plan` (host memory of
 * ar_adamw_plan_bytes bytes).  The caller copies all of it to device memory
 * (16-byte aligned) and passes both to the calls below, which read the host
 * plan's head and the device copy's tables; the device copy also holds the
 * norm's partial sums, so calls on one plan must be ordered on one stream (or
 * by events).  The tensors must stay where they are while the plan is used.
 * Everything is checked here: AR_ERROR_INVALID_ARGUMENT for NULL or
 * misaligned pointers, copies of some tensors only or of bfloat16 params,
 * scales missing (8) or given (32), a written range that overlaps any other
 * range; AR_ERROR_UNSUPPORTED for other types or state_bits, or more than
 * 2^22 - 1 tiles of (up to) 4,096 elements of one tensor (1.7e10 elements).
 * A tensor of count 0 is skipped, its pointers not looked at. */
ar_status_t ar_adamw_plan(const ar_adamw_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                          ar_dtype_t grad_dtype, int state_bits, void* plan, size_t bytes);

/* norm = |grad_scale| sqrt(sum g^2) over all tensors of the plan (products
 * and sums in 64 bits, in an order fixed by the plan), written as float32 to
 * the device address `norm` (may be NULL).  The plan keeps the factor
 * grad_scale min(1, max_norm / norm) (grad_scale where norm is NaN) for the
 * ar_adamw_step calls with `clip` that follow; it is NaN before the first
 * norm.  max_norm may be infinite (no clipping). */
ar_status_t ar_adamw_grad_norm(const void* plan, void* device_plan, double max_norm,
                               double grad_scale, float* norm, hipStream_t stream);

/* One AdamW step in place, with G = c grad_scale g (c = 1 without `clip`;
 * c grad_scale is one float32 factor):
 *   m' = beta1 m + (1 - beta1) G       v' = beta2 v + (1 - beta2) G^2
 *   p' = p - lr (weight_decay p + (m' / (1 - beta1^step)) /
 *                                 (sqrt(v' / (1 - beta2^step)) + eps))
 * rounded once to param's type, and to bfloat16 in `copy`.  With 32-bit
 * states in float32, with 8-bit states m' and v' in float64.  Any eps >= 0 is
 * taken; with one below about 4e-12 the updates are computed in float64, so
 * that an element whose v' float32 cannot hold moves as the formula says;
 * otherwise in float32, with a root and a reciprocal that are off by up to one
 * step of its last place.
 * With eps = 0 an element whose m' and v' are both 0 gets 0 / 0, a NaN.
 * AR_ERROR_INVALID_ARGUMENT: a factor that is not finite, lr, eps or
 * weight_decay negative, a beta outside [0, 1), step < 1.
 * AR_ERROR_UNSUPPORTED: `stream` is being captured (a replayed step would
 * repeat this step's bias corrections). */
ar_status_t ar_adamw_step(const void* plan, void* device_plan, const ar_adamw_step_t* args,
                          hipStream_t stream);

/* The values of `count` 8-bit codes (int8 for m when is_signed, else uint8
 * for v) as float32; code i belongs to scales[i / 256].
 * AR_ERROR_UNSUPPORTED: more than 4,096 (2^24 - 1) codes (6.9e10). */
ar_status_t ar_adamw_dequantize(const void* codes, const float* scales, size_t count,
                                int is_signed, float* out, hipStream_t stream);

#define AR_MAX_EXPERTS 1024
#define AR_MAX_TOP_K 8

/* Device memory of a router call's sums: AR_ROUTE_WORKSPACE bytes, 16-byte
 * aligned, all zero before its first call; a call leaves it ready for the
 * next, so one workspace serves any number of calls ordered on one stream.
 * Two streams need two. */
#define AR_ROUTE_WORKSPACE 2386432

/* Shape of a router call: `nranks` ranks (at most AR_MAX_RANKS) of `tokens`
 * tokens each, whose logits over `experts` experts lie `row_stride` elements
 * apart (row_stride >= experts).  nranks * tokens < 2^31. */
typedef struct {
  int nranks;
  size_t tokens;
  int experts;
  size_t row_stride;
  int top_k;          /* 1 .. min(experts, AR_MAX_TOP_K) */
  int renormalize;
  ar_dtype_t dtype;   /* of the logits: AR_FLOAT32 or AR_BFLOAT16 */
} ar_route_shape_t;

/* The router.  For each token with logits x: p = softmax(x); chosen are the
 * top_k largest x above -infinity, a tie to the lowest index;
 *   indices [nranks][tokens][top_k]  the chosen experts, largest first, -1
 *           where fewer than top_k are above -infinity
 *   weights [nranks][tokens][top_k]  their p, divided by their sum with
 *           `renormalize`; 0 where the index is -1
 *   counts  [nranks][experts]        tokens of the rank that chose the expert
 *   loss    E / (K T^2) sum_e C_e S_e, with C_e the counts' sum over ranks,
 *           S_e the sum of p_e over all tokens and T the tokens that live
 *   share   [experts]                E C_e / (K T^2), for ar_route_grad
 * `masks` (NULL, or one pointer a rank to `tokens` bytes): a token whose byte
 * is 0, or with every logit -infinity, is no token: index -1, weight 0,
 * nothing counted.  A token with a NaN or +infinite logit has NaN for every
 * weight and makes loss NaN; a NaN is never chosen.  p and weights are
 * computed in float32, with exponentials and reciprocals that are off by up to
 * one step of its last place (what is below its normal numbers may become 0);
 * the sums S are added up in float32 over the tokens of
 * a block, in float64 over some blocks and in fixed point (2^-32) beyond, in
 * ways that depend on the shape alone.  Outputs are written whole. */
ar_status_t ar_route(const void* const* logits, const uint8_t* const* masks,
                     const ar_route_shape_t* shape, int32_t* indices, float* weights,
                     int32_t* counts, float* loss, float* share, void* workspace,
                     hipStream_t stream);

/* Gradient of sum(dweights * weights) + dloss * loss with respect to the
 * logits, the counts held fixed: dlogits [nranks][tokens][experts],
 * contiguous, of the logits' type (one rounding), computed in float32 as
 * ar_route's weights are.  logits, masks and shape are the forward call's,
 * indices and share its outputs; dweights (NULL: 0) holds one pointer a rank
 * to [tokens][top_k] float32, dloss (NULL: 0) a float32 on the device.  0 for
 * a token that is none. */
ar_status_t ar_route_grad(const void* const* logits, const uint8_t* const* masks,
                          const ar_route_shape_t* shape, const int32_t* indices,
                          const float* share, const float* const* dweights, const float* dloss,
                          void* dlogits, hipStream_t stream);

/* ---- the experts' products ------------------------------------------------------
 *
 * What follows ar_route: the pairs (token, choice) in order by expert, matrix
 * products grouped by expert, the weighted sum back to the tokens, and the
 * gradients of all of it.  Pair p = token * top_k + choice.  Rows are the pairs
 * in order: by expert, within an expert by p, those without an expert behind
 * all others.  The counts stay on the GPU, no call waits for them.  Matrices
 * are bfloat16, products are added up in float32 and rounded once.  What the
 * device arrays `order`, `position` and `offsets` hold is bounds-checked by the
 * kernels (a row or token out of range is none).  What a call writes may not
 * overlap what it reads or writes elsewhere.
 */

/* Device memory that ar_expert_order needs for so many pairs and experts, in
 * bytes (16-byte aligned, any content); 0 for none. */
size_t ar_expert_order_workspace(size_t pairs, int experts);

/* The order of `pairs` choices (indices as ar_route writes them; a number
 * outside [0, experts) is no expert), stable:
 *   order    [pairs]        the pairs, -1 behind the last that has an expert
 *   position [pairs]        the row of each pair, -1 for none
 *   offsets  [experts + 1]  the row where each expert's pairs begin; the last is
 *            the number of pairs that have an expert
 * experts <= AR_MAX_EXPERTS, pairs < 2^31. */
ar_status_t ar_expert_order(const int32_t* indices, size_t pairs, int experts, int32_t* order,
                            int32_t* position, int32_t* offsets, void* workspace,
                            hipStream_t stream);

/* Operands of the products below.  Strides count elements.  `order` NULL: x has
 * a row for each pair, in order; else x has a row for each token (x_rows of
 * them), and the row of pair p is that of token p / top_k. */
typedef struct {
  const void* x;               /* [x_rows][in], rows x_stride apart */
  size_t x_rows;
  size_t x_stride;
  const int32_t* order;
  int top_k;
  const int32_t* offsets;
  size_t pairs;                /* < 2^31 */
  int experts;
  size_t in;
  size_t out;
  ar_dtype_t dtype;            /* AR_BFLOAT16 */
} ar_expert_rows_t;

/* y [pairs][out] (contiguous): y_i = x_i W_e for the rows i of expert e, 0 for
 * rows without an expert.  Element (k, n) of W_e lies at weight + e *
 * expert_stride + k * in_stride + n * out_stride; one of in_stride and
 * out_stride is 1 and the other at least the size along the first.  With the
 * two sizes and strides exchanged this is also the gradient with respect to x's
 * rows.  AR_ERROR_UNSUPPORTED: another dtype, or 2^23 tiles (of 16 x 64 to 256 x 256)
 * or more. */
ar_status_t ar_expert_matmul(const ar_expert_rows_t* rows, const void* weight,
                             size_t expert_stride, size_t in_stride, size_t out_stride, void* y,
                             hipStream_t stream);

/* Device memory that ar_expert_weight_grad needs for these sizes, in bytes
 * (16-byte aligned, any content); 0 for none. */
size_t ar_expert_weight_grad_workspace(size_t pairs, int experts, size_t in, size_t out);

/* dw [experts][in][out] (contiguous, AR_FLOAT32 or AR_BFLOAT16): dw_e = the sum
 * over the rows i of expert e of x_i^T dy_i, 0 for an expert without rows.  dy
 * has a row of `out` elements for each pair in order, dy_stride apart.  The
 * rows of an expert are added up in an order that the sizes alone decide.
 * AR_ERROR_INVALID_ARGUMENT also where dw meets what is read. */
ar_status_t ar_expert_weight_grad(const ar_expert_rows_t* rows, const void* dy, size_t dy_stride,
                                  void* dw, ar_dtype_t dw_dtype, void* workspace,
                                  hipStream_t stream);

/* out [tokens][size] (contiguous): out_t = the sum over the choices k of token t
 * that have a row of weights[t][k] * y_row, in the order of k (weights NULL: 1).
 * y has `pairs` rows, y_stride apart; position is [tokens][top_k].
 * AR_ERROR_UNSUPPORTED also for top_k > 2^31 - 4. */
ar_status_t ar_expert_combine(const void* y, size_t y_stride, size_t pairs, size_t size,
                              ar_dtype_t dtype, const int32_t* position, const float* weights,
                              size_t tokens, int top_k, void* out, hipStream_t stream);

/* Gradient of ar_expert_combine: dy [pairs][size] (contiguous, bfloat16), dy_row
 * = weights[t][k] * dout_t, 0 for rows behind offsets[experts]; dweights
 * [tokens][top_k] float32, dout_t . y_row, 0 for a pair without a row. */
ar_status_t ar_expert_combine_grad(const void* dout, size_t dout_stride, const void* y,
                                   size_t y_stride, size_t pairs, size_t size, ar_dtype_t dtype,
                                   const int32_t* position, const int32_t* offsets, int experts,
                                   const float* weights, size_t tokens, int top_k, void* dy,
                                   float* dweights, hipStream_t stream);

/* ---- Muon ------------------------------------------------------------------------
 *
 * The step of an optimiser for matrices, beside ar_adamw_*: the momentum is
 * orthogonalised (its singular values brought near 1) before it is applied.
 */

/* One tensor of a Muon plan: `count` matrices of rows x cols, contiguous, one
 * behind the other.
 *   param     AR_FLOAT32 or AR_BFLOAT16, updated in place
 *   grad      AR_FLOAT32 or AR_BFLOAT16, only read
 *   copy      bfloat16 working copy of a float32 param, rewritten by every step;
 *             NULL for none (all tensors of a plan or none)
 *   momentum  float32, updated in place */
typedef struct {
  void* param;
  const void* grad;
  void* copy;
  float* momentum;
  size_t count;
  size_t rows;
  size_t cols;
} ar_muon_tensor_t;

/* Hyperparameters of one step. */
typedef struct {
  double lr;
  double momentum;
  double eps;            /* added to the norm */
  double weight_decay;
  double grad_scale;     /* the gradients' factor, e.g. 1/N for a mean over N ranks */
  double match_rms;      /* 0: s = sqrt(max(1, rows / cols)), for matrices that stand as [out][in];
                          * else s = match_rms sqrt(max(rows, cols)), for either layout */
  int nesterov;
  int ns_steps;          /* 1 to 32 */
} ar_muon_step_t;

/* Bytes of a plan for these tensors; 0 for what ar_muon_plan refuses or when
 * the host runs out of memory. */
size_t ar_muon_plan_bytes(const ar_muon_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                          ar_dtype_t grad_dtype);

/* Writes the plan of these tensors into `plan` (host memory of
 * ar_muon_plan_bytes bytes).  The caller copies all of it to device memory
 * (256-byte aligned) and passes both to ar_muon_step; the device copy also holds
 * the norms, so steps on one plan must be ordered on one stream (or by events).
 * Everything is checked here: AR_ERROR_INVALID_ARGUMENT for NULL or misaligned
 * pointers, copies of some tensors only or of bfloat16 params, a written range
 * that overlaps any other range; AR_ERROR_UNSUPPORTED for other types, a matrix
 * whose sides, each rounded up to a multiple of 128, multiply to more than 2^30
 * or of which one exceeds 4,194,240, or more than 2^22 - 1 tiles (of 64 x 64 at
 * least) in all.  A tensor without elements is skipped. */
ar_status_t ar_muon_plan(const ar_muon_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                         ar_dtype_t grad_dtype, void* plan, size_t bytes);

/* Bytes of device memory (256-byte aligned, any content) for a step on this plan
 * to work in: 8 an element and 8 for each of the shorter sides' squares, all
 * sides rounded up to a multiple of 64, or of 128 from 256 tiles of 128 x 128 in
 * all on (so a matrix of 16 x 4,096 has that of 64 or 128 rows), and up to 34 MB
 * for products whose sums several blocks share. */
size_t ar_muon_workspace(const void* plan);

/* How many of them a step reads or writes: all, or none where every matrix has at
 * most 128 rows and 128 columns.  With none, any address that is aligned so, for
 * instance the device plan's, may be passed as the workspace. */
size_t ar_muon_workspace_used(const void* plan);

/* One step in place, per matrix, with G = grad_scale g:
 *   m' = momentum m + G;   u = G + momentum m' (nesterov) or m'
 *   X = u / (|u| + eps);   ns_steps times: A = X X^T, X = a X + (b A + c A A) X
 *   p' = p - lr (weight_decay p + s X)
 * with (a, b, c) = (3.4445, -4.7750, 2.0315), |u| the root of the sum of squares
 * and X X^T taken over the longer side.  m' and p' are computed in float32 (p'
 * rounded once to param's type, and to bfloat16 in `copy`), |u| in float64; X, A
 * and the polynomial are held in 22 bits and multiplied with float32 sums.  A
 * matrix with a NaN or an infinity in u gets NaN throughout; one of zeros is
 * not moved but by its decay, also where eps is 0.
 * AR_ERROR_INVALID_ARGUMENT: a value that is not finite, lr, eps, weight_decay
 * or match_rms negative, momentum outside [0, 1), ns_steps out of range.
 * May be captured into a graph (a replay repeats the step with these values). */
ar_status_t ar_muon_step(const void* plan, void* device_plan, void* workspace,
                         const ar_muon_step_t* args, hipStream_t stream);

/* ---- testing ---------------------------------------------------------------- */

/* For callers' tests of their AR_ERROR_HIP handling (the error path of the
 * "Errors" paragraph above, which a healthy GPU never takes): the k-th kernel
 * launch the library attempts from now on (k >= 1; a collective call makes
 * one launch, or one per step with AR_IMPL_STEP, or two for the two-launch
 * AllReduces, and none when it is a no-op) reports hipErrorLaunchFailure
 * instead of being enqueued.  That call then returns AR_ERROR_HIP with nothing more enqueued,
 * ar_last_hip_error() gives hipErrorLaunchFailure on its thread, the
 * launches it made before stay enqueued, and the counters are not updated.
 * The injection is spent by that launch; k == 0 disarms it.  Process-wide;
 * host only; AR_ERROR_INVALID_ARGUMENT for k < 0. */
ar_status_t ar_debug_fail_launch(int k);

#ifdef __cplusplus
}
#endif

#endif /* AR_H */
