/*
 * zero_partition.h -- C ABI of libzero_partition.so: one rank's share of a
 * ZeRO-DP optimizer step on an MI355X (gfx950).
 *
 * The method is described on the ZeRO explainer page ("ZeRO: Memory
 * Optimizations Toward Training Trillion Parameter Models", azimuth.plus):
 *   - model-states paragraph: per parameter the model states are an fp16
 *     parameter (2 bytes), an fp16 gradient (2 bytes) and an fp32 Adam state
 *     of master copy, momentum and variance (12 bytes), 16 bytes in all;
 *   - Stage 1 (P_os), Stage 2 (P_os+g) and Stage 3 (P_os+g+p) paragraphs:
 *     which of those kinds each of the N ranks keeps only 1/N of, that a
 *     rank reduces only its own gradient slice (reduce-scatter), updates only
 *     its own partition, and that the updated fp16 parameters are gathered
 *     from every rank afterwards;
 *   - constant-size buffers paragraph (ZeRO-R): small tensors are fused into
 *     one fixed-size buffer that does not grow with the model.
 *
 * Conventions
 *   - Every function returns ZERO_OK (0) or a negative zero_status.  A
 *     thread-local message for the last error is in zero_last_error().
 *   - Arguments are checked before anything is launched or written; on an
 *     argument error no host or device state is modified.  After a
 *     ZERO_ERR_HIP the device state reached by the failed call is undefined.
 *   - fp16 values cross the ABI as uint16_t bit patterns (IEEE binary16).
 *   - "device" pointers point into GPU memory of the current HIP device;
 *     "host" pointers into ordinary host memory.  The caller owns every
 *     buffer it passes; the library keeps no pointer beyond the call except
 *     the tensor tables given to zero_layout_bind_tensors,
 *     zero_layout_bind_contributions, zero_tensor_set_create and
 *     zero_tensor_set_bind_grads.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Device work is ordered on that stream, which must belong to the
 *     current device (a stream of another device is a STATE error).
 *   - Flat indices and sizes are int64_t.
 */
#ifndef ZERO_PARTITION_H
#define ZERO_PARTITION_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_PARTITION_VERSION 10000 /* 1.0.0 */

typedef enum zero_status {
    ZERO_OK = 0,
    ZERO_ERR_INVALID_ARG = -1,    /* a null pointer, a size or index out of range */
    ZERO_ERR_ALIGNMENT = -2,      /* a device pointer lacks the required alignment */
    ZERO_ERR_CAPACITY = -3,       /* an output array is too small; the needed count is reported */
    ZERO_ERR_INDEX_OVERFLOW = -4, /* a size or byte count does not fit in int64 */
    ZERO_ERR_HIP = -5,            /* a HIP runtime call failed; see zero_last_hip_error() */
    ZERO_ERR_OUT_OF_MEMORY = -6,  /* host or device allocation failed, or a table would be too large */
    ZERO_ERR_STATE = -7           /* call not valid in this state (e.g. pack before bind) */
} zero_status;

/* ------------------------------------------------------------------------ */
/* Partition layout (host only; no device work)                             */
/* ------------------------------------------------------------------------ */

/* Opaque layout handle, created by zero_partition_layout and freed by
 * zero_layout_destroy. */
typedef struct zero_layout zero_layout;

/* Summary of a layout.  Per-rank byte counts follow the model-states
 * paragraph (2 + 2 + 4 + 4 + 4 bytes per element) and the stage paragraphs:
 *   stage 0  nothing partitioned (plain data parallelism): every kind over Psi
 *   stage 1  master, momentum, variance over S; fp16 param and grad over Psi
 *   stage 2  additionally the fp16 gradient over S
 *   stage 3  additionally the fp16 parameter over S
 * Replicated kinds count the unpadded Psi, partitioned kinds the padded S. */
typedef struct zero_layout_info {
    int64_t psi;             /* total elements, sum of numel */
    int64_t shard_elems;     /* S = roundup(ceil(psi / n_ranks), align_elems) */
    int64_t padded_elems;    /* n_ranks * S */
    int64_t padding;         /* padded_elems - psi */
    int64_t n_tensors;
    int64_t align_elems;
    int64_t bucket_elems;    /* B; 0 when no bucket plan */
    int64_t n_fills;         /* ceil(psi / B); 0 when B == 0 */
    int64_t n_segments;
    int32_t n_ranks;
    int32_t stage;
    int64_t bytes_param16;   /* per-rank bytes of each kind at this stage */
    int64_t bytes_grad16;
    int64_t bytes_master;
    int64_t bytes_momentum;
    int64_t bytes_variance;
    int64_t bytes_total;
} zero_layout_info;

/* One piece of a tensor that lies inside one shard (and, with a bucket plan,
 * inside one bucket fill).  Segments are sorted by flat_off and tile
 * [0, psi) exactly; zero-sized tensors have no segment. */
typedef struct zero_segment {
    int32_t tensor;      /* index in the tensor list */
    int32_t owner;       /* rank owning this piece: flat_off / S */
    int64_t tensor_off;  /* element offset inside the tensor */
    int64_t flat_off;    /* element offset in the flattened vector */
    int64_t len;         /* elements, > 0 */
    int64_t shard_off;   /* flat_off - owner * S */
    int64_t fill;        /* flat_off / B, or -1 without a bucket plan */
    int64_t bucket_off;  /* flat_off - fill * B, or -1 without a bucket plan */
} zero_segment;

/* Build the layout of a list of tensors flattened in list order (no
 * per-tensor padding) and cut into n_ranks equal shards of S elements.
 *   numel        host, n_tensors sizes (>= 0); may be NULL when n_tensors == 0
 *   n_ranks      N >= 1
 *   stage        0..3 (which kinds are partitioned, for the byte counts)
 *   align_elems  A >= 1: S is a multiple of A
 *   bucket_elems B >= 0: with B > 0 segments are also cut at multiples of B
 *                (the fills of the constant-size bucket)
 *   out          receives the new handle
 * Errors: INVALID_ARG (ranges), INDEX_OVERFLOW (sum of sizes, or 16 * N * S
 * bytes, beyond int64), OUT_OF_MEMORY (more than 2^26 segments). */
int zero_partition_layout(const int64_t* numel, int64_t n_tensors, int32_t n_ranks,
                          int32_t stage, int64_t align_elems, int64_t bucket_elems,
                          zero_layout** out);

int zero_layout_destroy(zero_layout* layout); /* NULL is accepted; frees device tables too */

int zero_layout_get_info(const zero_layout* layout, zero_layout_info* info);

/* Flat offset of every tensor (host, n_tensors entries).  CAPACITY when
 * cap < n_tensors. */
int zero_layout_tensor_offsets(const zero_layout* layout, int64_t* out, int64_t cap);

/* Rank r owns [begin, end); [begin, real_end) are model elements and
 * [real_end, end) padding.  INVALID_ARG unless 0 <= rank < n_ranks. */
int zero_layout_rank_range(const zero_layout* layout, int32_t rank,
                           int64_t* begin, int64_t* real_end, int64_t* end);

/* Segment queries.  *n_out always receives the number of matching segments;
 * they are written to out (host) when cap is large enough, otherwise the call
 * returns CAPACITY and writes nothing (call with cap = 0 to size the array). */
int zero_layout_segments(const zero_layout* layout, zero_segment* out, int64_t cap,
                         int64_t* n_out);
int zero_layout_rank_segments(const zero_layout* layout, int32_t rank, zero_segment* out,
                              int64_t cap, int64_t* n_out);
int zero_layout_fill_segments(const zero_layout* layout, int64_t fill, zero_segment* out,
                              int64_t cap, int64_t* n_out);

/* ------------------------------------------------------------------------ */
/* Contiguous arena for one rank's buffers (memory defragmentation paragraph)*/
/* ------------------------------------------------------------------------ */

/* Buffer kinds of one rank, in the order of zero_arena_plan.offset/bytes. */
enum {
    ZERO_ARENA_PARAM16 = 0,      /* fp16 parameters: S at stage 3, else N*S    */
    ZERO_ARENA_GRAD16 = 1,       /* fp16 gradients: S at stages 2-3, else N*S  */
    ZERO_ARENA_MASTER = 2,       /* fp32 master: S at stages 1-3, else N*S     */
    ZERO_ARENA_MOMENTUM = 3,     /* fp32 momentum, as master                   */
    ZERO_ARENA_VARIANCE = 4,     /* fp32 variance, as master                   */
    ZERO_ARENA_MASTER_ALT = 5,   /* ping-pong alternates, as master            */
    ZERO_ARENA_MOMENTUM_ALT = 6,
    ZERO_ARENA_VARIANCE_ALT = 7,
    ZERO_ARENA_BUCKET = 8,       /* fp16 constant-size bucket: B               */
    ZERO_ARENA_CONTRIB0 = 9,     /* fp16 contribution r at CONTRIB0 + r: S     */
    ZERO_ARENA_KINDS = 25
};

typedef struct zero_arena_plan {
    int64_t total_bytes;                 /* size of the one allocation        */
    int64_t align_bytes;                 /* every buffer starts on a multiple */
    int64_t offset[ZERO_ARENA_KINDS];    /* byte offset, -1 when absent        */
    int64_t bytes[ZERO_ARENA_KINDS];     /* byte size, 0 when absent           */
} zero_arena_plan;

/* Lay out one rank's buffers in a single contiguous block (host only; the
 * caller allocates total_bytes once and carves the buffers).  Element sizes
 * follow the model-states paragraph and the partitioned kinds the stage
 * paragraphs, so the five model-state kinds add up to the page's per-rank
 * bytes (plus padding).  Order: fp32 state, alternates, fp16 gradients,
 * contributions, fp16 parameters, bucket.
 *   pingpong     1: also the alternate master/momentum/variance set
 *   n_contrib    0..16 fp16 contribution buffers of S elements
 *   with_bucket  1: one bucket of B elements (the layout needs a bucket plan)
 *   align_bytes  power of two >= 256 (0: 2 MiB)
 * Errors: INVALID_ARG, STATE (bucket requested without a bucket plan),
 * INDEX_OVERFLOW. */
int zero_arena_plan_for(const zero_layout* layout, int32_t pingpong, int32_t n_contrib,
                        int32_t with_bucket, int64_t align_bytes, zero_arena_plan* out);

/* ------------------------------------------------------------------------ */
/* Bucket pack (constant-size buffers paragraph)                             */
/* ------------------------------------------------------------------------ */

/* Record the device address of every tensor of the layout and upload the
 * gather tables the pack kernel reads (on the current device, ordered on
 * `stream`; the call waits for the upload).
 *   dev_ptrs  host array of n_tensors device pointers to fp16 data, each
 *             2-byte aligned; NULL entries are allowed for zero-sized tensors.
 *             Pointer i must address at least numel[i] elements (the sizes
 *             the layout was built with): the pack reads exactly that many,
 *             and device sizes cannot be checked here.
 * The tensors must stay allocated while the layout is used for packing.
 * Binding again replaces the previous table.  Errors: STATE (layout has no
 * bucket plan), INVALID_ARG, ALIGNMENT, HIP, OUT_OF_MEMORY. */
int zero_layout_bind_tensors(zero_layout* layout, const uint16_t* const* dev_ptrs,
                             void* stream);

/* Write fill `fill` of the bucket: bucket[j] = flat[fill * B + j] for
 * fill * B + j < psi and 0x0000 past the end, where flat is the concatenation
 * of the bound tensors in list order.  A bit copy (NaN payloads, -0 kept).
 *   bucket        device, B elements, 16-byte aligned
 *   packed_elems  optional host output: min(B, psi - fill * B)
 * Asynchronous on `stream`; must run on the device the layout was bound on.
 * Errors: STATE (not bound, or another device), INVALID_ARG (fill outside
 * [0, n_fills), or B above ZERO_MAX_SHARD_ELEMS), ALIGNMENT, HIP. */
int zero_pack_bucket(const zero_layout* layout, int64_t fill, uint16_t* bucket,
                     void* stream, int64_t* packed_elems);

/* ------------------------------------------------------------------------ */
/* Bucket reduce-to-owner (Stage 2 paragraph with the constant-size buffer)  */
/* ------------------------------------------------------------------------ */

/* Record R lists of device tensors, one list per reducing rank, each with
 * the layout's tensor sizes in list order, for zero_reduce_to_owner.
 *   R         1..16
 *   dev_ptrs  host array of R * n_tensors device pointers to fp16 data; row r
 *             (entries r*n_tensors ... r*n_tensors + n_tensors - 1) holds rank
 *             r's tensors; each 2-byte aligned; NULL allowed for empty ones;
 *             each must address at least numel[i] elements, as for
 *             zero_layout_bind_tensors.
 * Uploads the tables on the current device (the call waits for the upload).
 * The tensors must stay allocated while the layout reduces.  Binding again
 * replaces the previous contribution table; the pack binding is separate.
 * Errors: STATE (no bucket plan), INVALID_ARG, ALIGNMENT, HIP, OUT_OF_MEMORY. */
int zero_layout_bind_contributions(zero_layout* layout, int32_t R,
                                   const uint16_t* const* dev_ptrs, void* stream);

/* Owner's share of the reduce of bucket fill `fill`: for every flat index g
 * with fill*B <= g < (fill+1)*B, rank*S <= g < (rank+1)*S and g < psi,
 *   shard[g - rank*S] = fp16( c_0(g) + c_1(g) + ... + c_{R-1}(g) )
 * where c_r is rank r's bound tensor list laid back to back in list order,
 * the sum is formed in fp32 from contribution 0 up and rounded once to fp16
 * (nearest, ties to even); an infinite sum is written as fp16 infinity and a
 * NaN sum as an fp16 NaN (its payload bits are not specified).  Every other
 * element of `shard` is left as it is.
 *   shard    device, the owner's fp16 gradient shard (S values), 2-byte aligned
 *   written  optional host output: elements written (0 when the fill and the
 *            rank's shard do not meet)
 * Asynchronous on `stream`; must run on the device the contributions were
 * bound on.  Errors: STATE (no bucket plan, not bound, another device),
 * INVALID_ARG (fill or rank out of range, B above ZERO_MAX_SHARD_ELEMS),
 * ALIGNMENT, HIP. */
int zero_reduce_to_owner(const zero_layout* layout, int64_t fill, int32_t rank,
                         uint16_t* shard, void* stream, int64_t* written);

/* ------------------------------------------------------------------------ */
/* Fused shard step (Stage 1/2/3 paragraphs: the rank's own partition)        */
/* ------------------------------------------------------------------------ */

/* fp32 shard state of one rank.  Set [cur] is the live state.  When
 * p[1], m[1] and v[1] are all NULL the step runs in place (two passes over
 * the gradients: an overflow check, then the update).  When all three are
 * given the step reads set [cur] and writes set [1 - cur] in one pass, and
 * a taken step flips `cur` (ping-pong mode).  All six pointers are device
 * pointers to shard_elems floats, 16-byte aligned, and the sets may not
 * overlap. */
typedef struct zero_shard_state {
    int64_t shard_elems;   /* S */
    float* p[2];           /* fp32 master parameters */
    float* m[2];           /* fp32 momentum (first moment) */
    float* v[2];           /* fp32 variance (second moment) */
    int32_t cur;           /* live set: 0 or 1 (always 0 in place) */
    int32_t reserved;
    int64_t t;             /* Adam steps taken so far (skipped steps excluded) */
} zero_shard_state;

/* All finite; beta1, beta2 in [0, 1); eps > 0 (with eps = 0 a zero gradient
 * on a zero variance would divide 0 by 0). */
typedef struct zero_adam_hparams {
    float lr;
    float beta1;
    float beta2;
    float eps;
    float weight_decay;    /* L2 term added to the gradient; 0 disables it */
} zero_adam_hparams;

/* Dynamic loss scale.  A step is skipped when any reduced gradient value is
 * inf or NaN: then scale = max(scale * backoff, min_scale), good_steps = 0
 * and no state changes.  A taken step increments good_steps (saturating at INT32_MAX), and when it
 * reaches growth_interval (> 0) the scale is multiplied by growth (kept when
 * that product is not finite) and good_steps reset.
 *
 * scale and min_scale must be at least ZERO_MIN_LOSS_SCALE (2^-24); calls
 * with a smaller value fail with ZERO_ERR_INVALID_ARG.  At or above it
 * 1/scale is finite, and a finite sum of at most 16 fp16 values (below 2^20
 * in magnitude) unscales to |g| < 2^44, whose square stays far inside the
 * fp32 range: a clean step never turns a finite gradient into inf or NaN. */
#define ZERO_MIN_LOSS_SCALE 5.9604644775390625e-08f

/* Largest shard a step call takes, and largest bucket the pack and the
 * reduce-to-owner take (4096 * (2^24 - 1) elements, about 6.9e10): a pass is
 * one launch of 256-thread workgroups of 4096 elements each, and HIP takes
 * fewer than 2^32 work-items per grid dimension, so at most 2^24 - 1 of them.
 * Larger shard_elems (or bucket_elems) fail with ZERO_ERR_INVALID_ARG. */
#define ZERO_MAX_SHARD_ELEMS 68719472640LL
typedef struct zero_loss_scaler {
    float scale;           /* the contributions were multiplied by this */
    float backoff;
    float growth;
    float min_scale;
    int32_t growth_interval;
    int32_t good_steps;
} zero_loss_scaler;

/* One rank's shard step:
 *   sum   = grads[0] + grads[1] + ... + grads[R-1]   (fp16 inputs, fp32
 *           additions in that order)
 *   flag  = any element of sum is inf or NaN (over all S elements)
 *   if flag: skip (no state change), scaler backs off
 *   else, with t = st->t + 1:
 *     g = sum * (1 / scale) [+ weight_decay * p]
 *     m = beta1 * m + (1 - beta1) * g
 *     v = beta2 * v + (1 - beta2) * g * g
 *     p = p - lr * (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *     out_slot = fp16(p), round to nearest even
 *     st->t = t, scaler counts a good step
 *   grads     host array of R device pointers to S fp16 values each,
 *             16-byte aligned (the R contributions to this rank's slice)
 *   R         1..16
 *   out_slot  device, S fp16 values, 2-byte aligned: this rank's slot of the
 *             gather buffer (gather + rank * S)
 *   overflow  host output: 1 if the step was skipped, else 0 (may be NULL)
 * The call returns once the overflow decision is known: the last block of
 * the pass writes it into a pinned host word that the call polls, querying
 * `stream` meanwhile (an error on the stream, or a stream that drains
 * without the word written, ends the wait with an error).  In ping-pong mode
 * the pass may still be retiring when the call returns; in place the call
 * also waits for `stream`.  Everything the call enqueues (the passes, and
 * restoring the slot of a skipped ping-pong step) is ordered on `stream`:
 * order later readers of the state or the slot after it.  Calls on one
 * device are serialised by the library.
 * Errors: INVALID_ARG, ALIGNMENT, STATE, HIP. */
int zero_shard_step(zero_shard_state* st, const uint16_t* const* grads, int32_t R,
                    const zero_adam_hparams* hp, zero_loss_scaler* scaler,
                    uint16_t* out_slot, void* stream, int32_t* overflow);

/* zero_shard_step for callers that cannot allocate memory (code that must
 * not call hipMalloc or hipHostMalloc: tight serving loops, harnesses that
 * forbid allocation).  Same arguments, arithmetic, results, errors and
 * state/scaler updates as zero_shard_step, bit for bit, on the same kernels.
 * What differs: the flag word, the blocks-done counter and the decision word
 * live in a fixed 256-byte device array of the library (one copy per device
 * and process, kept until the process ends) instead of a workspace allocated
 * on a device's first call, and the call clears those words on `stream`
 * (with a one-block kernel),
 * copies the 8-byte decision back into host memory after the pass and waits
 * for `stream` (zero_shard_step instead polls a pinned host word).  The array
 * keeps the last call's contents; calls on one device are serialised by the
 * library within a process, so they never share the words at the same time.
 * The call allocates nothing (no hipMalloc, hipHostMalloc or event) and does
 * not take part in kernel timing.  The words are the same for every shard
 * size: the largest shard is ZERO_MAX_SHARD_ELEMS, as for zero_shard_step.
 * Errors: as zero_shard_step. */
int zero_shard_step_noalloc(zero_shard_state* st, const uint16_t* const* grads, int32_t R,
                            const zero_adam_hparams* hp, zero_loss_scaler* scaler,
                            uint16_t* out_slot, void* stream, int32_t* overflow);

/* Owner step: zero_shard_step in ping-pong mode with the sum taken straight
 * from the contribution lists bound by zero_layout_bind_contributions, so the
 * Stage 2 reduce of the rank's partition and its Stage 1 update are one pass
 * and no fp16 gradient shard is written in between.  With n = the rank's real
 * elements (min(S, psi - rank*S), or 0),
 *   sum(j) = c_0(rank*S + j) + ... + c_{R-1}(rank*S + j)   for j < n
 *   sum(j) = 0                                             for n <= j < S
 * (fp16 values, fp32 additions from contribution 0 up; c_r as for
 * zero_reduce_to_owner; no gradient reaches the padding), the flag, the Adam
 * arithmetic, the slot, the skip and the loss-scale rule are those of
 * zero_shard_step over all S elements: the result equals zero_shard_step fed
 * with the rank's windows of the R flattened lists, zero-filled past the end
 * of the model.  Padding that starts at 0 therefore stays 0 in the live set
 * and the slot, whatever the alternate set held.
 *   layout    bucket plan with contributions bound on the current device
 *   rank      0 .. n_ranks - 1: whose partition is updated
 *   st        ping-pong state (p[1], m[1], v[1] set), shard_elems = the
 *             layout's S; 16-byte aligned, pairwise disjoint, disjoint from
 *             every bound contribution tensor
 *   out_slot  device, S fp16 values, 2-byte aligned (gather + rank * S)
 *   overflow  host output: 1 if the step was skipped, else 0 (may be NULL)
 * Returns once the overflow decision is known (a one-thread kernel after the
 * pass writes it into the pinned host word the call polls, as for
 * zero_shard_step); the pass, and restoring the slot of a skipped step, are
 * ordered on `stream`.  Calls on one device are serialised by the library,
 * together with zero_shard_step.
 * Errors: INVALID_ARG (rank, in-place state, S mismatch, overlap),
 * ALIGNMENT, STATE (no bucket plan, not bound, another device), HIP. */
int zero_owner_step(const zero_layout* layout, int32_t rank, zero_shard_state* st,
                    const zero_adam_hparams* hp, zero_loss_scaler* scaler,
                    uint16_t* out_slot, void* stream, int32_t* overflow);

/* ------------------------------------------------------------------------ */
/* Tensor sets: AdamW over many tensors at once                              */
/* ------------------------------------------------------------------------ */

/* The update of a list of tensors of any sizes (the parameters of a model, or
 * the pieces of them that a rank's shard holds, zero_layout_rank_segments) in
 * one launch, with decoupled weight decay, parameter groups, clipping by the
 * global gradient norm and dynamic loss scaling.  A step is three calls, none
 * of which waits for the device:
 *
 *   zero_grad_sumsq   sum of squares of every gradient value, into device memory
 *                     (several sets and ranks add theirs up: pass accumulate = 1
 *                     for further sets, all-reduce the one double over ranks)
 *   zero_step_begin   decides from it, on the device, whether the step is taken
 *                     and what gradients are multiplied by; counts the step
 *   zero_adamw_step   the update of one set, in place
 *
 * Step count, loss scale and decision live in a zero_step_control in device
 * memory, so the three calls can be captured into a graph and replayed. */

/* Opaque handle, created by zero_tensor_set_create and freed by
 * zero_tensor_set_destroy. */
typedef struct zero_tensor_set zero_tensor_set;

/* Element types of a set's arrays. */
enum {
    ZERO_DTYPE_NONE = 0,
    ZERO_DTYPE_FP16 = 1,
    ZERO_DTYPE_BF16 = 2,
    ZERO_DTYPE_FP32 = 3,
    ZERO_DTYPE_MXFP8 = 4  /* states only, below */
};

#define ZERO_MAX_GROUPS 16
#define ZERO_STATE_BLOCK 32

/* One tensor.  Device pointers; only element alignment is required (4 bytes
 * for p and fp32 states and gradients, 2 for 16-bit ones, 1 for codes and
 * scales).  Pointers of an empty tensor are ignored. */
typedef struct zero_tensor {
    int64_t numel;       /* >= 0 */
    float* p;            /* fp32 master values */
    const void* grad;    /* gradient, grad_type */
    void* m;             /* momentum, state_type */
    void* v;             /* variance, state_type */
    uint8_t* m_scale;    /* MXFP8 only: ceil(numel / 32) scale bytes */
    uint8_t* v_scale;
    void* out;           /* 16-bit copy of p that a step writes, out_type */
    int32_t group;       /* index of the tensor's hyper-parameters, 0..15 */
    int32_t reserved;
} zero_tensor;

/* States in 8 bits (ZERO_DTYPE_MXFP8, the microscaling format MXFP8 E4M3): a
 * block is 32 consecutive elements of a tensor, from its first element on (the
 * last block may be shorter).  Element i of a block with scale byte s stands
 * for e4m3(code[i]) * 2^(s - 127).  An encoder takes the least scale that
 * brings the block's largest magnitude to 448 or below, and at least s = 1
 * (2^-126), so nothing saturates and a block that is decoded and encoded again
 * keeps its values.  All codes zero is the zero state whatever the scales; s = 255
 * is not a scale.
 *
 * A state that a step moves by less than half a unit of its code would be
 * frozen by rounding to nearest.  The variance is such a slow average, so a
 * step rounds v to one of its two neighbours at random, up with the probability
 * (to 2^-16) that keeps the mean, and only ever to zero when it is zero (a lost
 * v would divide a surviving m by eps).  m is rounded
 *   - to nearest, ties to even, where the group's beta1 is at most
 *     ZERO_NEAREST_BETA1.  An m without gradient then falls by a code a step
 *     until it is below 1/14000 of its block's largest, but one that moves
 *     towards a steady gradient stops short of it: at g = constant where
 *     (1 - beta1) |g - m| is half a unit, for beta1 = 0.9 at 0.62 to 0.8 of g
 *     (noise of the gradient's own size takes the mean of m on to g);
 *   - at random, as v is but also to zero, above it: 1.125 beta1 would be
 *     rounded back to 1.125, so an m without gradient would stay while v decays
 *     and the update m / sqrt(v) grow without end;
 *   - at random for every beta1 after zero_tensor_set_m_rounding(set, RANDOM),
 *     which keeps the mean of m there too.
 * The random bits are a function of the set's seed, the tensor's index, the
 * step count and the element (m's others than v's), so a run can be repeated
 * bit for bit.  The update of p uses the new m and v before they are rounded. */
#define ZERO_NEAREST_BETA1 0.9444f /* below 17/18 = 1.0625 / 1.125 */

enum {
    ZERO_M_ROUNDING_AUTO = 0,  /* by the group's beta1, as above */
    ZERO_M_ROUNDING_RANDOM = 1
};

/* Build a set of n tensors.
 *   grad_type   FP16, BF16 or FP32; NONE for a set that only converts states
 *   state_type  FP32 or MXFP8; NONE for a set that only sums squares
 *   out_type    FP16, BF16, or NONE (no 16-bit copies)
 *   seed        of the random rounding of MXFP8 states
 * Of the non-empty tensors, all or none have p, and all or none have grad (none:
 * zero_tensor_set_bind_grads comes first); m and v are set when state_type is
 * not NONE, the scales when it is MXFP8, out when out_type is not NONE, and are
 * NULL otherwise.  No two arrays that a step writes may overlap, nor a gradient
 * one of them.  Tables are uploaded on the current device, ordered on `stream`,
 * and the call waits for that.  The tensors must stay allocated while the set
 * is used, and the set must be kept until the work that uses it has finished
 * (graphs that captured it among it).
 * Errors: INVALID_ARG, ALIGNMENT, INDEX_OVERFLOW, OUT_OF_MEMORY (more than 2^25
 * tiles of 1024 elements, each tensor's first and last one counting as whole),
 * STATE (the stream is being captured, or another device's), HIP. */
int zero_tensor_set_create(const zero_tensor* tensors, int64_t n, int32_t grad_type,
                           int32_t state_type, int32_t out_type, uint32_t seed, void* stream,
                           zero_tensor_set** out);

/* Free a set (NULL is accepted), also while streams are being captured.  Waits
 * for the device.  Errors: HIP (the set is still there: call again later). */
int zero_tensor_set_destroy(zero_tensor_set* set);

/* How steps of a set with MXFP8 states round m (ZERO_M_ROUNDING_AUTO at first).
 * Holds for calls of zero_adamw_step from then on; a captured one keeps what it
 * was captured with.  Errors: INVALID_ARG, STATE (other states). */
int zero_tensor_set_m_rounding(zero_tensor_set* set, int32_t mode);

/* Replace every gradient address (host array of n pointers, as in
 * zero_tensor_set_create).  Ordered on `stream`: calls on it that were enqueued
 * before use the old addresses, later ones (replayed graphs too) the new.
 * Waits for the upload; on an error the old addresses stay.  No other call on
 * the set may run at the same time, nor work that uses it on another stream.
 * Errors: INVALID_ARG, ALIGNMENT, STATE (grad_type is NONE, another device, or
 * the stream is being captured), OUT_OF_MEMORY, HIP. */
int zero_tensor_set_bind_grads(zero_tensor_set* set, const void* const* grads, void* stream);

/* Sum of squares of every gradient value of the set, in fp64, into the device
 * double *sumsq (accumulate = 1: added to it).  The values are summed as they
 * are, with their loss scale.  The order of the sum is fixed by the tensors'
 * sizes and the gradients' type: equal values give equal bits, wherever the
 * tensors are and whatever else the set has.  inf and NaN values give an inf or NaN.
 *   sumsq   device, 8-byte aligned
 *   work    device, zero_grad_sumsq_work_bytes(set) bytes, 8-byte aligned, that
 *           nothing else uses until the call's work is done; may be NULL when
 *           that is 0.  Neither may overlap the other, an array of the set that
 *           a step writes, or (unchecked) a gradient.
 * Asynchronous on `stream`.  Errors: INVALID_ARG, ALIGNMENT, STATE (no
 * gradients, another device), HIP. */
int64_t zero_grad_sumsq_work_bytes(const zero_tensor_set* set);
int zero_grad_sumsq(const zero_tensor_set* set, double* sumsq, int32_t accumulate, void* work,
                    void* stream);

/* State of an optimizer's steps, in device memory (8-byte aligned).  The caller
 * writes t, skipped, scale, lr_mult and good_steps once at the start, and may
 * change lr_mult, scale and t between steps, ordered on the stream; sumsq
 * holds the sum of squares when zero_step_begin runs.  The rest is written by
 * zero_step_begin. */
typedef struct zero_step_control {
    int64_t t;             /* steps taken so far (skipped steps excluded) */
    int64_t skipped;       /* steps skipped so far */
    double sumsq;          /* in: sum of squares of all gradients, with their scale */
    float scale;           /* loss scale that the next gradients carry, >= 2^-24 */
    float lr_mult;         /* every group's lr is multiplied by it (a schedule) */
    int32_t good_steps;    /* taken steps since the scale last changed */
    int32_t skip;          /* out: 1 when the step is skipped, else 0 */
    float norm;            /* out: global norm of the unscaled gradients, 0 unchecked */
    float grad_mult;       /* out: what gradients are multiplied by: clip / scale */
    float group[ZERO_MAX_GROUPS][8];  /* out: the groups' constants for this step */
} zero_step_control;

/* Begin a step.  With S = ctl->scale, and check = 1:
 *   norm = sqrt(ctl->sumsq) / S;  c = max_norm / norm when max_norm > 0 and
 *   norm > max_norm, else 1.  The step is skipped unless norm * c < 2^62 (inf
 *   and NaN skip), c / S is at least 2^-126, S is at least 2^-24 and finite,
 *   lr_mult is finite and t is not negative.
 *   A skipped step leaves t and every tensor as they are.
 * With check = 0 sumsq is not read, norm is 0 and c is 1; max_norm must be 0,
 * and every gradient must be finite and below 2^62 S in magnitude.
 * A taken step counts t up and sets the constants of zero_adamw_step.
 *   groups    host, n_groups hyper-parameters (1..16), read during the call
 *   scaler    host, or NULL for a constant scale: a taken step counts
 *             good_steps, and at growth_interval (> 0) scale is multiplied by
 *             growth (kept when not finite) and good_steps reset; a skipped one
 *             sets scale = max(scale * backoff, min_scale) (min_scale when that
 *             is not finite), good_steps = 0.  Its own scale and good_steps are
 *             ignored.
 * Asynchronous on `stream`.  Errors: INVALID_ARG (as for zero_shard_step),
 * ALIGNMENT, STATE, HIP. */
int zero_step_begin(zero_step_control* ctl, const zero_adam_hparams* groups, int32_t n_groups,
                    float max_norm, int32_t check, const zero_loss_scaler* scaler, void* stream);

/* AdamW over the set's tensors, unless the begun step is skipped:
 *   g = grad_mult * grad
 *   m = beta1 * m + (1 - beta1) * g
 *   v = beta2 * v + (1 - beta2) * g * g
 *   p = p - (lr * weight_decay * p + lr / (1 - beta1^t) * (m / (sqrt(v) / sqrt(1 - beta2^t) + eps)))
 *   out = p rounded to nearest even
 * with the hyper-parameters of the tensor's group and lr * lr_mult for lr, in
 * fp32, one rounding an operation.  With MXFP8 states root and quotient are the
 * hardware's approximations, within 1 ulp each, and v counts as 2^-126 at least
 * under the root.  Several sets can follow one zero_step_begin.
 *   ctl       device, as zero_step_begin left it on this stream
 *   n_groups  as given to zero_step_begin; every tensor's group is below it
 * The set's gradients are part of the sum that a step begun with check = 1 went
 * by.  Asynchronous on `stream`.
 * Errors: INVALID_ARG, ALIGNMENT, STATE (no p, gradients or states, another
 * device), HIP. */
int zero_adamw_step(const zero_tensor_set* set, const zero_step_control* ctl, int32_t n_groups,
                    void* stream);

/* Write src's states to dst, in dst's type: FP32 to MXFP8 (both rounded to
 * nearest, a v above zero not to zero; values must be finite, v not negative)
 * or MXFP8 to FP32 (exact, save where the product leaves fp32's normal range).
 * The sets have the same number of tensors of the same sizes, different state
 * types, and the states do not overlap.  Asynchronous on `stream`.
 * Errors: INVALID_ARG, STATE (no states, another device), HIP. */
int zero_states_convert(const zero_tensor_set* dst, const zero_tensor_set* src, void* stream);

/* ------------------------------------------------------------------------ */
/* Activation checkpoints in 8 bits, and the gradients made from them        */
/* ------------------------------------------------------------------------ */

/* What a rank keeps of its forward pass for the backward one, a byte and a
 * thirty-second a value, and the parameter gradients that it makes from it:
 *
 *   zero_checkpoint_store, _load    a matrix to MXFP8 and back
 *   zero_activation, _grad          an activation that stores the checkpoint of
 *                                   its input in the same pass, and its gradient
 *   zero_weight_grad                the weight and bias gradient of a linear
 *                                   layer from the checkpoint of its input
 *   zero_embedding_lookup, _grad    rows of a table, and the table's gradient
 *
 * Gradients come in fp16, bf16 or fp32, the types that tensor sets read.  The
 * calls are asynchronous on `stream`, hold no state of their own and can be
 * captured into a graph.  Equal inputs give equal bits. */

/* A matrix in device memory: row r's element c is data[r * stride + c].  Only
 * element alignment is required.  A matrix that is read may have any stride >= 0
 * (0: every row the same); one that is written needs stride >= cols.  Pointers
 * of an empty matrix are ignored. */
typedef struct zero_matrix {
    void* data;
    int64_t rows;
    int64_t cols;
    int64_t stride;     /* elements from a row to the next */
    int32_t type;       /* ZERO_DTYPE_FP16, BF16 or FP32 */
    int32_t reserved;
} zero_matrix;

/* A matrix in 8 bits (MXFP8, as for states): blocks of 32 neighbouring values of
 * a row, the last of a row maybe shorter.  Element c of row r with scale byte
 * s = scale[r * B + c / 32] stands for e4m3(code[r * 32 B + c]) * 2^(s - 127), B
 * being ceil(cols / 32).  Storing takes the least s >= 1 that brings the block's
 * largest magnitude to 448 or below, rounds to nearest, ties to even (what is
 * beyond 1.875 2^127 to that), and pads rows of codes with zeros.  A block with
 * an inf or NaN gets s = 255 and codes 0x7F: all of it reads back as NaN.  Other
 * bytes than those that a store writes are not a checkpoint. */
typedef struct zero_checkpoint {
    uint8_t* code;      /* rows * 32 B bytes, 16-byte aligned */
    uint8_t* scale;     /* rows * B bytes */
    int64_t rows;
    int64_t cols;
} zero_checkpoint;

/* Bytes of a checkpoint's codes and scales; either pointer may be NULL.
 * Errors: INVALID_ARG (negative), INDEX_OVERFLOW (more than 2^48 codes, or 2^31
 * columns). */
int zero_checkpoint_bytes(int64_t rows, int64_t cols, int64_t* code_bytes, int64_t* scale_bytes);

/* Store x, and read a checkpoint back (exact in every type but for what leaves
 * its range: fp16 beyond 65504 becomes inf).  Shapes are equal and neither
 * overlaps the other.  Errors: INVALID_ARG, ALIGNMENT, INDEX_OVERFLOW, STATE (the
 * stream is another device's), HIP. */
int zero_checkpoint_store(const zero_matrix* x, const zero_checkpoint* c, void* stream);
int zero_checkpoint_load(const zero_checkpoint* c, const zero_matrix* out, void* stream);

enum {
    ZERO_ACT_RELU = 0,       /* z > 0 ? z : 0 (a NaN stays) */
    ZERO_ACT_SILU = 1,       /* z / (1 + exp(-z)) */
    ZERO_ACT_GELU = 2,       /* z (1 + erf(z / sqrt 2)) / 2 */
    ZERO_ACT_GELU_TANH = 3   /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
};

/* out = act(x), or act(x) * up where `up` is given (a gated layer), computed in
 * fp32 and rounded once; and in the same pass the checkpoints that the backward
 * pass needs: of x, of up where it is given, and of out (as rounded) where
 * `c_out` is, for the weight gradient of the layer that reads it.  c_x may be
 * NULL when nothing is kept (then c_up is NULL too).  x, up and out have one
 * type.  out may be x or up itself (the same place and stride); nothing else may
 * overlap what is written.  Errors: as for zero_checkpoint_store. */
int zero_activation(int32_t kind, const zero_matrix* x, const zero_matrix* up, const zero_matrix* out,
                    const zero_checkpoint* c_x, const zero_checkpoint* c_up, const zero_checkpoint* c_out,
                    void* stream);

/* The gradients of x and up from those of out, with x and up as the checkpoints
 * hold them:
 *   dx = dy * act'(x)    or, gated,    dx = dy * up * act'(x),  dup = dy * act(x)
 * in fp32, rounded once.  c_up and dup come together.  dy, dx and dup have one
 * type; dx or dup may be dy itself.  Errors: as for zero_checkpoint_store. */
int zero_activation_grad(int32_t kind, const zero_matrix* dy, const zero_checkpoint* c_x,
                         const zero_checkpoint* c_up, const zero_matrix* dx, const zero_matrix* dup,
                         void* stream);

/* Gradients of a linear layer y[t, n] = sum_k x[t, k] w[n, k] + b[n] from the
 * gradient of y and the checkpoint of x:
 *   dw[n, k] = sum_t dy[t, n] x[t, k]        bias[n] = sum_t dy[t, n]
 * added to what is there when accumulate is 1.  Sums are in fp32, in an order
 * fixed by the sizes; results are rounded once.  Products are exact for a dy in
 * bf16 or fp32 (what is below 2^-126 in x, and in the low bits of an fp32 dy, is
 * rounded to multiples of 2^-133).  For one in fp16 x is taken in fp16 too, with
 * a common scale for the tokens of each 32 columns, by which the largest of their
 * blocks (448 2^(s - 127) for scale byte s) becomes 57344: blocks down to 2^-22 of
 * that one keep all bits, the values of smaller ones are rounded to multiples of
 * 2^(s - 158).
 *   dy          fp16, bf16 or fp32, T rows, at most 2^40
 *   dw          fp16, bf16 or fp32, n by k; with transposed = 1 it is k by n (for a
 *               weight kept as inputs by outputs)
 *   bias        n values of dw's type, or NULL
 *   work        device, zero_weight_grad_work_bytes() bytes, 16-byte aligned, that
 *               nothing else uses until the call's work is done; may be NULL
 *               when that is 0
 * With T = 0 the sums are zero.  Nothing written may overlap anything else.
 * Errors: as for zero_checkpoint_store. */
int64_t zero_weight_grad_work_bytes(int64_t T, int64_t n, int64_t k, int32_t dy_type);
int zero_weight_grad(const zero_matrix* dy, const zero_checkpoint* x, const zero_matrix* dw, int32_t transposed,
                     void* bias, int32_t accumulate, void* work, void* stream);

/* out[i] = scale * table[tokens[i] - first], in fp32, rounded once.  A token that
 * names no row (tokens[i] - first outside 0 .. rows - 1) gives zeros: padding,
 * or another rank's part of a table cut by rows.
 *   tokens       device, out->rows of them (at most 2^40), int32 or int64 (token_bytes
 *                4 or 8)
 * out may not overlap the others.  Errors: as for zero_checkpoint_store. */
int zero_embedding_lookup(const zero_matrix* table, const void* tokens, int32_t token_bytes, int64_t first,
                          float scale, const zero_matrix* out, void* stream);

/* The table's gradient:
 *   dtable[r] = scale * (sum of dy[i] over the i with tokens[i] - first == r)
 * added to what is there when accumulate is 1 (rows without a token are not
 * touched then, and are zeros otherwise).  Tokens are sorted, each row's sum is
 * taken in fp32 in an order fixed by the tokens, and rounded once.
 *   dy           one row for each token, at most 2^30
 *   dtable       fewer than 2^27 rows
 *   work         device, zero_embedding_grad_work_bytes() bytes, 16-byte aligned,
 *                as for zero_weight_grad
 * Nothing written may overlap anything else.
 * Errors: as for zero_checkpoint_store. */
int64_t zero_embedding_grad_work_bytes(int64_t tokens, int64_t rows, int64_t cols);
int zero_embedding_grad(const zero_matrix* dy, const void* tokens, int32_t token_bytes, int64_t first, float scale,
                        const zero_matrix* dtable, int32_t accumulate, void* work, void* stream);

/* ------------------------------------------------------------------------ */
/* Kernel timing (profiling aid)                                            */
/* ------------------------------------------------------------------------ */

/* Per calling thread.  While enabled (enable != 0), zero_shard_step,
 * zero_owner_step, zero_pack_bucket, zero_reduce_to_owner, zero_grad_sumsq,
 * zero_adamw_step, zero_states_convert and the calls on checkpoints and
 * embeddings time their kernels with a pair of
 * HIP events that the launch itself records at the
 * start of their first kernel and at the end of their last (for
 * zero_shard_step: the fused pass, or the check and update passes in place;
 * for zero_owner_step: the pass, without the one-thread flag hand-over).
 * Those from zero_grad_sumsq on are not timed on a stream that is being
 * captured.
 * The pairs go into a ring of 4096 per thread, so calls can be timed back to
 * back without waiting on the events; enabling or disabling clears it.
 * zero_last_kernel_ms waits for the most recent pair's end event and returns
 * its elapsed milliseconds.  Errors: STATE (nothing recorded since enabling),
 * HIP. */
int zero_set_kernel_timing(int32_t enable);
int zero_last_kernel_ms(float* ms);

/* The elapsed milliseconds of every call timed since timing was enabled
 * (at most the last 4096), oldest first, into ms[0 .. *n); waits for their
 * events.  *n is always set; ms may be NULL when *n is 0.
 * Errors: INVALID_ARG (n NULL), CAPACITY (cap < *n), HIP. */
int zero_kernel_times(float* ms, int64_t cap, int64_t* n);

/* ------------------------------------------------------------------------ */
/* Misc                                                                      */
/* ------------------------------------------------------------------------ */

int zero_version(void);
const char* zero_last_error(void);     /* thread-local, never NULL */
int zero_last_hip_error(void);         /* hipError_t of the last ZERO_ERR_HIP */

/* sizeof of the ABI structs, for binding checks: 0 layout_info, 1 segment,
 * 2 shard_state, 3 adam_hparams, 4 loss_scaler, 5 arena_plan, 6 tensor,
 * 7 step_control, 8 matrix, 9 checkpoint; -1 otherwise. */
int64_t zero_abi_struct_size(int32_t which);

/* Architecture of the current device as a number (gfx950 -> 950) and its
 * memory size in bytes. */
int zero_device_info(int32_t* arch, int64_t* hbm_bytes);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_PARTITION_H */
