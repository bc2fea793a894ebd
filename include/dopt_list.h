/*
 * dopt_list.h -- the mixed-precision AdamW step over a list of separate
 * tensors, with fp32 or 8-bit Adam moments.
 *
 * dopt.h steps one rank's windows of flat, bucketed buffers.  The calls here
 * run the same step (unscale, inf/NaN check, global L2 norm and clip, AdamW,
 * copy-back to the 16-bit params, loss scale) over tensors that sit wherever
 * the caller has them: params kept out of the buckets, a job without
 * sharding, or, through dopt_list_from_layout, the rank's param shards of a
 * dopt_layout.  The moments may be held in 8 bits (below), which takes 2
 * bytes per element in place of 8.
 *
 * A dopt_list fixes the tensors' sizes and types.  Grads and params are given
 * by address at every call; the optimizer state is a few flat arrays in one
 * index space, the list's arena, in which tensor i's element j sits at
 * arena_offset(i) + j and every tensor starts on a multiple of
 * DOPT_LIST_BLOCK.  Arena slots between tensors belong to none; after
 * dopt_list_init no call writes them.
 *
 * 8-bit moments (DOPT_STATE_E4M3).  Each tensor is cut into blocks of
 * DOPT_LIST_BLOCK elements from its first; a block has one fp32 scale per
 * moment and every element one OCP e4m3 code per moment (1 sign, 4 exponent,
 * 3 mantissa bits; largest 448, smallest 2^-9):
 *     m = code * scale,     v = (code * scale)^2.
 * The second moment is held by its square root, which the update forms
 * anyway and whose range is half as many octaves.  After an update, with x =
 * m or sqrt(v) in fp32, A = max |x| over the block's elements and cap = 2^127
 * for m, the largest fp32 number below 2^64 for sqrt(v):
 *     scale = min(A, cap) * fp32(1/448), or 0 with codes 0 if A < 2^-100
 *     code  = e4m3(clamp(x * (1 / scale), -448, 448)), nearest, ties to even
 * and a nonzero sqrt(v) takes at least the smallest code, so that a moment
 * that has been seen never divides m by eps alone.  An element is thereby
 * within 2^-4 of its value, or within 2^-10 * scale if that is more (up to
 * 2^-9 * scale for a sqrt(v) raised to the smallest code).  A NaN in a block
 * makes its scale, and so every element of the block, NaN.
 *
 * Over a run, nearest rounding does not follow the grads: an update moves
 * sqrt(v) by (1 - beta2)/2 * (g^2/v - 1) of itself, 0.05% with beta2 = 0.999,
 * and what stays below half a step of its code (3 to 6%) is lost every time,
 * while the scale follows the block's largest element and takes the others with
 * it. Against fp32 moments, Gaussian grads: sqrt(v) is off by 0.63 to 1.6 times
 * (1st to 99th percentile) and stays so; where the grads of half a block fall
 * to a tenth, their sqrt(v) is 8.6 times too large (median) 6500 steps later.
 * DOPT_STATE_E4M3 is thus for a few updates at a time (grads whose size does
 * not move, a state that is loaded, updated and compared).
 *
 * DOPT_STATE_E4M3_SR holds the same codes and scales and is for whole runs: the
 * code is one of the two that x * (1 / scale) lies between, each with the
 * probability that keeps the mean, so that small changes add up.
 * sqrt(v) then stays within 0.7 to 1.4 times that of fp32 moments (1st to 99th
 * percentile) with a mean within 2%, and follows grads that grow or fall. A
 * nonzero sqrt(v) keeps a nonzero code here too. The random numbers are a
 * function of the list's seed (dopt_list_set_seed), the number of the step and
 * the element's place in the arena, and of nothing else: a run that is
 * repeated, resumed from its codes, scales, step count and seed, or replayed
 * from a captured graph takes the same ones, and replicas with one seed stay equal. With k the
 * element's arena index, w word k % 4 of Philox4x32-7 (Salmon, Moraes,
 * Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3, 2011) of counter {k
 * / 4, its high word, t, t's high word} and key {seed, its high word}, t the
 * step count after the step, and u = w mod 2^16 for m, w / 2^16 for sqrt(v):
 *     y = |q| + 2^-6 if |q| < 2^-6 else |q|,   q = clamp(x * (1 / scale), -448, 448)
 *     the bits of y, plus 16 u + 8, without their lowest 20, are those of the code's magnitude (+ 2^-6)
 * An element is thereby within a step of e4m3 of its value (2^-3 of it, or 2^-9 * scale).
 * dopt_list_import rounds to nearest in both kinds.
 *
 * A workspace belongs to the list it was initialised for (dopt_list_init):
 * another list's tables in it would lead the kernels astray.
 *
 * Conventions as in dopt.h: 0 or a negative DOPT_ERR_* code, stream-ordered,
 * nothing allocated on the device, no synchronization unless stated.  Calls
 * that use one workspace must not overlap in time.  dopt_list_stats,
 * _finalize, _prepare, _apply, _step (out == NULL), _export, _import and
 * _set_seed only launch kernels and may be captured into a HIP graph; a replay uses the
 * addresses and hyper-parameters that the captured call was given.  A tensor
 * without a grad in a step has no place in that step's list: a null grad is
 * refused.
 */
#ifndef DOPT_LIST_H
#define DOPT_LIST_H

#include "dopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- how the Adam moments are held ---- */
/* (_SR adds 2, unbiased rounding, to e4m3; fp32 moments have no such form.) */
enum { DOPT_STATE_F32 = 0, DOPT_STATE_E4M3 = 1, DOPT_STATE_E4M3_SR = 3 };

/* Elements per block of an 8-bit moment; every tensor's arena_offset is a multiple. */
#define DOPT_LIST_BLOCK 128

/* One tensor of a list. */
typedef struct dopt_tensor_desc {
    int64_t numel;       /* >= 0 */
    int32_t param_dtype; /* DOPT_F32 / DOPT_BF16 / DOPT_F16 */
    int32_t grad_dtype;
    int32_t hgroup;      /* optimizer param group, 0 <= hgroup < DOPT_MAX_HGROUPS */
    int32_t reserved;    /* 0 */
} dopt_tensor_desc;

typedef struct dopt_list dopt_list;

/*
 * dopt_list_build -- fix a list of n tensors (n >= 0) and how its moments
 * are held.  *out receives a list owned by the library; free it with
 * dopt_list_free.  It is immutable and may be shared by threads.
 * Errors: DOPT_ERR_INVALID (null pointers, n < 0 or n > 2^24, numel < 0, more
 * than 2^38 elements in all, bad dtype, hgroup or state kind), DOPT_ERR_NOMEM.
 */
int dopt_list_build(const dopt_tensor_desc *tensors, int64_t n, int32_t state_kind, dopt_list **out);

/*
 * dopt_list_from_layout -- the list of a rank's param shards: one tensor per
 * param with a shard, in model order, of the shard's length, types and
 * hyper-group.  Tensor i's param and grad are the buffers' arenas at
 * dopt_param_info.arena_offset of its param (dopt_list_tensor_info.param), and
 * the list's export order is the layout's model space (dopt_state_export).
 * Errors as dopt_list_build.
 */
int dopt_list_from_layout(const dopt_layout *layout, int32_t state_kind, dopt_list **out);

void dopt_list_free(dopt_list *list);

typedef struct dopt_list_info {
    int64_t n_tensors;
    int64_t numel;           /* elements over the tensors: length of the export arrays */
    int64_t arena_numel;     /* elements of every state array, a multiple of DOPT_LIST_BLOCK */
    int64_t n_blocks;        /* arena_numel / DOPT_LIST_BLOCK: elements of the scale arrays */
    int64_t workspace_bytes; /* device workspace the calls need (DOPT_PTR_ALIGN-aligned) */
    int64_t stats_record_offset; /* as dopt_stats_record_offset */
    int32_t state_kind;
    int32_t has_master;      /* 1: some param is 16-bit, so a master array is needed */
} dopt_list_info;

typedef struct dopt_list_tensor_info {
    int64_t numel;
    int64_t arena_offset;    /* where the tensor starts in the state arrays */
    int64_t export_offset;   /* where it starts in the export arrays */
    int64_t param;           /* index in the layout's params; -1 for a list of its own */
    int32_t param_dtype, grad_dtype, hgroup, reserved;
} dopt_list_tensor_info;

int dopt_list_query(const dopt_list *list, dopt_list_info *out);
int dopt_list_tensor(const dopt_list *list, int64_t i, dopt_list_tensor_info *out);

/* Device addresses of one tensor: contiguous, aligned to their element.
 * Both may be NULL for a tensor of no elements, and grad also for the calls
 * that read no grads.  No two params of a list may overlap, nor a param any
 * grad or state array. */
typedef struct dopt_list_ptrs {
    const void *grad; /* numel x grad dtype, read only */
    void *param;      /* numel x param dtype, written back */
} dopt_list_ptrs;

/* The optimizer state, device arrays in arena coordinates (DOPT_PTR_ALIGN-aligned). */
typedef struct dopt_list_state {
    float *master;           /* arena_numel fp32; NULL if no param is 16-bit (slots of fp32 params are unused) */
    void *exp_avg;           /* arena_numel: fp32, or e4m3 codes (1 byte each) */
    void *exp_avg_sq;        /* arena_numel: fp32 v, or e4m3 codes of sqrt(v) */
    float *exp_avg_scale;    /* DOPT_STATE_E4M3, _SR: n_blocks fp32; else NULL */
    float *exp_avg_sq_scale; /* DOPT_STATE_E4M3, _SR: n_blocks fp32; else NULL */
} dopt_list_state;

/*
 * dopt_list_init -- master = upcast of the 16-bit params, moments = 0, step
 * count 0, loss scale scaler->initial_scale, seed 0; loads the list's tables into the
 * workspace.  tensors: host array of n_tensors entries.  Synchronizes
 * `stream`.  Errors: DOPT_ERR_INVALID (null or misaligned pointers, bad
 * scaler), DOPT_ERR_HIP.
 */
int dopt_list_init(const dopt_list *list, const dopt_list_ptrs *tensors, const dopt_list_state *state,
                   const dopt_scaler_cfg *scaler, void *workspace, hipStream_t stream);

/*
 * dopt_list_step -- one step: dopt_list_prepare, then dopt_list_apply.  As
 * dopt_step: an inf/NaN grad skips the step (params, state and the step count
 * stay), max_grad_norm <= 0 disables clipping, out (host) may be NULL and
 * otherwise synchronizes `stream`.
 *
 * The parts, with the cross-rank seam of dopt_step_stats: dopt_list_stats
 * forms the grad-stats record {sum of squares, zero count} of this list's
 * grads; dopt_list_finalize takes the step's decision from the record;
 * dopt_list_prepare is both in one; dopt_list_apply updates.
 */
int dopt_list_step(const dopt_list *list, const dopt_list_ptrs *tensors, const dopt_list_state *state,
                   const dopt_hparams *hp, int32_t n_hgroups, double max_grad_norm, void *workspace,
                   hipStream_t stream, dopt_stats *out);
int dopt_list_prepare(const dopt_list *list, const dopt_list_ptrs *tensors, const dopt_hparams *hp,
                      int32_t n_hgroups, double max_grad_norm, void *workspace, hipStream_t stream);
int dopt_list_stats(const dopt_list *list, const dopt_list_ptrs *tensors, void *workspace, hipStream_t stream);
int dopt_list_finalize(const dopt_list *list, const dopt_hparams *hp, int32_t n_hgroups, double max_grad_norm,
                       void *workspace, hipStream_t stream);
int dopt_list_apply(const dopt_list *list, const dopt_list_ptrs *tensors, const dopt_list_state *state,
                    void *workspace, hipStream_t stream);

/*
 * Checkpoint of the state as three fp32 arrays of `numel` elements, the
 * tensors back to back in list order: master (for fp32 params the param), m
 * and v.  A list's 8-bit moments can thus be read into fp32 ones and the
 * reverse, and a dopt_list_from_layout list shares its format with
 * dopt_state_export.  _import also rewrites the params from the master, as the
 * step's copy-back would, and holds m and v in the list's kind (8 bits: as
 * after an update; a negative v is NaN).  The arrays need 4-byte alignment
 * only.  Refused with DOPT_ERR_INVALID: an array that overlaps the state or a
 * param (but for a master array whose elements are the fp32 param's own), and
 * arrays of an _export that overlap one another.  The workspace must have been
 * through dopt_list_init.
 */
int dopt_list_export(const dopt_list *list, const dopt_list_ptrs *tensors, const dopt_list_state *state,
                     float *master, float *exp_avg, float *exp_avg_sq, void *workspace, hipStream_t stream);
int dopt_list_import(const dopt_list *list, const dopt_list_ptrs *tensors, const dopt_list_state *state,
                     const float *master, const float *exp_avg, const float *exp_avg_sq, void *workspace,
                     hipStream_t stream);

/*
 * dopt_list_set_seed -- the seed of a DOPT_STATE_E4M3_SR list's rounding, from the next
 * step on. Errors: DOPT_ERR_INVALID (null or misaligned pointers, a list of
 * another kind), DOPT_ERR_HIP.
 */
int dopt_list_set_seed(const dopt_list *list, uint64_t seed, void *workspace, hipStream_t stream);

/* As dopt_state_scalars_get / _set and dopt_read_stats, of a list's workspace. */
int dopt_list_scalars_get(const dopt_list *list, const void *workspace, hipStream_t stream, dopt_state_scalars *out);
int dopt_list_scalars_set(const dopt_list *list, void *workspace, hipStream_t stream, const dopt_state_scalars *in);
int dopt_list_read_stats(const dopt_list *list, const void *workspace, hipStream_t stream, dopt_stats *out);

#ifdef __cplusplus
}
#endif
#endif
