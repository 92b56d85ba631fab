/*
 * zero_shard.h -- C ABI of libzero_shard.so: one data-parallel rank's share of
 * a ZeRO-1/2/3 mixed-precision AdamW step on an AMD Instinct MI355X (gfx950).
 *
 * What the step computes comes from these web pages on ZeRO (cited by title
 * and section):
 *   [Z] "【论文解读】ZeRO" (wkq9411.github.io)
 *   [X] "ZeRO 显存优化：ZeRO-1、ZeRO-2 与 ZeRO-3" (xiangdong0520.pages.dev)
 *   [O] operatorworld.com "ai-zero-optimizer-sharding"
 *   [D] "3、ZeRO技术概述：ZeRO三个阶段原理与对比" (5688vip.com DeepSpeed tutorial)
 *   [G] gitcode.csdn.net note on Megatron's distributed optimizer and ZeRO
 *
 * The rank's step, in call order:
 *   zero_shard_layout     which 1/N slice of the flat model state the rank owns
 *   zero_flatten_grads    per-tensor 16-bit grads -> the rank's contiguous shard
 *   zero_grad_sqnorm      local Σg² (fp64) and an inf/NaN flag over the shard
 *                         (zero_flatten_grads_sqnorm does both in one pass)
 *   zero_step_decision    global norm -> clip coefficient, loss scale, skip
 *   zero_adamw_step       fused AdamW on fp32 master/m/v + bf16 param writeback
 *
 * Conventions for every function:
 *   - Status: ZERO_OK (0) or a negative ZERO_ERR_*; zero_last_error() returns
 *     a message for the calling thread's last failure.  A status covers
 *     argument validation and kernel-launch errors only, not kernel results.
 *   - Memory: the caller allocates and frees every buffer (device buffers,
 *     workspace, segment tables).  The library never allocates or frees
 *     device memory.  Its only mutable global state is the per-thread error
 *     message and, for zero_flatten_grads_sqnorm_noalloc, one fixed-size
 *     scratch array per device (a static device variable) and its looked-up
 *     device addresses.
 *   - Device calls are asynchronous: they enqueue kernels on `stream` (a
 *     hipStream_t; NULL = the default stream) and return before completion.
 *   - Device buffers passed to one call must not overlap unless stated.
 *   - Sizes are element counts (int64); n = 0 is a valid no-op.
 */
#ifndef ZERO_SHARD_H
#define ZERO_SHARD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element counts are limited to 2^58 (ZERO_MAX_NUMEL): larger counts are
 * rejected with ZERO_ERR_INVALID, and the size queries return 0 for them. */
#define ZERO_MAX_NUMEL (INT64_MAX / 32)

enum {
  ZERO_OK = 0,
  ZERO_ERR_INVALID = -1,  /* bad argument (null pointer, negative or too large size, rank out of range, ...) */
  ZERO_ERR_CAPACITY = -2, /* caller-provided array too small; the required count is returned */
  ZERO_ERR_HIP = -3       /* the HIP runtime rejected a launch */
};

/* 16-bit floating-point formats.  Passed as a plain int32_t (an enum's size
 * and value range are implementation-defined across C and C++); any other
 * value is rejected with ZERO_ERR_INVALID. */
typedef int32_t zero_dtype;
enum { ZERO_BF16 = 0, ZERO_FP16 = 1 };

/* Message describing the calling thread's most recent failure ("" if none). */
const char* zero_last_error(void);

/* ------------------------------------------------------------------ layout
 *
 * [Z] section 四（一）: the optimizer state is split into N_d equal partitions
 * and rank i keeps and updates partition i; section 六（二） walks the same
 * rule on 8 parameters over 4 GPUs.  [Z] section 二（一） and [O]'s opening
 * equation give the ledger: 2 B param + 2 B grad (fp16/bf16) + 12 B fp32
 * master/m/v = 16 B per parameter; [X] section 三 and [Z] section 八 give the
 * per-rank bytes of DP / ZeRO-1 / ZeRO-2 / ZeRO-3.
 *
 * Reading where the pages assume N_d | Ψ: S = ceil(Ψ/N), every flat buffer
 * is padded with zeros to N·S, rank r owns flat elements [r·S, (r+1)·S).
 */
typedef struct zero_layout {
  int64_t psi;          /* Ψ: total parameters (sum of numels) */
  int64_t padded_numel; /* N·S */
  int64_t shard_numel;  /* S = ceil(Ψ/N) */
  int64_t shard_offset; /* r·S: first flat element of this rank's shard */
  int64_t shard_valid;  /* elements of the shard below Ψ; the rest is padding */
  int32_t world, rank;
  int64_t bytes_dp;     /* 16·Ψ */
  int64_t bytes_zero1;  /* 2·N·S + 2·N·S + 12·S */
  int64_t bytes_zero2;  /* 2·N·S + 14·S */
  int64_t bytes_zero3;  /* 16·S */
  /* Elements this rank sends per training step with ring collectives over the
   * padded flat space ([Z] section 六: a ring reduce-scatter or all-gather of
   * N·S elements sends (N-1)·S per rank; DP all-reduces the gradients (RS +
   * AG); ZeRO-1/2 reduce-scatter the gradients and all-gather the updated
   * parameters; ZeRO-3 also all-gathers the parameters once more, once for
   * forward and once for backward).  Multiply by the element size for bytes. */
  int64_t comm_dp;      /* 2·(N-1)·S */
  int64_t comm_zero1;   /* 2·(N-1)·S */
  int64_t comm_zero2;   /* 2·(N-1)·S */
  int64_t comm_zero3;   /* 3·(N-1)·S */
} zero_layout;

/* One piece of a tensor that lands in the shard. */
typedef struct zero_segment {
  int32_t tensor;     /* index into the tensor list */
  int32_t reserved;   /* 0 */
  int64_t src_offset; /* first element inside the tensor */
  int64_t dst_offset; /* first element inside the shard */
  int64_t numel;      /* > 0 */
} zero_segment;

/* Host only.  Tensors are laid end to end in list order (row-major each).
 * numels[n_tensors] >= 0; world >= 1; 0 <= rank < world; Σ numels <= 2^58.
 * Fills *out and up to segs_cap segments (sorted by dst_offset, contiguous,
 * covering [0, shard_valid)); *n_segs receives the full count.  If segs_cap
 * is too small, returns ZERO_ERR_CAPACITY after filling *out and *n_segs
 * (call again with a larger array).  segs may be NULL when segs_cap == 0. */
int zero_shard_layout(const int64_t* numels, int32_t n_tensors, int32_t world, int32_t rank, zero_layout* out,
                      zero_segment* segs, int32_t segs_cap, int32_t* n_segs);

/* ------------------------------------------------------------------ flatten
 *
 * [Z] section 五（三）: gradients are copied into a pre-allocated contiguous
 * region as they are produced; [Z] section 四（二）: a rank keeps only the
 * reduced gradients of its own partition (the buffer a reduce-scatter lands
 * in); [Z] section 二（二）: gradient norms flatten the gradients first.
 *
 * Device-side segment descriptor (32 bytes): element i of the piece is
 * src[src_offset + i] and goes to shard[dst_offset + i]. */
typedef struct zero_flat_seg {
  const void* src;    /* device address of the source tensor (16-bit elements) */
  int64_t src_offset;
  int64_t dst_offset;
  int64_t numel;
} zero_flat_seg;

/* Host only.  Packs layout segments and tensor base pointers into
 * descriptors: out[k] = {tensor_ptrs[segs[k].tensor], segs[k].src_offset,
 * segs[k].dst_offset, segs[k].numel}.  The caller copies `out` to device
 * memory for zero_flatten_grads. */
int zero_flatten_plan(const zero_segment* segs, int32_t n_segs, const void* const* tensor_ptrs, int32_t n_tensors,
                      zero_flat_seg* out);

/* Host only.  Constant-capacity buckets of the shard ([Z] section 五（二）:
 * fused buffers of a fixed capacity that does not grow with the model;
 * section 四（二）: gradients are bucketed and reduced bucket by bucket as
 * backward produces them).  Writes the parts of the layout's segments that
 * fall in the shard window [win_begin, win_begin + win_numel), with
 * dst_offset relative to the window, so that a bucket is flattened by
 * zero_flatten_grads[_sqnorm] on shard + win_begin with shard_numel =
 * win_numel.  Fills up to cap segments; *n_out receives the full count
 * (ZERO_ERR_CAPACITY when it exceeds cap).  Elements of the window past the
 * layout's shard_valid are padding (no segment covers them). */
int zero_bucket_segments(const zero_segment* segs, int32_t n_segs, int64_t win_begin, int64_t win_numel,
                         zero_segment* out, int32_t cap, int32_t* n_out);

/* Device.  segs_dev: n_segs descriptors in device memory, sorted by
 * dst_offset and non-overlapping, each inside [0, shard_numel).  Writes
 * shard[0, shard_numel): covered elements are bit copies of the source,
 * uncovered ones (padding) are +0.  Never writes outside the shard.  dt only
 * names the 16-bit format (the copy is bitwise).  The body of every piece
 * moves 16-byte vectors to 16-byte aligned destinations; when source and
 * destination differ in their position inside a 16-byte line, each vector is
 * assembled from the two aligned source lines it straddles (reads never leave
 * a 16-byte line that holds bytes of the piece).  Heads and tails shorter
 * than a vector are copied element by element. */
int zero_flatten_grads(const zero_flat_seg* segs_dev, int32_t n_segs, zero_dtype dt, void* shard_dev,
                       int64_t shard_numel, void* stream);

/* Device.  The same copy fused with the square-norm of the copied shard (one
 * pass over the gradients instead of two): writes the shard exactly as
 * zero_flatten_grads does and *sqnorm_dev / *nonfinite_dev exactly as
 * zero_grad_sqnorm would define them (padding contributes +0).  Deterministic
 * for a given shard_numel; the summation tree differs from
 * zero_grad_sqnorm's, so the two sums may differ in the last bits.  ws_dev
 * must hold zero_grad_sqnorm_workspace_bytes(shard_numel) bytes. */
int zero_flatten_grads_sqnorm(const zero_flat_seg* segs_dev, int32_t n_segs, zero_dtype dt, void* shard_dev,
                              int64_t shard_numel, void* ws_dev, size_t ws_bytes, double* sqnorm_dev,
                              int32_t* nonfinite_dev, void* stream);

/* Device.  For callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same fused flatten and norm as zero_flatten_grads_sqnorm, with the same
 * results bit for bit, but with its partials in a static scratch array of
 * ZERO_NOALLOC_SCRATCH_BYTES (6 MiB) per device instead of a caller
 * workspace.  That covers every shard size; a shard needing more scratch
 * than the array holds would be refused with ZERO_ERR_CAPACITY.  It calls no
 * allocating routine.  On its first call on a device the array's device
 * address is looked up (hipGetSymbolAddress) with that device current, so
 * call it with the stream's device current (a stream of another device is
 * refused with ZERO_ERR_INVALID).  Every call on one device shares that
 * device's array: calls that overlap in time on one device (two streams, two
 * threads) race on it and give wrong sums; serialize them.  The array keeps
 * the last call's partials; no call relies on its earlier contents (every
 * partial is written before it is read).  sqnorm_dev: 8-byte aligned;
 * nonfinite_dev: 4-byte aligned. */
#define ZERO_NOALLOC_SCRATCH_BYTES ((size_t)6 << 20)
int zero_flatten_grads_sqnorm_noalloc(const zero_flat_seg* segs_dev, int32_t n_segs, zero_dtype dt, void* shard_dev,
                                      int64_t shard_numel, double* sqnorm_dev, int32_t* nonfinite_dev, void* stream);

/* Bucketed norm.  With the shard split into constant-capacity windows
 * (zero_bucket_segments), each window is flattened as soon as its gradients
 * exist and leaves its per-workgroup partial square-sums and non-finite flags
 * side by side with the other windows'; one zero_sqnorm_reduce then folds
 * them all (fixed order: window by window, workgroup by workgroup), so a
 * bucket costs one launch.
 *
 * zero_flatten_partials_count: partials that zero_flatten_grads_partials
 * writes for a window of numel elements (0 for numel = 0).  Not monotone in
 * numel: size a shared partials buffer by summing the counts.
 *
 * zero_flatten_grads_partials (device): flattens the window exactly as
 * zero_flatten_grads does (dst_dev = the window's first shard element) and
 * writes the window's partials to part_sum_dev[0 .. count) (double, 8-byte
 * aligned) and part_flag_dev[0 .. count) (uint32, 4-byte aligned).  No final
 * reduction.
 *
 * zero_sqnorm_reduce (device): folds count partials into *sqnorm_dev and
 * *nonfinite_dev (0 or 1) in a fixed order (deterministic for a given
 * count), exactly as zero_flatten_grads_sqnorm folds its own.  Past 65536
 * partials the fold takes two levels and overwrites the partials: they are
 * scratch once reduced. */
int64_t zero_flatten_partials_count(int64_t numel);
int zero_flatten_grads_partials(const zero_flat_seg* segs_dev, int32_t n_segs, zero_dtype dt, void* dst_dev,
                                int64_t numel, double* part_sum_dev, uint32_t* part_flag_dev, void* stream);
int zero_sqnorm_reduce(double* part_sum_dev, uint32_t* part_flag_dev, int64_t count, double* sqnorm_dev,
                       int32_t* nonfinite_dev, void* stream);

/* ------------------------------------------------------------------ grad norm
 *
 * [G] table "AdamW全局grad_norm": inside optimizer.step() the global L2 norm
 * of the gradients is all-reduced before clipping and sets the clip
 * coefficient.  This call computes one rank's part: Σ g_j² over its shard,
 * accumulated in fp64 (each square is exact), and flags any element whose
 * exponent field is all ones (inf or NaN; bf16 0x7F80 mask, fp16 0x7C00).
 *
 * Deterministic: a fixed grid and fixed reduction tree give the same bits on
 * every run for the same n and pointer alignment.  The summation order is not
 * sequential, so results differ from a sequential fp64 sum by rounding only.
 * ws_dev: caller workspace of at least zero_grad_sqnorm_workspace_bytes(n)
 * bytes, 16-byte aligned.  Writes *sqnorm_dev (double) and *nonfinite_dev
 * (int32, 0 or 1); when the flag is set the sum is unspecified. */
size_t zero_grad_sqnorm_workspace_bytes(int64_t n);
int zero_grad_sqnorm(const void* shard_dev, zero_dtype dt, int64_t n, void* ws_dev, size_t ws_bytes,
                     double* sqnorm_dev, int32_t* nonfinite_dev, void* stream);

/* ------------------------------------------------------------------ host decision
 *
 * [G]: global norm -> clip coefficient.  The pages enable fp16 training
 * ([D] configuration) without describing loss scaling; readings:
 *   global = Σ_r rank_sqnorms[r] in rank order (the all-reduce's sum);
 *   nonfinite = OR of rank_flags;
 *   if nonfinite: *skip = 1, no update, *loss_scale halves, good steps reset;
 *   else: norm = sqrt(global / loss_scale²);
 *         coef = min(1, max_norm / (norm + 1e-6)) (max_norm <= 0: coef = 1);
 *         *grad_scale = coef / loss_scale; then growth_interval consecutive
 *         good steps double *loss_scale.
 * *global_norm receives the unscaled norm (NaN/inf when skipped).  For bf16
 * training pass loss_scale = 1 and growth_interval = INT32_MAX.
 * A loss scale that is not a positive finite number, or one so small that
 * loss_scale² underflows and the unscaled square-norm of a step without
 * overflow is not finite (after a long run of halvings), is refused with
 * ZERO_ERR_INVALID and nothing is written. */
int zero_step_decision(const double* rank_sqnorms, const int32_t* rank_flags, int32_t n_ranks, double max_norm,
                       double* loss_scale, int32_t* good_steps, int32_t growth_interval, double* grad_scale,
                       int32_t* skip, double* global_norm);

double zero_clip_coef(double global_sqnorm, double max_norm);
int zero_loss_scale_update(double* scale, int32_t nonfinite, int32_t* good_steps, int32_t growth_interval);
/* Half-cosine learning rate from lr_max at t = 1 to lr_min at t = total (reading). */
double zero_cosine_lr(int64_t t, int64_t total, double lr_max, double lr_min);

/* ------------------------------------------------------------------ AdamW
 *
 * [Z] section 四（一）: rank i updates only its partition of the optimizer
 * state and parameters, then parameters are all-gathered; [O] opening
 * equation and [Z] section 二（一）: bf16/fp16 weights and grads with fp32 m,
 * v and master weights.  The pages name AdamW ([O], [G]) but print no update
 * equations.  Reading: bias-corrected Adam with decoupled weight decay
 * p·(1 − lr·wd); host scalars are computed in fp64 and rounded once to fp32:
 *   b1 = β1, omb1 = 1−β1, b2 = β2, omb2 = 1−β2, eps, decay = 1 − lr·wd,
 *   step_size = lr / (1 − β1^t), bc2_sqrt = sqrt(1 − β2^t), gscale = grad_scale.
 * Per element, in fp32, round-to-nearest-even, no fused multiply-add, in
 * this order:
 *   g = gscale·g
 *   m = (b1·m) + (omb1·g)
 *   v = (b2·v) + (omb2·(g·g))
 *   d = ((sqrt(v) / bc2_sqrt) + eps)
 *   p = (p·decay) − (step_size·(m/d))
 *   param = p rounded to the parameter format pdt, nearest, ties to even:
 *           bf16, or IEEE binary16 for fp16 parameters ([Z] section 四（一）
 *           keeps fp16 parameters and gradients whole on every process; [D]
 *           trains with fp16 enabled); binary16 overflows to infinity and
 *           keeps subnormals.  NaN stays NaN.
 */
typedef struct zero_adamw_hparams {
  double lr;           /* >= 0 */
  double beta1, beta2; /* in [0, 1) */
  double eps;          /* >= 0 */
  double weight_decay; /* >= 0 */
  double grad_scale;   /* finite: clip coefficient / loss scale */
  int64_t step;        /* 1-based Adam step t */
} zero_adamw_hparams;

/* Device.  grad_dev: n gradients (bf16 or fp16, per gdt); master/m/v: n fp32
 * each, updated in place; param_dev: n 16-bit parameters in format pdt
 * (ZERO_BF16 or ZERO_FP16), written (never read).  Buffers
 * must be aligned to their element size.  When grad and param are 8-byte
 * aligned and master/m/v 16-byte aligned the kernel streams whole vectors;
 * otherwise (and for the last n mod 4 elements) it updates element by
 * element with identical results. */
int zero_adamw_step(const void* grad_dev, zero_dtype gdt, float* master_dev, float* m_dev, float* v_dev,
                    uint16_t* param_dev, zero_dtype pdt, int64_t n, const zero_adamw_hparams* hp, void* stream);

/* Tiled optimizer state: the same fp32 master / m / v, interleaved in tiles of
 * ZERO_STATE_TILE elements.  Tile k holds master[T·k .. T·k+T), then m[...],
 * then v[...] (T = ZERO_STATE_TILE, 12·T = 12 KiB per tile), so the update
 * streams three address ranges (grad, state, param) instead of five; on
 * MI355X the tiled update runs about 6% faster than the separate-array one
 * (6.66 against 6.27 TB/s on a 1.95e8-element shard).  A shard of n
 * elements needs zero_state_tiled_numel(n) floats (the last tile is padded).
 * zero_adamw_step_tiled computes exactly what zero_adamw_step computes (same
 * per-element operations, same bits); state_dev must be 16-byte aligned. */
#define ZERO_STATE_TILE 1024
int64_t zero_state_tiled_numel(int64_t n);
int zero_adamw_step_tiled(const void* grad_dev, zero_dtype gdt, float* state_dev, uint16_t* param_dev,
                          zero_dtype pdt, int64_t n, const zero_adamw_hparams* hp, void* stream);
/* Device bit copies between separate master/m/v arrays and the tiled state
 * (for initialisation and checkpoints); padding floats are left untouched.
 * All four buffers must be 4-byte aligned; NULL buffers (n > 0), n outside
 * [0, ZERO_MAX_NUMEL] or misalignment give ZERO_ERR_INVALID. */
int zero_state_tile(const float* master_dev, const float* m_dev, const float* v_dev, float* state_dev, int64_t n,
                    void* stream);
int zero_state_untile(const float* state_dev, float* master_dev, float* m_dev, float* v_dev, int64_t n, void* stream);

/* ------------------------------------------------------------------ device-resident decision
 *
 * The same decision (zero_step_decision) and scalar derivation (zero_adamw_step)
 * evaluated by one GPU thread, so a step needs no host round trip between the
 * norm and the update: flatten+norm -> zero_step_decision_dev ->
 * zero_adamw_step_[tiled_]dev, all enqueued back to back on one stream (and
 * capturable in a HIP graph: no memset, copy or host callback is involved).
 * The state lives in caller-allocated device memory; read it back at will.
 * The fp64 host arithmetic of the decision is repeated on the device with the
 * same IEEE operations (correctly rounded +, -, *, /, sqrt); beta^t uses the
 * device pow, which can differ from the host's in the last fp64 bit (then an
 * fp32 scalar may differ by one ulp, in about 1 of 10^9 steps). */
typedef struct zero_step_state {
  double loss_scale;      /* current dynamic loss scale */
  double global_norm;     /* unscaled global norm of the last decided step (NaN if skipped) */
  double grad_scale;      /* factor of the last decided step: coef / loss scale (0 if skipped) */
  int64_t adam_step;      /* Adam t of the last applied update */
  int64_t iteration;      /* steps decided so far, skipped or not */
  int32_t good_steps;     /* consecutive good steps since the last scale change */
  int32_t growth_interval;
  int32_t skip;           /* 1: the last decided step is skipped (the update kernels do nothing) */
  int32_t error;          /* 0, or ZERO_STEP_ERR_LOSS_SCALE for the last decided step */
  float scalars[12];      /* fp32 b1, 1-b1, b2, 1-b2, eps, 1-lr*wd, lr/(1-b1^t), sqrt(1-b2^t), gscale, 0, 0, 0 */
} zero_step_state;

/* The decision could not be taken: the loss scale is not a positive finite
 * number, or loss_scale² underflowed so that the unscaled square-norm of a
 * step without overflow is not finite (the cases zero_step_decision refuses
 * with ZERO_ERR_INVALID).  The step is skipped (skip = 1, grad_scale = 0,
 * global_norm = NaN); loss scale, good steps and Adam t are left as they
 * are.  The next decision sets error back to 0 if it can be taken. */
#define ZERO_STEP_ERR_LOSS_SCALE 1

/* Device.  Writes the initial state (loss scale, growth interval >= 1, t = 0,
 * error 0) with a one-thread kernel.  state_dev: 16-byte aligned. */
int zero_step_state_init(zero_step_state* state_dev, double loss_scale, int32_t growth_interval, void* stream);

/* Device.  rank_sqnorms_dev[n_ranks] (double) and rank_flags_dev[n_ranks]
 * (int32) as written by zero_grad_sqnorm / zero_flatten_grads_sqnorm; hp
 * supplies lr, beta1, beta2, eps and weight_decay (hp->step and
 * hp->grad_scale are ignored: t and the factor come from the state and the
 * decision).  Updates *state_dev as described above. */
int zero_step_decision_dev(const double* rank_sqnorms_dev, const int32_t* rank_flags_dev, int32_t n_ranks,
                           double max_norm, const zero_adamw_hparams* hp, zero_step_state* state_dev, void* stream);

/* Device.  zero_adamw_step / zero_adamw_step_tiled with the scalars taken
 * from the device state; when state_dev->skip is set the kernels return
 * without touching memory. */
int zero_adamw_step_dev(const void* grad_dev, zero_dtype gdt, float* master_dev, float* m_dev, float* v_dev,
                        uint16_t* param_dev, zero_dtype pdt, int64_t n, const zero_step_state* state_dev,
                        void* stream);
int zero_adamw_step_tiled_dev(const void* grad_dev, zero_dtype gdt, float* state_dev, uint16_t* param_dev,
                              zero_dtype pdt, int64_t n, const zero_step_state* step_state_dev, void* stream);

/* ------------------------------------------------------------------ lists of tensors
 *
 * The norm and the update over many tensors at once, where they lie: the
 * gradients are read from their own buffers and the parameters written to
 * theirs, with no flat copy in between (a list's step moves 30 B/param, the
 * flattened one 32).  A list can hold whole tensors (data parallelism without
 * sharding) or a rank's pieces of them (zero_shard_layout's segments).  The
 * tensors of a list may differ in size, format, state layout and group.
 * Calls are made with the device that holds the tensors current.  Host scalars
 * (zero_list_adamw*_step) are fixed in a captured graph; the _dev forms read
 * theirs at every replay.
 *
 *   zero_list_plan            checks a list and builds its device table
 *   zero_list_grad_sqnorm     fp64 sum of squares and inf/NaN flag
 *   zero_list_decision_dev    the decision, with the scalars of every group
 *   zero_list_adamw_step      AdamW with fp32 state
 *   zero_list_adamw8_step     AdamW with the moments held in 8 bits
 *   zero_list_state8_pack     fp32 moments -> 8 bits; _unpack: back
 */

/* Third format, of gradients and parameters in lists only. */
enum { ZERO_FP32 = 2 };

/* How a tensor's optimizer state is laid out. */
enum {
  ZERO_STATE_NONE = 0,   /* no state (norm only): state, m, v NULL */
  ZERO_STATE_ARRAYS = 1, /* state = fp32 master[numel], m[numel], v[numel]; 4-byte aligned */
  ZERO_STATE_TILED = 2,  /* state = zero_state_tiled_numel(numel) floats, 16-byte aligned; m, v NULL */
  ZERO_STATE_8BIT = 3    /* state = zero_state8_bytes(numel) bytes, 16-byte aligned; m, v NULL */
};

/* 8-bit state.  Moments are held in blocks of ZERO_STATE8_BLOCK elements with
 * one fp32 scale per block and moment:
 *   m = value4(code) * scale:  sign, 4 exponent and 3 fraction bits with
 *       subnormals (the OCP e4m3 format: bias 7, largest 448);
 *   v = value5(code) * scale:  5 exponent and 3 fraction bits, no sign, with
 *       subnormals (bias 31, largest 1.875): 32 octaves, as the second moment
 *       is a square.
 * The fp32 master stays.  A tile of ZERO_STATE8_TILE elements holds
 *   float master[4096]; uint8 m[4096]; uint8 v[4096]; float m_scale[16];
 *   float v_scale[16];                                  (24,704 bytes)
 * and a tensor's last tile is padded; padding is never written.
 *
 * Encoding a block (updates and pack): peak = the largest |m| (v) of the
 * block; a block whose peak is below 2^-110 is held as zeros, scale 0.
 * scale = peak / 448 (peak / 1.875, by a multiplication with the fp32
 * reciprocal of the constant), and x·(448/peak) (1.875/peak) is rounded to a
 * code.  A v that is not zero never takes code 0.  A NaN or infinity in a
 * block makes its scale NaN or infinite: the whole block then reads as not
 * finite (a step whose norm flagged it is to be skipped, as ever).  Packing
 * takes the magnitude of a v.
 *   Updates round stochastically: position p between two codes k and k+1 goes
 * to k+1 with probability p - k, so the expected value is the value, except for
 * a v below code 1 that is not zero, which is held as code 1.  With rounding to
 * nearest the second moment could grow but never decay: a step shrinks it by
 * at most 1 - beta2 of itself (0.1% at beta2 = 0.999), far below half the
 * distance of two codes (3 to 6%).  The dither is a counter hash, the same for the same arguments:
 *   base = mix(seed + G·t), key(b) = mix(base + G·(b + 1)), all mod 2^64,
 *   mix = SplitMix64's output function, G = 0x9E3779B97F4A7C15, t the Adam step,
 *   b = the block's number in the list (every tensor counts whole tiles: 16
 *   blocks each), and r(j) = (key(b) + j·0x9E3779B9) mod 2^32 for element j of
 *   the block: m takes the upper 20 bits of r, v the lower 20.
 *   Pack rounds to nearest. */
#define ZERO_STATE8_BLOCK 256
#define ZERO_STATE8_TILE 4096
/* Bytes of the 8-bit state of n elements (0 for n <= 0 or n > ZERO_MAX_NUMEL). */
int64_t zero_state8_bytes(int64_t n);

/* One tensor (or piece) of a list. */
typedef struct zero_list_tensor {
  const void* grad;  /* numel gradients in format gdt; NULL: no gradient in this step, the tensor is left as it is
                      * (Adam's t is the list's, not the tensor's: it counts the step all the same) */
  void* param;       /* numel parameters in format pdt, written by the updates (never read); NULL: none */
  void* state;       /* see the layouts above */
  float* m;          /* ZERO_STATE_ARRAYS only */
  float* v;
  int64_t numel;     /* in [0, 2^40] */
  zero_dtype gdt;    /* ZERO_BF16, ZERO_FP16 or ZERO_FP32 */
  zero_dtype pdt;
  int32_t layout;    /* ZERO_STATE_* */
  int32_t group;     /* which hyper-parameters: in [0, n_groups) */
} zero_list_tensor;

#define ZERO_LIST_MAX_GROUPS 64

/* A planned list, filled by zero_list_plan.  Host memory, the caller's.  Only
 * table_dev is for the caller to set: the device address of its copy of the
 * table (16-byte aligned), which must stay as planned while calls use it. */
typedef struct zero_list {
  const void* table_dev;
  int64_t table_bytes;   /* size of the table */
  int64_t grads_bytes;   /* its leading part, all that zero_list_repoint changes */
  int64_t numel;         /* elements of all tensors */
  int64_t norm_blocks;   /* workgroups of the norm */
  int64_t update_blocks; /* workgroups of the update (0 without state) */
  int64_t norm_offset;   /* where the table's parts begin, in bytes */
  int64_t update_offset;
  uint64_t shape;        /* fingerprint of the tensors' sizes */
  uint64_t check;        /* over the fields above but table_dev: a list that was not planned is refused */
  int32_t n_tensors;
  int32_t n_groups;
  int32_t state;         /* 0: none, 32: fp32 (arrays, tiled or both), 8: 8-bit */
  int32_t flags;         /* ZERO_LIST_* */
} zero_list;
enum {
  ZERO_LIST_HAS_PARAMS = 1, /* every tensor has a param */
  ZERO_LIST_WHOLE_STATE = 2 /* every tensor has master, m and v */
};

/* Host only.  Bytes of the table of these tensors (only the sizes and layouts
 * are looked at); 0 if they are not valid. */
int64_t zero_list_table_bytes(const zero_list_tensor* tensors, int32_t n_tensors);

/* Host only.  Checks the list, fills *out (table_dev NULL) and writes the
 * table to table_host (table_bytes >= zero_list_table_bytes, else
 * ZERO_ERR_CAPACITY), which the caller copies to the device.
 * Refused (ZERO_ERR_INVALID): unknown formats or layouts, fp32 and 8-bit
 * state in one list, buffers not aligned to their element size (tiled and
 * 8-bit state: 16 bytes), sizes or groups out of range, a state buffer
 * missing, and any overlap of a buffer that an update writes (state, params)
 * with another buffer of the list; gradients may share memory.
 *   With ZERO_STATE_ARRAYS any of state, m and v may be NULL: such a list can
 * only be the source or target of a conversion (a NULL target part is not
 * written, a NULL source part reads as zeros).  Tensors of no elements are
 * valid and are passed over.  A list holds at most 2^23 chunks of 16,384
 * elements, counted by tensor. */
int zero_list_plan(const zero_list_tensor* tensors, int32_t n_tensors, int32_t n_groups, void* table_host,
                   int64_t table_bytes, zero_list* out);

/* Host only.  The same list with other addresses (the next step's gradients,
 * some of them perhaps NULL): checks it and rewrites the first
 * list->grads_bytes bytes of table_host, which the caller copies over the
 * device table's.  Sizes, layouts and groups must be the planned ones. */
int zero_list_repoint(const zero_list_tensor* tensors, int32_t n_tensors, void* table_host, int64_t table_bytes,
                      const zero_list* list);

/* Device.  What zero_grad_sqnorm does, over the gradients of every tensor that
 * has one.  Deterministic for a given list.  ws_dev: 16-byte aligned, at least
 * zero_list_grad_sqnorm_workspace_bytes(list) bytes; calls that may overlap in
 * time need a workspace each. */
size_t zero_list_grad_sqnorm_workspace_bytes(const zero_list* list);
int zero_list_grad_sqnorm(const zero_list* list, void* ws_dev, size_t ws_bytes, double* sqnorm_dev,
                          int32_t* nonfinite_dev, void* stream);

/* Device.  zero_adamw_step's operations, bit for bit, on every tensor that has
 * a gradient; hp[list->n_groups] on the host, one for each group (the
 * parameter is rounded to its format as ever, ZERO_FP32 takes the master).
 * The list must have params and whole fp32 state. */
int zero_list_adamw_step(const zero_list* list, const zero_adamw_hparams* hp, void* stream);

/* Device.  The same with 8-bit state: the moments are decoded, take
 * zero_adamw_step's operations bit for bit and are encoded again; master and
 * parameter come from the new moments before they are rounded.  The step that
 * the master takes may differ from zero_adamw_step's by 14·2^-24 of itself and
 * its rounding by one unit (hardware root and reciprocals, 1 ulp each, and
 * fused products; a second moment below 2^-126 may count as 0 under the root).
 * eps >= 1e-16 for every group (a second moment whose block is held as zeros
 * reads as 0).  Every group's hp must have the same step, which with seed sets
 * the dither. */
int zero_list_adamw8_step(const zero_list* list, const zero_adamw_hparams* hp, uint64_t seed, void* stream);

/* Scalars of one group on the device: those of zero_step_state. */
typedef struct zero_group_scalars {
  float scalars[12];
} zero_group_scalars;

/* Device.  zero_step_decision_dev for n_groups groups: the same decision into
 * *state_dev (whose own scalars become group 0's), and, unless the step is
 * skipped, the scalars of every group into groups_dev[n_groups] (16-byte
 * aligned).  hp[n_groups] on the host: lr, beta1, beta2, eps and weight_decay
 * are used, and are fixed in a captured graph.  n_groups in
 * [1, ZERO_LIST_MAX_GROUPS]. */
int zero_list_decision_dev(const double* rank_sqnorms_dev, const int32_t* rank_flags_dev, int32_t n_ranks,
                           double max_norm, const zero_adamw_hparams* hp, int32_t n_groups,
                           zero_step_state* state_dev, zero_group_scalars* groups_dev, void* stream);

/* Device.  The updates with the scalars and the Adam step taken from the
 * device (groups_dev[list->n_groups]); when state_dev->skip is set they return
 * without touching memory.  With 8-bit state an eps below 1e-16 counts as
 * 1e-16. */
int zero_list_adamw_step_dev(const zero_list* list, const zero_step_state* state_dev,
                             const zero_group_scalars* groups_dev, void* stream);
int zero_list_adamw8_step_dev(const zero_list* list, const zero_step_state* state_dev,
                              const zero_group_scalars* groups_dev, uint64_t seed, void* stream);

/* Device.  Conversion between a list with fp32 state and a list of the same
 * sizes with 8-bit state (masters are copied; gradients and parameters are not
 * touched).  The two lists' states must not overlap. */
int zero_list_state8_pack(const zero_list* from32, const zero_list* to8, void* stream);
int zero_list_state8_unpack(const zero_list* from8, const zero_list* to32, void* stream);

/* ------------------------------------------------------------------ the ends of a model
 *
 * Where the gradients come from that the step above takes, at the two ends of
 * a language model and at its norms: the token embedding with its table's
 * gradient, layer norm with its backward pass, and the softmax cross entropy
 * of the output head, whose gradients carry the loss scale that
 * zero_step_state holds on the device.  Weight gradients are written where
 * the flatten or a list of tensors reads them, in a format of their own,
 * replacing what is there or added to it (a table that is also the head; the
 * micro-batches of one step).
 *
 *   zero_embed_forward        rows of a table for tokens, scaled
 *   zero_embed_grad           the table's gradient, by sorted tokens
 *   zero_layernorm_forward    layer norm, with or without the mean
 *   zero_layernorm_grad       its three gradients
 *   zero_loss_head            losses of the head, without keeping its scores
 *   zero_loss_head_grad       the same, and both gradients
 *
 * Sums and statistics are held in fp32; each result is rounded once to its
 * format, and every sum has one order: the same arguments give the same bits.
 * Calls are made with the device that holds the buffers current.  A workspace
 * belongs to one call at a time; what it holds between calls is of no
 * meaning, so it needs no initial value.  What a call writes overlaps nothing
 * else of it, but that y may be x, and x_grad x or y_grad, the same rows at the
 * same place. */

/* Rows in device memory: row r begins at element r·stride of data.  cols >= 1,
 * rows and cols at most 2^31 - 1, stride >= cols, rows·stride <= 2^40.  data
 * is aligned to its elements (no more is needed; rows of whole 16-byte lines
 * are fastest) and may be NULL where rows = 0. */
typedef struct zero_rows {
  void* data;
  int64_t rows;
  int64_t cols;
  int64_t stride;
  zero_dtype dt;    /* ZERO_BF16, ZERO_FP16 or ZERO_FP32 */
  int32_t reserved; /* 0 */
} zero_rows;

/* Device.  out[t] = scale · table[ids[t] - first_row], rounded to out's
 * format, for out->rows tokens; zeros where that row is not one of the
 * table's (a rank that holds a slice of the vocabulary adds up the slices'
 * outputs).  id_bytes: 4 (int32) or 8 (int64).  scale: finite in fp32, as are
 * the other factors below and eps.  table and out: any formats, the same cols. */
int zero_embed_forward(const zero_rows* table, int64_t first_row, const void* ids_dev, int32_t id_bytes, double scale,
                       const zero_rows* out, void* stream);

/* Bytes of zero_embed_grad's workspace (16-byte aligned) for up to n_tokens
 * tokens and a table of table_rows rows of cols elements; 0 if a size is out
 * of range. */
size_t zero_embed_grad_workspace_bytes(int64_t n_tokens, int64_t table_rows, int64_t cols);

/* Device.  table_grad[v] = scale · (sum of out_grad[t] over the tokens t with
 * ids[t] - first_row = v), in fp32 and in an order that only the tokens
 * decide, rounded once; rows that no token names become zeros.  With
 * accumulate the sum is added to what table_grad holds, in fp32, and rows
 * that no token names are not touched.  Tokens outside the table are passed
 * over, with their out_grad unread.  Sizes whose launch would have 2^24
 * workgroups or more are refused: rows/64 (without accumulate) and cols/512 for
 * each of up to 512 tokens, or of the 8192 parts at most that more are split into. */
int zero_embed_grad(const void* ids_dev, int32_t id_bytes, int64_t first_row, const zero_rows* out_grad, double scale,
                    const zero_rows* table_grad, int32_t accumulate, void* ws_dev, size_t ws_bytes, void* stream);

/* Device.  Layer norm of each row of x:
 *   center = 1:  y = (x - mean)·rstd·weight + bias,  rstd = 1/sqrt(mean((x - mean)²) + eps)
 *   center = 0:  y = x·rstd·weight + bias,           rstd = 1/sqrt(mean(x²) + eps)
 * weight_dev, and bias_dev (NULL: none): cols elements of format wdt, which is
 * x's or ZERO_FP32.  y: x's shape and format.  mean_dev, rstd_dev: fp32 per
 * row, for the backward pass; either may be NULL (mean_dev is not written
 * where center = 0).  eps >= 0.  cols at most ZERO_LAYERNORM_MAX_COLS (a row
 * stays in registers between its statistics and its result). */
#define ZERO_LAYERNORM_MAX_COLS 16384
int zero_layernorm_forward(const zero_rows* x, const void* weight_dev, const void* bias_dev, zero_dtype wdt, double eps,
                           int32_t center, const zero_rows* y, float* mean_dev, float* rstd_dev, void* stream);

/* Bytes of zero_layernorm_grad's workspace (16-byte aligned) for up to n_rows
 * rows of cols elements; 0 if a size is out of range. */
size_t zero_layernorm_grad_workspace_bytes(int64_t n_rows, int64_t cols);

/* Device.  With h = (x - mean)·rstd and d = y_grad·weight:
 *   x_grad      = rstd·(d - mean(d) - h·mean(d·h))     (without mean(d) where center = 0)
 *   weight_grad = sum of y_grad·h over the rows
 *   bias_grad   = sum of y_grad over the rows
 * mean_dev and rstd_dev as the forward pass left them (mean_dev is not read
 * where center = 0).  y_grad and x_grad: x's shape and format.  weight_grad
 * and bias_grad: cols elements of format gdt (any), added to what they hold
 * with accumulate.  Each of the three results may be left out (NULL). */
int zero_layernorm_grad(const zero_rows* x, const zero_rows* y_grad, const void* weight_dev, zero_dtype wdt,
                        int32_t center, const float* mean_dev, const float* rstd_dev, const zero_rows* x_grad,
                        void* weight_grad_dev, void* bias_grad_dev, zero_dtype gdt, int32_t accumulate, void* ws_dev,
                        size_t ws_bytes, void* stream);

/* Bytes of the workspace (256-byte aligned) of zero_loss_head (gradients = 0)
 * and zero_loss_head_grad (gradients = 1) for up to n_tokens tokens, whatever
 * the strides; 0 if a size is out of range.  Scores exist for one block of
 * tokens at a time, and the size does not grow with n_tokens past a block: as
 * many tokens as have 256 MiB of 16-bit scores or 1 GiB of hidden rows at 8
 * bytes an element, whichever are fewer, but 256 at least. */
size_t zero_loss_head_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t cols, int32_t gradients);

/* The same for calls with this table alone (its place, stride and format; 0
 * where the calls would refuse it).  Less by a copy of the table where its
 * rows can be read where they are: cols a multiple of 64, stride of 8 and below
 * 2^22, data on a 16-byte line. */
size_t zero_loss_head_workspace_bytes_for(int64_t n_tokens, const zero_rows* table, int32_t gradients);

/* Device.  Scores z = x·tableᵀ of x->rows tokens over table->rows words, and
 *   losses[t] = log(sum of exp(z[t])) - z[t][labels[t]]
 *   *loss     = sum of losses / count,  *count = number of tokens that count
 * A label outside [0, table->rows) does not count: its loss is 0, its
 * gradients zeros.  Where none counts, *loss is 0.  x and table: the same
 * 16-bit format and cols (fp32 is refused: the products take 16-bit factors).
 * label_bytes: 4 (int32) or 8 (int64).  losses_dev (x->rows), loss_dev: fp32.
 * Scores are sums in fp32, never rounded to fewer bits for the losses, and the
 * loss of a token that is all but sure of its label keeps its digits.  A
 * score that is NaN or +inf makes its token's loss (and gradients) NaN; one of
 * -inf is a word of probability 0.  table->rows in [1, 2^22], cols at most
 * 2^16, rows·cols (rows rounded up to 256, cols to 64) below 2^36. */
int zero_loss_head(const zero_rows* x, const zero_rows* table, const void* labels_dev, int32_t label_bytes,
                   float* losses_dev, float* loss_dev, int64_t* count_dev, void* ws_dev, size_t ws_bytes, void* stream);

/* Device.  The same, and the gradients of *loss times the loss scale:
 *   G = (softmax(z) - onehot(label))·scale·loss_scale/count   (zeros for tokens that do not count)
 *   x_grad     = G·table     (x's shape and format)
 *   table_grad = Gᵀ·x        (table's shape and format), or added to what it
 *                            holds with accumulate
 * loss_scale is state_dev->loss_scale when the kernels run (1 where state_dev
 * is NULL), so a captured step follows the scale that the decision moves.  The
 * factors softmax - onehot are rounded to the 16-bit format for the products,
 * from scores held to 2^-12 of an octave (a word more than 32 octaves below the
 * largest of its 64 neighbours counts as 0 there).
 * A token that does not count has no part in the gradients, whatever its row
 * of x holds. */
int zero_loss_head_grad(const zero_rows* x, const zero_rows* table, const void* labels_dev, int32_t label_bytes,
                        double scale, const zero_step_state* state_dev, float* losses_dev, float* loss_dev,
                        int64_t* count_dev, const zero_rows* x_grad, const zero_rows* table_grad, int32_t accumulate,
                        void* ws_dev, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ measurement aid
 *
 * Not a step of the method: the read-modify-write ceiling of the tiled
 * update's own access pattern.  Device.  Exactly the loads and stores of
 * zero_adamw_step_tiled over n elements (same launches of at most 2^25
 * elements, same workgroup-to-tile mapping, same non-temporal hints: read 2 B
 * of gradient and 12 B of tiled state, write the 12 B of state back and 2 B
 * of parameter per element), with the arithmetic replaced by an XOR with key:
 * state words become state ^ key, each 32-bit pair of parameters becomes the
 * gradient pair ^ key.  With key = 0 the state keeps its bits and the
 * parameters receive the gradient bits.  Only whole groups of four elements
 * are touched (n mod 4 trailing elements are left alone).  Same alignment
 * rules as the vector path of zero_adamw_step_tiled (grad and param 8-byte,
 * state 16-byte aligned), otherwise ZERO_ERR_INVALID. */
int zero_calibrate_tiled_rmw(const void* grad_dev, float* state_dev, uint16_t* param_dev, int64_t n, uint32_t key,
                             void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_SHARD_H */
