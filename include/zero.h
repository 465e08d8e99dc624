/*
 * zero.h -- C ABI of the GB300 ZeRO sharded mixed-precision optimizer step.
 *
 * One process, one GPU, N *virtual* data-parallel ranks: rank q's gradient
 * replica and rank r's optimizer shard are separate caller-owned buffers in
 * the same HBM.  The library owns only the partition plan (host memory).
 * Every tensor argument is caller-owned memory the GPU can address: device
 * memory (for example a torch tensor's data_ptr()), or host memory mapped
 * into the GPU's address space at the same address (pinned with
 * cudaHostAlloc / cudaHostRegister under unified addressing).  Host buffers
 * are read and written by the kernels across the host link (NVLink-C2C on
 * Grace-Blackwell), which replaces an explicit copy; they run at the link's
 * bandwidth instead of HBM's.  Every stream argument is a cudaStream_t passed
 * as void* (NULL = the legacy default stream).  Compute calls are
 * asynchronous on that stream, except the three that run the optimizer on
 * host threads (zero_cpu_adamw_shard_step, zero_offload_step,
 * zero_offload_step_amp), which return when the host work is done.
 *
 * Sources (page title, section) for what each call computes:
 *  [ZeRO-2 blog]   "DeepSpeed ZeRO-2 ... DeepSpeedZeroOptimizer" (discosf.com):
 *                  §2.1 and §4.1 flatten + near-equal partition + fp32 master
 *                  cloned from the 16-bit partition; §2.2 and §4.2 bucketed
 *                  reduce-scatter leaving each rank the averaged gradient of
 *                  its partition; §4.3 local update of the rank's partition;
 *                  §4.4 all-gather of the updated partitions.
 *  [cookllm ZeRO]  "ZeRO 优化器" (cookllm.com): 参数分配策略 (tensor i owned
 *                  by rank i % world_size), 梯度同步 (reduce = sum to the
 *                  owner), the per-stage memory tables.
 *  [ZeRO report]   "ZeRO / DeepSpeed 深度解读报告" (zako-mio.github.io) §3.3:
 *                  per-device memory 16P, 4P+12P/N, 2P+14P/N, 16P/N.
 *  [wmrh tutorial] "ZeRO ... 实操" (wmrh.cn) §3.1: AdamW hyper-parameters.
 *
 * Conventions common to every call:
 *  - Every call returns a zero_status and never throws or aborts.  On
 *    failure, zero_last_error() returns a message (thread-local storage,
 *    valid until the next call on the same thread).
 *  - All arguments are validated before anything is launched; a call that
 *    fails validation launches nothing and leaves every output untouched.
 *  - Device pointers must be 16-byte aligned (ZERO_ERR_ALIGN otherwise)
 *    unless the call says otherwise; torch allocations are 256-byte aligned.
 *  - Asynchronous device errors surface as ZERO_ERR_CUDA from the next call
 *    or from zero_sync().
 *  - At most 64 virtual ranks; rank_mask bit r selects rank r.  Pointer
 *    arrays are indexed by rank and have n_ranks entries; entries of ranks
 *    outside rank_mask, or whose shard is empty, are not read and may be
 *    NULL.  Likewise any buffer of zero length (a group whose tensors are
 *    all empty has an empty flat buffer) may be NULL.
 *  - Flat indices f run over the gathered flat buffer (length `padded` from
 *    zero_plan_total); shard indices i run over rank r's shard buffers
 *    (length from zero_plan_shard).
 *  - A call may make several launches (one per bucket, and more when a
 *    bucket holds more runs than one launch carries).  Launches of one call
 *    that touch disjoint elements may run concurrently on the GPU; all of
 *    them complete, with their writes visible, before work enqueued on the
 *    stream after the call starts, so stream order between calls holds as
 *    for single kernels (also inside captured CUDA graphs).
 */
#ifndef ZERO_GB300_H_
#define ZERO_GB300_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ZERO_OK = 0,
  ZERO_ERR_INVALID = 1,     /* bad argument: null, out of range, size mismatch   */
  ZERO_ERR_ALIGN = 2,       /* a device pointer is not 16-byte aligned           */
  ZERO_ERR_CUDA = 3,        /* CUDA runtime error (launch or asynchronous)       */
  ZERO_ERR_OOM = 4,         /* host allocation failed                            */
  ZERO_ERR_TIMEOUT = 5,     /* a bounded wait on the device gave up (zero_sync)   */
  ZERO_ERR_UNSUPPORTED = 6  /* valid request this build does not implement       */
} zero_status;

/* ZERO_FP32 belongs to the gradient-list, block, expert, embedding and head calls
 * below; the optimizer's calls take the two 16-bit types. */
typedef enum { ZERO_FP16 = 0, ZERO_BF16 = 1, ZERO_FP32 = 2 } zero_dtype;
typedef enum { ZERO_PART_FLAT = 0, ZERO_PART_ROUND_ROBIN = 1 } zero_part_mode;
typedef enum { ZERO_REDUCE_SUM = 0, ZERO_REDUCE_AVG = 1 } zero_reduce_op;

/*
 * AdamW hyper-parameters as the caller holds them (binary64).  The library
 * forms the step's binary32 constants in binary64 and rounds each once:
 *   d = 1 - lr*weight_decay, c1 = 1 - beta1, c2 = 1 - beta2,
 *   ss = lr / (1 - beta1^t), sb = sqrt(1 - beta2^t).
 * Requirements: all finite, lr >= 0, weight_decay >= 0, eps > 0,
 * 0 <= beta1 < 1, 0 <= beta2 < 1.
 */
typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
} zero_adamw_hparams;

typedef struct zero_plan zero_plan; /* opaque, host memory, owned by the library */

/* ------------------------------------------------------------------------ */
/* Partition plan (host only; no GPU needed)                                */
/* ------------------------------------------------------------------------ */

/*
 * Build the partition plan of one parameter group.
 *  numel[k], k < n_tensors: element counts of the group's tensors in
 *    named_parameters() order (>= 0; n_tensors >= 1).
 *  ZERO_PART_FLAT ([ZeRO-2 blog] §2.1, §4.1): the tensors are concatenated
 *    with no gap into one flat buffer of phi = sum(numel) elements, padded at
 *    the tail with zeros to P = ceil(phi / (n_ranks*align_elems)) *
 *    n_ranks*align_elems; rank r owns flat range [r*S, (r+1)*S), S = P/n_ranks.
 *    align_elems must be a power of two in [1, 4096].
 *  ZERO_PART_ROUND_ROBIN ([cookllm ZeRO] 参数分配策略): tensor k is owned
 *    whole by rank k % n_ranks; the flat buffer is the unpadded concatenation
 *    (P = phi) and rank r's shard packs its tensors in increasing k.
 *    align_elems is ignored.
 *  n_ranks in [1, 64].  On success *out receives a plan that the caller
 *  releases with zero_plan_destroy.
 */
zero_status zero_plan_partitions(const int64_t* numel, int32_t n_tensors, int32_t n_ranks,
                                 zero_part_mode mode, int32_t align_elems, zero_plan** out);

/* Release a plan (NULL is allowed). */
void zero_plan_destroy(zero_plan* plan);

/* phi = real element count, padded = length of the gathered flat buffer. */
zero_status zero_plan_total(const zero_plan* plan, int64_t* phi, int64_t* padded);

/* Number of virtual ranks and the partition mode of a plan. */
zero_status zero_plan_info(const zero_plan* plan, int32_t* n_ranks, int32_t* mode,
                           int32_t* align_elems, int32_t* n_tensors);

/*
 * Rank r's shard: *len = its element count; *flat_off = the flat index of its
 * first element in flat mode, or -1 in round-robin mode (shards are not
 * contiguous in the flat buffer there).
 */
zero_status zero_plan_shard(const zero_plan* plan, int32_t rank, int64_t* flat_off,
                            int64_t* len);

/*
 * Ownership map of rank r: the segments (tensor_idx, tensor_off, flat_off,
 * shard_off, len) in increasing flat order.  A segment is a maximal run of
 * elements that lies in one tensor and in rank r's shard; flat-mode tail
 * padding is reported with tensor_idx = -1.  Each output array holds `cap`
 * entries; *n_out receives the number of segments (which may exceed cap: call
 * once with cap = 0 to size the arrays).  Output arrays may be NULL when
 * cap == 0.
 */
zero_status zero_plan_segments(const zero_plan* plan, int32_t rank, int64_t* tensor_idx,
                               int64_t* tensor_off, int64_t* flat_off, int64_t* shard_off,
                               int64_t* len, int64_t cap, int64_t* n_out);

/* Human-readable dump of the plan into buf (NUL-terminated, truncated to cap). */
zero_status zero_plan_describe(const zero_plan* plan, char* buf, int64_t cap);

/*
 * Per-rank model-state bytes of mixed-precision Adam training ([ZeRO report]
 * §3.3; [cookllm ZeRO] stage tables): 2 B/param 16-bit params, 2 B/param
 * 16-bit grads, 12 B/param fp32 master + m + v.  stage 0 (DDP) 16 phi;
 * 1: 4 phi + 12 phi/N; 2: 2 phi + 14 phi/N; 3: 16 phi/N.  Returned as the
 * exact reduced fraction *num / *den.  ZERO_ERR_INVALID if the numerator
 * would overflow int64.
 */
zero_status zero_memory_bytes(int32_t stage, int64_t phi, int32_t n_ranks, int64_t* num,
                              int64_t* den);

/* ------------------------------------------------------------------------ */
/* Device calls                                                             */
/* ------------------------------------------------------------------------ */

/*
 * Optimizer-state initialisation ([ZeRO-2 blog] §4.1: each rank clones its
 * fp32 master from its own 16-bit partition):
 *   master[r][i] = float(full_flat16[f]), m[r][i] = v[r][i] = +0
 * for every (f, i) owned by a rank in rank_mask.  The widening is exact.
 *  full_flat16: device, `padded` 16-bit elements of `dtype` (read).
 *  master/m/v:  n_ranks device pointers, each to that rank's shard length of
 *               float (written).
 */
zero_status zero_init_shards(const zero_plan* plan, const void* full_flat16, zero_dtype dtype,
                             float* const* master, float* const* m, float* const* v,
                             uint64_t rank_mask, void* stream);

/*
 * Reduce-scatter ([ZeRO-2 blog] §2.2, §4.2; [cookllm ZeRO] 梯度同步):
 *   grad_shards[r][i] = G_0[f] + G_1[f] + ... + G_{N-1}[f]
 * accumulated in binary32 in rank order, then divided by N for
 * ZERO_REDUCE_AVG.  grads[q] (n_ranks entries, all required) points to rank
 * q's flat gradient replica of `dtype`; it is read only at the flat indices
 * owned by ranks in rank_mask (so a caller holding only those ranges may pass
 * correspondingly offset pointers).  grad_shards[r]: device float[shard len].
 *  bucket_elems > 0 splits the work into buckets of that many flat indices,
 *  one launch each (like the reduce_bucket_size of the pages); <= 0 means one
 *  bucket.  Results do not depend on the bucketing.
 */
zero_status zero_reduce_scatter(const zero_plan* plan, const void* const* grads,
                                zero_dtype dtype, zero_reduce_op op, float* const* grad_shards,
                                uint64_t rank_mask, int64_t bucket_elems, void* stream);

/*
 * zero_reduce_scatter restricted to the flat index range [flat_lo, flat_hi)
 * (0 <= flat_lo <= flat_hi <= padded): one gradient bucket.  This is the call
 * a backward pass makes as soon as every rank's replica holds a bucket's
 * gradients ("DeepSpeed ZeRO-2 ..." §2.2, §4.2: IPG buckets of
 * reduce_bucket_size reduced on a side stream while the backward pass goes
 * on, overlap_comm).  Only grad_shards elements whose flat index falls in the
 * range are written; an empty intersection launches nothing.
 */
zero_status zero_reduce_scatter_range(const zero_plan* plan, const void* const* grads,
                                      zero_dtype dtype, zero_reduce_op op,
                                      float* const* grad_shards, uint64_t rank_mask,
                                      int64_t flat_lo, int64_t flat_hi, void* stream);

/*
 * Local AdamW step on each masked rank's shard ([ZeRO-2 blog] §4.3), one
 * binary32 rounding per operation, in this order (t = step >= 1):
 *   p = p*d;  m = b1*m + c1*g;  v = b2*v + c2*(g*g);
 *   den = sqrt(v)/sb + eps;  p = p - ss*(m/den)
 * and, when out16_shard is non-NULL, out16_shard[r][i] = p rounded to
 * nearest even in `dtype` (entries may be NULL to skip a rank).
 *  master/m/v: device float[shard len] (read-modify-write).
 *  grad_shards: device float[shard len] (read).
 */
zero_status zero_adamw_shard_step(const zero_plan* plan, float* const* master, float* const* m,
                                  float* const* v, const float* const* grad_shards,
                                  void* const* out16_shard, zero_dtype dtype,
                                  const zero_adamw_hparams* hp, int64_t step,
                                  uint64_t rank_mask, void* stream);

/*
 * ZeRO-Offload's CPU optimizer ([ZeRO-2 blog] §4.5: offload_optimizer to the
 * CPU, DeepSpeedCPUAdam, pinned buffers): the update of
 * zero_adamw_shard_step computed by host threads on HOST buffers (master, m,
 * v, grad_shards and out16_shard are host memory, pinned or not), with the
 * same binary32 operations in the same order, so the results equal the GPU
 * update bit for bit.  It runs only when called: the usual offload step is
 * zero_reduce_scatter into pinned host grad_shards, zero_sync, this call,
 * then zero_allgather from the pinned host 16-bit shards (zero_offload_step
 * runs that sequence overlapped).  Synchronous; the masked ranks' shards are
 * split into n_threads equal slices (n_threads <= 0: every hardware thread;
 * the calling thread takes the first slice).
 */
zero_status zero_cpu_adamw_shard_step(const zero_plan* plan, float* const* master,
                                      float* const* m, float* const* v,
                                      const float* const* grad_shards, void* const* out16_shard,
                                      zero_dtype dtype, const zero_adamw_hparams* hp,
                                      int64_t step, uint64_t rank_mask, int32_t n_threads);

/*
 * ZeRO-Offload with the CPU optimizer, pipelined ([ZeRO-2 blog] §4.5:
 * offload_optimizer to the CPU, DeepSpeedCPUAdam, pinned-memory gradient
 * buffers; the pipelining is this library's).  The result is that of
 *   zero_reduce_scatter(grads -> grad_shards); zero_sync;
 *   zero_cpu_adamw_shard_step(master, m, v, grad_shards -> out16_shard);
 *   zero_allgather(out16_shard -> full_flat16)
 * element for element and bit for bit, but the flat index space is cut into
 * chunks of chunk_elems elements: the device reduces every chunk in turn,
 * host threads update chunk k as soon as its reduction has completed (while
 * the device still reduces the chunks after it), and chunk k's all-gather is
 * enqueued as soon as the host has written its 16-bit values.
 *  grads: the N flat replicas (device, or pinned host memory); or NULL when
 *    grad_shards already hold the reduced gradients (reduced bucket by bucket
 *    during backward): then nothing is reduced, `op` is not used, and the
 *    host update starts once the work enqueued on `stream` before the call
 *    has completed (the update and the gathers still overlap).
 *  grad_shards, out16_shard: PINNED (or managed) host memory the device
 *    writes (fp32 reduced gradient) and reads (16-bit shard) across the host
 *    link; checked with cudaPointerGetAttributes (ZERO_ERR_INVALID otherwise).
 *  master, m, v: host memory (pinned or not; never device memory), updated
 *    by the host threads only.
 *  full_flat16: device memory, or NULL for no gather (the 16-bit shards are
 *    still written).
 *  chunk_elems <= 0: one chunk (no overlap); at most 4096 chunks.
 *  n_threads: host threads that update (at most 1024); <= 0: every hardware
 *    thread but one, which is left to the calling thread (it sleeps on the
 *    device's events and launches the gathers).
 * Each thread updates an equal slice of every chunk, so the host part takes
 * what streaming 30 bytes per element through host memory takes; the device
 * traffic across the host link shares that memory.
 * Blocking: returns when every host update is done and every gather is
 * enqueued on `stream` (the gathers complete asynchronously; zero_sync or a
 * later call on `stream` orders after them).  It waits for the device in the
 * middle, so it cannot be captured in a CUDA graph (ZERO_ERR_UNSUPPORTED
 * while `stream` is capturing).  A ZERO_ERR_CUDA during the call may leave
 * some chunks updated and others not.
 */
zero_status zero_offload_step(const zero_plan* plan, const void* const* grads, zero_dtype dtype,
                              zero_reduce_op op, float* const* grad_shards, float* const* master,
                              float* const* m, float* const* v, void* const* out16_shard,
                              void* full_flat16, const zero_adamw_hparams* hp, int64_t step,
                              uint64_t rank_mask, int64_t chunk_elems, int32_t n_threads,
                              void* stream);

/*
 * All-gather ([ZeRO-2 blog] §4.4): full_flat16[f] = shards16[r][i] for every
 * (f, i) owned by a rank in rank_mask.  Flat-mode tail padding belongs to
 * the last rank's shard and is copied like any other element.
 */
zero_status zero_allgather(const zero_plan* plan, const void* const* shards16,
                           zero_dtype dtype, void* full_flat16, uint64_t rank_mask,
                           void* stream);

/*
 * The fused step: reduce-scatter, AdamW, cast and all-gather in one pass
 * over HBM (one read of the N gradient replicas and of master/m/v, one write
 * of master/m/v and of the 16-bit parameters).  The results are bit-identical
 * to zero_reduce_scatter -> zero_adamw_shard_step -> zero_allgather.
 *  full_flat16 (nullable): gathered flat 16-bit buffer, written at the flat
 *    indices of masked ranks.
 *  out16_shard (nullable, entries nullable): each rank's 16-bit shard (the
 *    ZeRO-3 layout, where the shard is the next all-gather's source).
 *  bucket_elems: as for zero_reduce_scatter.
 */
zero_status zero_step(const zero_plan* plan, const void* const* grads, zero_dtype dtype,
                      zero_reduce_op op, float* const* master, float* const* m, float* const* v,
                      void* full_flat16, void* const* out16_shard, const zero_adamw_hparams* hp,
                      int64_t step, uint64_t rank_mask, int64_t bucket_elems, void* stream);

/* ------------------------------------------------------------------------ */
/* ZeRO-3 layer stream with prefetch                                        */
/* ------------------------------------------------------------------------ */
/*
 * ZeRO-3 keeps only 16-bit shards of every layer and gathers a layer's full
 * parameters just before it is used, releasing them afterwards ("ZeRO 优化器"
 * (cookllm.com), ZeRO Stage 3: per-layer gather -> compute -> release;
 * "ZeRO / DeepSpeed 深度解读报告" §2.4; "DeepSpeed ZeRO-2 ..." §5 names the
 * prefetch bucket).  One layer of a stack that shares one plan: */
typedef struct {
  const void* const* grads; /* n_ranks 16-bit flat gradient replicas of the layer   */
  float* const* master;     /* n_ranks fp32 shards (read-modify-write)               */
  float* const* m;          /* n_ranks fp32 shards (read-modify-write)               */
  float* const* v;          /* n_ranks fp32 shards (read-modify-write)               */
  void* const* shards16;    /* n_ranks 16-bit shards: gather source, step output     */
} zero_layer;

/*
 * One pass over n_layers layers: for layer l, zero_allgather(shards16 ->
 * layer_bufs[l % n_bufs]) on gather_stream, then zero_step(grads, master, m,
 * v, full_flat16 = NULL, out16_shard = shards16) on step_stream for step
 * `step`.  Ordering, enforced with events (no host waits):
 *   - the gather of layer l starts after the step of layer l - n_bufs
 *     finished (the layer buffer it overwrites is released then);
 *   - the step of layer l starts after the gather of layer l (the step
 *     rewrites the shards the gather reads);
 *   - the first gather starts after all work already queued on step_stream.
 * So with two streams and n_bufs >= 2 the gathers of the next layers run
 * ahead (prefetch) while earlier layers update; with gather_stream ==
 * step_stream the pass is serial.  All work of the pass is complete once
 * step_stream reaches the point after the call.  Results do not depend on
 * n_bufs or the streams.  n_bufs in [1, 64]; every layer buffer holds
 * `padded` 16-bit elements.
 */
zero_status zero_zero3_pass(const zero_plan* plan, const zero_layer* layers, int32_t n_layers,
                            void* const* layer_bufs, int32_t n_bufs, zero_dtype dtype,
                            zero_reduce_op op, const zero_adamw_hparams* hp, int64_t step,
                            void* gather_stream, void* step_stream);

/* ------------------------------------------------------------------------ */
/* Mixed-precision controls: dynamic loss scaling, overflow skip, clipping  */
/* ------------------------------------------------------------------------ */
/*
 * The pages give these as configuration only ("ZeRO ... 实操" (wmrh.cn) §3.1
 * and §3.3, ds_config: fp16 loss_scale 0 (dynamic), loss_scale_window,
 * hysteresis, min_loss_scale; gradient_clipping).  What the library does:
 *  - the gradient replicas carry the loss scale S; they are reduced as by
 *    zero_reduce_scatter into binary32 shards, and the squared L2 norm of
 *    the reduced gradient over every masked rank is accumulated (binary32
 *    squares; sums in a fixed order with about 48 significant bits, kept as
 *    pairs of binary32 numbers, squares of 2^64 and above in a second pair
 *    scaled by 2^-64, so the sum of finite squares is finite);
 *  - a non-finite norm (an inf or NaN anywhere) skips the update: no
 *    parameter, moment or step count changes; if more than one overflow is
 *    still tolerated the tolerance drops by one, else S halves (not below
 *    min_scale); the run of good steps restarts;
 *  - otherwise norm = sqrt(sumsq)/S; the clip factor is
 *    min(1, max_norm/(norm + 1e-6)) when max_norm > 0 (as
 *    torch.nn.utils.clip_grad_norm_), else 1; every element's gradient is
 *    g * coef with coef = clip/S rounded once to binary32, and AdamW runs as
 *    zero_adamw_shard_step for step t = state.step + 1, followed by the cast
 *    and the all-gather of zero_step; after `window` consecutive good steps S
 *    doubles and the overflow tolerance is restored.
 * Every decision is taken on the device: no call waits for the host, so a
 * sequence of steps needs no synchronisation.
 */
typedef struct {
  double init_scale;  /* loss scale of the first gradients (finite, > 0)           */
  double min_scale;   /* floor of the loss scale (finite, > 0)                       */
  int32_t window;     /* good steps before the scale doubles; 0 = never grows        */
  int32_t hysteresis; /* overflows tolerated before the scale halves (>= 1)          */
  double max_norm;    /* clip threshold of the unscaled global norm; <= 0 = no clip  */
} zero_amp_config;

/* State of the controls; lives in caller-owned DEVICE memory (16-byte aligned),
 * written by zero_amp_init and by every zero_step_amp; copy it to the host to
 * read it. */
typedef struct {
  double scale;            /* loss scale the next gradients are expected to carry */
  double norm;             /* unscaled global L2 norm of the last call (inf/NaN on overflow) */
  int64_t step;            /* AdamW steps applied (skipped calls not counted)     */
  int64_t skipped;         /* calls skipped because of a non-finite gradient      */
  int32_t good_steps;      /* good steps since the scale last changed             */
  int32_t hysteresis_left; /* overflows still tolerated before the scale halves   */
  int32_t overflow;        /* 1 if the last call skipped its update               */
  float coef;              /* gradient multiplier of the last applied update      */
  float sc[8];             /* binary32 AdamW constants of the last applied update */
} zero_amp_state;

/* Write the initial state (scale = init_scale, everything else 0, tolerance =
 * hysteresis) into d_state, asynchronously on `stream`. */
zero_status zero_amp_init(void* d_state, const zero_amp_config* cfg, void* stream);

/* Bytes of device workspace zero_step_amp needs for this plan, mask and
 * bucketing: an 8 KB head (copies of the step's decision record, the
 * decision kernel's partial sums) plus one 16-byte partial sum of squares
 * per 2048-element tile. */
zero_status zero_amp_workspace_bytes(const zero_plan* plan, uint64_t rank_mask,
                                     int64_t bucket_elems, int64_t* bytes);

/*
 * One mixed-precision step (see above).  Arguments as zero_step, plus:
 *  grad_shards: n_ranks device pointers to float[shard len], written with the
 *    reduced (still scaled) gradient, the partitioned gradient of ZeRO-2;
 *  cfg: host pointer, read during the call;
 *  d_state: the device state (read-modify-write);
 *  workspace: caller-owned device scratch of at least
 *    zero_amp_workspace_bytes(plan, rank_mask, bucket_elems), 16-byte aligned.
 * Launches the reduction (one launch per bucket), the decision kernel and
 * the update; calls must not overlap on the device when they share d_state
 * or workspace.
 */
zero_status zero_step_amp(const zero_plan* plan, const void* const* grads, zero_dtype dtype,
                          zero_reduce_op op, float* const* grad_shards, float* const* master,
                          float* const* m, float* const* v, void* full_flat16,
                          void* const* out16_shard, const zero_adamw_hparams* hp,
                          const zero_amp_config* cfg, void* d_state, void* workspace,
                          int64_t workspace_bytes, uint64_t rank_mask, int64_t bucket_elems,
                          void* stream);

/*
 * The mixed-precision step from gradients that are already reduce-scattered:
 * grad_shards[r] (read only) holds rank r's reduced, still loss-scaled fp32
 * gradient, as zero_reduce_scatter or zero_reduce_scatter_range leave it --
 * the flow of a training loop that reduces gradient buckets while the
 * backward pass runs ("DeepSpeed ZeRO-2 ..." §2.2, §4.2: overlap_comm and the
 * reduction stream) and then checks for overflow, clips and updates the
 * partitions.  Everything else (norm, skip, loss scale, clip, AdamW, cast,
 * gather, workspace, state) is as zero_step_amp; the workspace size is
 * zero_amp_workspace_bytes(plan, rank_mask, bucket_elems) for the same
 * bucket_elems.  The results equal zero_reduce_scatter followed by this call
 * and zero_step_amp on the replicas, bit for bit.
 */
zero_status zero_step_amp_shards(const zero_plan* plan, zero_dtype dtype,
                                 float* const* grad_shards, float* const* master, float* const* m,
                                 float* const* v, void* full_flat16, void* const* out16_shard,
                                 const zero_adamw_hparams* hp, const zero_amp_config* cfg,
                                 void* d_state, void* workspace, int64_t workspace_bytes,
                                 uint64_t rank_mask, int64_t bucket_elems, void* stream);

/*
 * One gradient bucket of a mixed-precision training step: the reduce-scatter
 * of zero_reduce_scatter_range over the flat range
 * [bucket_index * bucket_elems, min((bucket_index + 1) * bucket_elems,
 * padded)) (bucket_elems <= 0: one bucket, the whole buffer), which also
 * writes that bucket's per-tile sums of squares into `workspace`, numbered
 * exactly as zero_step_amp numbers its tiles for the same plan, rank_mask
 * and bucket_elems -- the reduction the pages overlap with the backward pass
 * ("DeepSpeed ZeRO-2 ..." §2.2, §4.2: reduce_bucket_size, overlap_comm),
 * with the overflow check's and the clipping norm's first pass folded into
 * it, so that zero_step_amp_reduced needs no pass over the gradient shards
 * for them.  Buckets may be reduced in any order, on any stream ordered
 * before the step.  The launch holding the step's first tile also prepares
 * the decision (it reads d_state's step count: no step on this state may be
 * in flight).
 *  hp: host pointer, read during the call (beta1, beta2);
 *  d_state: the device state of zero_amp_init (read);
 *  workspace: as zero_step_amp's, of at least
 *    zero_amp_workspace_bytes(plan, rank_mask, bucket_elems) bytes.
 * Errors: bucket_index outside the buckets, an undersized workspace, and
 * the argument errors of zero_reduce_scatter_range (ZERO_ERR_INVALID /
 * ZERO_ERR_ALIGN), before any launch.  A bucket whose range holds no element
 * of a masked rank launches nothing.
 */
zero_status zero_reduce_scatter_bucket_amp(const zero_plan* plan, const void* const* grads,
                                           zero_dtype dtype, zero_reduce_op op,
                                           float* const* grad_shards,
                                           const zero_adamw_hparams* hp, const void* d_state,
                                           void* workspace, int64_t workspace_bytes,
                                           uint64_t rank_mask, int64_t bucket_elems,
                                           int64_t bucket_index, void* stream);

/*
 * The mixed-precision step after every bucket of the plan was reduced by
 * zero_reduce_scatter_bucket_amp into grad_shards and `workspace` with the
 * same rank_mask and bucket_elems since the last step on this state: only
 * the decision kernel and the update run (no pass over the gradient shards
 * for the norm: 30 bytes per element instead of zero_step_amp_shards's 34).
 * Arguments and results as zero_step_amp_shards; the results equal
 * zero_step_amp on the replicas with the same bucket_elems, bit for bit.
 * Calling it without those reductions decides on whatever the workspace
 * holds (nothing checks this on the device).
 */
zero_status zero_step_amp_reduced(const zero_plan* plan, zero_dtype dtype,
                                  float* const* grad_shards, float* const* master,
                                  float* const* m, float* const* v, void* full_flat16,
                                  void* const* out16_shard, const zero_adamw_hparams* hp,
                                  const zero_amp_config* cfg, void* d_state, void* workspace,
                                  int64_t workspace_bytes, uint64_t rank_mask,
                                  int64_t bucket_elems, void* stream);

/*
 * The mixed-precision step with the optimizer offloaded to the host
 * ([ZeRO-2 blog] §4.5 with the fp16 controls above): the device reduces
 * (grads non-NULL, as zero_step_amp; or grads NULL, the shards and the
 * workspace's sums of squares written by zero_reduce_scatter_bucket_amp with
 * this bucket_elems, as zero_step_amp_reduced) and takes the decision in
 * d_state; the host reads the decision and, unless it skips the step, host
 * threads apply the update of zero_step_amp (gradient times the decision's
 * coef, then AdamW with its constants) to the host master/m/v and write the
 * host 16-bit shards, chunk by chunk, each chunk's gather into full_flat16
 * (nullable) enqueued as soon as it is written.  Buffers, chunk_elems,
 * n_threads, blocking and capture as zero_offload_step; d_state and
 * workspace are device memory as for zero_step_amp.  A skipped step changes
 * nothing on the host and launches no gather.  Results equal zero_step_amp's
 * bit for bit.
 */
zero_status zero_offload_step_amp(const zero_plan* plan, const void* const* grads,
                                  zero_dtype dtype, zero_reduce_op op, float* const* grad_shards,
                                  float* const* master, float* const* m, float* const* v,
                                  void* const* out16_shard, void* full_flat16,
                                  const zero_adamw_hparams* hp, const zero_amp_config* cfg,
                                  void* d_state, void* workspace, int64_t workspace_bytes,
                                  uint64_t rank_mask, int64_t bucket_elems, int64_t chunk_elems,
                                  int32_t n_threads, void* stream);

/*
 * zero_step_amp without a workspace argument, for callers that cannot
 * allocate device memory: code whose device memory all comes from a fixed
 * budget or pool it does not control, or that runs where a cudaMalloc /
 * cudaFree (and the device-wide synchronisation a cudaFree can imply) is not
 * allowed, or that has nowhere to keep a workspace alive between calls.
 * The pages describe no such call; it is a convenience of this library.
 *
 * Same arguments and results as zero_step_amp, minus workspace and
 * workspace_bytes.  The scratch is instead a fixed 2 MiB array compiled into
 * the library, present on every GPU that loads it until the process exits;
 * this call allocates nothing (no cudaMalloc, no cudaFree, no allocating
 * library routine).  Limits and rules:
 *  - the step may span at most 130,560 tiles of 2048 elements, i.e.
 *    zero_amp_workspace_bytes(plan, rank_mask, bucket_elems) <= 2 MiB (about
 *    267 million owned elements per call); larger steps are rejected with
 *    ZERO_ERR_INVALID and a message, and nothing is launched;
 *  - the first call on a device looks up the array's device address with
 *    that device current and caches it; make that first call before any
 *    stream capture begins.  With CUDA's lazy module loading (the default)
 *    that lookup is also what loads the library's device code on that
 *    device and commits the 2 MiB array, so the first call can fail with
 *    ZERO_ERR_CUDA (out of memory) on a device that is already full; later
 *    calls commit nothing;
 *  - the cached address belongs to the device's current context: do not call
 *    cudaDeviceReset on that device between calls of this function;
 *  - every call on a device shares the one array, which keeps what the last
 *    call left there (each call writes everything it reads, so nothing needs
 *    clearing): calls whose work overlaps on the GPU (different streams,
 *    not ordered by events) race on it and must be serialised by the caller.
 */
zero_status zero_step_amp_noalloc(const zero_plan* plan, const void* const* grads,
                                  zero_dtype dtype, zero_reduce_op op, float* const* grad_shards,
                                  float* const* master, float* const* m, float* const* v,
                                  void* full_flat16, void* const* out16_shard,
                                  const zero_adamw_hparams* hp, const zero_amp_config* cfg,
                                  void* d_state, uint64_t rank_mask, int64_t bucket_elems,
                                  void* stream);

/* ------------------------------------------------------------------------ */
/* Gradient norm and clipping over many tensors                             */
/* ------------------------------------------------------------------------ */
/*
 * The pages' gradient_clipping ("ZeRO ... 实操" (wmrh.cn) §3.1) for gradients
 * that are still one tensor each (a training loop without the loss-scaled
 * step, gradients accumulated in fp32, parameters outside the plan):
 *   norm = sqrt(sum of g^2) over all elements of all tensors (ZERO_NORM_L2),
 *          or max |g| (ZERO_NORM_INF);
 *   coef = min(1, max_norm / (norm + 1e-6)), formed in binary32; 1 when the
 *          norm is not finite;
 *   dst[i] = src[i] * coef, the product in binary32, rounded once to dst.
 * A non-finite norm (an infinity or NaN anywhere) is flagged in the record
 * and scales nothing, so that the caller can skip the step as zero_step_amp
 * does.  No finite gradients make the norm infinite (squares are summed in
 * two exactly scaled ranges); values below 2^-83 may count as zero in it.
 * Sums run in a fixed order: the same call gives the same bits.  Nothing is
 * read back by the host.
 */
typedef enum { ZERO_NORM_L2 = 0, ZERO_NORM_INF = 1 } zero_norm_kind;

/* One tensor.  Pointers need their element's alignment only (a view into a
 * flat buffer at any offset).  dst (clipping only): src itself, for clipping
 * in place with equal types, or memory that overlaps no tensor's src or dst,
 * of any of the three types.  An empty tensor's pointers may be NULL. */
typedef struct {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t src_dtype, dst_dtype;
} zero_grad_tensor;

/* The record a call leaves in caller-owned DEVICE memory (16-byte aligned). */
typedef struct {
  double norm;       /* 0 for an empty list                          */
  float norm32;      /* norm rounded to binary32                     */
  float coef;        /* 1 after zero_grad_norm                       */
  int32_t nonfinite; /* 1: the norm is infinite or NaN               */
  int32_t pad_[3];
} zero_norm_result;

/* Device workspace of either call for this list. */
zero_status zero_grad_norm_workspace_bytes(const zero_grad_tensor* tensors, int32_t n_tensors,
                                           int64_t* bytes);

/* The norm alone (dst and dst_dtype are not read).  `tensors` is host memory,
 * read during the call; workspace: 16-byte aligned device scratch. */
zero_status zero_grad_norm(const zero_grad_tensor* tensors, int32_t n_tensors, int32_t kind,
                           void* d_result, void* workspace, int64_t workspace_bytes,
                           void* stream);

/* Norm and clipping.  max_norm: finite, >= 0. */
zero_status zero_clip_grad_norm(const zero_grad_tensor* tensors, int32_t n_tensors, int32_t kind,
                                double max_norm, void* d_result, void* workspace,
                                int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Block join: norms before and after a block, its gate and residual scale  */
/* ------------------------------------------------------------------------ */
/*
 * Between two blocks of a model, for every row of `hidden` channels:
 *   u = N_post(b)     b: the block's output; u = b without w_post
 *   o = x + scale * g * u   x: the residual stream; g = 1 without a gate
 *   n = N_pre(o)      the next block's input, from o before its rounding
 *   N(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps) * w + bias
 * ZERO_JOIN_RMS has no mean and no bias.  Statistics, products and sums are
 * binary32; o and n are rounded once.  With b NULL, o = x: the norm alone.
 * Pointers need their element's alignment only; rows of 16-byte multiples on
 * 16-byte boundaries take the wide path.  Outputs overlap no input and no
 * other output but for the forms named below.
 */
typedef enum { ZERO_JOIN_RMS = 0, ZERO_JOIN_LAYER = 1 } zero_join_kind;
typedef enum {
  ZERO_GATE_NONE = 0,
  ZERO_GATE_CHANNEL = 1, /* gate[hidden], shared by the rows    */
  ZERO_GATE_ROW = 2,     /* one number a row                    */
  ZERO_GATE_FULL = 3     /* one number an element               */
} zero_gate_kind;

typedef struct {
  int64_t rows, hidden;
  int32_t act_dtype;   /* b, n, d_n, db                                   */
  int32_t res_dtype;   /* x, o, d_o, dx: act_dtype or ZERO_FP32           */
  int32_t param_dtype; /* weights and biases: act_dtype or ZERO_FP32      */
  int32_t gate_dtype;  /* act_dtype or ZERO_FP32                          */
  int32_t kind, gate_kind;
  double eps;          /* > 0                                             */
  double scale;
  /* elements between rows of the inputs (outputs are contiguous); of row
   * gates, between two rows' numbers */
  int64_t x_stride, b_stride, gate_stride, do_stride, dn_stride;
} zero_join_desc;

typedef struct {
  const void *x, *b, *gate;
  const void *w_post, *bias_post; /* NULL: no post norm / no bias */
  const void *w_pre, *bias_pre;   /* NULL: no pre norm / no bias  */
} zero_join_inputs;

/* Any entry may be NULL: that gradient is not formed.  dgate has the gate's
 * type and (contiguous) shape, the parameters' gradients the parameters'. */
typedef struct {
  void *dx, *db, *dgate, *dw_post, *dbias_post, *dw_pre, *dbias_pre;
} zero_join_grads;

/* o (res_dtype) and n (act_dtype, needs w_pre): [rows, hidden], one of them
 * may be NULL.  o may be x and n may be b, each with contiguous rows, when
 * nothing is kept for a backward pass.  stats (nullable, 16-byte aligned):
 * float[rows][4], which the backward pass takes.  rows == 0 does nothing. */
zero_status zero_block_join(const zero_join_desc* desc, const zero_join_inputs* inputs, void* o,
                            void* n, float* stats, void* stream);

/* Device workspace of the backward call (16-byte aligned). */
zero_status zero_block_join_workspace_bytes(const zero_join_desc* desc, int64_t* bytes);

/* The gradients of the same inputs from d_o and d_n (either may be NULL: no
 * gradient comes that way) and the forward call's stats.  x and b still hold
 * what the forward call read.  dx may be d_o and db may be d_n, each with
 * contiguous rows.  The parameters' gradients are summed over the rows in a
 * fixed order; with rows == 0 they are zero.  The workspace is needed when any
 * of them, or a channel gate's, is wanted. */
zero_status zero_block_join_backward(const zero_join_desc* desc, const zero_join_inputs* inputs,
                                     const void* d_o, const void* d_n, const float* stats,
                                     const zero_join_grads* grads, void* workspace,
                                     int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Expert permutation: tokens sorted by expert, brought back with weights   */
/* ------------------------------------------------------------------------ */
/*
 * Choice k of token t is pair p = t*topk + k, of expert ids[p]; a choice
 * outside [0, n_experts) is dropped.  The kept pairs in order of (expert,
 * pair) take the rows 0 .. M-1 of a buffer of tokens*topk rows:
 *   offsets[e] = first row of expert e (n_experts + 1 entries, the last is M)
 *   rows[p]    = the row of pair p, -1 when dropped
 *   pairs[i]   = the pair of row i, -1 for i >= M
 * ids: int32 (id_bytes 4) or int64 (8).  n_experts at most 4096, tokens*topk
 * below 2^31.  The order is stable.  workspace: 4-byte aligned device scratch
 * (NULL when zero_expert_sort_workspace_bytes says 0).  Outputs of this call
 * and the next four overlap no input and no other output.  Nothing is read
 * back by the host.
 */
zero_status zero_expert_sort(const void* ids, int32_t id_bytes, int64_t tokens, int32_t topk,
                             int32_t n_experts, int32_t* offsets, int32_t* rows, int32_t* pairs,
                             void* workspace, int64_t workspace_bytes, void* stream);
zero_status zero_expert_sort_workspace_bytes(int64_t tokens, int32_t topk, int32_t n_experts,
                                             int64_t* bytes);

/* xs[rows[p]] = x[t]; the rows of xs past M are zero.  x_stride: elements
 * between rows of x; xs is [tokens*topk, hidden], contiguous. */
zero_status zero_expert_dispatch(const void* x, int64_t x_stride, zero_dtype dtype, int64_t tokens,
                                 int32_t topk, int64_t hidden, const int32_t* offsets,
                                 int32_t n_experts, const int32_t* rows, void* xs, void* stream);

/* dx[t] = sum of dxs[rows[p]] over the token's kept pairs, in binary32, k in
 * order, rounded once.  The rows of dxs past M are not read. */
zero_status zero_expert_dispatch_backward(const void* dxs, zero_dtype dtype, int64_t tokens,
                                          int32_t topk, int64_t hidden, const int32_t* rows,
                                          void* dx, void* stream);

/* y[t] = sum of weights[p] * ys[rows[p]] over the token's kept pairs, in
 * binary32, k in order, rounded once; zero for a token without any.  weights:
 * [tokens, topk] of weight_dtype (dtype or ZERO_FP32).  The rows of ys past M
 * are not read. */
zero_status zero_expert_combine(const void* ys, zero_dtype dtype, const void* weights,
                                zero_dtype weight_dtype, int64_t tokens, int32_t topk,
                                int64_t hidden, const int32_t* rows, void* y, void* stream);

/* dys[rows[p]] = weights[p] * dy[t], zero past M; dweights[p] (nullable) =
 * <dy[t], ys[rows[p]]> in binary32, zero for a dropped pair. */
zero_status zero_expert_combine_backward(const void* dy, int64_t dy_stride, const void* ys,
                                         zero_dtype dtype, const void* weights,
                                         zero_dtype weight_dtype, int64_t tokens, int32_t topk,
                                         int64_t hidden, const int32_t* offsets,
                                         int32_t n_experts, const int32_t* rows, void* dys,
                                         void* dweights, void* stream);

/* ------------------------------------------------------------------------ */
/* Router: probabilities, choices, counts and balance of sparse experts     */
/* ------------------------------------------------------------------------ */
/*
 * What makes the ids and weights that the calls above take, from every token's
 * scores z of the experts:
 *   p = softmax(z), lse = log(sum exp z); a token whose scores are all -inf is
 *     left out: no choice, p and lse 0
 *   ids[t][k]     = the expert of the k-th largest score, of equal scores the
 *                   lowest expert; -inf is never chosen: -1 (dropped by the
 *                   sort).  NaN counts as +inf.
 *   weights[t][k] = p of the choice, with normalize divided by the sum of the
 *                   token's; 0 for -1
 *   counts[e]     = how often expert e was chosen, n = tokens not left out
 *   losses[0]     = n_experts / (topk max(n,1)^2) sum_e counts[e] sum_t p[t][e],
 *                   1 when the experts are chosen evenly
 *   losses[1]     = sum_t lse[t]^2 / max(n,1)
 *   stats[t] = lse[t], stats[tokens] = n
 * Sums are binary32 in a fixed order.  n_experts at most 1024, topk at most 32,
 * tokens 2^24.  logits_stride: elements between rows.  Pointers need their
 * element's alignment only.  workspace: 4-byte aligned device scratch (NULL when
 * zero_expert_route_workspace_bytes says 0).  Outputs overlap no input and no
 * other output.
 */
zero_status zero_expert_route(const void* logits, int64_t logits_stride, zero_dtype dtype,
                              int64_t tokens, int32_t n_experts, int32_t topk, int32_t normalize,
                              int32_t* ids, float* weights, int32_t* counts, float* losses,
                              float* stats, void* workspace, int64_t workspace_bytes, void* stream);
zero_status zero_expert_route_workspace_bytes(int64_t tokens, int32_t n_experts, int64_t* bytes);

/* d_logits (dtype, contiguous) from the gradients of the weights and of the two
 * losses (either may be NULL: no gradient comes that way); the counts and the
 * choices are constants.  A left-out token's row is zero. */
zero_status zero_expert_route_backward(const void* logits, int64_t logits_stride, zero_dtype dtype,
                                       int64_t tokens, int32_t n_experts, int32_t topk,
                                       int32_t normalize, const int32_t* ids, const float* weights,
                                       const int32_t* counts, const float* stats,
                                       const float* d_weights, const float* d_losses,
                                       void* d_logits, void* stream);

/* ------------------------------------------------------------------------ */
/* Token embedding and the gradient of its table                            */
/* ------------------------------------------------------------------------ */
/*
 * y[t] = scale * table[ids[t]], zero for an id outside [0, vocab), the product
 * in binary32 and rounded once.  ids: int32 (id_bytes 4) or int64 (8); y is
 * contiguous, of table_dtype or ZERO_FP32.  Pointers need their element's
 * alignment only.  Outputs overlap no input and no other output.  tokens at most
 * 2^28, vocab 2^22, hidden 2^20.
 */
zero_status zero_embedding(const void* ids, int32_t id_bytes, int64_t tokens, const void* table,
                           int64_t table_stride, zero_dtype table_dtype, int64_t vocab,
                           int64_t hidden, double scale, void* y, zero_dtype y_dtype, void* stream);

/* dtable[v] = scale * sum of dy[t] over the tokens with ids[t] = v, zero for an
 * id that no token has; accumulate: on top of what dtable holds, and only the
 * rows of the tokens' ids are touched (a table that is also the head's takes
 * both gradients so).  Sums are binary32 in a fixed order (the same call gives
 * the same bits), rounded once.  dtable is contiguous; it and dy have one type,
 * or one of them ZERO_FP32.  workspace: 256-byte aligned device scratch. */
zero_status zero_embedding_backward(const void* dy, int64_t dy_stride, zero_dtype dy_dtype,
                                    const void* ids, int32_t id_bytes, int64_t tokens,
                                    int64_t vocab, int64_t hidden, double scale, int32_t accumulate,
                                    void* dtable, zero_dtype dtable_dtype, void* workspace,
                                    int64_t workspace_bytes, void* stream);
zero_status zero_embedding_workspace_bytes(int64_t tokens, int64_t vocab, int64_t hidden,
                                           int64_t* bytes);

/* ------------------------------------------------------------------------ */
/* Linear softmax cross entropy over a vocabulary                           */
/* ------------------------------------------------------------------------ */
/*
 * The loss of a language model's head, without its logits in memory:
 *   z = scale * x w^T                 x [tokens, hidden], w [vocab, hidden]
 *   lse[t] = log(sum_v exp(z[t][v]))
 *   losses[t] = lse[t] - z[t][targets[t]]
 * A token whose target lies outside [0, vocab) is left out: its losses and lse
 * are 0, nothing of its row of x is read, and it costs next to nothing.
 *   total = {sum / max(count, 1), sum, count} of the losses that are not left out
 *   rows[0 .. n) = the tokens that are not left out, in order, then -1;
 *   rows[tokens] = n
 * x and w are 16-bit; products are summed in binary32, and so are the
 * exponentials.  targets: int32 (id_bytes 4) or int64 (8).  Pointers need their
 * element's alignment only, the workspace 256 bytes; w with rows off 16-byte
 * boundaries is copied to the workspace first.  tokens at most 2^24, hidden
 * 2^20, vocab 2^22; |scale| in [1e-6, 1e6].  Outputs and workspace overlap no
 * input and no other output.  The same call gives the same bits.  Where a bounded
 * wait on the device gave up, in this call or in one that zero_sync has not
 * reported yet, the losses, lse and gradients of kept tokens, the total and dw
 * are NaN.
 */
typedef enum { ZERO_LOSS_NONE = 0, ZERO_LOSS_SUM = 1, ZERO_LOSS_MEAN = 2 } zero_loss_reduction;

typedef struct {
  int64_t tokens, hidden, vocab;
  int64_t x_stride, w_stride; /* elements between rows                 */
  zero_dtype dtype;           /* x, w, dx: ZERO_FP16 or ZERO_BF16      */
  zero_dtype dw_dtype;        /* dw: dtype or ZERO_FP32                */
  int32_t id_bytes;
  double scale;
} zero_linear_ce_desc;

/* Device workspace of the call (backward 0) or of its gradient (1). */
zero_status zero_linear_cross_entropy_workspace_bytes(const zero_linear_ce_desc* desc, const void* w,
                                                      int32_t backward, int64_t* bytes);

/* losses, lse: float[tokens]; rows: int32[tokens + 1]; total: float[3]. */
zero_status zero_linear_cross_entropy(const zero_linear_ce_desc* desc, const void* x, const void* w,
                                      const void* targets, float* losses, float* lse, int32_t* rows,
                                      float* total, void* workspace, int64_t workspace_bytes,
                                      void* stream);

/* The same with one more output: rest[t] = 1 - p[targets[t]], the others'
 * probability, 0 for a left-out token; float[tokens]. */
zero_status zero_linear_cross_entropy_rest(const zero_linear_ce_desc* desc, const void* x, const void* w,
                                           const void* targets, float* losses, float* lse, float* rest,
                                           int32_t* rows, float* total, void* workspace,
                                           int64_t workspace_bytes, void* stream);

/* dx [tokens, hidden] and dw [vocab, hidden], contiguous, either may be NULL,
 * from the forward call's lse and rows; x, w and targets still hold what it
 * read.  d_loss (device): of ZERO_LOSS_NONE float[tokens], the gradients of the
 * losses; else one float, of their sum or of their mean (total[1], total[0]).
 * The logits are formed again, a piece of the vocabulary at a time, p of them to
 * 2^-22 |lse| of itself; their
 * gradient is rounded to dtype between its two products, scaled by the power of
 * two that brings the largest finite |d_loss| to [2^13, 2^14) (for dx in fp16
 * every token's own, once they lie 2^16 apart); for a dw in binary32 it is rounded
 * to two numbers of dtype that hold 16 or 22 bits of it, which doubles dw's
 * product.  So to an fp16 call's dw a token adds nothing where its |d_loss| p is
 * below 2^-39 of the largest |d_loss|, and of less than 11 bits where it is below
 * 2^-27.  dx and dw are rounded once. */
zero_status zero_linear_cross_entropy_backward(const zero_linear_ce_desc* desc, const void* x,
                                               const void* w, const void* targets, const float* lse,
                                               const int32_t* rows, const float* d_loss,
                                               int32_t reduction, void* dx, void* dw,
                                               void* workspace, int64_t workspace_bytes,
                                               void* stream);

/* The same with the rest that zero_linear_cross_entropy_rest left: the gradient
 * of the target's logit is -rest, to its last places.  The call above forms it
 * as p - 1 from lse, off by up to 2^-22 |lse|, which is all of it where the
 * target is that certain. */
zero_status zero_linear_cross_entropy_rest_backward(const zero_linear_ce_desc* desc, const void* x,
                                                    const void* w, const void* targets,
                                                    const float* lse, const float* rest,
                                                    const int32_t* rows, const float* d_loss,
                                                    int32_t reduction, void* dx, void* dw,
                                                    void* workspace, int64_t workspace_bytes,
                                                    void* stream);

/*
 * Measurement helper; the pages have no counterpart.  Launches, on `stream`,
 * kernels with exactly the grid, job table and memory accesses zero_step
 * would use for the same arguments (same plan, mask and buckets), but with
 * none of its arithmetic, so that a benchmark can time the floor a launch of
 * that shape reaches on this GPU:
 *   kind 0  the launches alone (every CTA returns at once);
 *   kind 1  every load of the step (the N gradient replicas, master, m, v),
 *           no store;
 *   kind 2  every load and every store of the step: master/m/v are written
 *           back unchanged and full_flat16 (nullable) receives the master
 *           rounded to 16 bits, which is what a step leaves there anyway.
 * No buffer changes value.  Arguments, layouts, ownership and errors as for
 * zero_step (no hyper-parameters, no shard outputs); kind outside 0..2 is
 * ZERO_ERR_INVALID.  Asynchronous on `stream`.
 */
zero_status zero_floor_probe(const zero_plan* plan, int32_t kind, const void* const* grads,
                             zero_dtype dtype, float* const* master, float* const* m,
                             float* const* v, void* full_flat16, uint64_t rank_mask,
                             int64_t bucket_elems, void* stream);

/* Synchronize `stream` and report any asynchronous device error, and
 * ZERO_ERR_TIMEOUT if a kernel gave up a bounded wait since the last check
 * (the device error word is then cleared). */
zero_status zero_sync(void* stream);

/*
 * Self-test of the timeout path: one kernel waits on a barrier that nothing
 * ever completes, gives up after limit_ns nanoseconds (1e3 .. 1e10) and
 * raises the device error word, so the next zero_sync(stream) returns
 * ZERO_ERR_TIMEOUT.  No fault and no hang: the context stays usable.  The
 * library's waiting kernels (the cross entropy's products) give up the same way,
 * after two seconds.
 */
zero_status zero_selftest_wait_timeout(int64_t limit_ns, void* stream);

/* Message of the last failed call on this thread ("" if none). */
const char* zero_last_error(void);

/* Number of kernel launches the library issued since load (all threads). */
int64_t zero_launch_count(void);

/* Library version string. */
const char* zero_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_GB300_H_ */
