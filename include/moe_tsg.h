/*
 * moe_tsg.h - C ABI of the tile-signalled grouped MoE expert-combine path (sm_103a).
 *
 * The path follows the TileMoE notes (zhongzhuzhou.org, "Fine-grained
 * Computation-Communication Overlap via Tile-level Signaling and Scheduling
 * for Mixture-of-Experts"):
 *   routing (section 2.2 step 1) -> expert problem construction and combine
 *   plan (section 4.2 row layout, 4.4 remote-first schedule / Algorithm 1,
 *   4.5 combine plan) -> overlapped execution: a persistent grouped expert-FFN
 *   producer that sets one ready flag per finished output tile, and a consumer
 *   on a disjoint set of SMs that polls the flags and copies finished segments
 *   (section 5.1-5.3) -> gated weighted sum (scale, section 2.2 step 5).
 * The consumer signals each (sender, destination) group once, after one
 * fence, as in the decoupled signalling of the Perseus summary
 * (papercache.org, section 4.1, Algorithm 1).
 *
 * Everything runs on ONE GPU. The W expert-parallel ranks of the pages are
 * logical: each has its own device allocations (token input, weights,
 * rank workspace, receive buffer, output), and the combine all-to-all is a
 * device-memory copy between those allocations.
 *
 * Conventions
 *  - All pointers are device pointers unless stated. The caller owns all
 *    memory; the library never allocates device memory and owns no stream.
 *  - Tensors are dense, row-major, bf16 unless stated; every tensor's base
 *    pointer (bf16, int32 and fp32 alike) must be 16-byte aligned, or the call
 *    returns MOE_ERR_ARG. d_model and d_ff must be multiples of 128.
 *  - Return value 0 (MOE_OK) or a negative MOE_ERR_* for errors detected on
 *    the host before anything is enqueued. Errors detected on the device
 *    (bad routing ids, a device wait that ran out of time) are sticky in the
 *    plan workspace and are read with moe_status().
 *  - Every call is asynchronous on the given stream(s) except moe_status(),
 *    moe_timings() and the pure-host queries.
 */
#ifndef MOE_TSG_H
#define MOE_TSG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st *moe_stream_t;

/* Largest number of logical ranks one plan can hold. */
#define MOE_MAX_RANKS 8

/* moe_cfg.consumer_ctas value: the combine copy runs inside the pair producer. */
#define MOE_CONSUMER_FUSED (-1)

/* moe_gate splits value: for E <= 16, CTAs small enough to share an SM with a running
 * producer CTA (a gate that runs beside the previous batch's combine). */
#define MOE_GATE_BESIDE (-1)

enum moe_error {
  MOE_OK = 0,
  MOE_ERR_ARG = -1,         /* invalid configuration or argument */
  MOE_ERR_WORKSPACE = -2,   /* a workspace is smaller than moe_workspace_size() */
  MOE_ERR_CUDA = -3,        /* a CUDA runtime call failed (no device, launch error) */
  MOE_ERR_UNSUPPORTED = -4, /* the device is not sm_103 / the shape is outside the kernels' limits */
  /* Device-side codes, reported through moe_status(). */
  MOE_DEV_ROUTING = 1,      /* an expert id is out of range or repeated within a token */
  MOE_DEV_TIMEOUT = 2       /* a device-side wait exceeded cfg.timeout_ns */
};

/* Configuration of one MoE layer split over W logical ranks.
 * Expert e is owned by rank e / L (local index e % L), the placement of
 * Figure 2b of the TileMoE notes. */
typedef struct moe_cfg {
  int W;             /* logical expert-parallel ranks, 1..MOE_MAX_RANKS */
  int L;             /* experts per rank (E = W*L, 1..1024) */
  int topk;          /* experts per token, 1..min(E, 32) */
  int T;             /* tokens per rank, >= 1 */
  int d_model;       /* D, multiple of 128, at most 10240 (a token row fits one 20 KB
                        copy chunk; larger gives MOE_ERR_UNSUPPORTED) */
  int d_ff;          /* F, expert hidden size, multiple of 128 */
  int tb_M;          /* row-band height of the layout: 64, 128 or 256 */
  int mgb;           /* row bands merged into one middle segment (section 5.2), >= 1 */
  int consumer_ctas; /* consumer CTAs running beside the producer (cCTA of section 5.3).
                        0 = serial: the producer uses every SM, then the consumer runs
                        on every SM after it, on the producer stream.
                        MOE_CONSUMER_FUSED (-1, with producer_pairs = 1): no consumer
                        kernel; one warp of every producer CTA polls the flags and
                        copies, on every SM. */
  long long timeout_ns; /* bound on every device-side wait; <= 0 selects 2 s */
  int producer_pairs; /* 0: one producer CTA per 128-row tile (tcgen05.mma, M = 128).
                         1: CTA pairs (clusters of two): each task covers two 128-row
                         tiles of one expert, rows estart + 256 i and estart + 256 i + 128
                         of its block, with one tcgen05.mma of M = 256 (cta_group::2);
                         each CTA loads its own rows and half of the weight rows. */
} moe_cfg;

/* Opaque host-side handle; holds the configuration, the carved workspace
 * pointers and a few CUDA events. Created by moe_plan_create(). */
typedef struct moe_plan moe_plan;

/* Sizes of the caller-provided memory for cfg (pure host arithmetic).
 *  plan_bytes:  one device allocation shared by all ranks (plan arrays, flags).
 *  rank_bytes:  one device allocation per rank (its expert input X, hidden
 *               activations and expert outputs Y, sized for the worst case).
 *  recv_rows:   rows of the receive buffer every rank needs ([recv_rows, D] bf16);
 *               the worst case T*topk.
 * Any output pointer may be NULL. */
int moe_workspace_size(const moe_cfg *cfg, size_t *plan_bytes, size_t *rank_bytes,
                       int *recv_rows);

/* Bind a configuration to its workspaces. plan_ws: plan_bytes; rank_ws: W pointers,
 * each rank_bytes. Queries the current device; fails with MOE_ERR_UNSUPPORTED
 * on anything other than compute capability 10.3. *out must be released with
 * moe_plan_destroy(). Host memory only; enqueues nothing. */
int moe_plan_create(const moe_cfg *cfg, void *plan_ws, size_t plan_ws_bytes,
                    void *const *rank_ws, size_t rank_ws_bytes, moe_plan **out);
void moe_plan_destroy(moe_plan *plan);

/* Routing (TileMoE notes section 2.1 and 2.2 step 1): for every token, softmax over
 * the E gate logits, then the topk experts with the largest logits in descending
 * order (equal logits: the lower expert id first). The weights are the softmax
 * probabilities at the chosen ids, not renormalised.
 *  logits:     [W][T][E] fp32.
 *  forced_ids: NULL, or [W][T][topk] int32 prescribed routing; then ids = forced_ids
 *              and the weights are the probabilities at those ids.
 *  topk_ids:   out [W][T][topk] int32.   topk_w: out [W][T][topk] fp32. */
int moe_route(moe_plan *plan, const float *logits, const int32_t *forced_ids,
              int32_t *topk_ids, float *topk_w, moe_stream_t stream);

/* Gate from the token rows (TileMoE notes section 2.1: a small gating network;
 * 2.2 step 1: every rank gates its own tokens), in one kernel: the router's
 * scores logits[s][t][e] = sum_c x_s[t][c] * w_router[e][c] (bf16 operands, fp32
 * sums on the tensor cores), then the routing of moe_route on those scores.
 *  x:          W pointers, rank s's tokens [T][D] bf16, 16-byte aligned.
 *  w_router:   [E][D] bf16 (nn.Linear layout), one copy shared by every rank,
 *              16-byte aligned.
 *  forced_ids, topk_ids, topk_w: as moe_route.
 *  logits:     NULL, or out [W][T][E] fp32: the scores the routing used.
 *  splits:     0 picks the kernel: for E <= 16 one that streams the token rows
 *              from HBM into registers and takes the scores with mma.sync (the
 *              contraction is 8 or 16 columns wide and the launch a one-shot read
 *              of x), in CTAs of 32 tokens and 8 warps (16 tokens and 4 warps with
 *              9-16 experts) when there are enough of them to fill every SM, else in
 *              larger CTAs that spread the tokens over one wave; above, the tcgen05
 *              kernel with the K split it picks. 1, 2, 4 or 8 force the tcgen05
 *              kernel with that split (that many CTAs of one cluster share a
 *              128-token tile, each summing a range of D).
 *              MOE_GATE_BESIDE: for E <= 16 always the small CTAs, which fit in what a
 *              pair-producer CTA leaves of its SM, so the gate of the next batch runs
 *              beside a running combine instead of waiting for its SMs; above, as 0.
 * Both kernels add each score's partial sums in a fixed order, so a given choice
 * gives the same bits on every call; the two kernels' scores differ by rounding
 * only. A tcgen05 tile holds as many tokens (a multiple of 8, at most 128) as fill
 * one wave of CTAs.
 * The routing tail also sets the plan's token bitmaps (prescribed ids out of range
 * or repeated set MOE_DEV_ROUTING), for a following moe_plan_build(plan, NULL, ...).
 * E <= 256; larger E, or a split the GPU cannot hold, gives MOE_ERR_UNSUPPORTED.
 * The caller owns every buffer. Timed in slot [0] of moe_timings, its device-clock
 * span in slot [9]. */
int moe_gate(moe_plan *plan, const void *const *x, const void *w_router,
             const int32_t *forced_ids, int32_t *topk_ids, float *topk_w, float *logits,
             int splits, moe_stream_t stream);

/* Expert problem construction and combine plan (TileMoE notes section 4.2, 4.4
 * Algorithm 1, 4.5, 5.2) for all ranks, then the layout gather that fills each
 * owner's expert input X with its tokens' rows (zero rows for padding).
 *  topk_ids: [W][T][topk] int32, ids distinct within a token; or NULL: the routing of
 *            the last moe_gate on this plan (no moe_route or moe_plan_build since),
 *            whose routing tail already set the plan's token bitmaps, so the bitmap
 *            kernel is skipped; MOE_ERR_ARG if there is none.
 *  x:        W pointers, rank s's tokens [T][D] bf16.
 * Ids out of range or repeated set MOE_DEV_ROUTING; the offending assignments are
 * skipped. No device-to-host transfer: every size is read on the device. */
int moe_plan_build(moe_plan *plan, const int32_t *topk_ids, const void *const *x,
                   moe_stream_t stream);

/* Overlapped expert FFN and combine (TileMoE notes section 5.1-5.3).
 * The producer walks the remote-first schedule: per 128-row tile of X,
 * h = SiLU(X Wg^T) * (X Wu^T) (bf16), then Y = h Wd^T (bf16), fp32 accumulation,
 * and after each finished Y tile it sets that tile's ready flag. The consumer
 * (consumer_ctas CTAs on a high-priority stream, or after the producer in serial
 * mode) polls the flags and copies each finished segment's valid rows into the
 * destination rank's receive buffer at the planned offset. Padding rows are never
 * copied. Local rows stay in the owner's Y.
 *  w_gate, w_up: W pointers, [L][F][D] bf16.  w_down: W pointers, [L][D][F] bf16.
 *  recv:         W pointers, [recv_rows][D] bf16 (moe_workspace_size).
 *  producer, consumer: streams; the consumer stream should have higher priority.
 *  When consumer_ctas == 0 or both streams are equal, the call runs serially on
 *  `producer`. On return, work enqueued later on `producer` is ordered after both
 *  kernels. */
int moe_expert_combine(moe_plan *plan, const void *const *w_gate, const void *const *w_up,
                       const void *const *w_down, void *const *recv,
                       moe_stream_t producer, moe_stream_t consumer);

/* Scale (TileMoE notes section 2.2 step 5): out_s[t] = sum_j w[s][t][j] * y_j, where
 * y_j is token (s,t)'s output of its j-th expert, read from rank s's receive buffer
 * (remote expert) or rank s's own Y (local expert). fp32 accumulation in slot order,
 * bf16 result.
 *  topk_w: [W][T][topk] fp32.  recv: W pointers as given to moe_expert_combine.
 *  out:    W pointers, [T][D] bf16. */
int moe_scale(moe_plan *plan, const float *topk_w, const void *const *recv, void *const *out,
              moe_stream_t stream);

/* Scale overlapped with the combine (TileMoE notes section 2.2 step 5; the Perseus
 * summary, section 4.1, Algorithm 1: the receiver acts on the one signal of each
 * (sender, destination) group). Same arguments and the same results, bit for bit,
 * as moe_scale, for the routing of the last moe_expert_combine. Enqueue it on that
 * call's producer stream right after it: the kernel is launched with programmatic
 * stream serialization, so it starts once every CTA of the kernel before it on the
 * stream (the producer; the consumer in the serial schedule) is running, and works
 * beside it. A token's sum waits on the device until its rows are final: the signal
 * of each remote slot's (sender, destination) group and the ready flags of each
 * local slot's row band; tokens whose slots are all remote go first. Any other work
 * between the combine and this call on the stream (an event, a wait) makes it start
 * after the combine instead, with the same results. Waits are bounded by timeout_ns
 * (MOE_DEV_TIMEOUT); a status already set makes the kernel return. One call per
 * moe_expert_combine, on its producer stream (MOE_ERR_ARG otherwise). No CUDA events are recorded around it
 * (they would keep it from overlapping); with moe_set_timing(plan, 2) the device clock
 * records its span (moe_timings slots 7 and 8). */
int moe_scale_gated(moe_plan *plan, const float *topk_w, const void *const *recv,
                    void *const *out, moe_stream_t stream);

/* Overlap of the combine copy with the expert FFN in the last moe_expert_combine made
 * while device-clock records were on (moe_set_timing 1 or 2), the quantity of the TileMoE
 * notes' section 7.3 (overlap ratio of the second all-to-all): *landed_frac is the share
 * of the combine's bytes whose copies had landed when the producer finished its last
 * output tile, *tail_us how long after that tile the last copy landed (negative if
 * before), *copy_bytes the bytes copied. Synchronises the device. MOE_ERR_ARG if no
 * such combine was recorded; MOE_ERR_UNSUPPORTED if host memory for copies of the
 * segment records and stamps cannot be had. Any output pointer may be NULL. */
int moe_combine_overlap(moe_plan *plan, double *landed_frac, double *tail_us,
                        double *copy_bytes);

/* The device-clock intervals of the producer launches recorded while device-clock
 * records were on (moe_set_timing 1 or 2), oldest first: start_ns[i], end_ns[i] are
 * the i-th launch's first CTA start and last CTA end on the GPU's global timer
 * (nanoseconds; comparable across the plans of one device, so a caller running
 * several plans in turn can take the union of their launches). At most max_records of
 * the last 1024 launches; *count receives how many were written. Synchronises the
 * device. MOE_ERR_ARG without records. */
int moe_producer_spans(moe_plan *plan, unsigned long long *start_ns, unsigned long long *end_ns,
                       int max_records, int *count);

/* Plan build that allocates nothing, for callers that cannot call cudaMalloc (for
 * example a serving loop that reserved all of its device memory up front, or a
 * runtime whose device memory comes from an allocator it does not own). The pages
 * have no counterpart. It runs moe_plan_build's plan kernels on the same routing
 * and writes the same plan, but not the layout gather (X is not filled).
 *  topk_ids: [W][T][topk] int32 (input).
 *  plan_out: caller buffer of at least the plan_bytes of moe_workspace_size(),
 *            256-byte aligned; the plan arrays are written where moe_plan_build
 *            writes them in a plan workspace (moe_field() reports the public ones).
 *            Bad routing ids set the MOE_PLAN_STATUS word inside plan_out, which
 *            this call never clears. A plan handle created on plan_out
 *            (moe_plan_create) can then run moe_expert_combine and moe_scale on it,
 *            given rank workspaces whose X a moe_plan_build of the same routing
 *            filled. The regions of the plan kernels' internal arrays (token
 *            bitmaps, word prefixes, per-band and per-tile orderings, segment
 *            indices) are left untouched in plan_out, as is the per-combine region.
 * Those internal arrays live in a fixed 1 MiB array inside the library, which every
 * GPU that loads the library holds until the process exits; shapes whose internal
 * arrays exceed it return MOE_ERR_UNSUPPORTED. No cudaMalloc, cudaFree or
 * allocating library call is made. The first call on each device looks up that
 * array's device address (cudaGetSymbolAddress, with the device current) and may
 * load the library's kernels: make it before any stream capture. Every call shares
 * the one array, so calls that overlap on the GPU (other streams, other threads)
 * race; serialise them. Host threads may make calls at the same time. */
int moe_plan_build_noalloc(const moe_cfg *cfg, const int32_t *topk_ids, void *plan_out,
                           size_t plan_out_bytes, moe_stream_t stream);

/* Changes the schedule of an existing plan: the consumer partition (consumer_ctas of
 * moe_cfg; 0 = serial) and the segment merge width (mgb of moe_cfg, section 5.2). Host
 * only; a new mgb takes effect at the next moe_plan_build, a new consumer_ctas at the
 * next moe_expert_combine. Same limits as in moe_cfg: MOE_ERR_ARG for values out of
 * range, MOE_ERR_UNSUPPORTED if a segment of mgb bands would exceed the copy-chunk limit.
 * The workspaces are unchanged (their sizes do not depend on either value). */
int moe_set_schedule(moe_plan *plan, int consumer_ctas, int mgb);

/* How moe_expert_combine splits the GPU for this plan (pure host query; the
 * occupancy is read once by moe_plan_create).
 *  producer_ctas:   CTAs of one producer launch in the overlapped schedule (even
 *                   with producer_pairs: clusters of two that fit on the GPU at once).
 *  consumer_ctas:   CTAs of one consumer launch in the overlapped schedule.
 *  num_sms:         SMs of the device.
 *  pair_clusters:   clusters of two CTAs of the pair producer that fit on an idle
 *                   GPU at once (0 if the runtime could not tell).
 * Any output pointer may be NULL. */
int moe_launch_info(moe_plan *plan, int *producer_ctas, int *consumer_ctas, int *num_sms,
                    int *pair_clusters);

/* Synchronises `stream` and reads the device status word: *code is 0 or a
 * MOE_DEV_* value, *detail the first failing item (token, band or tile index).
 * The status stays set until moe_status_clear(). */
int moe_status(moe_plan *plan, moe_stream_t stream, int *code, int *detail);
int moe_status_clear(moe_plan *plan, moe_stream_t stream);

/* Named arrays of the plan workspace and the rank workspaces, for inspection:
 * byte offset of the array inside its workspace and its element count. Elements
 * are int32 except MOE_RANK_X/H/Y (bf16). Pure host arithmetic. */
enum moe_field {
  MOE_PLAN_CNT = 0,          /* [E][W] rows of expert e from rank s */
  MOE_PLAN_GROUP_START,      /* [E][W] first row of group (e, s) in expert e's block */
  MOE_PLAN_RECV_OFF,         /* [E][W] first receive row of (e, s) at rank s, -1 if local */
  MOE_PLAN_EXPERT_START,     /* [E]    first row of expert e's block in its owner's X */
  MOE_PLAN_ROWS_ALLOC,       /* [E]    rows of expert e's block (multiple of tb_M) */
  MOE_PLAN_NRB,              /* [E]    remote row bands of expert e */
  MOE_PLAN_RANK_ROWS,        /* [W]    rows of each owner's X */
  MOE_PLAN_RANK_NREMOTE,     /* [W]    remote prefix length of each owner's schedule */
  MOE_PLAN_RECV_ROWS,        /* [W]    rows received by each rank */
  MOE_PLAN_RANK_NSEG,        /* [W]    segments of each owner */
  MOE_PLAN_BAND_EXPERT,      /* [W][NBmax] per rank-local band: expert */
  MOE_PLAN_BAND_DST,         /* [W][NBmax] destination rank */
  MOE_PLAN_BAND_VALID,       /* [W][NBmax] valid (non-padding) rows */
  MOE_PLAN_BAND_DST_ROW,     /* [W][NBmax] first receive row at the destination, -1 if local */
  MOE_PLAN_SCHEDULE,         /* [W][NBmax] S: rank-local band ids in schedule order */
  MOE_PLAN_SEG_FIRST,        /* [W][NBmax] first schedule index of each segment */
  MOE_PLAN_SEG_NBANDS,       /* [W][NBmax] bands of each segment */
  MOE_PLAN_XSRC,             /* [W][RowsMax] per X row: source token s*T+t, or -1 */
  MOE_PLAN_SCALE_SRC,        /* [W][T][topk] >= 0: receive row; < 0: row -v-1 of own Y */
  MOE_PLAN_TOTALS,           /* [8] 0: tiles, 1: segments, 2: tile units, 3: bands,
                                4: consumer copy chunks, 5: producer CTA pairs */
  MOE_PLAN_TILE_ROW,         /* [tiles] per 128-row producer tile: rank*2^24 + first X row */
  MOE_PLAN_TILE_EXPERT,      /* [tiles] expert of each producer tile */
  MOE_PLAN_SEG_ORDER,        /* [segments] consumer order: rank*NBmax + segment */
  MOE_PLAN_STATUS,           /* [4] device status word */
  MOE_PLAN_FLAGS,            /* [W][NBmax][D/tile_N] ready flags of the last combine */
  MOE_PLAN_GROUP_SIG,        /* [W][W] group signals (sender, destination) of the last combine */
  MOE_PLAN_PAIR,             /* [pairs][4] producer CTA pairs in pair order: the earlier tile of
                                the tile order, its partner or -1, the earlier tile's
                                rank*2^24 + first X row, and its local expert + 2^16 if the
                                partner's rows lie 128 above */
  MOE_PLAN_NFIELDS,
  MOE_RANK_X = 100,          /* [RowsMax][D] bf16 expert input */
  MOE_RANK_H,                /* [RowsMax][F] bf16 hidden activation */
  MOE_RANK_Y                 /* [RowsMax][D] bf16 expert output */
};
int moe_field(const moe_cfg *cfg, int field, size_t *byte_offset, size_t *count);

/* Device time in ms of the kernels the calls enqueue, measured with CUDA events
 * recorded on the stream each kernel ran on: the mean over the calls made since
 * timing was last enabled (the most recent 64 of them). Synchronises on those
 * events. Order: [0] route (moe_route or moe_gate), [1] plan (all plan kernels and the gather),
 * [2] producer, [3] consumer, [4] scale, [5] gather only. Then, from the device clock,
 * means over the last 1024 combines: [6] the producer's execution span (its first CTA's
 * start to its last CTA's end; unlike [2] it excludes time spent queued behind other
 * kernels, for example those of another batch in flight, and the launch latency CUDA
 * events include), [7] the span of the scale (moe_scale or moe_scale_gated) after the
 * combine, [8] the part of [7] before the producer's end, [9] the span of moe_gate,
 * [10] the span of the consumer kernel (not the fused copy warp), [11] the span of the
 * layout gather of moe_plan_build. A slot with no measurement is -1. Instrumentation only: moe_set_timing(plan, 1) records the events
 * and the device-clock records, 2 only the device-clock records (no CUDA event enters
 * the streams, so kernels keep overlapping as without timing), 0 nothing; enabling
 * resets the counts. */
int moe_set_timing(moe_plan *plan, int enable);
int moe_timings(moe_plan *plan, float *ms, int n);

/* ---------------------------------------------------------------------------
 * Operators of the transformer block around the routed experts. They need no plan:
 * every call takes its tensors, works on the current device (compute capability 10.3,
 * else MOE_ERR_UNSUPPORTED) and is asynchronous on `stream`. Matrices are row-major
 * with a leading dimension ld_* in elements (at least the row's length). Base pointers
 * need the alignment of their element type only, unless stated. Inputs and outputs of
 * a call do not overlap. n = 0 rows is a call that does nothing (gradients of weights
 * are then zero). The first call on a device loads the kernels: make it before a
 * stream capture; every later call may be captured.
 * ------------------------------------------------------------------------- */
enum moe_dtype {
  MOE_BF16 = 0,
  MOE_FP16 = 1,
  MOE_FP32 = 2
};

enum moe_score {
  MOE_SCORE_SOFTMAX = 0, /* exp(l_e) / sum_i exp(l_i) */
  MOE_SCORE_SIGMOID = 1  /* 1 / (1 + exp(-l_e)) */
};

/* Routing to experts from their scores l (moe_router). */
typedef struct moe_router_cfg {
  int E;           /* experts, 1..1024 */
  int topk;        /* experts chosen for each token, 1..min(E, 32) */
  int score;       /* enum moe_score */
  int groups;      /* groups of E / groups consecutive experts (1..32, divides E); 1: none */
  int topk_groups; /* groups that stay, 1..groups; topk <= topk_groups * E / groups */
  int group_top;   /* a group is judged by the sum of its 1 or 2 largest s + bias */
  int renorm;      /* 1: the chosen experts' scores are divided by their sum */
  float scale;     /* factor of every weight, finite */
} moe_router_cfg;

/* For every token: s = score(l), c = s + bias; the topk_groups best groups stay, and of
 * their experts the topk with the largest c, in descending order (equal c: the lower id;
 * equal groups: the lower group). weight = s at the chosen id (without the bias), divided
 * by the sum of the chosen s with renorm, times scale. The choice is that of 64-bit arithmetic.
 * Without a bias the order of the c, and of groups judged by one of them, is that of the l: scores
 * that even 64 bits round to the same (a sigmoid beyond 37; 0 for l = -inf and for a very low
 * l) are told apart there, where with a bias they tie.
 * l = -inf masks an expert (s = 0); bias = -inf keeps it from being chosen while another
 * is left. A token whose chosen s are all 0 has weights 0 and valid, distinct ids. A NaN
 * score counts as -inf in the order, and the weights computed from it are NaN.
 *  plan:   NULL, or the plan whose moe_plan_build reads these ids next: then E, topk and
 *          n = W*T are the plan's, ids and w are 16-byte aligned, the call is timed in
 *          slot [0] of moe_timings, and the routing of an earlier moe_gate is forgotten.
 *  logits: [n][E] of `dtype` (enum moe_dtype), leading dimension ld.
 *  bias:   NULL or [E] fp32.   ids: out [n][topk] int32.   w: out [n][topk] fp32. */
int moe_router(moe_plan *plan, const moe_router_cfg *cfg, const void *logits, int dtype,
               long long n, long long ld, const float *bias, int32_t *ids, float *w,
               moe_stream_t stream);

/* Gradient of the scores from the gradient of the weights, for the ids that moe_router
 * chose (the choice itself, and so the bias, has none): d_logits, out [n][E] of `dtype`,
 * leading dimension ld_d, written whole. d_w: [n][topk] fp32. The ids of a token are
 * distinct; one out of range has no gradient. */
int moe_router_backward(const moe_router_cfg *cfg, const float *d_w, const void *logits,
                        const int32_t *ids, int dtype, long long n, long long ld,
                        void *d_logits, long long ld_d, moe_stream_t stream);

/* Layer norm of n rows of D elements, forward and backward. */
typedef struct moe_norm_args {
  long long n;      /* rows */
  int D;            /* elements of a row, 1..2^24 */
  int dtype;        /* enum moe_dtype of the matrices */
  int wtype;        /* of w, b, dw and db: dtype or MOE_FP32 */
  float eps;        /* >= 0, finite (forward) */
  const void *x;    /* forward: in [n][D] */
  const void *r;    /* forward: in [n][D], the residual stream, or NULL */
  const void *w;    /* in [D], or NULL: ones */
  const void *b;    /* forward: in [D], or NULL: zeros */
  void *y;          /* forward: out [n][D] */
  void *z;          /* forward: out [n][D], x + r, or NULL; backward: in, the normalised rows */
  float *mean;      /* [n]: forward: out or NULL; backward: in */
  float *rstd;      /* [n]: forward: out or NULL; backward: in */
  const void *dy;   /* backward: in [n][D], gradient of y */
  const void *dz;   /* backward: in [n][D], gradient of z from elsewhere, or NULL */
  void *dx;         /* backward: out [n][D], gradient of x (and of r) */
  void *dw;         /* backward: out [D] or NULL */
  void *db;         /* backward: out [D] or NULL */
  long long ld_x, ld_r, ld_y, ld_z, ld_dy, ld_dz, ld_dx;
} moe_norm_args;

/* z = x + r, y = (z - mean) * rstd * w + b with mean and rstd = 1 / sqrt(variance + eps)
 * of each row of z (fp32; the variance is the mean squared distance). y, and z where it is
 * stored, are rounded once from fp32. */
int moe_layer_norm(const moe_norm_args *args, moe_stream_t stream);

/* dx = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dz with g = dy * w and
 * xhat = (z - mean) * rstd; dw = sum over rows of dy * xhat; db = sum over rows of dy.
 * workspace: at least moe_layer_norm_workspace(n, D) bytes (pure host arithmetic), 16-byte
 * aligned, used
 * until the call has run on the stream. The sums are added in a fixed order. */
size_t moe_layer_norm_workspace(long long n, int D);
int moe_layer_norm_backward(const moe_norm_args *args, void *workspace, size_t workspace_bytes,
                            moe_stream_t stream);

enum moe_act {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU,
  MOE_ACT_GELU,      /* 0.5 z (1 + erf(z / sqrt(2))) */
  MOE_ACT_GELU_TANH, /* 0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
  MOE_ACT_SILU       /* z / (1 + exp(-z)) */
};

/* Matrix product with an epilogue, forward and backward. dtype is MOE_BF16 or MOE_FP16. x
 * and w (and dy, to be read in place) have 16-byte aligned bases and leading dimensions
 * that are multiples of 8; M, N and K are any, and the other matrices may lie anywhere. */
typedef struct moe_linear_args {
  long long M, N, K; /* M >= 0, N >= 1, K >= 1 */
  int dtype;         /* of x, w, r, z, dy and dx */
  int ytype;         /* of y: dtype or MOE_FP32 */
  int btype;         /* of b and db: dtype or MOE_FP32 */
  int dwtype;        /* of dw: dtype or MOE_FP32 */
  int act;           /* enum moe_act */
  const void *x;     /* in [M][K] (backward: only for dw) */
  const void *w;     /* in [N][K] (backward: only for dx) */
  const void *b;     /* forward: in [N] or NULL */
  const void *r;     /* forward: in [M][N], the residual, or NULL */
  void *y;           /* forward: out [M][N] */
  void *z;           /* forward: out [M][N] or NULL; backward: in, if act is not none */
  const void *dy;    /* backward: in [M][N], gradient of y (and of r) */
  void *dx;          /* backward: out [M][K] or NULL */
  void *dw;          /* backward: out [N][K] or NULL */
  void *db;          /* backward: out [N] or NULL */
  long long ld_x, ld_w, ld_r, ld_y, ld_z, ld_dy, ld_dx, ld_dw;
  const uint8_t *z_scales; /* backward: in [M][ceil(N / 32)] where z are the codes of an 8-bit
                              checkpoint (moe_checkpoint), else NULL */
  const uint8_t *x_scales; /* backward: in [M][ceil(K / 32)] where x are such codes, rows of K bytes
                              (K a multiple of 8, 8-byte aligned), else NULL */
} moe_linear_args;

/* z = x w^T + b, y = act(z) + r: fp32 sums, y and z rounded once from fp32. */
int moe_linear(const moe_linear_args *args, moe_stream_t stream);

/* dz = dy * act'(z); db = sum over rows of dz; dx = dz w; dw = dz^T x. The products take
 * dz rounded to dtype, db takes it in fp32; all sums are fp32, in a fixed order. Those of dw are long:
 * the tensor cores lose about 1.2e-9 of dw's norm for each row that is summed at once (which is some or
 * all of the M), 1e-5 for 65536 rows of 256 x 512, 1.5e-4 for 1048576.
 * workspace: at least moe_linear_workspace(M, N) bytes (pure host arithmetic), 256-byte
 * aligned, used until the call has run on the stream; where dw is made from a checkpoint of x, and
 * moe_linear_kept_bytes(M, K) more, for x in dtype. */
size_t moe_linear_workspace(long long M, long long N);
size_t moe_linear_kept_bytes(long long M, long long K);
int moe_linear_backward(const moe_linear_args *args, void *workspace, size_t workspace_bytes,
                        moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Tokens as rows in the order of their experts, and back. n = T * topk slots: slot
 * t * topk + j is choice j of token t.
 * ------------------------------------------------------------------------- */

/* The stable order of the n slots by expert: offsets, out [E + 1]: expert e has the rows
 * offsets[e] .. offsets[e + 1] - 1; rows, out [n]: the row of each slot, -1 where ids is not in
 * 0 .. E - 1; slots, out [n]: the slot of each row, -1 behind the last. A token may choose an
 * expert twice. n is below 2^30, E at most 1024. workspace: at least
 * moe_sort_experts_workspace(n, E) bytes (pure host arithmetic; 0 for few slots), 16-byte aligned,
 * used until the call has run on the stream. */
size_t moe_sort_experts_workspace(long long n, int E);
int moe_sort_experts(const int32_t *ids, long long n, int E, int32_t *slots, int32_t *rows,
                     int32_t *offsets, void *workspace, size_t workspace_bytes,
                     moe_stream_t stream);

typedef struct moe_rows_args {
  long long T, D;          /* tokens; elements of a row */
  int topk, E;             /* topk 1..32, T * topk below 2^30; E 1..1024 */
  int dtype;               /* enum moe_dtype of the matrices */
  const int32_t *rows;     /* in [T][topk], of moe_sort_experts; outside 0 .. n - 1: no row */
  const int32_t *offsets;  /* in [E + 1]; the rows from offsets[E] on have no slot */
  const float *w;          /* combine, backward: in [T][topk]; combine: or NULL, ones */
  const void *x;           /* rows: in [T][D]; backward: in, the gradient of y */
  void *y;                 /* combine: out [T][D] */
  const void *r;           /* combine, backward: in [n][D]; backward: of dtype or e4m3 codes */
  const uint8_t *r_scales; /* backward: in [n][ceil(D / 32)], the scales of codes, or NULL */
  void *dr;                /* rows, backward: out [n][D] */
  float *dw;               /* backward: out [T][topk] */
  long long ld_x, ld_y, ld_r, ld_scales, ld_dr;
} moe_rows_args;

/* dr[rows[t][j]] = x[t]; rows without a slot are zero. */
int moe_expert_rows(const moe_rows_args *args, moe_stream_t stream);

/* y[t] = sum over j of w[t][j] * r[rows[t][j]], in the order of j in fp32, rounded once; slots without
 * a row have no part in it. With w = NULL it is the gradient of moe_expert_rows. */
int moe_combine_experts(const moe_rows_args *args, moe_stream_t stream);

/* dr[rows[t][j]] = w[t][j] * x[t] (rows without a slot: zero) and dw[t][j] = the product of x[t]
 * and r[rows[t][j]] (0 without a row), fp32 sums in a fixed order. */
int moe_combine_experts_backward(const moe_rows_args *args, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Checkpoints in 8 bits: what a backward pass needs of a forward pass, in half the bytes.
 * Blocks of 32 elements of a row (the last one of a row may be shorter) share a scale 2^s, stored
 * as s + 127, with the least s in -127 .. 127 for which the block's largest finite |x| is at most
 * 448 * 2^s; the code of an element is x * 2^-s rounded to e4m3, to nearest, ties to even, NaN
 * where x is not finite, and the code below where that one would stand for more than dtype holds
 * (|x| from 63488 on in fp16, from 1.9375 * 2^127 on in the others). Restored in dtype, an element is
 * within 2^-4 of itself, or within 2^-10 * 2^s.
 * ------------------------------------------------------------------------- */
typedef struct moe_checkpoint_args {
  long long n, c;   /* rows; elements of a row */
  int dtype;        /* enum moe_dtype of x */
  void *x;          /* checkpoint: in [n][c]; restore: out */
  void *codes;      /* checkpoint: out [n][c] e4m3; restore: in */
  uint8_t *scales;  /* checkpoint: out [n][ceil(c / 32)]; restore: in */
  long long ld_x, ld_codes, ld_scales;
} moe_checkpoint_args;
int moe_checkpoint(const moe_checkpoint_args *args, moe_stream_t stream);
/* x = code * 2^s, rounded once to dtype (exact in fp32). */
int moe_restore(const moe_checkpoint_args *args, moe_stream_t stream);

/* Gated activation of n rows of c elements. dtype is MOE_BF16 or MOE_FP16. The scales' rows are
 * ceil(c / 32) bytes apart, the codes' rows c. */
typedef struct moe_gated_args {
  long long n, c;
  int dtype;            /* of the matrices that are not codes */
  int act;              /* enum moe_act */
  const void *gate;     /* in [n][c]; backward: of dtype, or codes with gate_scales */
  const void *up;       /* in [n][c], as gate */
  void *h;              /* out [n][c], act(gate) * up; backward: or NULL */
  void *gate_codes, *up_codes;       /* forward: out, 8-bit checkpoints of gate and up, or all NULL */
  uint8_t *gate_scales, *up_scales;  /* forward: out; backward: in, or NULL: gate and up of dtype */
  const void *dh;       /* backward: in [n][c] */
  void *dgate, *dup;    /* backward: out [n][c] */
  long long ld_gate, ld_up, ld_h, ld_dh, ld_dgate, ld_dup;
} moe_gated_args;
/* h = act(gate) * up, rounded once from fp32. */
int moe_gated(const moe_gated_args *args, moe_stream_t stream);
/* dgate = dh * up * act'(gate), dup = dh * act(gate), h = act(gate) * up once more. */
int moe_gated_backward(const moe_gated_args *args, moe_stream_t stream);

/* The experts' matrix products: rows sorted by expert (moe_sort_experts), each expert with its own
 * weights. dtype is MOE_BF16 or MOE_FP16; N and K are multiples of 8, E is at most 1024. All
 * matrices have 16-byte aligned bases and leading dimensions (and strides from expert to
 * expert) that are multiples of 8. */
typedef struct moe_expert_linear_args {
  long long n, N, K;      /* rows; features of y; features of x */
  int E;
  int dtype;              /* of all matrices but dw */
  int dwtype;             /* of dw: dtype or MOE_FP32 */
  const int32_t *offsets; /* in [E + 1], on the device, ascending: expert e has the rows offsets[e] to
                             offsets[e + 1] - 1; what lies outside 0 .. n is left out */
  const void *x;          /* in [n][K] (backward: only for dw) */
  const void *w;          /* in [E][N][K] (backward: only for dx) */
  void *y;                /* forward: out [n][N] */
  const void *dy;         /* backward: in [n][N] */
  const void *add;        /* backward: in [n][K], or NULL */
  void *dx;               /* backward: out [n][K] or NULL */
  void *dw;               /* backward: out [E][N][K] or NULL */
  long long ld_x, ld_w, stride_w, ld_y, ld_dy, ld_add, ld_dx, ld_dw, stride_dw;
} moe_expert_linear_args;

/* y[r] = w[e] x[r] for the rows of every expert e, fp32 sums, rounded once; rows before offsets[0] and
 * from offsets[E] on are zero. workspace: at least moe_expert_linear_workspace(n, N, K, E) bytes (pure host arithmetic;
 * 0 but for few rows and a long sum), 16-byte aligned, used until the call has run on the stream. */
size_t moe_expert_linear_workspace(long long n, long long features, long long sum, int E);
int moe_expert_linear(const moe_expert_linear_args *args, void *workspace, size_t workspace_bytes,
                      moe_stream_t stream);

/* dx[r] = w[e]^T dy[r] + add[r] (rows before offsets[0] and from offsets[E] on: add alone, or zero);
 * dw[e] = sum over its rows of dy[r] x[r]^T (zero without rows). fp32 sums in a fixed order, rounded
 * once. In fp32 dw is summed by parts of the rows and within 1.2e-6 of its norm up to a million rows of
 * an expert; in 16 bits all rows are one sum, which loses 1.2e-9 of the norm for each: as much as the
 * rounding to fp16 at some 170000 rows of one expert, to bf16 at 1.4 million. workspace: for dx, at
 * least moe_expert_linear_workspace(n, K, N, E) bytes, as above. */
int moe_expert_linear_backward(const moe_expert_linear_args *args, void *workspace,
                               size_t workspace_bytes, moe_stream_t stream);

/* The device waits of the products and of layer norm are bounded; one that runs out sets a
 * sticky status of the device (its results are void). Synchronises `stream` and reads the
 * status of that stream's device, whichever is current (of the current one for a default
 * stream): *code is 0 or MOE_DEV_TIMEOUT, *detail the wait. */
int moe_ops_status(moe_stream_t stream, int *code, int *detail);
int moe_ops_status_clear(moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TSG_H */
