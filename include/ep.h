/*
 * ep.h -- C ABI of libep: deterministic MoE expert-parallel dispatch layout,
 * dispatch (scatter + copy epilogue) and combine on one GPU's share of the
 * work, the router before it, the experts' products inside it and the
 * gradients of all three, as HIP kernels for CDNA4 (gfx950).
 *
 * Sources (DeepEP v2 pages):
 *   [DET] "DeepEP v2: Kernel-side deterministic dispatch for the non-expand
 *         layout" (PR #753): sections Motivation, Approach, Direct vs hybrid
 *         dispatch, Compatibility, New API.
 *   [DRX] "DeepEP v2: Add experimental direct recv_x dispatch path" (PR #690):
 *         sections Background, Direct Recv X design, Implementation, and the
 *         review's buffer-size and guardrail comments.
 *   [UNO] "Add unordered hybrid kernels for transports without ordered
 *         delivery" (PR #732): section Changes (combine reduce epilogue).
 *
 * Model.  S source partitions ("source ranks") each hold T tokens; every token
 * routes to K experts out of E, and expert e lives on logical rank e / El,
 * El = E / R.  All S sources and all R destinations are partitions of the one
 * GPU's HBM: a "send" is a local store, and stream order replaces the pages'
 * signals and release atomics.
 *
 * Conventions for every call:
 *   - pointers named *_dev are device pointers the caller allocated (for
 *     example with torch.empty(..., device="cuda")); the library never
 *     allocates or frees, and keeps nothing between calls but the per-GPU
 *     array of ep_layout_no_alloc and cached device properties;
 *   - all arrays are dense row-major; rows of x, staging and recv are 16-byte
 *     aligned (the base pointers must be 16-byte aligned, and the row size in
 *     bytes is a multiple of 16);
 *   - `stream` is a hipStream_t (NULL = the default stream); calls only
 *     enqueue work on it and never synchronise;
 *   - argument errors are detected on the host before anything is enqueued
 *     and return a negative ep_status; a failed launch returns EP_ERR_HIP;
 *   - data errors found on the device (a top-k id >= E) set bit 0 of
 *     *error_flags and the lane is then treated as masked (id < 0); bit 1
 *     reports a timed-out one-launch layout (EP_FLAG_LAYOUT_ONE_LAUNCH);
 *   - calls on different streams with disjoint buffers may run concurrently.
 */
#ifndef EP_H
#define EP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum ep_status {
    EP_OK = 0,
    EP_ERR_INVALID_ARG = -1, /* a size, dtype or pointer is not acceptable    */
    EP_ERR_CAPACITY = -2,    /* Nmax < T, or a buffer is smaller than needed  */
    EP_ERR_UNSUPPORTED = -3, /* outside the limits below                      */
    EP_ERR_HIP = -4          /* the HIP runtime refused a launch              */
};

enum ep_dtype {
    EP_DTYPE_BF16 = 0,        /* rows of H bf16                                */
    EP_DTYPE_FP8_E4M3FN = 1,  /* rows of H OCP e4m3fn bytes + H/128 fp32 scales */
    EP_DTYPE_FP32 = 2         /* the router's logits only                      */
};

/* Phases of ep_dispatch.  The pages time the sender's dispatch kernel and the
 * receiver's copy epilogue separately ([DET] Performance, [DRX] Background);
 * a caller may enqueue them in two calls (for example with its own event
 * between them).  EP_PHASE_ALL runs both. */
enum ep_phase {
    EP_PHASE_SCATTER = 1,
    EP_PHASE_EPILOGUE = 2,
    EP_PHASE_ALL = 3
};

/* Option bits of ep_config_t.flags. */
enum ep_flags {
    /* Direct Recv X ([DRX] Direct Recv X design): the scatter writes each hidden
     * row straight into its compact receive row recv_base[d] + recv_psum[d][s]
     * + j instead of the staging row; staging keeps the scales and metadata,
     * and the epilogue produces recv_sf and the metadata tensors but copies no
     * hidden bytes.  staging_x is not used (may be NULL).  Compact layout only
     * (EP_ERR_UNSUPPORTED with expand), as on the page. */
    EP_FLAG_DIRECT_RECV_X = 1,
    /* ep_layout of the compact layout as one launch, the form [DET] Approach
     * describes (a cooperative two-pass scan whose passes exchange their
     * counts grid-wide), used when its whole grid fits on the device at once
     * (checked on the host before the launch; otherwise the separate count
     * and slot launches run).  Same tables as the default two launches, which
     * measured faster on MI355X (8.3 against 9-11 us back to back at 4096
     * tokens, top-8 of 256 on 16 ranks): the device's kernel boundary is
     * cheaper than the exchange.  Its waits are bounded (far above any normal
     * duration); a layout whose exchange times out sets bit 1 of
     * *error_flags, and its tables are then not valid. */
    EP_FLAG_LAYOUT_ONE_LAUNCH = 2
};

/* Limits (checked on the host): 1 <= R <= 64, 1 <= K <= 32, E % R == 0,
 * E <= 1024, S <= 65535, T <= 2^30, H <= 262144, S * Nmax < 2^31,
 * S * T * K < 2^31, H * element size a multiple of 16 bytes, fp8 needs
 * H % 128 == 0.  Outside them a call returns EP_ERR_UNSUPPORTED. */
#define EP_MAX_RANKS 64
#define EP_MAX_TOKENS (1 << 30)
#define EP_MAX_TOPK 32
#define EP_MAX_EXPERTS 1024
#define EP_MAX_HIDDEN 262144

typedef struct ep_config {
    int32_t num_src_ranks;            /* S >= 1                                  */
    int32_t num_tokens;               /* T >= 0, tokens per source               */
    int32_t hidden;                   /* H                                       */
    int32_t num_topk;                 /* K                                       */
    int32_t num_experts;              /* E                                       */
    int32_t num_ranks;                /* R, destination ranks                    */
    int32_t num_max_tokens_per_rank;  /* Nmax >= T, else EP_ERR_CAPACITY: the
                                         rows a source may fill at one
                                         destination ([DET] Approach)            */
    int32_t x_dtype;                  /* enum ep_dtype                           */
    int32_t expand;                   /* 0: compact receive layout; 1: one row
                                         per valid (token, top-k) lane, grouped
                                         by expert                               */
    int32_t expert_alignment;         /* A >= 1; expand segments are padded to a
                                         multiple of A (ignored if !expand)      */
    int32_t num_layout_cus;           /* workgroups of the layout pass; 0 = auto
                                         (the pages' num_prologue_sms, [DET] New
                                         API); never changes any result          */
    int32_t flags;                    /* enum ep_flags bits; others must be 0    */
    int32_t num_scaleout_ranks;       /* 0 or 1: direct path.  > 1: hybrid path
                                         ([DET] Direct vs hybrid dispatch): the
                                         S source ranks are num_scaleout_ranks x
                                         num_scaleup_ranks, rank s = (s / n_up,
                                         s % n_up); S must be a multiple.  The
                                         row base of a slot is the sender's
                                         scale-out index, and a destination's
                                         staging buffer is read in row form:
                                         segment = scale-up index, offset =
                                         scale-out index * Nmax + row slot.
                                         Receive rows are the same as on the
                                         direct path.                            */
} ep_config_t;

/* Byte sizes of every caller-allocated buffer for a configuration (0 = not
 * used).  recv_rows is the receive capacity in rows: S*T*min(K,R) for the
 * compact layout, the largest count a destination-sum of deduplicated rows can
 * reach; S*T*K + E*(A-1) for expand. */
typedef struct ep_sizes {
    uint64_t dst_slot, tokens_per_rank, tokens_per_expert, recv_psum, recv_base;
    uint64_t expert_base, expand_pos, error_flags, layout_scratch, recv_psum_scaleup;
    uint64_t staging_x, staging_sf, staging_meta;
    uint64_t recv_rows;
    uint64_t recv_x, recv_sf, recv_src_idx, recv_topk_idx, recv_topk_weights;
    uint64_t y, out;
} ep_sizes_t;

/* Layout tables ("handle"): written by ep_layout, read by ep_dispatch and
 * ep_combine.  All device pointers, int32:
 *   dst_slot          [S][T][K]  row_base*Nmax + the number of earlier tokens
 *                                of source s that reach the same destination,
 *                                on the lowest valid lane of each destination
 *                                of a token; -1 on every other lane
 *                                ([DET] Motivation and Approach); row_base is
 *                                s (direct) or s / n_up (hybrid)
 *   tokens_per_rank   [S][R]     deduplicated tokens source s sends to rank d
 *   tokens_per_expert [S][E]     valid lanes of source s routed to expert e
 *   recv_psum         [R][S+1]   exclusive prefix over sources of
 *                                tokens_per_rank[.][d]: the base of source s
 *                                in destination d's compact receive rows
 *                                ([DRX] Direct Recv X design)
 *   recv_base         [R+1]      exclusive prefix over destinations of the
 *                                deduplicated row totals recv_psum[d][S];
 *                                recv_base[R] = rows in the compact layout
 *   expert_base       [E+1]      expand only: first row of expert e, segments
 *                                padded to a multiple of A
 *   expand_pos        [S][T][K]  expand only: receive row of a valid lane
 *                                (ascending (s,t,k) inside the expert), else -1
 *   recv_psum_scaleup [R][n_up+1] hybrid only: per destination, exclusive
 *                                prefix over scale-up segments of the rows
 *                                each segment holds (the per-segment part of
 *                                the pages' extended psum)
 *   error_flags       [1]        bit 0: some top-k id was >= E
 *   scratch           bytes      ep_sizes_t.layout_scratch, private to the
 *                                library; contents need no initialisation.
 *                                Compact layouts and expand layouts with
 *                                alignment 1: its head holds the receive-row
 *                                index (8 bytes per receive row, rounded up
 *                                to 256 bytes) that the copy epilogue reads,
 *                                written by a dispatch's scatter (compact) or
 *                                by the layout (expand, ep_layout_no_alloc
 *                                included when a scratch is given); the
 *                                layout's own words follow.  Required by
 *                                ep_layout; may be NULL for ep_dispatch (the
 *                                epilogue then searches the receiver tables
 *                                for each row's source: slower) and for
 *                                ep_combine, which do not allocate it.  */
typedef struct ep_layout {
    int32_t *dst_slot_dev;
    int32_t *tokens_per_rank_dev;
    int32_t *tokens_per_expert_dev;
    int32_t *recv_psum_dev;
    int32_t *recv_base_dev;
    int32_t *expert_base_dev;   /* NULL unless expand */
    int32_t *expand_pos_dev;    /* NULL unless expand */
    int32_t *error_flags_dev;
    void *scratch_dev;
    int32_t *recv_psum_scaleup_dev; /* NULL unless hybrid */
} ep_layout_t;

/* Staging ([R][S][Nmax] rows: destination d's receive buffer holds one Nmax-row
 * region per source, [DET] Direct vs hybrid dispatch) and receive buffers.
 *   staging_x     [R][S][Nmax][row bytes]; on the hybrid path the S regions
 *                 of a destination are ordered [n_up segments][n_out]
 *   staging_sf    [R][S][Nmax][H/128] fp32 (fp8 only, else NULL)
 *   staging_meta  [R][S][Nmax][1+2K] int32: token index t, the token's K
 *                 expert ids (masked/invalid as -1), the K weights' fp32 bits
 *   compact layout (expand == 0), row i of destination d's source s slot j is
 *   i = recv_base[d] + recv_psum[d][s] + j:
 *     recv_x [recv_rows][row bytes], recv_sf [recv_rows][H/128],
 *     recv_src_idx [recv_rows] (= s*T + t), recv_topk_idx [recv_rows][K]
 *     (local expert id on d, else -1), recv_topk_weights [recv_rows][K]
 *     (weight, else +0)
 *   expand layout: recv_x, recv_sf, recv_src_idx as above at expand_pos rows,
 *     recv_topk_weights [recv_rows] (the lane's weight); recv_topk_idx unused;
 *     padding rows get zero bytes, src -1 and weight +0.
 * Rows beyond the filled ones are left untouched. */
typedef struct ep_recv {
    void *staging_x_dev;
    float *staging_sf_dev;
    int32_t *staging_meta_dev;
    void *recv_x_dev;
    float *recv_sf_dev;
    int32_t *recv_src_idx_dev;
    int32_t *recv_topk_idx_dev;
    float *recv_topk_weights_dev;
    int64_t recv_capacity_rows;       /* rows allocated; must be >= recv_rows */
} ep_recv_t;

/* Host only (no HIP call): validate cfg and fill *sizes.  Returns EP_OK or the
 * validation error ([DRX] review: the buffer sizes are derived in one place). */
int ep_query_sizes(const ep_config_t *cfg, ep_sizes_t *sizes);

/* Deterministic layout prologue ([DET] Approach): a two-pass scan over
 * topk_idx_dev (int64 [S][T][K]) producing every table of *layout.  The result
 * is a pure function of topk_idx; num_layout_cus changes only the speed. */
int ep_layout(const ep_config_t *cfg, const int64_t *topk_idx_dev, const ep_layout_t *layout,
              void *stream);

/* Size of the layout scratch the library keeps on each GPU for
 * ep_layout_no_alloc. */
#define EP_NO_ALLOC_SCRATCH_BYTES (4u << 20)

/* ep_layout for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same launches and the same tables as ep_layout, but the scratch is an
 * EP_NO_ALLOC_SCRATCH_BYTES array the library holds on each GPU it runs on
 * until the process ends, so layout->scratch_dev is not required (may be
 * NULL; when given, only the receive-row index at its head is written).
 * The call allocates and frees nothing.  A configuration whose layout words
 * (ep_sizes_t.layout_scratch less the receive-row index at its head, which
 * the array does not hold) exceed EP_NO_ALLOC_SCRATCH_BYTES returns
 * EP_ERR_CAPACITY before anything is enqueued; EP_ERR_HIP if the array's
 * device address cannot be obtained.  Every call on one GPU uses that GPU's
 * one array: calls that overlap on one GPU (on different streams, or from
 * different host threads without ordering) race and may produce wrong tables,
 * so order them (for example, one stream).  The array needs no clearing
 * between calls. */
int ep_layout_no_alloc(const ep_config_t *cfg, const int64_t *topk_idx_dev, const ep_layout_t *layout,
                       void *stream);

/* Dispatch: scatter ([DET] Direct vs hybrid dispatch: senders replay the
 * layout's slots) of every token's row, scales and metadata into the staging
 * rows, then the copy epilogue ([DRX] Background) into the receive buffers.
 *   x_dev            [S][T][row bytes] (bf16, or e4m3fn bytes)
 *   x_sf_dev         [S][T][H/128] fp32 (fp8 only, else NULL)
 *   topk_idx_dev     int64 [S][T][K];  topk_weights_dev fp32 [S][T][K]
 *   phases           enum ep_phase mask; the epilogue reads the staging rows
 *                    the scatter of the same layout wrote (and, when the
 *                    layout's scratch is given, the receive-row index that
 *                    scatter wrote at its head: give both phases the same
 *                    layout). */
int ep_dispatch(const ep_config_t *cfg, const void *x_dev, const float *x_sf_dev,
                const int64_t *topk_idx_dev, const float *topk_weights_dev,
                const ep_layout_t *layout, const ep_recv_t *recv, int32_t phases, void *stream);

/* Layout and dispatch in one call: ep_layout followed by ep_dispatch with
 * EP_PHASE_ALL, with the same arguments, checks and results (the pages'
 * dispatch runs its deterministic prologue itself when no cached handle is
 * given, [DET] Approach and New API).  For one small source in the compact
 * layout (T*K <= 2048, rows of at most 1 KiB, no Direct Recv X) everything
 * runs as one kernel: each workgroup lays out the whole source in LDS and
 * dispatches its share of the tokens; otherwise the layout's and the
 * dispatch's launches are enqueued as the two calls would. */
int ep_layout_dispatch(const ep_config_t *cfg, const void *x_dev, const float *x_sf_dev,
                       const int64_t *topk_idx_dev, const float *topk_weights_dev, const ep_layout_t *layout,
                       const ep_recv_t *recv, void *stream);

/* Combine ([UNO] Changes: the reduce epilogue brings expert outputs back to
 * token order): out[s][t] = bf16(sum over valid lanes k of w[s][t][k] *
 * Y(s,t,k)), accumulated in fp32 and rounded to nearest-even once.  Y is, in
 * the compact layout, row recv_base[d] + recv_psum[d][s] + run of y_dev for
 * the lane's rank d (lanes sharing a rank weight the same row); in the expand
 * layout, row expand_pos[s][t][k].  A token with no valid lane gives +0.
 * Arithmetic order (fixed, so results are bitwise reproducible): in the
 * compact layout the weights of the lanes that share a rank are first summed
 * in fp32 in ascending lane order, then each distinct row is applied with one
 * fp32 fused multiply-add, rows in the order of their owner (lowest) lanes; in
 * the expand layout each valid lane's row is applied with one fused
 * multiply-add in ascending lane order.  The result is therefore within one
 * bf16 rounding of the exact sum, not bitwise that of a per-lane fp32 loop.
 *   y_dev   bf16 [rows][H] in the receive row order (at least recv_rows rows)
 *   out_dev bf16 [S][T][H] */
int ep_combine(const ep_config_t *cfg, const ep_layout_t *layout, const int64_t *topk_idx_dev,
               const float *topk_weights_dev, const void *y_dev, void *out_dev, void *stream);

/* Combine plus bias ([DET] Performance runs the combine with num_bias = 2):
 * out[s][t] = bf16(sum over valid lanes of w * Y + bias0[s][t] + bias1[s][t]),
 * the bias rows added in fp32 before the one rounding.  bias0_dev / bias1_dev
 * are bf16 [S][T][H] (16-byte aligned), either may be NULL; with both NULL
 * this is ep_combine. */
int ep_combine_bias(const ep_config_t *cfg, const ep_layout_t *layout, const int64_t *topk_idx_dev,
                    const float *topk_weights_dev, const void *y_dev, const void *bias0_dev,
                    const void *bias1_dev, void *out_dev, void *stream);

/* Gradients of ep_combine for the y_dev of that call and the gradient d_out of
 * its output (ep_combine_bias has the same ones, and d_out is the gradient of
 * each bias tensor):
 *   d_y[row] = bf16(w_row * d_out[s][t]), w_row the fp32 sum in ascending lane
 *              order of the weights of the lanes of (s,t) that read the row
 *              (one lane in the expand layout), so every filled row has exactly
 *              one token and is written once; padding rows of an expand layout
 *              with alignment > 1 are written as zeros, rows beyond the filled
 *              ones are left untouched;
 *   d_topk_weights[s][t][k] = fp32 sum over the row of Y(s,t,k) * d_out[s][t]
 *              on a valid lane, +0 on a masked one.  The order of the sum is
 *              fixed: results are bitwise reproducible.
 * Either gradient may be NULL (not both); y_dev is needed for d_topk_weights
 * only and topk_weights_dev for d_y only.  bf16 d_y_dev [rows][H], d_out_dev
 * [S][T][H], y_dev as in ep_combine; 16-byte aligned. */
int ep_combine_backward(const ep_config_t *cfg, const ep_layout_t *layout, const int64_t *topk_idx_dev,
                        const float *topk_weights_dev, const void *y_dev, const void *d_out_dev, void *d_y_dev,
                        float *d_topk_weights_dev, void *stream);

/* ---- Router: the topk_idx and topk_weights that ep_layout, ep_dispatch and
 * ep_combine take, from the logits of S x T tokens over E experts. ---- */

enum ep_scoring {
    EP_SCORING_SOFTMAX = 0, /* s = exp(l - max) / sum over the token's experts */
    EP_SCORING_SIGMOID = 1  /* s = 1 / (1 + exp(-l))                           */
};

/* Limits as above: 1 <= K <= 32, K <= E <= 1024, S <= 65535, T <= 2^30,
 * S * T * K < 2^31. */
typedef struct ep_route_config {
    int32_t num_src_ranks;  /* S >= 1                                          */
    int32_t num_tokens;     /* T >= 0, tokens per source                       */
    int32_t num_experts;    /* E                                               */
    int32_t num_topk;       /* K <= E                                          */
    int32_t logits_dtype;   /* EP_DTYPE_FP32 or EP_DTYPE_BF16                  */
    int32_t scoring;        /* enum ep_scoring                                 */
    float scale;            /* finite; the weights of a token sum to it        */
} ep_route_config_t;

/* Byte sizes of the buffers of ep_route_t. */
typedef struct ep_route_sizes {
    uint64_t topk_idx, topk_weights, tokens_per_expert, tokens_valid, balance_loss, scratch;
} ep_route_sizes_t;

/* Outputs of ep_route.  tokens_per_expert, tokens_valid, balance_loss and
 * scratch serve the balance loss: all four, or all NULL.
 *   topk_idx          int64 [S][T][K], best first; -1 on the lanes of a token
 *                     with fewer than K valid experts
 *   topk_weights      fp32 [S][T][K], scale * s_k / (sum of s_k + 1e-20); +0
 *                     on a lane of -1
 *   tokens_per_expert int32 [S][E], lanes of source s that chose expert e
 *   tokens_valid      int32 [S], tokens with a valid expert, V
 *   balance_loss      fp32 [S], sum over e of f_e * P_e with
 *                     f_e = tokens_per_expert[e] * E / (K * max(V, 1)) and
 *                     P_e = sum over tokens of p_e / max(V, 1); p = s (softmax)
 *                     or s / (sum of the token's s + 1e-20) (sigmoid)
 *   scratch           16-byte aligned, private to the library, needs no
 *                     initialisation */
typedef struct ep_route {
    int64_t *topk_idx_dev;
    float *topk_weights_dev;
    int32_t *tokens_per_expert_dev;
    int32_t *tokens_valid_dev;
    float *balance_loss_dev;
    void *scratch_dev;
} ep_route_t;

int ep_query_route_sizes(const ep_route_config_t *cfg, ep_route_sizes_t *sizes);

/* Scores, choice and weights.  An expert of a token is valid if the token's
 * mask byte is not 0 (token_mask_dev uint8 [S][T], may be NULL) and its logit is
 * above the type's lowest value: -inf, that value and NaN are masked; +inf
 * counts as the type's largest value.  The K experts are those with the largest
 * key, ties to the lowest index.  Without a bias (bias_dev NULL) the key is the
 * logit; with one (fp32 [E]) it is s + bias[e] to 64-bit accuracy, so that the
 * choice does not depend on rounding; an expert whose bias is NaN or -inf is
 * not chosen.  The weights use s without the bias. */
int ep_route(const ep_route_config_t *cfg, const void *logits_dev, const float *bias_dev,
             const uint8_t *token_mask_dev, const ep_route_t *route, void *stream);

/* Gradient of the logits (same type, [S][T][E]) from the gradients of the
 * weights (d_topk_weights_dev fp32 [S][T][K], may be NULL) and of the balance
 * losses (d_balance_loss_dev fp32 [S], may be NULL; needs the counts), of the
 * ep_route call with the same logits, mask and route.  The choice and the
 * counts are constants; masked experts get +0.  Reads topk_idx,
 * tokens_per_expert and tokens_valid of *route. */
int ep_route_backward(const ep_route_config_t *cfg, const void *logits_dev, const uint8_t *token_mask_dev,
                      const ep_route_t *route, const float *d_topk_weights_dev, const float *d_balance_loss_dev,
                      void *d_logits_dev, void *stream);

/* ---- Experts' products: rows grouped by expert times their expert's weights,
 * for the receive rows of the expand layout (expert_base) or any other rows
 * grouped the same way. ---- */

enum ep_activation {
    EP_ACTIVATION_NONE = 0,
    EP_ACTIVATION_RELU = 1,
    EP_ACTIVATION_GELU = 2,   /* v * Phi(v), the exact form                    */
    EP_ACTIVATION_SILU = 3,   /* v / (1 + exp(-v))                             */
    EP_ACTIVATION_SWIGLU = 4  /* silu(gate) * up: Nw = 2N weight rows, the gate's
                                 first                                         */
};

#define EP_MAX_EXPERT_ROWS 2147483647ll

/* Limits: E <= 1024, I and N <= 262144, N a multiple of 8, I of 8 (bf16) or of
 * 128 (fp8).  Outside them a call returns EP_ERR_UNSUPPORTED. */
typedef struct ep_expert_config {
    int32_t num_experts;   /* E                                                */
    int32_t in_features;   /* I                                                */
    int32_t out_features;  /* N                                                */
    int32_t x_dtype;       /* EP_DTYPE_BF16 or EP_DTYPE_FP8_E4M3FN: x and w    */
    int32_t activation;    /* enum ep_activation                               */
    int32_t reserved;      /* 0                                                */
    int64_t num_rows;      /* rows allocated, >= expert_base[E]                */
} ep_expert_config_t;

/* Byte sizes of the buffers of a configuration (0 = not used). */
typedef struct ep_expert_sizes {
    uint64_t x, x_sf, w, w_sf, bias, out, pre, backward_scratch;
} ep_expert_sizes_t;

int ep_query_expert_sizes(const ep_expert_config_t *cfg, ep_expert_sizes_t *sizes);

/* Rows of the tiles that the products of a configuration are computed in (32,
 * 64, 128 or 256; 0 without rows, and for the gradients of fp8): which of the
 * kernels a profile or a test of that configuration shows. */
typedef struct ep_expert_tiles {
    int32_t forward, d_x, d_w;
} ep_expert_tiles_t;

int ep_query_expert_tiles(const ep_expert_config_t *cfg, ep_expert_tiles_t *tiles);

/* For each expert e and each of its rows r in [expert_base[e],
 * expert_base[e+1]):  pre[r] = x[r] W_e^T + bias[e],
 * out[r] = act(pre[r]) + residual[r].
 *   expert_base_dev int32 [E+1], not decreasing (an entry outside the rows is
 *                   taken as the nearest row); other rows are left untouched
 *   x_dev           [num_rows][I];  w_dev [E][Nw][I], Nw = N, or 2N for swiglu
 *   x_sf_dev        fp32 [num_rows][I/128] and
 *   w_sf_dev        fp32 [E][ceil(Nw/128)][I/128], one scale per 128 x 128
 *                   block: fp8 only, else NULL
 *   bias_dev        fp32 [E][Nw] or NULL;  residual_dev bf16 [num_rows][N] or
 *                   NULL (may be out_dev itself)
 *   out_dev         bf16 [num_rows][N];  pre_dev bf16 [num_rows][Nw] or NULL:
 *                   the pre-activation that the backward pass reads
 * Products are summed in fp32, the epilogue works on the fp32 sum, and out and
 * pre are each rounded once.  All pointers but the scales and expert_base
 * 16-byte aligned. */
int ep_expert_mm(const ep_expert_config_t *cfg, const int32_t *expert_base_dev, const void *x_dev,
                 const float *x_sf_dev, const void *w_dev, const float *w_sf_dev, const float *bias_dev,
                 const void *residual_dev, void *out_dev, void *pre_dev, void *stream);

/* Gradients of a bf16 ep_expert_mm with d_out (bf16 [num_rows][N]) the gradient
 * of out (the residual's is d_out itself):
 *   d = act'(pre) d_out,  d_x[r] = d[r] W_e  (bf16 [num_rows][I]),
 *   d_w[e] = sum over the expert's rows of d[r]^T x[r]  (bf16 [E][Nw][I]),
 *   d_bias[e] = sum of d[r]  (fp32 [E][Nw]);
 * an expert without rows gets zeros.  Each gradient may be NULL (not all, unless
 * num_rows is 0).
 * pre_dev is not needed without an activation, x_dev only for d_w.  The
 * matrix units take d rounded to bf16; d_bias sums the unrounded values, in a
 * fixed order.  Padding rows count like others: ep_combine_backward writes
 * zeros there.  scratch_dev: backward_scratch bytes, contents need no
 * initialisation. */
int ep_expert_mm_backward(const ep_expert_config_t *cfg, const int32_t *expert_base_dev, const void *x_dev,
                          const void *w_dev, const void *pre_dev, const void *d_out_dev, void *d_x_dev, void *d_w_dev,
                          float *d_bias_dev, void *scratch_dev, void *stream);

/* Static description of a status code. */
const char *ep_status_string(int status);

/* Library version, MAJOR*10000 + MINOR*100 + PATCH. */
int ep_version(void);

#ifdef __cplusplus
}
#endif
#endif /* EP_H */
