/*
 * ep.h -- C ABI of libep.so: the single-GPU data-parallel core of
 * expert-parallel MoE dispatch and combine on AMD Instinct MI355X (gfx950).
 *
 * Sources (web pages, cited by title and section):
 *   [V2]   "DeepEP V2 深度深潜：统一接口、SM 估算本质与 TopK 复制机制"
 *   [PIPE] "07: DeepEP Intra/Inter-node 协调 — NVLink Scale-up + RDMA
 *          Scale-out 三阶段流水线的代码实证"
 *   [MEGA] "06_06: NVLink Scale-up + RDMA Scale-out — DeepEP 三阶段流水线 vs
 *          DeepGEMM 对称内存"
 *   [ASC]  "Ascend Send Ordering"
 *
 * Model. One GPU holds T tokens of one source rank. R logical destination
 * ranks (E / R experts each, rank of expert e = e / (E / R)) are partitions of
 * this GPU's HBM; for the two-level path the R ranks form G scale-out groups
 * of P = R / G scale-up peers, rank r = g * P + peer ([PIPE]
 * is_nvlink_accessible). Each destination rank owns a compact region of
 * receive rows; regions are laid end to end in rank order (rank_offsets), and
 * inside a region rows follow ascending source token.
 *
 * Conventions for every entry point:
 *   - Every pointer is a DEVICE pointer unless stated, allocated and owned by
 *     the caller. The library allocates and frees no device memory and keeps
 *     no global state; calls on distinct workspaces are independent.
 *   - Work is enqueued asynchronously on `stream` (NULL = default stream).
 *     Inputs must stay valid until the work completes.
 *   - Arrays are row-major and densely packed. bf16 values are passed as their
 *     16-bit patterns (uint16_t), FP8 values as e4m3 bytes.
 *   - Alignment: hidden rows (bf16, FP8), receive rows and chunk buffers need
 *     16 B aligned base pointers; other arrays their element alignment.
 *   - With T = 0 the per-token arrays (topk_idx, x, weights, slot, ...) and
 *     buffers of zero capacity may be NULL; the layout calls then write zero
 *     counts and offsets, and no call writes a row.
 *   - Return value: EP_OK, or a negative EP_ERR_* status. Nothing is enqueued
 *     when a host-side check fails. Problems only visible on the device set
 *     bits in the workspace's error words (read with ep_check_errors and
 *     ep_check_sticky_errors, which return EP_ERR_DEVICE when a bit is set).
 */
#ifndef EP_H
#define EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define EP_OK 0
#define EP_ERR_ARG (-1)         /* null / misaligned pointer, bad shape, bad size */
#define EP_ERR_UNSUPPORTED (-2) /* shape outside the supported limits below */
#define EP_ERR_HIP (-3)         /* a HIP runtime call or launch failed */
#define EP_ERR_DEVICE (-4)      /* the device reported an error: ep_check_errors /
                                   ep_check_sticky_errors return it when error bits are
                                   set and write the bits (EP_DEVERR_*) to *bits */
#define EP_ERR_SCRATCH (-5)     /* ep_get_layout_noalloc: the shape's count tables do not
                                   fit the static scratch (EP_LAYOUT_SCRATCH_BYTES) */

/* Device error bits (workspace error words). */
#define EP_DEVERR_EXPERT_ID 1u  /* an expert id < -1 or >= E (treated as -1) */
#define EP_DEVERR_CAPACITY 2u   /* a row index >= the given buffer capacity (not written / not read) */
#define EP_DEVERR_FLAG 4u       /* a 512 B chunk flag != epoch (row dropped / skipped) */
#define EP_DEVERR_TIMEOUT 8u    /* a bounded wait for a batch flag gave up (batch not forwarded) */
#define EP_DEVERR_LOGIT 16u     /* a router logit or bias is NaN (taken as -infinity) */

/* Payload pieces present in a token record (ep_record_bytes). */
#define EP_SEG_BF16 1
#define EP_SEG_FP8 2
#define EP_SEG_SCALES 4

/* Row formats accepted by ep_combine. */
#define EP_FMT_PLAIN 0    /* rows of H bf16 values at a fixed byte stride */
#define EP_FMT_CHUNKED 1  /* chunked token records (see ep_hierarchical_dispatch) */

/* Two-level dispatch steps. */
#define EP_HIER_SCALEOUT 1 /* step 1: one write per (token, destination group) */
#define EP_HIER_FORWARD 2  /* step 2: forward group rows to scale-up peers */

/* Order of an expert's weight matrix (ep_expert_matmul): rows of the
 * contracted index, or rows of the produced one. */
#define EP_WEIGHT_NK 0 /* w[e][n][k]: y = x * w[e]^T (forward) */
#define EP_WEIGHT_KN 1 /* w[e][k][n]: y = x * w[e]   (gradient of the rows) */

/* Element type of a weight gradient (ep_expert_wgrad). */
#define EP_GRAD_BF16 0
#define EP_GRAD_F32 1

/* Element type of the residual stream (ep_rms_norm, ep_rms_norm_grad). */
#define EP_STREAM_BF16 0
#define EP_STREAM_F32 1

/* Scores that a router makes of its logits (ep_route). */
#define EP_SCORE_SOFTMAX 0 /* exp(l[e]) / sum over all experts e' of exp(l[e']) */
#define EP_SCORE_SIGMOID 1 /* 1 / (1 + exp(-l[e])) */

/* Forms of 4-bit weights (ep_moe_few_w4). */
#define EP_W4_INT 0  /* code - 8, times a bf16 scale for each row and 128 columns */
#define EP_W4_E2M1 1 /* e2m1 (sign, 2 bits of exponent, 1 of fraction), times 2^(s - 127) for each
                        row and 32 columns, s one byte (255: NaN) */

/* Supported limits (EP_ERR_UNSUPPORTED beyond them). */
#define EP_FEW_MAX_TOKENS 128 /* tokens of ep_moe_few */
#define EP_MAX_DIM (1 << 20)  /* columns of the expert products' matrices */
#define EP_MAX_TOPK 64
#define EP_MAX_RANKS 1024
#define EP_MAX_GROUPS 256
#define EP_MAX_EXPERTS 4096

/* Problem shape. T >= 0 tokens; H hidden size (H % 8 == 0; H % 128 == 0 when
 * FP8 scales are used); K in [1, 64] experts per token; E experts; R ranks
 * with E % R == 0; G groups with R % G == 0 (G = 1 for the flat path). */
typedef struct ep_shape {
    int32_t T, H, K, E, R, G;
} ep_shape;

/* Layout arrays written by ep_get_layout and read by the other calls
 * ([V2] §3.3 阶段1: per-expert counts, per-rank counts after rank
 * deduplication, prefix sums; [V2] §3.3 阶段2: one slot per token and
 * destination; the is-token-in-rank mask of [PIPE]'s RDMA sender). */
typedef struct ep_layout {
    int32_t *tokens_per_expert;  /* [E]   valid lanes per expert (not deduplicated) */
    int32_t *tokens_per_rank;    /* [R]   tokens per rank, each token counted once */
    int32_t *tokens_per_group;   /* [G]   tokens per group, each token counted once */
    int32_t *expert_offsets;     /* [E+1] exclusive prefix sum of tokens_per_expert */
    int32_t *rank_offsets;       /* [R+1] exclusive prefix sum; rank_offsets[R] = N rows */
    int32_t *group_offsets;      /* [G+1] exclusive prefix sum of tokens_per_group */
    uint8_t *is_token_in_rank;   /* [T*R] 1 if token t sends to rank r, else 0 */
    uint8_t *is_token_in_group;  /* [T*G] 1 if token t sends to group g, else 0 */
    int32_t *slot;               /* [T*K] receive row of (t, rank of lane k); -1 if lane skipped */
    int32_t *group_slot;         /* [T*K] group-region row of (t, group of lane k); -1 if skipped */
    int32_t *expert_slot;        /* [T*K] expand-mode row of (t, k); -1 if skipped (needs
                                    expert_offsets) */
} ep_layout;

/* Send side: per-token payload and routing of the T local tokens ([V2] §3.5). */
typedef struct ep_tokens {
    const uint16_t *x;            /* [T*H] bf16 hidden rows, or NULL */
    const uint8_t *x_fp8;         /* [T*H] e4m3 hidden rows, or NULL */
    const float *x_scales;        /* [T*H/128] one fp32 scale per 128 channels, or NULL */
    const int64_t *topk_idx;      /* [T*K] expert ids, -1 = no expert (required) */
    const float *topk_weights;    /* [T*K] routing weights, or NULL */
} ep_tokens;

/* Receive side of the direct dispatch: `capacity` rows each ([V2] §3.5
 * outputs recv_x / recv_topk_idx / recv_topk_weights; [PIPE] NVL receivers
 * write recv_x[row] and recv_x_scales[row * H/128]). */
typedef struct ep_recv {
    uint16_t *x;               /* [cap*H] or NULL (needs ep_tokens.x) */
    uint8_t *x_fp8;            /* [cap*H] or NULL (needs ep_tokens.x_fp8) */
    float *x_scales;           /* [cap*H/128] or NULL (needs ep_tokens.x_scales) */
    int32_t *src_idx;          /* [cap] source token of each row, or NULL */
    int32_t *topk_idx;         /* [cap*K] the token's expert ids as int32 (invalid -> -1), or NULL */
    float *topk_weights;       /* [cap*K] the token's weights, bit for bit, or NULL */
    int64_t capacity;          /* rows available; rows >= capacity are not written */
} ep_recv;

/* Bytes of workspace the calls need for `shape` (host only, no GPU work).
 * Layout: two u32 error words at offset 0 (word 0: errors of the current
 * pass of calls, cleared by the layout calls; word 1: errors since the last
 * ep_clear_errors, cleared by nothing else; undefined in a new workspace
 * until its first ep_clear_errors), then per-block partial counts. The
 * workspace may be reused by successive calls on one stream. */
size_t ep_workspace_bytes(const ep_shape *shape);

/* Byte length P of a packed token record with pieces `seg_flags`
 * (EP_SEG_*): [bf16 H*2][fp8 H][scales (H/128)*4][topk_idx K*4][topk_w K*4]
 * [src 4], each present piece padded to 16 B ([V2] §3.4 TokenLayout; the
 * metadata pieces are always present). Host only. Returns -1 on bad args. */
int64_t ep_record_bytes(const ep_shape *shape, int seg_flags);

/* Row stride of a chunked record: 512 * ceil(P / 480) bytes ([ASC] 导言 and
 * 能省多少: 512 B blocks of 480 B payload + 32 B flag). Host only. */
int64_t ep_chunked_record_bytes(const ep_shape *shape, int seg_flags);

/* Layout ([V2] §3.3 阶段1 notify warps and the slot rule of 阶段2).
 * For each token t and lane k with a valid expert e = topk_idx[t*K+k]:
 * rank r = e / (E/R), group g = r / (R/G). Counts: tokens_per_expert per lane;
 * tokens_per_rank / tokens_per_group once per token. Offsets: exclusive
 * prefix sums. Slot: slot[t*K+k] = rank_offsets[r] + #{t' < t : token t'
 * sends to r} (repeated ranks in a token share the row); group_slot likewise
 * with groups. Every output pointer except the workspace may be NULL to skip
 * that output. Also clears workspace error word 0 first, so a pass of
 * calls starts with a clean word. Ids < -1 or >= E set EP_DEVERR_EXPERT_ID
 * and count as -1. ws: at least ep_workspace_bytes(shape) bytes, 256 B
 * aligned. */
int ep_get_layout(const ep_shape *shape, const int64_t *topk_idx, const ep_layout *layout,
                  void *ws, size_t ws_bytes, void *stream);

/* Allocation-free layout, for callers that cannot allocate device memory at
 * call time (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc): ep_get_layout with the same outputs, bit for bit,
 * but its per-workgroup count tables live in a static device array of
 * EP_LAYOUT_SCRATCH_BYTES inside the library instead of a workspace. Each GPU
 * the library runs on holds one such array until the process ends (its
 * address is looked up on the first call on that GPU); every call on a GPU
 * shares it, so calls that overlap on one GPU (several streams, several host
 * threads) race and must be serialised by the caller. The call allocates and
 * frees nothing. Limit: the count tables, 256 + a(4 * (nb + 1) * (2 * R4 + G4))
 * + a(4 * (nb + 1) * E) bytes (nb = ceil(T / 256), R4 and G4 = R and G rounded up to
 * multiples of 4, a() rounds up to a multiple of 256), must not exceed
 * EP_LAYOUT_SCRATCH_BYTES (4 MiB: e.g. 262,144 tokens with E = 256 and R =
 * 64 need 1.6 MB, 16,384 tokens with E = 2048 and R = 256 need 0.66 MB),
 * else EP_ERR_SCRATCH and nothing is enqueued.
 * errors: device pointer to two u32 error words with the meaning of the
 * workspace's (word 0 cleared by this call, then EP_DEVERR_EXPERT_ID set for
 * invalid ids in both); passing a workspace's base makes ep_check_errors on
 * that workspace read them. Other arguments and checks as ep_get_layout. */
#define EP_LAYOUT_SCRATCH_BYTES (4u << 20)
int ep_get_layout_noalloc(const ep_shape *shape, const int64_t *topk_idx, const ep_layout *layout,
                          uint32_t *errors, void *stream);

/* Expand-mode rows ([V2] §3.3 阶段3: the copy epilogue with expand, where a
 * received token gets one row per chosen expert, grouped by expert for the
 * expert GEMMs). When layout->expert_slot is non-NULL, ep_get_layout also
 * writes expert_slot[t*K+k] = expert_offsets[e] + #{lanes (t', k') before
 * (t, k) in token-then-lane order with the same expert e}, -1 for skipped
 * lanes; the rows of expert e are [expert_offsets[e], expert_offsets[e+1]),
 * expert_offsets[E] rows in all. Requires layout->expert_offsets
 * (EP_ERR_ARG without it). */

/* Direct dispatch ([V2] §3.3 阶段2 and §3.5; [PIPE] RDMA sender / NVL
 * sender record fields). Each token is read once and its record (present
 * pieces of ep_tokens plus src index, topk ids and weights) is written to
 * every receive row it owns: recv row layout->slot[t*K+k] for the first lane
 * k of each distinct rank. Needs layout->slot from ep_get_layout with the
 * same topk_idx. Receive pointers may be NULL to skip that piece. Rows >=
 * recv->capacity are not written and set EP_DEVERR_CAPACITY. */
int ep_dispatch(const ep_shape *shape, const ep_layout *layout, const ep_tokens *tokens,
                const ep_recv *recv, void *ws, size_t ws_bytes, void *stream);

/* Expand-mode dispatch: like ep_dispatch, but the token's record goes to the
 * row layout->expert_slot[t*K+k] of every valid lane k (one row per lane, no
 * rank deduplication). recv->capacity counts expand rows. */
int ep_dispatch_expand(const ep_shape *shape, const ep_layout *layout, const ep_tokens *tokens,
                       const ep_recv *recv, void *ws, size_t ws_bytes, void *stream);

/* Two-level dispatch ([V2] §3.6; [PIPE] hybrid scale-out stage and forward
 * warps) with chunked records ([ASC] data-as-flag 512 B blocks).
 * A record (ep_record_bytes, pieces = the non-NULL ones among x, x_fp8,
 * x_scales; x is required, topk_weights required) is cut into 512 B blocks:
 * block c holds record bytes [480c, 480c+480) (zero past the end) and then
 * eight u32 flag words equal to `epoch`. Row stride = ep_chunked_record_bytes.
 *  step EP_HIER_SCALEOUT: each token writes its chunked record once per
 *    destination group g, at row layout->group_slot of group_buf.
 *  step EP_HIER_FORWARD: each row n < min(group_offsets[G], group_cap) of
 *    group_buf is read once; if any block flag != epoch the row is dropped
 *    (EP_DEVERR_FLAG); else its record is written, flags = epoch, to
 *    peer_buf row layout->slot[src*K+k] for the first lane k of each distinct
 *    rank of the row's group.
 * `steps` is EP_HIER_SCALEOUT, EP_HIER_FORWARD or both (two launches, stream
 * ordered). epoch >= 1 (zeroed memory never passes the flag check). Needs
 * layout->slot, group_slot and group_offsets. Rows >= a buffer's capacity are
 * not written (EP_DEVERR_CAPACITY). After both steps the unpacked peer rows
 * equal what ep_dispatch writes for the same pieces. */
int ep_hierarchical_dispatch(const ep_shape *shape, const ep_layout *layout,
                             const ep_tokens *tokens, uint32_t epoch, int steps,
                             void *group_buf, int64_t group_cap, void *peer_buf,
                             int64_t peer_cap, void *ws, size_t ws_bytes, void *stream);

/* Both two-level steps in one persistent launch, forwarders consuming each
 * batch of records once its flag is published ([ASC] 方案一 and the
 * hierarchical Stage1: the batch's payload written without ordering, then
 * one ordered flag per batch; [PIPE] forward warps: records taken from the
 * scale-out buffer as they arrive, each wait bounded by a time limit).
 * Batch b = tokens [b * tile, (b+1) * tile). A workgroup writing batch b's
 * group rows (as step EP_HIER_SCALEOUT) stores them with device scope, waits
 * until they are acknowledged, then stores flag b = epoch; a workgroup
 * forwarding batch b waits for that flag (at most timeout_us; then the
 * batch's rows are not forwarded and EP_DEVERR_TIMEOUT is set) and forwards
 * the group rows of the batch's tokens (as step EP_HIER_FORWARD, block flags
 * checked). Jobs are handed out in order and job i writes batch i, then
 * forwards batch i - 64, so each group row is read back shortly after it was
 * written. The results are those of ep_hierarchical_dispatch with both
 * steps, byte for byte. Same arguments and requirements as
 * ep_hierarchical_dispatch with steps = 3; the workspace (ep_workspace_bytes)
 * also holds the batch flags, the ring's batch-freed words and the work
 * counters, which the call zeroes first with a small kernel (no memset), so
 * calls on one workspace must not overlap. opts may be NULL (defaults);
 * all-zero fields mean the defaults. */
typedef struct ep_fused_opts {
    int32_t tile_tokens;    /* tokens per batch, 1..64 (0: 2) */
    uint32_t timeout_us;    /* longest wait for one batch flag (0: 100000 us; in ring
                               mode scaled by the batch's generation, below) */
    uint32_t test_flags;    /* EP_FUSED_WITHHOLD: batch `withhold_batch`'s flag is never
                               published, to test the bounded wait (its group rows are
                               still written; it is not forwarded; EP_DEVERR_TIMEOUT) */
    int32_t withhold_batch;
    int32_t ring_batches;   /* 0: group rows at their group-region rows (group_slot), as
                               ep_hierarchical_dispatch writes them. > 64: group_buf is a
                               ring of this many batches instead ([PIPE] the scale-out
                               receive buffer with flow control: a sender waits until the
                               forwarder has freed the slots it reuses). Token i of batch b
                               puts its j-th distinct group's record at row
                               ((b mod ring) * tile + i) * min(K, G) + j; the producer of
                               batch b waits until batch b - ring was forwarded. With
                               n = b / ring, the producer waits at most (n + 1/2) *
                               timeout_us (then writes anyway and sets
                               EP_DEVERR_TIMEOUT) and the forwarder (n + 1) * timeout_us,
                               so a lost flag stops only its own batch, and a broken run
                               lasts at most about (nbatch / ring + 1) * timeout_us.
                               Needs group_cap >= ring * tile * min(K, G) (< 2^31); the
                               peer rows are those of ring 0, byte for byte; group_buf's
                               contents afterwards are unspecified (the last pass over the
                               ring), and group_slot's capacity check does not apply.
                               A ring too short for the whole grid runs with a shorter
                               lag (down to 16 batches) and at most ring - lag
                               workgroups, so it also bounds the work in flight (slower).
                               Other values: EP_ERR_ARG. */
} ep_fused_opts;
#define EP_FUSED_WITHHOLD 1u
int ep_hierarchical_dispatch_fused(const ep_shape *shape, const ep_layout *layout,
                                   const ep_tokens *tokens, uint32_t epoch, void *group_buf,
                                   int64_t group_cap, void *peer_buf, int64_t peer_cap,
                                   const ep_fused_opts *opts, void *ws, size_t ws_bytes,
                                   void *stream);

/* Combine ([MEGA] combine write of BF16 expert outputs per (token, top-k);
 * [ASC] BF16 hidden with FP32 top-k weights): the inverse gather plus a
 * weighted reduction back to token order:
 *   out[t][h] = bf16_rne(acc), acc = +0.0f, then for k = 0..K-1 with
 *   s = layout->slot[t*K+k] >= 0:  acc = fmaf(topk_weights[t*K+k], y[s][h], acc)
 * (fp32, one rounding per step, ascending k; a row shared by two lanes is read
 * once and used twice). y: `y_rows` rows at `y_row_stride` bytes; format
 * EP_FMT_PLAIN (H bf16 at the start of each row; stride % 16 == 0) or
 * EP_FMT_CHUNKED (chunked records whose first piece is the bf16 hidden;
 * stride % 512 == 0; a row whose hidden-carrying blocks do not all have
 * flag == epoch is skipped with EP_DEVERR_FLAG). s >= y_rows is skipped with
 * EP_DEVERR_CAPACITY. A token with no usable lane gets zeros. */
int ep_combine(const ep_shape *shape, const ep_layout *layout, const void *y, int64_t y_rows,
               int64_t y_row_stride, int y_format, uint32_t epoch, const float *topk_weights,
               uint16_t *out, void *ws, size_t ws_bytes, void *stream);

/* Expand-mode combine: ep_combine over expand rows, s = layout->expert_slot
 * instead of layout->slot (each lane has its own row). */
int ep_combine_expand(const ep_shape *shape, const ep_layout *layout, const void *y,
                      int64_t y_rows, int64_t y_row_stride, int y_format, uint32_t epoch,
                      const float *topk_weights, uint16_t *out, void *ws, size_t ws_bytes,
                      void *stream);

/* Byte stride of a partial row of the two-level combine: the bf16 hidden row
 * alone in 512 B data-as-flag blocks, 512 * ceil(2H / 480). Host only. */
int64_t ep_partial_row_bytes(const ep_shape *shape);

/* Two-level combine: the two-level dispatch run backwards (the combine roles
 * of [MEGA]'s legacy internode walk-through: scale-up reduce, then
 * scale-out; [V2] §3.6 groups). y holds the per-(token, rank) expert outputs
 * at layout->slot rows (EP_FMT_PLAIN or EP_FMT_CHUNKED as for ep_combine).
 *  step 1 (steps & 1): for each token t and group g it sends to, partial =
 *    bf16_rne(acc), acc = +0.0f, then for the usable lanes k of t whose rank
 *    lies in g, ascending k: acc = fmaf(topk_weights[t*K+k], y[slot][h], acc);
 *    written with flags = epoch as a chunked row (stride
 *    ep_partial_row_bytes) at row layout->group_slot[t*K+k0] of group_buf (k0
 *    = first lane of g). Rows >= group_cap are not written
 *    (EP_DEVERR_CAPACITY).
 *  step 2 (steps & 2): out[t][h] = bf16_rne(acc), acc = +0.0f, then for the
 *    groups of t in ascending g: acc = acc + partial[t, g][h] (fp32 add); a
 *    partial row with a flag != epoch is skipped (EP_DEVERR_FLAG).
 * Needs layout->slot, layout->group_slot, tokens' topk_idx; epoch >= 1.
 * Usable lanes are as in ep_combine. With G = 1 the result equals
 * ep_combine bit for bit. With steps = 3, K <= 8, H <= 3,840 or
 * 5,760 < H <= 7,680 (a row's 512 B blocks cut into 1, 2 or 4 slices of 8
 * blocks) and group_cap partial rows of at least 512 MB (smaller ones stay
 * in the MALL between two launches anyway), both steps run as one persistent
 * launch with one flag per batch of tokens in the workspace (as for
 * ep_hierarchical_dispatch_fused; calls on one workspace must not overlap):
 * job i reduces batch i's groups, publishes it, then sums batch i - 128
 * across groups, so the partial rows are read back shortly after they were
 * written. A batch whose flag does not come
 * within 100 ms is not summed (EP_DEVERR_TIMEOUT). The results equal the two
 * launches' bit for bit. */
int ep_combine_two_level(const ep_shape *shape, const ep_layout *layout, const int64_t *topk_idx,
                         const void *y, int64_t y_rows, int64_t y_row_stride, int y_format,
                         uint32_t epoch, const float *topk_weights, void *group_buf,
                         int64_t group_cap, int steps, uint16_t *out, void *ws, size_t ws_bytes,
                         void *stream);

/* Several source ranks on one GPU ([V2] §3.3 阶段2: each source hands out,
 * per destination rank, the next slot of its own region there, addressed as
 * rank * capacity + slot; 阶段3: the copy epilogue finds each received row's
 * source from the prefix sum of tokens received per source rank
 * (psum_num_recv_tokens_per_scaleup_rank) and copies the row out of that
 * source's region). Source s owns tokens [s*Ts, min((s+1)*Ts, T)), Ts =
 * ceil(T / S). The staging buffer holds one region of `capacity` chunked
 * rows per (destination rank r, source s), region index r*S + s. */
typedef struct ep_sources {
    int32_t S;               /* source ranks, 1 <= S <= EP_MAX_RANKS */
    int64_t capacity;        /* rows per (rank, source) region; R*S*capacity <= INT32_MAX */
    int32_t *counts;         /* [S*R] tokens source s sends to rank r, each token once */
    int32_t *recv_offsets;   /* [R*S+1] rank-major exclusive prefix of counts: the dense rows
                                of region (r, s) start at recv_offsets[r*S+s]; [R*S] = N */
    int32_t *src_slot;       /* [T*K] staging row (r*S+s)*capacity + j of (t, rank r of lane
                                k), j = #{earlier tokens of s sending to r}; -1 if skipped */
} ep_sources;

/* Workspace bytes of the several-source calls (>= ep_workspace_bytes; the
 * error word is at the same place). Host only; 0 on bad args. */
size_t ep_source_workspace_bytes(const ep_shape *shape, int32_t S);

/* Per-source counts, the counts exchange (recv_offsets, what every
 * destination learns from an all-to-all of counts) and src_slot. Clears the
 * workspace error word 0 first. j >= capacity sets EP_DEVERR_CAPACITY and the
 * lane gets -1; invalid ids set EP_DEVERR_EXPERT_ID. Deterministic: with
 * contiguous sources, region (r, s) of the dense rows is exactly the part of
 * rank r's region (ep_get_layout) that holds source s's tokens, so dense row
 * recv_offsets[r*S+s] + j == layout slot of the same (t, r). */
int ep_source_layout(const ep_shape *shape, const int64_t *topk_idx, const ep_sources *sources,
                     void *ws, size_t ws_bytes, void *stream);

/* Send step: each token's chunked record (pieces as for
 * ep_hierarchical_dispatch; x and topk_weights required) goes once to each
 * distinct staging row src_slot[t*K+k] >= 0, flags = epoch (>= 1). staging:
 * R*S*capacity rows of ep_chunked_record_bytes. */
int ep_source_dispatch(const ep_shape *shape, const ep_sources *sources, const ep_tokens *tokens,
                       uint32_t epoch, void *staging, void *ws, size_t ws_bytes, void *stream);

/* Copy epilogue: dense row i < N = recv_offsets[R*S] of region (r, s)
 * (recv_offsets[r*S+s] <= i < recv_offsets[r*S+s+1]) is staging row
 * (r*S+s)*capacity + (i - recv_offsets[r*S+s]); its record (pieces
 * `seg_flags`, as written by ep_source_dispatch) is unpacked into row i of
 * the receive arrays (NULL ones skipped; a piece must be in the record to be
 * asked for). A row whose flags are not all epoch is skipped
 * (EP_DEVERR_FLAG); rows >= recv->capacity and region rows >= capacity are
 * skipped (EP_DEVERR_CAPACITY). The result equals ep_dispatch's receive
 * rows. The combine of this layout is ep_combine with layout->slot =
 * src_slot over y rows indexed like the staging buffer. */
int ep_copy_epilogue(const ep_shape *shape, const ep_sources *sources, const void *staging,
                     uint32_t epoch, int seg_flags, const ep_recv *recv, void *ws,
                     size_t ws_bytes, void *stream);

/* Send and copy epilogue in one persistent launch: the same staging rows and
 * receive rows as ep_source_dispatch followed by ep_copy_epilogue with the
 * pieces of `tokens` (EP_SEG_BF16, plus EP_SEG_FP8 / EP_SEG_SCALES when
 * tokens carry them), with the destinations consuming each batch of records
 * once its flag is published ([V2] §3.3 阶段2 and 阶段3; [ASC] 方案一: a
 * batch's records written without ordering, then one ordered flag). Jobs are
 * handed out in order: job i sends the records of tokens [4i, 4i+4) and
 * publishes the batch, then unpacks the staging rows of batch i - 64 into
 * their dense rows recv_offsets[r*S+s] + j, while those rows are still in the
 * MALL. That pays off only when the staging rows are well past the MALL:
 * at 4,096 tokens over 32 ranks and 32 sources, 0.95 times the two calls'
 * time at H = 7,168 (473 MB of staging rows), 1.05 times at H = 4,096 and
 * up to 1.26 times at H = 1,024. A batch whose flag does not come within
 * 100 ms is not unpacked (EP_DEVERR_TIMEOUT); rows >= recv->capacity are skipped
 * (EP_DEVERR_CAPACITY). Needs the arguments of both calls; the workspace
 * (ep_source_workspace_bytes) also holds the batch flags, which the call
 * zeroes first with a small kernel, so calls on one workspace must not
 * overlap. */
int ep_source_dispatch_fused(const ep_shape *shape, const ep_sources *sources, const ep_tokens *tokens,
                             uint32_t epoch, void *staging, const ep_recv *recv, void *ws,
                             size_t ws_bytes, void *stream);

/* ---- Expert products -------------------------------------------------------
 * What runs between dispatch and combine: the experts' two-layer network with
 * a SwiGLU gate,
 *   expert(x) = W2 (silu(G) * U),  [G; U] = W13 x,  silu(v) = v / (1 + exp(-v)),
 * on the expand-mode rows that ep_dispatch_expand writes ([V2] §3.3 阶段3: rows
 * grouped by expert for the expert GEMMs), its gradients, and for a few
 * tokens the whole layer in two launches without dispatch and combine.
 *
 * Rows of expert e are [expert_offsets[e], expert_offsets[e+1]) of the given
 * arrays, which hold `rows` rows; rows at and past expert_offsets[E] are
 * neither read nor written, rows >= `rows` are left out and set
 * EP_DEVERR_CAPACITY, and so do offsets that decrease or are negative
 * (ep_expert_matmul and ep_expert_swiglu then compute nothing, ep_expert_wgrad
 * sums the rows that exist of each expert's own range). An expert may have no
 * rows. Sums are held in 32 bits and rounded once to the output's type (round
 * to nearest even). Matrix dimensions are multiples of 8 up to EP_MAX_DIM; all
 * arrays here need 16 B aligned base pointers, except topk_weights and its
 * gradient (4 B). Outputs must not overlap inputs. Calls that only use the
 * workspace for its error words (all but ep_moe_few) may overlap on one
 * workspace.
 *
 * A whole training step of a layer, from these calls:
 *   forward   ep_get_layout, ep_dispatch_expand, ep_expert_swiglu (act and the
 *             8-bit checkpoint), ep_expert_matmul (W2, NK), ep_combine_expand
 *   backward  ep_dispatch_expand of the output's gradient (rows d_y),
 *             ep_expert_matmul (d_y, W2, KN -> d_act), ep_swiglu_grad (-> d_gu,
 *             w * act, d_topk_weights), ep_expert_wgrad (d_y, w * act -> dW2),
 *             ep_expert_wgrad (d_gu, x -> dW13; x the dispatched bf16 or FP8
 *             rows), ep_expert_matmul (d_gu, W13, KN -> d_x rows),
 *             ep_combine_expand of those with weights of 1. */

/* Rows times the experts' matrices: for each row i of expert e,
 *   y[i][n] = bf16_rne(sum_k x[i][k] * w[e][n][k])   (EP_WEIGHT_NK)
 *   y[i][n] = bf16_rne(sum_k x[i][k] * w[e][k][n])   (EP_WEIGHT_KN)
 * x: [rows][k_dim] bf16, y: [rows][n_dim] bf16. Needs layout->expert_offsets. */
int ep_expert_matmul(const ep_shape *shape, const ep_layout *layout, const uint16_t *x, int64_t rows,
                     int32_t k_dim, const uint16_t *w, int32_t n_dim, int w_order, uint16_t *y,
                     void *ws, size_t ws_bytes, void *stream);

/* Gate/up product with SwiGLU in one pass, and the 8-bit checkpoint that its
 * gradient reads: for each row i of expert e, in 32 bits,
 *   g = x[i] * w13[e][0:F]^T, u = x[i] * w13[e][F:2F]^T,
 *   act[i] = bf16_rne(silu(g) * u);
 * and, when gu_fp8 is non-NULL, for every block of 128 values of [g, u]:
 *   gu_scales = m / 448, m the block's largest magnitude (1 if m < 1e-33)
 *   gu_fp8 = e4m3_rne(v * (1 / gu_scales)).
 * A NaN reads back as NaN; all values of a block with an infinity do.
 * x: [rows][H], w13: [E][2F][H] (gate rows, then up rows), act: [rows][F] bf16;
 * gu_fp8: [rows][2F], gu_scales: [rows][2F/128], both or neither (F % 128 ==
 * 0 with them). 4 * F * H must stay below 2^31 - 16 (EP_ERR_UNSUPPORTED). */
int ep_expert_swiglu(const ep_shape *shape, const ep_layout *layout, const uint16_t *x, int64_t rows,
                     const uint16_t *w13, int32_t F, uint16_t *act, uint8_t *gu_fp8, float *gu_scales,
                     void *ws, size_t ws_bytes, void *stream);

/* Gradient of the SwiGLU from the checkpoint. For each lane (t, k) with row i
 * = layout->expert_slot[t*K+k] >= 0 and weight w = topk_weights[t*K+k], with g
 * and u the values that the checkpoint stands for, s = 1 / (1 + exp(-g)) and d
 * = d_act[i] (the gradient of the row's expert output, without w, times W2):
 *   d_gu[i]  = bf16_rne([w d u s (1 + g (1 - s)), w d g s])
 *   act_w[i] = bf16_rne(w g s u)         (the rows that W2's gradient takes)
 *   d_topk_weights[t*K+k] = sum_f d g s u  (0 for a lane without a row)
 * gu_fp8, gu_scales as written by ep_expert_swiglu; d_act, act_w: [rows][F];
 * d_gu: [rows][2F]; d_topk_weights: [T*K] fp32. act_w and d_topk_weights may
 * be NULL. F % 128 == 0. A slot >= rows is left out (EP_DEVERR_CAPACITY) and
 * its d_topk_weights is 0. */
int ep_swiglu_grad(const ep_shape *shape, const ep_layout *layout, int32_t F, const uint8_t *gu_fp8,
                   const float *gu_scales, const uint16_t *d_act, int64_t rows,
                   const float *topk_weights, uint16_t *d_gu, uint16_t *act_w, float *d_topk_weights,
                   void *ws, size_t ws_bytes, void *stream);

/* Rows of ep_expert_wgrad's second operand: x, or x_fp8 with x_scales. */
typedef struct ep_rows {
    const uint16_t *x;      /* [rows][k_dim] bf16, or NULL */
    const uint8_t *x_fp8;   /* [rows][k_dim] e4m3, or NULL */
    const float *x_scales;  /* [rows][k_dim/128] fp32, with x_fp8 */
} ep_rows;

/* Weight gradient: for every expert e (0 for one without rows)
 *   dw[e][n][k] = sum over rows i of e of dy[i][n] * x[i][k]
 * dy: [rows][n_dim] bf16; x: bf16 rows, or the FP8 rows with their scales
 * that dispatch delivers (k_dim % 128 == 0; each value q * scale is rounded
 * to bf16 for the matrix instruction, by 2^-8 of it at most, for results of
 * either type). dw: [E][n_dim][k_dim], bf16 or fp32
 * (dtype EP_GRAD_*), overwritten. */
int ep_expert_wgrad(const ep_shape *shape, const ep_layout *layout, const uint16_t *dy, int64_t rows,
                    int32_t n_dim, const ep_rows *x, int32_t k_dim, void *dw, int dtype, void *ws,
                    size_t ws_bytes, void *stream);

/* Weights of the experts: bf16 matrices, or e4m3 ones with one fp32 scale for
 * each row and 128 columns (the same form for both matrices). */
typedef struct ep_experts {
    int32_t F;                 /* inner size, F % 8 == 0 (F % 128 == 0 and H % 128 == 0 for FP8) */
    const uint16_t *w13;       /* [E][2F][H] bf16: gate rows, then up rows; or NULL */
    const uint16_t *w2;        /* [E][H][F] bf16, or NULL */
    const uint8_t *w13_fp8;    /* [E][2F][H] e4m3, or NULL */
    const float *w13_scales;   /* [E][2F][H/128] */
    const uint8_t *w2_fp8;     /* [E][H][F] e4m3, or NULL */
    const float *w2_scales;    /* [E][H][F/128] */
} ep_experts;

/* Bytes of workspace of ep_moe_few (>= 256; error words at offset 0 as in
 * ep_workspace_bytes). Host only; 0 on bad args (T > EP_FEW_MAX_TOKENS too). */
size_t ep_few_workspace_bytes(const ep_shape *shape, int32_t F);

/* The whole expert layer for at most EP_FEW_MAX_TOKENS tokens (decoding),
 * without layout, dispatch and combine:
 *   out[t] = bf16_rne(sum over the distinct experts e of t's lanes of
 *            w * W2[e] (silu(g) * u)),  w = the sum of the weights of t's
 *            lanes with expert e, [g; u] = W13[e] x[t]
 * silu(g) * u enters the second product as two bf16 values, itself rounded and
 * what that leaves (off by 2^-16 of it at most, where |silu(g) * u| > 1e-33).
 * tokens: x, topk_idx and topk_weights required. A token without a valid lane
 * gets zeros. An expert's non-finite results reach only its own tokens. Starts
 * a pass: clears error word 0, then sets EP_DEVERR_EXPERT_ID for ids < -1 or
 * >= E (treated as -1). out: [T*H] bf16. ws: ep_few_workspace_bytes, 256 B
 * aligned, needs no initialisation besides ep_clear_errors; calls on one
 * workspace must not overlap. */
int ep_moe_few(const ep_shape *shape, const ep_tokens *tokens, const ep_experts *experts,
               uint16_t *out, void *ws, size_t ws_bytes, void *stream);

/* ---- Before the dispatch: norm and router ----------------------------------
 * What makes the rows and the routing that ep_dispatch, ep_dispatch_expand and
 * ep_moe_few take, and takes the gradients that the backward pass hands back.
 * One layer, in calls (l = the router's product y W^T in 32 bits, a plain
 * matrix product that the caller makes):
 *   forward   ep_rms_norm (y bf16 and / or y_fp8 with y_scales, the stream h,
 *             rstd), l, ep_route, ep_get_layout, ..., ep_combine_expand -> x of
 *             the next ep_rms_norm (which adds it to the stream)
 *   backward  ..., ep_swiglu_grad (d_topk_weights) -> ep_route_grad (d_logits;
 *             ep_expert_matmul and ep_expert_wgrad with one expert take them
 *             on in bf16, E % 8 == 0), d_y = the rows' and the router's part ->
 *             ep_rms_norm_grad -> the stream's gradient and the gain's
 * No call writes a row past shape->T. Sums are held in 32 bits. */

/* Outputs of ep_rms_norm; NULL ones are left out. */
typedef struct ep_norm_out {
    void *h;          /* [T*H] the stream with x added, in the stream's type; may be `residual` itself */
    uint16_t *y;      /* [T*H] bf16 */
    uint8_t *y_fp8;   /* [T*H] e4m3, with y_scales (H % 128 == 0) */
    float *y_scales;  /* [T*H/128] */
    float *rstd;      /* [T] for ep_rms_norm_grad */
} ep_norm_out;

/* Root-mean-square norm of a residual stream: for each token t < T
 *   h[t] = x[t] + residual[t], rounded to the stream's type (x[t] alone
 *          where residual is NULL),
 *   rstd[t] = 1 / sqrt(mean over H of h[t]^2 + eps),
 *   v = h[t] * rstd[t] * gain,
 *   y[t] = bf16_rne(v), and for every 128 channels, m their largest |v|,
 *   y_scales = m / 448 (1 if m < 1e-33), y_fp8 = e4m3_rne(v * (1 / y_scales)).
 * x: [T*H] bf16, residual: [T*H] of stream_type (EP_STREAM_*) or NULL, gain:
 * [H] bf16, eps > 0 and finite, H <= EP_MAX_DIM. The norm is that of h as
 * stored, so its gradient needs h alone. A row whose mean square passes 32
 * bits has rstd 0. x, residual, gain, h, y and y_fp8 need 16 B aligned base
 * pointers. out->h may be residual (same address); apart from that outputs
 * must not overlap inputs or each other. At least one output. */
int ep_rms_norm(const ep_shape *shape, const uint16_t *x, const void *residual, int stream_type,
                const uint16_t *gain, float eps, const ep_norm_out *out, void *stream);

/* Bytes of workspace of ep_rms_norm_grad (>= 256). Host only; 0 on bad args. */
size_t ep_norm_workspace_bytes(const ep_shape *shape);

/* Gradient of ep_rms_norm: with a = dy[t] * gain, r = rstd[t],
 *   d = d_stream[t] + r * (a - h[t] * r^2 * mean over H of a * h[t])
 *   d_h[t] = d in the stream's type (the gradient of residual, and of x),
 *   d_x[t] = bf16_rne(d) (for x where the stream has 32 bits),
 *   d_gain = sum over t of dy[t] * h[t] * r.
 * h: [T*H] of stream_type as ep_rms_norm stored it (x itself for a bf16 stream
 * without residual); dy: [T*H] bf16; d_stream: [T*H] of stream_type, the
 * gradient that h has from the layers after, or NULL; d_h: like d_stream, may
 * be it (same address); d_x: [T*H] bf16; d_gain: [H] fp32, overwritten (0 with
 * T = 0). d_h, d_x and d_gain may be NULL, not all of them; apart from d_h =
 * d_stream, outputs must not overlap inputs or each other. The sum over t is
 * made in a fixed order: calls repeat bit for bit. 16 B aligned base pointers;
 * rstd 4 B. ws: ep_norm_workspace_bytes, 256 B aligned, needs no
 * initialisation; calls on one workspace must not overlap. */
int ep_rms_norm_grad(const ep_shape *shape, const void *h, int stream_type, const uint16_t *gain,
                     const float *rstd, const uint16_t *dy, const void *d_stream, void *d_h,
                     uint16_t *d_x, float *d_gain, void *ws, size_t ws_bytes, void *stream);

/* How a router chooses and weighs. */
typedef struct ep_router {
    int32_t score;      /* EP_SCORE_* */
    int32_t top_groups; /* groups of shape->G that a token's experts may lie in, 1..G (G: any);
                           less than G: G <= 64 (EP_ERR_UNSUPPORTED) */
    int32_t group_top;  /* a group ranks by the sum of its 1 or 2 largest keys */
    int32_t normalize;  /* 1: weights of a token add up to `scale`; 0: they are scores times scale */
    float scale;        /* finite */
    const float *bias;  /* [E] added to the scores for the choice alone, or NULL */
} ep_router;

/* Router: K experts of each token and their weights from its logits.
 *   s[e] = the score (EP_SCORE_*) of l = logits[t*E + e]
 *   key[e] = s[e] + bias[e], in 64 bits; where bias is NULL and the groups do
 *            not rank by sums of two, the logit itself (which orders alike)
 *   groups (top_groups < G; group g holds experts [g*E/G, (g+1)*E/G), as in
 *            the layout): the top_groups groups with the largest sums of
 *            their group_top largest keys
 *   topk_idx[t*K + k] = the expert with the k-th largest key of those groups
 *   topk_weights[t*K + k] = scale * s / (sum of the K chosen s + 1e-20)  (normalize)
 *                           scale * s                                    (otherwise)
 * Equal keys go to the lower id. A masked expert, whose logit or key is
 * -infinity, is never chosen and counts for nothing in a group's sum; lanes
 * left without an expert get -1 and weight 0, as do all of a token without
 * unmasked experts. Experts with a logit of +infinity share a softmax evenly.
 * NaN logits and biases are taken as -infinity and set EP_DEVERR_LOGIT.
 * logits: [T*E] fp32, topk_idx: [T*K], topk_weights: [T*K] fp32 (may be NULL).
 * ws: ep_workspace_bytes(shape), for its error words; the call clears none
 * (ep_get_layout clears word 0, word 1 keeps the report). */
int ep_route(const ep_shape *shape, const float *logits, const ep_router *router, int64_t *topk_idx,
             float *topk_weights, void *ws, size_t ws_bytes, void *stream);

/* Gradient of ep_route's weights for the logits, the choice held fixed (bias,
 * groups and keys have none): with g[k] = scale * d_topk_weights[t*K + k],
 * S = sum of the chosen s + 1e-20,
 *   d_s[k] = (g[k] - sum_j g[j] s[j] / S) / S  (normalize),  g[k]  (otherwise)
 *   d_logits[t*E + e] = s[e] * (d_s[e] - sum_k d_s[k] s[k])  (softmax)
 *                       s[e] * (1 - s[e]) * d_s[e]           (sigmoid)
 * d_s[e] summed over the lanes that hold e, 0 for the others. Lanes with -1
 * have no part; ids < -1 or >= E neither, and set EP_DEVERR_EXPERT_ID. Masked
 * experts get 0. d_logits: [T*E], bf16 or fp32 (dtype EP_GRAD_*), 16 B
 * aligned. ws as in ep_route. */
int ep_route_grad(const ep_shape *shape, const float *logits, const ep_router *router,
                  const int64_t *topk_idx, const float *d_topk_weights, void *d_logits, int dtype,
                  void *ws, size_t ws_bytes, void *stream);

/* Weights of the experts in 4 bits: of a row's columns c the code of an even
 * one lies in the low half of byte c / 2, of an odd one in the high half. */
typedef struct ep_experts_w4 {
    int32_t F;               /* inner size; EP_W4_INT: F and H % 128 == 0, EP_W4_E2M1: % 32 */
    int32_t form;            /* EP_W4_* */
    const uint8_t *w13;      /* [E][2F][H/2]: gate rows, then up rows */
    const void *w13_scales;  /* [E][2F][H/128] bf16 or [E][2F][H/32] bytes */
    const uint8_t *w2;       /* [E][H][F/2] */
    const void *w2_scales;   /* [E][H][F/128] bf16 or [E][H][F/32] bytes */
} ep_experts_w4;

/* Bytes of workspace of ep_moe_few_w4, as ep_few_workspace_bytes. */
size_t ep_few_w4_workspace_bytes(const ep_shape *shape, int32_t F);

/* ep_moe_few with 4-bit weights: the same result for the values that codes and
 * scales stand for (these are exact in the products, sums are held in 32
 * bits), the same tokens, errors, workspace rules and limits, and T * K * F <
 * 2^29. Longer batches go in parts of EP_FEW_MAX_TOKENS. Base pointers 16 B
 * aligned. EP_W4_E2M1 values past bf16's range (scale bytes of 253 and 254)
 * are infinite. */
int ep_moe_few_w4(const ep_shape *shape, const ep_tokens *tokens, const ep_experts_w4 *experts,
                  uint16_t *out, void *ws, size_t ws_bytes, void *stream);

/* Clear both workspace error words (a stream-ordered kernel, no memset
 * node). */
int ep_clear_errors(void *ws, void *stream);

/* Synchronise `stream`, then copy error word 0 (the errors since the last
 * ep_get_layout / ep_source_layout call on this workspace) to *bits (host
 * pointer). Returns EP_OK when no bit is set, EP_ERR_DEVICE when one is
 * ([V2] §3.5: the caller learns of a failed pass from the call, not only
 * from the data), EP_ERR_ARG / EP_ERR_HIP when the word could not be read
 * (*bits is then left unchanged). */
int ep_check_errors(void *ws, void *stream, uint32_t *bits);

/* As ep_check_errors, for error word 1: every error any call on this
 * workspace reported since the last ep_clear_errors, across passes (a pass
 * that follows a failed one does not hide it). */
int ep_check_sticky_errors(void *ws, void *stream, uint32_t *bits);

/* Static description of a status code. */
const char *ep_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* EP_H */
