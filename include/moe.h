/*
 * moe.h -- C ABI of the OEA MoE decode layer for one GB300 (sm_103a).
 *
 * The layer is the decode-time Mixture-of-Experts block described on the
 * page "Opportunistic Expert Activation (OEA)" (zhaifeiyue.github.io,
 * papers/2511.02237/detail.html):
 *   1. router scores and per-token top-k (section 2, Q1/Q2);
 *   2. optionally the OEA two-phase re-route: each token keeps its top-n_i
 *      experts, n_i = min(k0, t_i) with t_i an adaptive top-p count, the
 *      batch union S_base of those baselines is formed, and each token then
 *      adds experts from its own ranked list only if they are already in
 *      S_base, so T = |S_base| does not grow; kept scores are renormalised
 *      (section 2 Q2, section 3);
 *   3. grouping of (token, slot) pairs by expert (the per-expert loads
 *      cnt_e of the cost model, section 4);
 *   4. the expert FFN of every activated expert, each expert's weights read
 *      from HBM once (section 2 Q1, section 4 check 4), in the SwiGLU form
 *      of the Qwen3 experts the page measures:
 *      y = W_down (silu(W_gate x) * (W_up x));
 *   5. the weighted combine out_i = sum_j w_ij y_{e_ij}(x_i).
 *
 * Conventions shared by every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller, 16-byte
 *     aligned, row-major and densely packed.  Buffers whose size is a
 *     multiple of B may be NULL when B == 0.  The library allocates no
 *     device memory; per-call scratch lives in the caller's workspace.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default
 *     stream).  Nothing synchronises except moe_device_status().
 *   - Arguments are checked on the host before anything is launched; a bad
 *     argument returns MOE_ERR_ARG and launches nothing.  Conditions only
 *     the GPU can see (a non-finite router score, a wait that timed out)
 *     set bits in a flag word in the workspace and never trap; read them
 *     with moe_device_status().
 *   - Results are deterministic: the same inputs give the same bits.
 *   - Not thread-safe per workspace: calls that share a workspace must be
 *     ordered on one stream.
 */
#ifndef OEA_MOE_H
#define OEA_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream. */
typedef struct CUstream_st *moe_stream_t;

typedef enum {
    MOE_OK = 0,
    MOE_ERR_ARG = 1,          /* invalid argument; nothing was launched       */
    MOE_ERR_CUDA = 2,         /* a CUDA runtime call failed                   */
    MOE_ERR_DEVICE_CHECK = 3, /* the GPU raised a flag (moe_device_status)    */
    MOE_ERR_WORKSPACE = 4,    /* workspace missing, misaligned or too small   */
    MOE_ERR_UNSUPPORTED = 5   /* valid but not supported on this device       */
} moe_status;

typedef enum { MOE_MODE_TOPK = 0, MOE_MODE_OEA = 1 } moe_mode;

/* Element type of hidden states, router and expert weights and output. */
typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F32 = 1 } moe_dtype;

/* Device flag bits reported by moe_device_status(). */
#define MOE_FLAG_NONFINITE_SCORE 0x1u  /* a router score was NaN or +-inf     */
#define MOE_FLAG_WAIT_TIMEOUT 0x2u     /* an in-kernel wait gave up           */
#define MOE_FLAG_BAD_INDEX 0x4u        /* an index failed its range check     */

/* Size limits. */
#define MOE_MAX_TOKENS 256
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_SLOTS 32

/*
 * Routing parameters (OEA page, section 2 Q2; sections 4-5 and 7 for maxP,
 * k^max and the padding mask).
 *   B        tokens in the batch, 0..MOE_MAX_TOKENS.
 *   B_valid  tokens 0..B_valid-1 are real; tokens B_valid..B-1 are padding
 *            and select no expert, so they cannot enlarge T (OEA page,
 *            section 7, implementation detail 1).  Negative: B.
 *   d        hidden size; a multiple of 64.
 *   N        experts, 1..MOE_MAX_EXPERTS.
 *   k        experts per token of the plain router, 1..min(N, 32).
 *   mode     MOE_MODE_TOPK or MOE_MODE_OEA.
 *   k0       OEA baseline cap, 1..k; <= 0 chooses it from the batch
 *            (section 7, implementation detail 2: piggybacking adds nothing
 *            for a single token, and smaller batches want a larger, safer
 *            k0): B_valid <= 1 routes as plain top-k (k0 = k, top-p off),
 *            2..15 real tokens take k0 = ceil(5k/8), 16 or more
 *            ceil(3k/8) -- for k = 8 the page's settings 5 and 3.
 *   p        OEA top-p threshold in (0, 1]; p >= 1 switches top-p off
 *            (t_i = N), as in the simplified router of section 5.
 *   maxP     OEA: deepest rank of the token's own list that phase 2 may
 *            take an expert from; <= 0 or >= N means N (no limit).
 *   kmax     OEA: experts per token after phase 2 (k^max); <= 0 means k;
 *            otherwise k0..min(N, 32).
 *   dtype    moe_dtype of hidden, router weights, expert weights and output.
 * Slots per token: kslots = k for MOE_MODE_TOPK, kmax for MOE_MODE_OEA
 * (moe_num_slots()).
 */
typedef struct {
    int32_t B;
    int32_t B_valid;
    int32_t d;
    int32_t N;
    int32_t k;
    int32_t mode;
    int32_t k0;
    float p;
    int32_t maxP;
    int32_t kmax;
    int32_t dtype;
} moe_route_params;

/*
 * Routing results: device buffers owned by the caller, written by
 * moe_route().  Ranks and ties: experts are ranked by score, larger first,
 * equal scores by the lower expert id.
 *   expert_idx [B][kslots] int32  chosen experts in rank order, -1 in unused
 *                                 slots (a token keeps min(kmax, T) experts
 *                                 in OEA mode; padding tokens keep none).
 *   weights    [B][kslots] fp32   renormalised scores (softmax over the kept
 *                                 scores), 0 in unused slots.
 *   T          [1] int32          number of distinct activated experts.
 *   active     [N] int32          activated experts, ascending id; entries
 *                                 T..N-1 are -1.
 *   counts     [N] int32          cnt_e, tokens routed to expert e.
 *   offsets    [N+1] int32        exclusive prefix sum of counts.
 *   perm       [B*kslots] int32   token*kslots+slot grouped by expert
 *                                 (ascending id), tokens ascending within an
 *                                 expert; entries offsets[N].. are unused.
 *   n_base     [B] int32          nullable; n_i (k in top-k mode, 0 for
 *                                 padding tokens).
 *   logits     [B][N] fp32        nullable; router scores (bias included).
 */
typedef struct {
    int32_t *expert_idx;
    float *weights;
    int32_t *T;
    int32_t *active;
    int32_t *counts;
    int32_t *offsets;
    int32_t *perm;
    int32_t *n_base;
    float *logits;
} moe_routing;

/* Slots per token for these parameters (k or kmax), or -1 if invalid. */
int32_t moe_num_slots(const moe_route_params *params);

/*
 * Kernels that one moe_decode_layer() call launches for these parameters
 * and expert FFN width on the current device, or -1 if the parameters are
 * invalid.  bf16 batches of up to 32 tokens with N <= 128 score and route
 * in one cluster launch, so a layer is two kernels.  Otherwise the router
 * and the routing are separate launches: three kernels with bf16 experts,
 * five on the fp32 path (three expert kernels).  An empty batch launches
 * only the routing kernel.
 */
int32_t moe_layer_launches(const moe_route_params *params, int32_t d_ff);

/*
 * Bytes of device workspace needed by moe_route / moe_expert_ffn /
 * moe_decode_layer for these parameters and expert FFN width d_ff (pass
 * d_ff = 0 when only moe_route is used).  Returns 0 if the parameters are
 * invalid.  The workspace must be 256-byte aligned and zero-filled once
 * before its first use; the library leaves it ready for the next call.
 */
size_t moe_workspace_bytes(const moe_route_params *params, int32_t d_ff);

/*
 * Router + routing (steps 1-3 above).
 *   hidden      [B][d]  dtype   token hidden states.
 *   w_router    [N][d]  dtype   router (gate) weights.
 *   router_bias [N]     fp32    nullable; added to every score.
 *   routing                     outputs, see moe_routing.
 * Scores are accumulated in fp32.  Routing decisions compare those fp32
 * scores exactly; the top-p prefix is computed in fp32.
 */
moe_status moe_route(const void *hidden, const void *w_router, const float *router_bias,
                     const moe_route_params *params, const moe_routing *routing,
                     void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Expert FFN + weighted combine (steps 4-5) for a batch routed by
 * moe_route() with the same params and the same workspace: besides the
 * routing outputs it reads the per-pair positions, per-expert records and
 * per-(token, 128 rows of d) combine counters that moe_route left in the
 * workspace, so no other call may use that workspace in between.  A
 * completed call leaves them as it found them, so it may be repeated on the
 * same routing.  Reads only activated experts, each expert's three
 * matrices once from HBM.  With OEA routing of up to 64 tokens, the call
 * starts on the activated experts' weights as soon as the preceding
 * moe_route() on this workspace and stream has fixed them (its phase 1),
 * before that routing call's kernel ends; it recognises that call's
 * published set by a per-call tag the library keeps for the workspace.
 *   hidden  [B][d]        dtype  the hidden states given to moe_route.
 *   w_gate  [N][d_ff][d]  dtype  expert gate projections.
 *   w_up    [N][d_ff][d]  dtype  expert up projections.  bf16: where w_gate
 *           and w_up are distinct and less than 2^40 bytes apart (two halves
 *           of one allocation always are), one tensor map reads both and a
 *           pipeline stage of an expert tile is a single copy; otherwise
 *           (for instance separate allocations in distant address ranges)
 *           each stage takes 16 smaller copies, and such tiles run about
 *           20 % slower.  Results are the same.
 *   w_down  [N][d][d_ff]  dtype  expert down projections.
 *   d_ff    expert FFN width, a multiple of 64.
 *   routing the results of moe_route (expert_idx, weights, T, active,
 *           counts, offsets, perm are read).
 *   out     [B][d]        dtype  written; padding tokens get zeros.
 * bf16: products in fp32 on tensor cores, the SwiGLU activation h rounded
 * to bf16 before the down projection, sums in fp32, output rounded once.
 * fp32: all arithmetic in fp32 on CUDA cores.
 */
moe_status moe_expert_ffn(const void *hidden, const void *w_gate, const void *w_up,
                          const void *w_down, int32_t d_ff, const moe_route_params *params,
                          const moe_routing *routing, void *out, void *workspace,
                          size_t workspace_bytes, moe_stream_t stream);

/*
 * Mixed-precision experts (DynaExq page, section 3.2: frequently used experts
 * in high precision, the others in a 4-bit version).  Hot experts keep bf16
 * weights in w_gate / w_up / w_down (laid out as for moe_expert_ffn, with
 * n_hot experts); cold experts are INT4 with one bf16 scale per row and
 * 128-column group of the contraction dimension (d for W_gate / W_up, d_ff
 * for W_down): w = q * s, q in -7..7.  An INT4 expert is
 * 3 * (d * d_ff / 2 + d * d_ff / 64) bytes (moe_pack_int4 makes images).
 *   slot    [N] int32, device: for expert e, slot[e] >= 0 is its index among
 *           the bf16 experts, slot[e] < 0 means INT4 expert -1 - slot[e].
 *           An out-of-range slot raises MOE_FLAG_BAD_INDEX.
 *   q_gate, q_up  [n_cold] packed images of the [d_ff][d] matrices,
 *   q_down        [n_cold] packed images of the [d][d_ff] matrices.
 * Packed image of a matrix [rows][cols] with chunk height rb (64 for W_gate
 * and W_up, 128 for W_down): chunks of rb rows x 128 columns (one scale
 * group) in row-block-major, column-group order; a chunk is rb*64 bytes of
 * codes then rb bf16 scales (one per row: the row's scale of the group).
 * In a chunk row, local column c is the 4-bit field at bit
 * 4*((c%8)/2) + 16*(c%2) of little-endian 32-bit word c/8 of the row's 64
 * bytes, holding q + 8.
 * Requirements: dtype bf16, d and d_ff multiples of 128, n_hot >= 1,
 * 16-byte aligned images.  Results as moe_expert_ffn; each INT4 weight is
 * decoded to q exactly and multiplied by its group scale with one rounding
 * to bf16 before the tensor-core products (fp32 accumulation).
 */
typedef struct {
    const int32_t *slot;
    const void *q_gate;
    const void *q_up;
    const void *q_down;
    int32_t n_hot;
    int32_t n_cold;
} moe_mixed_experts;

moe_status moe_expert_ffn_mixed(const void *hidden, const void *w_gate, const void *w_up, const void *w_down,
                                const moe_mixed_experts *mixed, int32_t d_ff, const moe_route_params *params,
                                const moe_routing *routing, void *out, void *workspace, size_t workspace_bytes,
                                moe_stream_t stream);

/*
 * Makes the packed INT4 image of one bf16 matrix on the device: the 4-bit
 * version of an expert matrix that moe_expert_ffn_mixed reads (DynaExq
 * page, section 3.2, INT4 tier; section 2.4: a new version is prepared
 * off the request path and only then published, here by writing the
 * expert's slot).  Per row and 128-column group:
 *   s = max|w| / 7, the quotient taken in double and rounded to nearest
 *       even, first to fp32, then to bf16;
 *   q = rint(w / s) in double (ties to even), clamped to -7..7; q = 0
 *       where s = 0.
 *   w     [rows][cols] bf16, device, 16-byte aligned.
 *   rows  a multiple of rb.  cols: a multiple of 128.
 *   rb    chunk height of the image: 64 for W_gate / W_up, 128 for W_down
 *         (any multiple of 8 is accepted).
 *   out   rows*cols/2 + rows*(cols/128)*2 bytes, device, 16-byte aligned.
 * Asynchronous on `stream`; allocates nothing.
 */
moe_status moe_pack_int4(const void *w, int32_t rows, int32_t cols, int32_t rb, void *out, moe_stream_t stream);

/*
 * The whole layer with mixed-precision experts in one call: moe_route, then
 * moe_expert_ffn_mixed, on the same stream and workspace.  `mixed` is the
 * per-expert descriptor of the DynaExq page's stable expert handles
 * (section 2.2; section 3.2 for the precision tiers): for every expert id,
 * its slot says where its current version lives -- a bf16 expert of
 * w_gate / w_up / w_down, or a packed INT4 image -- so the kernels resolve
 * each activated expert through the table and a caller switches an
 * expert's version by rewriting its slot (and image) between calls.
 * Arguments, layouts and results as moe_route and moe_expert_ffn_mixed;
 * every argument, the descriptor included, is checked before anything is
 * launched.  With OEA routing of up to 64 tokens the expert kernel starts
 * on the activated experts before the routing kernel ends, as for
 * moe_expert_ffn.
 */
moe_status moe_decode_layer_mixed(const void *hidden, const void *w_router, const float *router_bias,
                                  const void *w_gate, const void *w_up, const void *w_down,
                                  const moe_mixed_experts *mixed, int32_t d_ff,
                                  const moe_route_params *params, const moe_routing *routing, void *out,
                                  void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Expert residency at run time (DynaExq page, sections 2.2-2.5 and 3.2-3.5):
 * which experts of one layer keep their bf16 version, decided from the
 * routing as the layer runs, and changed without stopping it.
 *   - Handles: `slot` is the table moe_expert_ffn_mixed / moe_decode_layer_mixed
 *     read (pass it as moe_mixed_experts.slot with n_hot = n_hot, n_cold = N
 *     and INT4 images of all N experts, image i = expert i).  The kernels
 *     resolve every activated expert through it at every call.
 *   - Pools: the caller's bf16 pool of n_hot slots (fixed budget) and INT4
 *     images of all experts, which stay resident as the version every handle
 *     can fall back to.
 *   - Hotness (section 2.5): moe_residency_observe adds a call's per-expert
 *     counts (moe_routing.counts) on the device; every update_every calls the
 *     interval's counts c are copied to `snapshot` (pinned host memory) and
 *     cleared, without waiting; when they have arrived,
 *     S_e <- alpha S_e + (1 - alpha) c_e (S starts at 0).
 *   - Selection with hysteresis (section 3.5): while the best expert outside
 *     the bf16 set (highest S, ties to the lower id) scores more than
 *     `margin` above the weakest member (lowest S, ties to the higher id),
 *     the two swap places (moe_residency_select).  A selection runs only
 *     when no transition is pending.
 *   - Transitions (sections 2.4, 3.4): a demotion redirects the handle to
 *     the INT4 image on the caller's stream, then the freed slot receives
 *     the promoted expert's bf16 weights: an asynchronous copy from the
 *     caller's pinned host memory on the residency's own migration stream,
 *     which waits for the redirect.  The handle is pointed at the new slot
 *     only after that copy's completion event has been seen (by a later
 *     observe or flush), so no kernel reads a partly copied version; until
 *     then the expert runs in INT4.  At most max_inflight copies are in
 *     flight; further swaps wait in a queue.
 * The library allocates no device memory for this: the accumulator and the
 * snapshot are the caller's.  Not thread-safe; calls on one residency must
 * use one stream.
 * Reading of the page: the update interval is counted in routing calls
 * (the page uses a time interval); the INT4 images of all experts stay on
 * the device, so a demotion moves no data.
 */
typedef struct {
    int32_t N;             /* experts, 2..MOE_MAX_EXPERTS                          */
    int32_t n_hot;         /* bf16 slots (the budget), 1..N-1                      */
    int32_t d, d_ff;       /* multiples of 128                                     */
    double alpha;          /* weight of the old score, 0 <= alpha < 1              */
    double margin;         /* hysteresis margin, in selections per interval, >= 0 */
    int32_t update_every;  /* routing calls per update interval, >= 1             */
    int32_t max_inflight;  /* promotion copies in flight at once, >= 1            */
    int32_t *slot;         /* [N] device: the handle table                         */
    uint32_t *counts_acc;  /* [N] device: counts of the current interval           */
    uint32_t *snapshot;    /* [N] pinned host: counts of the last interval         */
    void *hot_gate;        /* device bf16 pool: [n_hot][d_ff][d]                   */
    void *hot_up;          /*                   [n_hot][d_ff][d]                   */
    void *hot_down;        /*                   [n_hot][d][d_ff]                   */
    const void *host_gate; /* pinned host bf16 weights of all experts: [N][d_ff][d] */
    const void *host_up;   /*                                          [N][d_ff][d] */
    const void *host_down; /*                                          [N][d][d_ff] */
} moe_residency_config;

typedef struct moe_residency moe_residency;

/* Residency states reported by moe_residency_query. */
#define MOE_RESIDENT_LO 0
#define MOE_RESIDENT_HI 1
#define MOE_PROMOTING 2

/*
 * Creates a residency whose bf16 set starts as initial_hot[n_hot] (expert
 * initial_hot[k] in slot k; the caller has filled the pool accordingly).
 * Writes the handle table and clears the accumulator on `stream` and waits
 * for them.
 */
moe_status moe_residency_create(const moe_residency_config *cfg, const int32_t *initial_hot,
                                moe_residency **out, moe_stream_t stream);

/* After a routing call on `stream`: adds its counts[N] (device), publishes
 * completed promotions, updates the scores when a snapshot has arrived,
 * selects and issues transitions.  Never waits for the GPU. */
moe_status moe_residency_observe(moe_residency *r, const int32_t *counts, moe_stream_t stream);

/* Waits for every queued and in-flight transition and publishes it. */
moe_status moe_residency_flush(moe_residency *r, moe_stream_t stream);

/* Host copies of the per-expert state (MOE_RESIDENT_*, nullable [N]), the
 * scores S (nullable [N]) and, in stats[5] (nullable): routing calls seen,
 * score updates, promotions, demotions, transitions queued or in flight. */
moe_status moe_residency_query(const moe_residency *r, int32_t *state, double *scores, uint64_t *stats);

moe_status moe_residency_destroy(moe_residency *r);

/*
 * The selection step alone, on the host: in_hot[N] (0/1) is updated in
 * place and the swaps are written to promote / demote (nullable, [N]) in
 * the order they are made.  Returns their number, or -1 for bad arguments.
 */
int32_t moe_residency_select(const double *S, int32_t N, double margin, uint8_t *in_hot, int32_t *promote,
                             int32_t *demote);

/* moe_route followed by moe_expert_ffn on the same stream. */
moe_status moe_decode_layer(const void *hidden, const void *w_router, const float *router_bias,
                            const void *w_gate, const void *w_up, const void *w_down,
                            int32_t d_ff, const moe_route_params *params,
                            const moe_routing *routing, void *out, void *workspace,
                            size_t workspace_bytes, moe_stream_t stream);

/*
 * Routing for models whose router is not a plain top-k of the scores: the
 * experts are scored by a softmax or a sigmoid, a per-expert bias (learnt to
 * balance the experts' load) shifts the selection but not the weights, and
 * the selection may be limited to the best few of n_group equal groups of
 * consecutive experts.  For a token with router scores x[N]:
 *   p_e   = softmax(x)_e or 1 / (1 + exp(-x_e));
 *   v_e   = p_e + bias_e, the selection value;
 *   group value: the sum of the group's group_top (1 or 2) largest v; the
 *           topk_group groups of largest value stay, equal values by the
 *           lower group;
 *   the k largest v_e of the groups that stay are chosen, in that order,
 *           equal values by the lower expert id;
 *   w_e   = p_e, over the sum of the chosen p if renormalise (0 where that
 *           sum is 0), times scale.
 * A softmax without a bias and with group_top 1 is ranked by x itself,
 * which it keeps in order.  An expert whose x or v is not finite is never
 * chosen (a token may then keep fewer than k experts) and raises
 * MOE_FLAG_NONFINITE_SCORE; what the scores of padding tokens (B_valid and on)
 * hold does not matter.  All arithmetic is fp32.
 * MOE_MODE_TOPK only: OEA's two phases are defined on the softmax of the scores
 * over all experts, and what they should be with groups or a balance bias is not.
 */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

#define MOE_MAX_GROUPS 32

typedef struct {
    int32_t score;       /* moe_score                                             */
    int32_t n_group;     /* groups, 1..MOE_MAX_GROUPS, a divisor of N             */
    int32_t topk_group;  /* groups that stay, 1..n_group                          */
    int32_t group_top;   /* 1 or 2 (at most N / n_group): values in a group's sum */
    int32_t renormalise; /* 0 or 1                                                */
    float scale;         /* factor of the weights, finite                         */
} moe_select_params;

/*
 * Selection and grouping (as above) of the caller's router scores.
 *   scores      [B][N] fp32.
 *   select_bias [N] fp32, nullable.
 *   params      mode must be MOE_MODE_TOPK; k at most the experts of the
 *               groups that stay.
 *   routing     as for moe_route (logits is not written).
 * Afterwards moe_expert_ffn or moe_expert_ffn_mixed may follow on the same
 * workspace, as after moe_route.
 */
moe_status moe_route_scores(const float *scores, const float *select_bias, const moe_route_params *params,
                            const moe_select_params *select, const moe_routing *routing, void *workspace,
                            size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_route with this selection: router scores (router_bias added to the
 * scores, select_bias to the selection values), selection and grouping.
 */
moe_status moe_route_grouped(const void *hidden, const void *w_router, const float *router_bias,
                             const float *select_bias, const moe_route_params *params,
                             const moe_select_params *select, const moe_routing *routing, void *workspace,
                             size_t workspace_bytes, moe_stream_t stream);

/* moe_route_grouped followed by moe_expert_ffn on the same stream. */
moe_status moe_decode_layer_grouped(const void *hidden, const void *w_router, const float *router_bias,
                                    const float *select_bias, const void *w_gate, const void *w_up,
                                    const void *w_down, int32_t d_ff, const moe_route_params *params,
                                    const moe_select_params *select, const moe_routing *routing, void *out,
                                    void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * The attention half of a decoder block, for tokens that are decoded or
 * drafted: keys and values live in pages, moe_kv_append rotates a step's
 * queries and keys and writes its keys and values into their pages, and
 * moe_tree_attention attends from the step's tokens to the cache.  No page
 * of the method describes them; they are the library's own addition.
 *
 * A cache holds, for every page, key head and row of the page, one vector
 * of head_dim components:
 *   k, v        [n_pages][kv_heads][page_size][head_dim] dtype, device,
 *               16-byte aligned.
 *   page_table  [n_requests][max_pages] int32, device: entry j of a request
 *               is the page of its positions j * page_size and on.  Read by
 *               moe_tree_attention only (NULL is allowed for moe_kv_append).
 *   head_dim    a multiple of 8, 8..256.  page_size: 1..65536.
 */
typedef struct {
    void *k;
    void *v;
    const int32_t *page_table;
    int32_t n_pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t n_requests;
    int32_t max_pages;
    int32_t dtype;
} moe_kv_cache;

#define MOE_MAX_HEAD_DIM 256
#define MOE_MAX_PAGE 65536
#define MOE_MAX_REQUESTS 1024

/*
 * Rotation angles: position m turns pair i (0 <= i < rot / 2) by m * f_i,
 * f_i = base^(-2 i / rot), or scaled for contexts longer than a model was
 * trained on:
 *   MOE_ROPE_LINEAR  f_i / factor (positions are interpolated);
 *   MOE_ROPE_NTK     base * factor^(rot / (rot - 2)) in place of base;
 *   MOE_ROPE_YARN    (Peng et al., "YaRN", 2023) pairs that turn more than
 *                    beta_fast times over original_len positions keep f_i,
 *                    pairs that turn less than beta_slow times take
 *                    f_i / factor, with a linear ramp over the pair index
 *                    between the two (its ends rounded outwards to whole
 *                    indices); cosines and sines are multiplied by
 *                    0.1 ln(factor) + 1, unless `magnitude` is positive.
 *   magnitude        factor of every cosine and sine; <= 0: 1 (YaRN: the
 *                    value above).
 */
typedef enum { MOE_ROPE_PLAIN = 0, MOE_ROPE_LINEAR = 1, MOE_ROPE_NTK = 2, MOE_ROPE_YARN = 3 } moe_rope_scaling;

typedef struct {
    int32_t rot;         /* rotated components, even, 2..MOE_MAX_HEAD_DIM (NTK: 4..) */
    int32_t scaling;     /* moe_rope_scaling                                         */
    double base;         /* > 1                                                      */
    double factor;       /* >= 1 (not read by MOE_ROPE_PLAIN)                        */
    double original_len; /* YaRN: > 0                                                */
    double beta_fast;    /* YaRN: > beta_slow                                        */
    double beta_slow;    /* YaRN: > 0                                                */
    double magnitude;
} moe_rope_params;

/*
 * Writes the table that moe_kv_append reads: table[n_pos][rot] fp32, row m
 * the rot/2 cosines of position m's angles, then their sines (angles and
 * functions in fp64, rounded once).  Made once per model.
 */
moe_status moe_rope_table(const moe_rope_params *params, int32_t n_pos, float *table, moe_stream_t stream);

/*
 * Rotates the queries and keys of T tokens and writes keys and values into
 * the cache.
 *   q [T][heads][head_dim], k and v [T][kv_heads][head_dim], dtype of the
 *             cache: components of a head are adjacent; *_tok and *_head
 *             are the distances, in elements, between tokens and between
 *             heads (slices of one projection's output serve as they are),
 *             each a multiple of 16 bytes.  16-byte aligned.
 *             q and q_out may both be NULL (keys and values only).
 *   rope      [n_pos][rot] fp32 (moe_rope_table); components rot.. of a
 *             head are not rotated.  rot 0: no rotation, rope NULL.
 *   interleaved  0: pair i is (i, i + rot/2); 1: (2i, 2i + 1).
 *   positions [T] int32: rows of rope.  One outside 0..n_pos-1 raises
 *             MOE_FLAG_BAD_INDEX and the nearest row is taken.  Not read
 *             with rot 0.
 *   slots     [T] int64: page * page_size + row of the page.  A negative
 *             slot writes no key and value (padding); one past the cache
 *             raises MOE_FLAG_BAD_INDEX and writes none.  Two tokens of a
 *             call must not share a slot.
 *   q_out     rotated queries; may be q itself with the same distances.
 * A pair (a, b) becomes (a cos - b sin, b cos + a sin) in fp32, rounded
 * once.  The workspace holds the flag word: MOE_ATTENTION_WORKSPACE_MIN
 * bytes (or more), these zero-filled once before its first use.
 */
typedef struct {
    int32_t T;
    int32_t heads;
    int32_t rot;
    int32_t n_pos;
    int32_t interleaved;
    int64_t q_tok, q_head;
    int64_t k_tok, k_head;
    int64_t v_tok, v_head;
    int64_t out_tok, out_head;
} moe_append_params;

#define MOE_ATTENTION_WORKSPACE_MIN 512

moe_status moe_kv_append(const void *q, const void *k, const void *v, const float *rope, const int32_t *positions,
                         const int64_t *slots, const moe_append_params *params, const moe_kv_cache *cache,
                         void *q_out, void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Attention of the step's tokens to their requests' caches.
 *   q          [T][heads][head_dim], cache's dtype, distances as above.
 *              Query head h reads key head h / (heads / kv_heads).
 *   q_offsets  [n_requests + 1] int32, device: tokens q_offsets[r] ..
 *              q_offsets[r + 1] - 1 are request r's, in the order in which
 *              they sit in its cache.  Ascending from 0, the last at most T.
 *   ctx_len    [n_requests] int32, device: positions before the step.  The
 *              request's token i is at position ctx_len + i, written before
 *              the call (moe_kv_append).
 *   mask       [T][mask_words] uint32, device, nullable: token t sees every
 *              position before ctx_len, and its request's token j if bit
 *              j % 32 of word j / 32 of its row is set (a draft tree: its
 *              ancestors and itself); tokens past 32 * mask_words are not
 *              seen.  NULL: token i sees tokens 0..i.
 *   scale      positive and finite.
 *   out        [T][heads][head_dim], dense: sum_j softmax(scale q.k)_j v_j.
 *   lse        [T][heads] fp32, nullable: ln sum_j exp(scale q.k_j).
 * A token that sees nothing gets zeros and an lse of -inf.  Tokens past
 * q_offsets[n_requests] are not written.  What lies in positions that a
 * token does not see, and in rows of its request's pages past its length,
 * has no influence on it whatever its value; a token that sees a drafted
 * token whose value (V) is not finite may become NaN in all components, and one
 * that sees such a value in the context infinite or NaN in that component.
 * A request whose length does not fit max_pages, whose page is outside
 * 0..n_pages-1, or whose q_offsets or ctx_len are out of range raises
 * MOE_FLAG_BAD_INDEX; its output is unspecified, other requests are not
 * affected.  A wait that passes moe_set_wait_timeout_us raises
 * MOE_FLAG_WAIT_TIMEOUT; the call's output is not valid then, and the
 * workspace is ready for the next call.
 * Lengths, offsets, table and mask are read on the device, so a captured
 * call follows their contents.  Results repeat bit for bit.
 * Products and sums are fp32.  Tensor cores (bf16, heads of 64 or 128, pages
 * that are a multiple of 8 and divide 128 or are a multiple of it): the
 * exponentials are rounded before the product with V, their sum is not; to two
 * bf16 numbers each (2^-16 of it) while the requests have few rows a key head
 * (tokens times heads / kv_heads), to one (2^-8 of it) with more.  Few are up to
 * 48 on average, T over n_requests; up to 64 for one request, or where T is at
 * most n_requests.  Other heads and pages, and fp32, run on CUDA cores, without
 * that rounding.
 * T and n_requests (the page table's height) choose the tiles as well: a table
 * with many rows for requests that have no tokens in the step, or a T with many
 * tokens past q_offsets[n_requests], costs time (3 requests of 64 tokens at 4000
 * positions in a table of 256 rows 94 us, of 3 rows 30), not correctness.
 * n_requests at most MOE_MAX_REQUESTS, max_pages * page_size at most 2^30.
 * One call takes up to 2^31 - 2^25 pairs of a tile of query rows (tokens times
 * heads / kv_heads, of one request and key head; the shorter the requests, the
 * smaller the tiles) and a tile of keys: minutes of work, such as a prompt of
 * 2^20 tokens with 64 heads, tiles of 256 rows and 128 keys, or on CUDA cores one
 * of 2^18 (64 rows, 32 keys).  From 2^31 on MOE_FLAG_BAD_INDEX is raised and no
 * output of the call is written.
 */
typedef struct {
    int32_t T;
    int32_t heads;
    int32_t mask_words;
    float scale;
    int64_t q_tok, q_head;
} moe_attention_params;

/* Workspace for up to T tokens of `heads` query heads on this cache (its
 * buffers are not read); 0 if the arguments are invalid.  256-byte aligned,
 * its first MOE_ATTENTION_WORKSPACE_MIN bytes zero-filled once before its
 * first use.  It serves moe_kv_append too. */
size_t moe_attention_workspace_bytes(int32_t T, int32_t heads, const moe_kv_cache *cache);

moe_status moe_tree_attention(const void *q, const int32_t *q_offsets, const int32_t *ctx_len, const uint32_t *mask,
                              const moe_attention_params *params, const moe_kv_cache *cache, void *out, float *lse,
                              void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Norms of the heads before the rotation: a row x of q or k becomes
 * x / sqrt(mean(x^2) + eps) * (w + offset), in fp32, rounded once after the
 * rotation.
 *   q_weight, k_weight  [head_dim], or [heads][head_dim] and [kv_heads]
 *             [head_dim] with per_head 1; dtype of q and k, 16-byte aligned;
 *             NULL: ones (offset is not read then).
 *   eps       positive and finite (moe_kv_append_q8: eps * head_dim too).
 *   offset    0, or 1 for models that keep the weights less 1; finite.
 */
typedef struct {
    const void *q_weight, *k_weight;
    float eps;
    float offset;
    int32_t per_head;
} moe_head_norm;

/* moe_kv_append with norms of queries and keys before the rotation. */
moe_status moe_kv_append_norm(const void *q, const void *k, const void *v, const float *rope, const int32_t *positions,
                              const int64_t *slots, const moe_append_params *params, const moe_head_norm *norm,
                              const moe_kv_cache *cache, void *q_out, void *workspace, size_t workspace_bytes,
                              moe_stream_t stream);

/*
 * A cache in 8 bits: a component is code * scale, the code an e4m3 number
 * (sign, 4 exponent and 3 fraction bits, largest 448, NaN 0x7f and 0xff).
 *   k, v        [n_pages][kv_heads][page_size][head_dim] e4m3, device,
 *               16-byte aligned.  head_dim: a multiple of 16, 16..256.
 *   k_scale, v_scale  [n_pages][kv_heads][page_size / block] fp32, device: one
 *               for each key head and `block` consecutive rows of a page.
 *               block: a divisor of page_size.
 *   dtype       of the queries, keys, values and results that are not in the
 *               cache: moe_dtype.
 * The rest as in moe_kv_cache.
 */
typedef struct {
    void *k;
    void *v;
    float *k_scale;
    float *v_scale;
    const int32_t *page_table;
    int32_t n_pages;
    int32_t page_size;
    int32_t block;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t n_requests;
    int32_t max_pages;
    int32_t dtype;
} moe_kv_cache_q8;

/*
 * moe_kv_append into a cache in 8 bits; norm may be NULL (no norms).  Keys
 * and values are quantised from their fp32 values, rounded to nearest even.
 * Of each block and key head that the call writes rows of, k and v apart, let
 * `most` be the largest finite magnitude among the components written:
 *   - need = the smallest power of two with most <= 448 need, 2^-64 at least;
 *   - a block whose first row the call writes begins anew: scale = need;
 *   - another keeps its scale if that is finite and at least need, else scale
 *     = need, and the codes of its other rows become the e4m3 numbers nearest
 *     to code * old / need (where the old scale is not positive and finite: 0).
 * So the rows of a block are to be written in order, from its first (with
 * block 1 in any order).  Rows past those that were written may be written
 * again (drafted tokens that were not kept); a block's scale does not shrink
 * before it begins anew.  Components that are not finite get the code NaN.
 *   slots     as for moe_kv_append, and tokens that write the same block must
 *             follow one another in the call (a request's tokens do): between
 *             two of them may lie none that writes another block, and up to
 *             255 that write nothing.  The rows and the scale of a block for
 *             which they do not are unspecified.
 */
moe_status moe_kv_append_q8(const void *q, const void *k, const void *v, const float *rope, const int32_t *positions,
                            const int64_t *slots, const moe_append_params *params, const moe_head_norm *norm,
                            const moe_kv_cache_q8 *cache, void *q_out, void *workspace, size_t workspace_bytes,
                            moe_stream_t stream);

/*
 * Reads T rows of a cache in 8 bits: out = code * scale, rounded once to
 * dtype (bf16 holds the product of a code and a power of two exactly).
 *   slots     [T] int64: page * page_size + row of the page, in any order, the
 *             same more than once too.  A negative one leaves its token's rows
 *             of k_out and v_out as they were; so does one past the cache,
 *             which raises MOE_FLAG_BAD_INDEX.
 *   k_out, v_out  [T][kv_heads][head_dim] dtype, distances between tokens and
 *             heads as for moe_kv_append, 16-byte aligned; one of them may be
 *             NULL.
 * The workspace as for moe_kv_append.
 */
typedef struct {
    int32_t T;
    int64_t k_tok, k_head;
    int64_t v_tok, v_head;
} moe_read_params;

moe_status moe_kv_read_q8(const int64_t *slots, const moe_read_params *params, const moe_kv_cache_q8 *cache, void *k_out,
                          void *v_out, void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_tree_attention over a cache in 8 bits: arguments, limits, masks, flags
 * and results as there, with q and out of the cache's dtype and its keys and
 * values code * scale.  Scales of positions that are seen are 0 to 2^120 (the
 * largest that an append begins a block with); those of values may count as
 * 2^-64 below that.  What lies in positions that a token does not see, their
 * scales too, has no influence on it.
 * Tensor cores (heads and pages as there): up to 64 rows a key head on average,
 * queries are taken exactly but for 2^-21 of the largest component of the rows
 * that are worked on together (up to 32 of a request and key head), and weights
 * times values' scales are off by up to 2^-11 + 2^-14 of themselves and 2^-28 of
 * the row's largest among 128 positions; the weights' sum is not.  With more
 * rows, weights are rounded to bf16 (2^-8 of each, their sum is not), and so are
 * values whose scale is no power of two.
 */
size_t moe_attention_q8_workspace_bytes(int32_t T, int32_t heads, const moe_kv_cache_q8 *cache);

moe_status moe_tree_attention_q8(const void *q, const int32_t *q_offsets, const int32_t *ctx_len, const uint32_t *mask,
                                 const moe_attention_params *params, const moe_kv_cache_q8 *cache, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_decode_layer for callers that cannot allocate device memory.  The
 * pages have no counterpart: this is a property of the library, not of the
 * method.  A plugin whose host engine owns all device memory, a runtime
 * that freezes allocation after start-up, or code without access to its
 * framework's allocator may have no way to provide a workspace.  This call
 * takes its scratch from one fixed array in the library's own device memory
 * (MOE_STATIC_SCRATCH_BYTES, held by every GPU that loads the library until
 * the process exits) and allocates nothing.  Inputs, routing buffers and
 * output are the caller's, exactly as for moe_decode_layer.
 *   - A batch whose workspace (moe_workspace_bytes) exceeds
 *     MOE_STATIC_SCRATCH_BYTES is rejected with MOE_ERR_WORKSPACE before
 *     anything is launched.
 *   - Every call looks up the array's device address on the current device
 *     (no allocation).  The first call on a device may load the library's
 *     device code, so make it before any stream capture.  After a reset of
 *     the device (cudaDeviceReset, or the primary context torn down and
 *     recreated) the next call finds the array again, zeroed.
 *   - All calls on a device share its array, which keeps the last call's
 *     contents; the counters at its front are cleared on `stream` at every
 *     call.  Calls that overlap on the GPU (for example on two streams) race
 *     with each other: serialise them.
 *   - Device flags raised by these calls accumulate in the array until
 *     moe_device_status_static() reads and clears them.
 */
#define MOE_STATIC_SCRATCH_BYTES (32u << 20)
moe_status moe_decode_layer_static(const void *hidden, const void *w_router, const float *router_bias,
                                   const void *w_gate, const void *w_up, const void *w_down,
                                   int32_t d_ff, const moe_route_params *params,
                                   const moe_routing *routing, void *out, moe_stream_t stream);

/*
 * moe_device_status for moe_decode_layer_static: synchronises `stream`,
 * returns the device flag word (MOE_FLAG_*) that calls of
 * moe_decode_layer_static raised on the current device since the last
 * read, and clears it.  Returns MOE_ERR_DEVICE_CHECK if any flag was set.
 * Allocates nothing.  (No counterpart on the pages.)
 */
moe_status moe_device_status_static(moe_stream_t stream, uint32_t *flags);

/*
 * Synchronises `stream`, returns the device flag word (MOE_FLAG_*) that the
 * calls on this workspace raised since the last read, and clears it.
 * Returns MOE_ERR_DEVICE_CHECK if any flag was set.
 */
moe_status moe_device_status(void *workspace, moe_stream_t stream, uint32_t *flags);

/*
 * Bound, in microseconds, of every wait inside the library's kernels: the
 * expert kernel's CTAs wait for one another (hidden states copied, h rows
 * written, y slices stored) and, with the early start, for the routing
 * kernel's published union.  A healthy layer's waits last microseconds.  A
 * wait that reaches the bound gives up: the kernel raises
 * MOE_FLAG_WAIT_TIMEOUT, every later wait in the same CTA returns at once,
 * the call's output is not valid, and the kernel still ends and leaves the
 * workspace ready for the next call.  Default 2,000,000 (two seconds);
 * 0 restores it.  The bound is counted in SM clock cycles at 2,000 per
 * microsecond (the clock runs at up to 2.07 GHz), so it lasts at least
 * about the given time.  Applies to calls launched afterwards, process
 * wide.  Short bounds are for tests of the failure path: a layer whose CTA
 * is delayed for longer than the bound (for example by a long kernel on
 * another stream occupying its SM) would fail with the flag.
 * (No counterpart on the pages.)
 */
moe_status moe_set_wait_timeout_us(uint32_t microseconds);

/*
 * Seeded synthetic tensor fill (for benchmarks and tests; not part of the
 * layer).  Writes elements start..start+n-1 of the counter-based stream:
 * SplitMix64 (Steele, Lea & Flood, OOPSLA 2014) output i for initial state
 * `seed`, its four 16-bit fields summed and centred (an Irwin-Hall sum),
 * times `scale` in fp32, rounded to bf16 (nearest even) when dtype is bf16.
 * dst must hold n elements of dtype.
 */
moe_status moe_synth_normal(void *dst, int32_t dtype, uint64_t n, uint64_t start, uint64_t seed,
                            float scale, moe_stream_t stream);

/* Human-readable name of a status, and the last error detail on this thread. */
const char *moe_status_string(moe_status status);
const char *moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* OEA_MOE_H */
