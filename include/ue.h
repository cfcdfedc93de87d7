/*
 * ue.h -- C ABI of the MI355X (gfx950) per-layer MoE expert-rebalancing
 * library (libue.so).
 *
 * The library implements the data-parallel hot path of an exact-load,
 * real-time expert balancer: count each expert's load from the post-gating
 * routing, plan replicas of hot experts onto spare slots of expert-parallel
 * ranks under a quota, expand logical expert ids to physical replica ids
 * with the stable dispatch permutation, copy master weights into replicas,
 * and sum replica gradients into the masters.
 *
 * Sources: the gitdiagram page "How dots-infra/ultraep works" (summary and
 * connection list: the framework registers expert pointers and passes
 * routing; the manager profiles loads, updates placement, syncs weights,
 * reroutes tokens and reduces gradients); the UltraEP news write-up
 * ("UltraEP ot Xiaohongshu: balansirovka MoE-ekspertov za 300 mks"), section
 * on how balancing in 300 microseconds works (quota-driven scheduler, every
 * microbatch and layer, right after gating; persistent tile streaming of
 * expert state); the UltraEP abstract, arXiv 2606.04101 ("exact-load,
 * real-time balancer").
 *
 * Conventions for every call:
 *  - Pointers named as device pointers must point to device memory of the
 *    current HIP device (e.g. torch CUDA tensors on ROCm). Host pointers are
 *    read before the call returns and not kept, unless stated.
 *  - `stream` is a hipStream_t passed as void*; NULL means the null stream.
 *    Every call is asynchronous and stream-ordered; results are valid once
 *    the stream reaches that point. No call synchronises with the host.
 *  - The return value is UE_OK (0) or a negative ue_status. Every argument
 *    is validated before anything is launched or written: a refused call
 *    leaves all outputs untouched. The reason is in ue_last_error().
 *  - A context is not thread-safe: one host thread at a time. Its routing
 *    calls (ue_load, ue_plan, ue_reroute, ue_rebalance) use the context's
 *    workspace and must not overlap one another in time on different
 *    streams. Calls of ue_moe_tokens have a workspace of their own and must
 *    not overlap one another, replays of captured ones included.
 *    ue_weight_sync, ue_grad_reduce, ue_gather_rows, ue_gate,
 *    ue_gate_backward, ue_quantize_rows, ue_matmul_i8 and the calls of the
 *    training step (ue_balance to ue_combine_backward_all) use no workspace but
 *    what they are given, and may run on another stream beside them (the next layer's
 *    rebalance beside this layer's sync), while kernel timing is off and
 *    the registered tables are not replaced meanwhile.
 *  - All shapes are int32; the number of assignments per layer, T*k, must
 *    stay below 2^30.
 *  - The workgroups of ue_reroute combine per-tile counts through bounded
 *    waits on each other (decoupled lookback); no other call waits across
 *    workgroups (ue_load and ue_rebalance count every tile on its own and
 *    scan the counts in the planner's launch). A wait that outlasts the
 *    context's wait limit (ue_set_wait_limit) gives up, and every kernel
 *    still runs to its end; the layer is then marked poisoned: bit 30
 *    (0x40000000, UE_POISONED) is set in that layer's `faults` word, the
 *    other bits keep their counts, and the layer's other outputs are
 *    unspecified.
 */
#ifndef UE_H
#define UE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ue_status {
    UE_OK = 0,
    UE_EINVAL = -1,       /* null pointer, bad alignment, bad value       */
    UE_ESHAPE = -2,       /* dimensions outside what the context allows   */
    UE_ENOMEM = -3,       /* device allocation failed                     */
    UE_EHIP = -4,         /* a HIP runtime call failed                    */
    UE_EUNSUPPORTED = -5, /* configuration outside what the kernels cover */
    UE_ESTATE = -6        /* call made in the wrong state (e.g. unregistered) */
} ue_status;

/* Shape of the simulated expert-parallel machine and the size limits of
 * one context.
 *   num_experts E      logical experts, 1..1024
 *   num_ranks R        expert-parallel ranks, divides E; N = E / R experts
 *                      live natively on each rank (expert e on rank e / N,
 *                      native slot e mod N)
 *   spare_per_rank S   empty replica slots per rank, 0..64; physical slot id
 *                      p = r*(N+S) + s, natives s < N, spares N <= s < N+S;
 *                      P = R*(N+S) <= 4096
 *   topk k             experts per token, 1..E
 *   max_tokens         largest T of any call (T*k < 2^30)
 *   max_layers         largest L (layers or microbatches) of any call
 *   plan_policy        rule of the planner (see ue_plan):
 *                      UE_PLAN_LEAST_LOADED (0), UE_PLAN_BEST_FIT (1),
 *                      UE_PLAN_BEST_FIT_COVER (2) or
 *                      UE_PLAN_BEST_FIT_ASCENDING (3)
 *   quota_mode         how the planner sets the quota (see ue_plan):
 *                      UE_QUOTA_FIXED (0) or UE_QUOTA_SEARCH (1)           */
typedef struct ue_config {
    int32_t num_experts;
    int32_t num_ranks;
    int32_t spare_per_rank;
    int32_t topk;
    int32_t max_tokens;
    int32_t max_layers;
    int32_t plan_policy;
    int32_t quota_mode;
} ue_config;

enum {
    UE_PLAN_LEAST_LOADED = 0,  /* every chunk to the least-loaded rank     */
    UE_PLAN_BEST_FIT = 1,      /* a chunk the least-loaded rank would not
                                  fill goes to the eligible rank with the
                                  smallest headroom that holds it          */
    UE_PLAN_BEST_FIT_COVER = 2, /* best fit, candidates in covering order:
                                  amounts one rank can take first, smallest
                                  first, then the rest, largest first      */
    UE_PLAN_BEST_FIT_ASCENDING = 3 /* best fit, candidates by their amount
                                  at Q0, smallest first                   */
};

enum {
    UE_QUOTA_FIXED = 0,        /* Q = ceil(sum(counts) / R)                 */
    UE_QUOTA_SEARCH = 1        /* the lowest of Q0 + j*ceil(Q0/256), j < 64,
                                  at which nothing is left over (else Q0)   */
};

/* Bit of a layer's invalid / faults word marking a wait that gave up. */
#define UE_POISONED 0x40000000

typedef struct ue_ctx ue_ctx;

/* Creates a context on the current HIP device and allocates its device
 * workspace once (per-tile scan state and counters, sized from the
 * limits). *out is set only on success. Errors: UE_EINVAL (null),
 * UE_EUNSUPPORTED (limits above), UE_ENOMEM, UE_EHIP. */
int ue_create(const ue_config *cfg, ue_ctx **out);

/* Frees the workspace and the context. Registered expert memory is the
 * caller's and is not freed. Waits for the device to finish pending work
 * of the context. NULL is accepted. */
void ue_destroy(ue_ctx *ctx);

/* Last error message of the context ("" if none); valid until the next
 * call on the context. With ctx NULL: the message of the calling thread's
 * last ue_rebalance_static call. */
const char *ue_last_error(const ue_ctx *ctx);

/* Short name of a status code. */
const char *ue_status_name(int status);

/* ---------------------------------------------------------------------
 * Placement block: one per layer, int32 words at fixed offsets.
 * ue_get_placement_layout() reports the offsets (in int32 words from the start
 * of a layer's block) and the block size. Fields:
 *   quota        Q = ceil(sum(counts) / R)
 *   exhausted    1 if overloaded ranks kept excess because no rank had a
 *                free spare slot and load < Q, else 0
 *   residual     sum over ranks of max(0, load_after - Q)
 *   n_rep        entries used in the replica table (masters included)
 *   rep_off[E+1] replica table offsets per expert (CSR)
 *   rep_slot[P]  physical slot of each replica; per expert the master
 *                (native slot) first, then replicas in creation order;
 *                entries >= n_rep hold -1
 *   rep_cap[P]   assignments routed to each replica (0 beyond n_rep)
 *   slot_expert[P] logical expert held by each slot, -1 for an unused spare
 *   slot_cap[P]  assignments routed to each slot (0 if unused)
 *   slot_off[P+1] exclusive prefix sum of slot_cap: where each slot's
 *                assignments start in the dispatch permutation
 *   load_before[R], load_after[R]  rank loads under the native placement
 *                and after the plan                                        */
typedef struct ue_placement_layout {
    int32_t words;          /* int32 words per layer block */
    int32_t quota, exhausted, residual, n_rep;
    int32_t rep_off, rep_slot, rep_cap;
    int32_t slot_expert, slot_cap, slot_off;
    int32_t load_before, load_after;
} ue_placement_layout;

int ue_get_placement_layout(const ue_ctx *ctx, ue_placement_layout *out);

/* Bytes of one layer's placement block (words * 4). 0 for a NULL ctx. */
size_t ue_placement_bytes(const ue_ctx *ctx);

/* ---------------------------------------------------------------------
 * Exact per-expert load ("Load computation"; the balancer is exact-load).
 *   routing  device, int32 [L, T, k], logical expert ids, flat assignment
 *            order a = t*k + j within a layer
 *   counts   device, int32 [L, E] out: counts[l][e] = #{a : routing = e}
 *   invalid  device, int32 [L] out, may be NULL: ids outside [0, E) per
 *            layer (such ids are not counted)
 * L in 1..max_layers, T in 0..max_tokens. */
int ue_load(ue_ctx *ctx, const int32_t *routing, int32_t L, int32_t T,
            int32_t *counts, int32_t *invalid, void *stream);

/* Quota replica plan ("Placement planning", the quota-driven scheduler),
 * per layer, from counts alone:
 *   Q = ceil(sum(counts)/R); experts of ranks whose load exceeds Q are
 *   visited heaviest first (count desc, id asc); each spills its rank's
 *   excess, chunk by chunk, into the lowest free spare slot of the
 *   least-loaded rank (ties: lowest id) that has a free spare slot and load
 *   < Q; chunk = min(source excess, expert remainder, destination
 *   headroom); with no such rank the plan stops (exhausted = 1).
 *   Under UE_PLAN_BEST_FIT, when the amount left (min of source excess and
 *   expert remainder) is below the least-loaded rank's headroom, it goes
 *   whole to the eligible rank with the smallest headroom >= the amount
 *   (ties: lowest id) instead.
 *   UE_PLAN_BEST_FIT_COVER places chunks as UE_PLAN_BEST_FIT does but
 *   visits the candidates in covering order, fixed at Q0: a candidate's
 *   amount at a quota is what its rank must shed below it that the rank's
 *   heavier experts (count desc, id asc) do not; H0 is the largest
 *   headroom Q0 - load among ranks with a spare slot; candidates whose
 *   amount at Q0 is at most H0 come first (amount asc, id asc), then the
 *   others (amount desc, id asc); each places its amount at the pass's
 *   quota. With one spare slot per rank every destination takes one
 *   chunk, and this order keeps the small pieces for the small amounts.
 *   UE_PLAN_BEST_FIT_ASCENDING is the same with every candidate in the
 *   first group: all amounts at Q0 ascending (ties: lowest id), so the
 *   large amounts too go smallest first and the largest, which needs the
 *   most pieces, is placed last, into what the others left.
 *   Under UE_QUOTA_SEARCH the plan above is made at the quotas
 *   Q0 + j*ceil(Q0/256), j = 0..63 (Q0 = ceil(sum(counts)/R)), in order,
 *   and the first that leaves nothing over is kept; with none, Q0 stands.
 *   The placement's quota field holds the quota used.
 *   counts     device, int32 [L, E] (e.g. from ue_load); every count >= 0
 *              and each layer's sum below 2^30 (ue_load's counts always
 *              are). A layer that breaks this is not planned: its block
 *              gets exhausted = -1 and an empty replica table (rep_off all
 *              0, n_rep 0), so every assignment of a later ue_reroute with
 *              it is a fault.
 *   placement  device, L blocks of ue_placement_bytes() bytes, out
 * Fully on the device; nothing returns to the host. */
int ue_plan(ue_ctx *ctx, const int32_t *counts, int32_t L, void *placement,
            void *stream);

/* Routing expansion and dispatch layout ("Routing expansion": physical
 * routing for token dispatch). For every assignment a of layer l with
 * logical expert e, j = number of earlier assignments of e in flat order;
 * the replica of e whose capacity prefix (master first) covers j gets it:
 *   phys        device, int32 [L, T, k] out: physical slot id
 *   rank_counts device, int32 [L, R] out: assignments per rank, counted
 *               from phys
 *   perm        device, int32 [L, T*k] out: perm[pos] = a, the stable sort
 *               of assignments by physical slot (pos = slot_off[p] + j -
 *               prefix)
 *   inv_perm    device, int32 [L, T*k] out, may be NULL: inv_perm[a] = pos
 *   faults      device, int32 [L] out, may be NULL: assignments that could
 *               not be placed (id outside [0, E), or beyond the plan's
 *               capacity for its expert); their phys and inv_perm are -1
 * The placement must come from ue_plan on the counts of this routing; with
 * faults > 0 perm is unspecified. */
int ue_reroute(ue_ctx *ctx, const int32_t *routing, const void *placement,
               int32_t L, int32_t T, int32_t *phys, int32_t *rank_counts,
               int32_t *perm, int32_t *inv_perm, int32_t *faults,
               void *stream);

/* One rebalance of L layers in one call: ue_load, ue_plan and ue_reroute
 * with the same arguments and results as those three calls in a row (every
 * output of each is an output here; invalid and inv_perm may be NULL). The
 * pages rebalance right after gating, on the critical path, for every
 * microbatch and layer; this entry point is that path as three launches
 * with no host work between them. The reroute reuses the per-tile expert
 * prefixes the load kernel publishes, so it reads the routing once more but
 * never waits on another workgroup; and since the plan is made from these
 * very counts, rank_counts and faults follow from it (the plan's loads
 * after, and the ids out of range) and the planner's launch writes them.
 * Arguments are validated before the first launch; a refusal leaves every
 * output untouched. */
int ue_rebalance(ue_ctx *ctx, const int32_t *routing, int32_t L, int32_t T,
                 int32_t *counts, int32_t *invalid, void *placement,
                 int32_t *phys, int32_t *rank_counts, int32_t *perm,
                 int32_t *inv_perm, int32_t *faults, void *stream);

/* Rank loads under an earlier plan: the periodic, historical-load
 * balancing that the UltraEP abstract (arXiv 2606.04101) and the news
 * write-up (section on the problem UltraEP solves) contrast with exact-load
 * balancing. Each layer's placement block (from ue_plan on earlier counts)
 * is applied to that layer's new counts: the plan keeps its replicas and
 * their proportions, so of expert e's n new assignments, with old
 * capacities c_1..c_m (master first, then replicas in table order) summing
 * to C, replica i takes floor(n * c_<=i / C) - floor(n * c_<i / C); an
 * expert the plan saw no tokens of (C = 0) stays whole on its master.
 *   placement   device, L blocks from ue_plan (on other counts)
 *   counts      device, int32 [L, E], the new counts (each >= 0, the sum of
 *               a layer below 2^30)
 *   rank_loads  device, int32 [L, R] out: assignments per rank
 * Exact integer arithmetic; the same covering rule as ue_reroute with the
 * capacities rescaled. Errors: UE_EINVAL (null or misaligned pointers),
 * UE_ESHAPE (L outside 1..max_layers). */
int ue_stale_loads(ue_ctx *ctx, const void *placement, const int32_t *counts,
                   int32_t L, int32_t *rank_loads, void *stream);

/* Polls one cross-workgroup wait of ue_reroute may take before it gives up
 * and marks its layer poisoned (see the conventions above); default
 * 4,194,304, far beyond any wait of a healthy device. 0 makes every wait
 * give up without polling, so every layer of more than one routing tile is
 * marked: a way to exercise the error path with every kernel still ending
 * normally. Applies to later calls on the context. */
int ue_set_wait_limit(ue_ctx *ctx, uint32_t polls);

/* ue_rebalance without a context and without allocating: for callers
 * that cannot allocate device memory where they rebalance (code under
 * stream capture, tight serving loops, harnesses that forbid allocation).
 * Same arguments, outputs and results as ue_rebalance, with the context
 * replaced by its configuration (validated as ue_create does: the same
 * UE_EUNSUPPORTED cases; L <= max_layers and T <= max_tokens).
 * Its scratch is one device array of UE_STATIC_SCRATCH_BYTES (16 MiB) in
 * the library, which every device the library runs on holds until the
 * process ends. A call needs, with tiles = max(1, ceil(T*k / 2048)) and
 * groups = ceil(tiles / 8), each term rounded up to 256 bytes:
 *   4 L groups E + 2 L (tiles + groups) E
 * bytes (the 58-layer dsv3 rebalance, E=256, T=65536, k=8: 10.5 MB). A call
 * needing more is refused with UE_ESHAPE before anything is launched.
 * Every scratch word a call reads it has written itself, so nothing is
 * cleared between calls (and the call may be captured in a graph). Calls
 * share the array: calls that overlap in time on one device race and give
 * wrong results; order them on one stream. The first call on a device
 * looks up the array's address there (hipGetSymbolAddress).
 * Calls no allocation routine. Error text: ue_last_error(NULL). */
#define UE_STATIC_SCRATCH_BYTES (16u << 20)
int ue_rebalance_static(const ue_config *cfg, const int32_t *routing,
                        int32_t L, int32_t T, int32_t *counts,
                        int32_t *invalid, void *placement, int32_t *phys,
                        int32_t *rank_counts, int32_t *perm,
                        int32_t *inv_perm, int32_t *faults, void *stream);

/* Kernel timing. With timing enabled, every call records a HIP event on its
 * stream before its first kernel and after each kernel it launches.
 * ue_kernel_times waits for the latest call's last event and writes the
 * duration in milliseconds of each of its kernels, in launch order, to
 * ms[0 .. *n-1] (at most max_n values; *n is the number that call launched; a
 * kernel that takes several launches, for more rows than the threads of one
 * reach, counts as one).
 * Off by default; enabling it costs one event per kernel. Errors:
 * UE_ESTATE if timing is off or no call has run since it was enabled. */
int ue_set_timing(ue_ctx *ctx, int enable);
int ue_kernel_times(ue_ctx *ctx, float *ms, int32_t max_n, int32_t *n);

/* ---------------------------------------------------------------------
 * Expert state ("registers expert pointers"). Stores device pointers to
 * n_experts master experts and n_buffers replica buffers, each made of
 * n_mats matrices; matrix m has mat_elems[m] elements in every expert and
 * buffer. Weights are bf16 (2 bytes per element), gradients fp32.
 *   mat_elems  host, int64 [n_mats]
 *   master_w   host array of device pointers [n_experts * n_mats], index
 *              e*n_mats + m; master_g likewise (float*)
 *   spare_w    host array of device pointers [n_buffers * n_mats];
 *              spare_g likewise
 * Every pointer must be 16-byte aligned. The memory stays the caller's;
 * the context keeps the pointers (copied to the device) until the next
 * registration or ue_destroy. n_mats in 1..16. Any of master_g/spare_g
 * may be NULL (then ue_grad_reduce is refused), any of master_w/spare_w
 * may be NULL (then ue_weight_sync is refused). */
int ue_register_experts(ue_ctx *ctx, int32_t n_experts, int32_t n_mats,
                        const int64_t *mat_elems, void *const *master_w,
                        float *const *master_g, int32_t n_buffers,
                        void *const *spare_w, float *const *spare_g);

/* Replica weight sync ("Replica weight sync": replicas receive the master
 * weights before expert compute). Replica table as device CSR:
 *   rep_off  device, int32 [n_experts + 1]
 *   rep_buf  device, int32 [rep_off[n_experts]]; for expert e the entries
 *            rep_off[e] .. rep_off[e+1]-1: the first stands for the master
 *            and is ignored, the others are replica buffer indices
 * Every matrix of every replica becomes a bitwise copy of its master's.
 * The master is read once per tile and written to all its replicas.
 * n_experts must not exceed the registered count; buffer indices must be
 * < n_buffers (entries outside are skipped). Replica buffers that the table
 * names must not alias masters or each other.
 * A placement block's rep_off and rep_slot fields (ue_plan) form such a
 * table when buffer p is registered for physical slot p (n_buffers = P):
 * its first entry per expert is the native slot, the others are spare
 * slots. Buffers of native slots are never named as replicas, so they may
 * be the masters themselves. The plan then drives the sync (and, before
 * backward, the restore: the same call with the saved plan) and the
 * gradient reduction without leaving the device. */
int ue_weight_sync(ue_ctx *ctx, const int32_t *rep_off, const int32_t *rep_buf,
                   int32_t n_experts, void *stream);

/* Replica gradient reduction ("Replica gradient reduction": replica
 * gradients are summed into master gradients during backward). Same CSR as
 * ue_weight_sync. Per element, with the running sum in binary64 and no
 * reassociation: g = master; g += replica_1; g += replica_2; ...; then
 * master = g rounded once to binary32 (nearest even). The fp32 gradient is
 * thus within one rounding of the exact sum (unless the binary64 partial
 * sums themselves round, which takes terms some 2^29 apart in magnitude),
 * also where replicas cancel the master. Replica gradients are left
 * unchanged. */
int ue_grad_reduce(ue_ctx *ctx, const int32_t *rep_off, const int32_t *rep_buf,
                   int32_t n_experts, void *stream);

/* Token dispatch into physical-expert order on one device: out[pos, :] =
 * x[perm[pos] div k, :], done source-major through the inverse
 * permutation (every token row is read once and written to its k
 * positions).
 *   x        device, bf16 [T, H], 16-byte aligned rows (H % 8 == 0)
 *   inv_perm device, int32 [T*k] (from ue_reroute, one layer)
 *   out      device, bf16 [T*k, H]
 * Positions outside [0, T*k) are skipped. */
int ue_gather_rows(ue_ctx *ctx, const void *x, const int32_t *inv_perm,
                   int32_t T, int32_t k, int32_t H, void *out, void *stream);

/* ---------------------------------------------------------------------
 * The expert layer around a rebalance: the router's choice, which makes the
 * routing the calls above take; products of 8-bit integers over the rows of
 * a dispatch; and the whole layer for a few tokens, where a rebalance does
 * not pay. Rows of a matrix argument are `ld` elements apart and contiguous
 * inside. */
enum {
    UE_F32 = 0,
    UE_BF16 = 1,
    UE_I8 = 2
};

enum {
    UE_SCORE_SOFTMAX = 0,      /* p = softmax(logits); ranked by the logit   */
    UE_SCORE_SIGMOID = 1       /* p = 1/(1+exp(-logit)); ranked by p + bias  */
};

/* Expert choice from router logits (E and k are the context's). Per token:
 *   ids      the k experts with the highest rank, best first, equal ranks
 *            lowest id first; an expert whose logit is -inf or NaN (or
 *            whose p + bias is) is never taken, and where fewer than k are
 *            left the remaining ids are -1 (ue_load counts such ids as
 *            invalid) and their weights 0
 *   weights  scale * p_j, or with renorm scale * p_j / sum over the chosen
 *            (sigmoid: that sum plus 1e-20)
 * A logit of +inf counts as the largest float in the softmax. A NaN among a
 * token's logits makes that token's weights NaN.
 *   logits   device, [T] rows of E, UE_F32 or UE_BF16, ld apart (ld >= E)
 *   bias     device, fp32 [E], added to the sigmoid's p for the ranking only;
 *            may be NULL; must be NULL with the softmax
 *   ids      device, int32 [T, k] out: a layer's routing for ue_load
 *   weights  device, fp32 [T, k] out
 * T in 0..max_tokens. Scores and sums are fp32: equal ranks are ranks equal in
 * fp32 (a sigmoid above 16.7 is 1). Errors: UE_EINVAL, UE_ESHAPE. */
int ue_gate(ue_ctx *ctx, const void *logits, int32_t type, int64_t ld,
            int32_t T, int32_t score, int32_t renorm, float scale,
            const float *bias, int32_t *ids, float *weights, void *stream);

/* Gradient of the logits from the gradient of ue_gate's weights, at the
 * choice `ids` (not differentiated; ids outside [0, E) take no part, and a
 * token's ids must be distinct). Every element of dlogits is written: 0
 * where nothing flows (an expert not chosen, except for the softmax without
 * renorm, whose denominator holds every logit).
 *   dweights  device, fp32 [T, k]
 *   dlogits   device, out, [T] rows of E of the logits' type, ld_out apart */
int ue_gate_backward(ue_ctx *ctx, const void *logits, int32_t type, int64_t ld,
                     int32_t T, int32_t score, int32_t renorm, float scale,
                     const int32_t *ids, const float *dweights, void *dlogits,
                     int64_t ld_out, void *stream);

/* Rows as 8-bit integers: with top = max |x| of a row, q = rint(x * (127 /
 * top)) (to even) and scale = top / 127; a row of zeros (or one so small
 * that 127 / top overflows) has q = 0 and scale 0. The factor 127 / top is
 * rounded to fp32, and so is its product with x: an x that lies half way
 * between two steps (top / 2, common in bf16) may go to either. A row that
 * holds an infinity or a NaN has q = 0 and scale NaN, so that its products are
 * NaN.
 *   x      device, [M] rows of K, UE_F32 or UE_BF16, ldx apart
 *   q      device, int8, out, 16-byte aligned rows ldq apart (ldq a multiple
 *          of 16, at least K rounded up to 16; bytes K .. that are set to 0)
 *   scale  device, fp32 [M] out
 * K in 1..65536. */
int ue_quantize_rows(ue_ctx *ctx, const void *x, int32_t type, int64_t ldx,
                     int32_t M, int32_t K, int8_t *q, int64_t ldq,
                     float *scale, void *stream);

/* Product of 8-bit integers with a scale per row and per channel:
 *   out[m, n] = a_scale[r] * w_scale[e, n] * sum_k a[r, k] * w[e, n, k]
 * The sums are exact. Row m uses row r of a: m, or with `index` row
 * index[m] / index_div (a dispatch permutation and its top-k: the gather of
 * tokens into dispatch order happens inside; an entry outside a's rows gives
 * a row of zeros). Rows are grouped by `offsets` (a placement block's
 * slot_off, or any prefix sums): rows offsets[g] .. offsets[g+1]-1 use matrix
 * e = expert_of[g] (slot_expert), or g without it; rows of a group whose e is
 * outside [0, n_mats), and rows no group holds, are left as they are. Groups
 * may be empty or of any length; entries are clamped to 0..M, and should not
 * decrease (rows two groups claim are undefined). Without offsets all
 * rows use matrix 0. With `gated`, w has 2 N channels, gate then up, and
 *   out[m, n] = silu(gate) * up,  silu(v) = v / (1 + exp(-v)).
 *   a        device, int8, 16-byte aligned rows, lda a multiple of 16
 *   w        device, int8, likewise; matrices w_stride apart (multiple of 16)
 *   w_scale  device, fp32, matrices ws_stride apart
 * For a and w the bytes of a row up to K rounded up to 16 must be readable.
 * out is UE_BF16 or UE_F32, ldo >= N. K in 1..65536; one matrix of w is below
 * 4 GiB and lda below 16 MiB; rows of out times channels are limited by a
 * launch of fewer than 2^32 threads (UE_ESHAPE): 512 for a tile of 256 x 256
 * results, 256 for a begun tile of 32 x 64 where groups are that short. */
typedef struct ue_i8_product {
    const int8_t *a;
    const float *a_scale;
    const int8_t *w;
    const float *w_scale;
    const int32_t *offsets;     /* int32 [groups + 1] or NULL */
    const int32_t *expert_of;   /* int32 [groups] or NULL     */
    const int32_t *index;       /* int32 [M] or NULL          */
    void *out;
    int64_t lda, ldw, w_stride, ws_stride, ldo;
    int32_t a_rows, n_mats, groups, index_div;
    int32_t M, N, K;
    int32_t gated, out_type;
} ue_i8_product;

int ue_matmul_i8(ue_ctx *ctx, const ue_i8_product *p, void *stream);

/* The layer of ue_moe_tokens: the context's E experts with their router.
 *   router     device, bf16 [E, hidden]
 *   gate_up    device, [E] matrices [2 inter, hidden] (gate rows, then up
 *              rows), gate_up_stride elements apart
 *   down       device, [E] matrices [hidden, inter], down_stride apart
 *   weight_type  UE_BF16, or UE_I8 with gate_up_scale fp32 [E, 2 inter] and
 *              down_scale fp32 [E, hidden] (the weights of ue_matmul_i8)
 *   bias, score, renorm, scale   as in ue_gate
 * All matrices 16-byte aligned; hidden and inter multiples of 8 (bf16) or 16
 * (int8), strides likewise, an expert's gate_up below 4 GiB. The memory stays
 * the caller's; the context keeps the pointers until the next registration or
 * ue_destroy. The call waits for the device (it cannot be captured) and
 * allocates a workspace for min(max_tokens, UE_MOE_MAX_TOKENS) tokens, unless
 * an earlier layer's is large enough. Workspaces live until ue_destroy: a
 * captured graph of ue_moe_tokens keeps working after further registrations,
 * with the layer it was captured with, as long as the caller keeps that
 * layer's memory (and replays do not overlap other calls of ue_moe_tokens). */
#define UE_MOE_MAX_TOKENS 64
typedef struct ue_layer {
    const void *router;
    const float *bias;
    const void *gate_up, *down;
    const float *gate_up_scale, *down_scale;
    int64_t gate_up_stride, down_stride;
    int32_t hidden, inter, weight_type;
    int32_t score, renorm;
    float scale;
} ue_layer;

int ue_register_layer(ue_ctx *ctx, const ue_layer *layer);

/* A mixture-of-experts layer for a few tokens (the decode step of a served
 * model), from the registered layer:
 *   logits = x router^T;  (ids, weights) = ue_gate(logits)
 *   out_t = sum_j weights_tj (silu(x_t G^T) * (x_t U^T)) D^T
 * over the matrices of expert ids_tj; ids of -1 add nothing. Sums are fp32; the
 * hidden activations silu() * () go from the first product to the second as
 * a sum of two bf16 numbers, 16 bits of them; out is rounded once. The result
 * does not depend on timing (no atomics on values).
 *   x        device, bf16 [T] rows of hidden, 16-byte aligned, ldx apart
 *            (a multiple of 8, at most 2^24)
 *   out      device, bf16, ldo apart
 *   ids      device, int32 [T, k] out: the routing, as ue_load takes it
 *   weights  device, fp32 [T, k] out
 * T in 0..min(max_tokens, UE_MOE_MAX_TOKENS). UE_ESTATE without a registered
 * layer. Uses the context's workspace. */
int ue_moe_tokens(ue_ctx *ctx, const void *x, int64_t ldx, int32_t T,
                  void *out, int64_t ldo, int32_t *ids, float *weights,
                  void *stream);

/* ---------------------------------------------------------------------
 * The training step of the expert layer: the loss that keeps the routing
 * even, activations kept in 8 bits for the backward pass, the gradients of the
 * slots' matrices (which ue_grad_reduce then sums into the masters'), and the
 * sum of the experts' rows back to their tokens. None of these calls uses the
 * context's workspace: they may run beside any other call on another stream,
 * two calls that are given the same `workspace` excepted. */

/* Balance loss of packed sequences (E and k are the context's). With p the
 * softmax of a token's logits, or its sigmoids over their sum plus 1e-20, and
 * for sequence s of n tokens:
 *   counts[s, e] = number of its assignments to e (ids outside [0, E) are none)
 *   prob[s, e]   = (1 / n) sum_t p[t, e]
 *   loss[s]      = (E / (k n)) sum_e counts[s, e] prob[s, e]
 * which is 1 where the choice is even. An empty sequence has 0 everywhere. An
 * expert whose logit is -inf has p = 0, a token with no other has p = 0
 * everywhere; +inf counts as the largest float in the softmax; a NaN among a
 * token's logits makes its sequence's prob and loss NaN.
 *   logits   device, [T] rows of E, UE_F32 or UE_BF16, ld apart (ld >= E)
 *   ids      device, int32 [T, k] (from ue_gate)
 *   offsets  device, int32 [n_seq + 1]: sequence s is tokens offsets[s] ..
 *            offsets[s + 1] - 1; NULL: one sequence of all T tokens (n_seq 1).
 *            Entries are clamped to 0..T and must not decrease (results are
 *            undefined if they do). Tokens no sequence holds (padding) take no
 *            part.
 *   counts   device, int32 [n_seq, E] out;  prob  device, fp32 [n_seq, E] out
 *   loss     device, fp32 [n_seq] out
 *   workspace  device, 16-byte aligned, ue_balance_workspace(ctx, T, n_seq)
 *            bytes, overwritten; may be NULL where that is 0 (few tokens). Calls
 *            given the same one must not overlap, replays of captured ones
 *            included.
 * T in 0..max_tokens, n_seq in 0..2^20. Sums are fp32 in a fixed order (no
 * atomics on values): results repeat bit for bit. */
size_t ue_balance_workspace(const ue_ctx *ctx, int32_t T, int32_t n_seq);
int ue_balance(ue_ctx *ctx, const void *logits, int32_t type, int64_t ld,
               int32_t T, int32_t score, const int32_t *ids,
               const int32_t *offsets, int32_t n_seq, int32_t *counts,
               float *prob, float *loss, void *workspace, void *stream);

/* Gradient of the logits from that of the losses (counts are constants):
 *   d[t, e] = dloss[s] (E / (k n^2)) p_e (counts[s, e] - sum_j p_j counts[s, j])
 * times 1 - sigmoid(logit) for the sigmoid.
 *   counts   device, int32 [n_seq, E], from ue_balance (or summed over several
 *            devices that share the batch, with dloss scaled to match)
 *   dloss    device, fp32 [n_seq]
 *   dlogits  device, of the logits' type, [T] rows of E, ld_out apart: with
 *            `accumulate` the gradient is added to it (in fp32, rounded once;
 *            the gradient ue_gate_backward wrote, say) and rows of tokens no
 *            sequence holds stay as they are; else every element is written,
 *            0 in those rows. May be the logits' own memory. */
int ue_balance_backward(ue_ctx *ctx, const void *logits, int32_t type,
                        int64_t ld, int32_t T, int32_t score,
                        const int32_t *offsets, int32_t n_seq,
                        const int32_t *counts, const float *dloss,
                        void *dlogits, int64_t ld_out, int32_t accumulate,
                        void *stream);

/* Packed rows: 8 bits per element and one power of two per row and 32 columns
 * (a block; the last one of a row may be shorter). With top the block's largest
 * magnitude, e the smallest exponent from -126 with top <= 127 * 2^e:
 *   q = rint(x / 2^e) (to even),  scale = e + 127 as a byte
 * so |x - q 2^e| <= 2^(e-1), every quotient is exact, and q 2^e is a bf16
 * number. e is at most 121, so that q 2^e is finite: of larger magnitudes than
 * 127 * 2^121 (3.376e38) q is +-127, less than a step away. A block of zeros has scale 1. A block that holds an infinity or a NaN
 * has q = 0 and scale 255 and stands for NaNs.
 *   x      device, [M] rows of K, UE_F32 or UE_BF16, ldx apart
 *   q      device, int8, 16-byte aligned rows ldq apart (a multiple of 16, at
 *          least K rounded up to 32; bytes K .. that are set to 0)
 *   scale  device, bytes, rows of ceil(K / 32), lds apart
 * K in 1..2^20. ue_unpack_rows writes the values q 2^e stands for. */
#define UE_PACK_BLOCK 32
int ue_pack_rows(ue_ctx *ctx, const void *x, int32_t type, int64_t ldx,
                 int32_t M, int32_t K, int8_t *q, int64_t ldq, uint8_t *scale,
                 int64_t lds, void *stream);
int ue_unpack_rows(ue_ctx *ctx, const int8_t *q, int64_t ldq,
                   const uint8_t *scale, int64_t lds, int32_t M, int32_t K,
                   void *x, int32_t type, int64_t ldx, void *stream);

/* Gated activation that keeps its inputs in 8 bits, and its backward pass from
 * what was kept:
 *   h = silu(gate) up,  silu(v) = v / (1 + exp(-v))
 *   gu     device, [M] rows of 2 I: gate, then up; UE_F32 or UE_BF16, ldgu
 *          apart
 *   h      device, out, of the same type, [M] rows of I, ldh apart
 *   q, scale  out, or both NULL (nothing is kept): gate and up as packed rows
 *          side by side, each half padded to whole blocks: with P = I rounded up
 *          to 32, q has gate in bytes 0 .. I-1 and up in P .. P+I-1 of a row of
 *          2 P (ldq >= 2 P), scale P / 32 bytes for each (lds >= P / 16)
 * Backward, with gate and up the values that q and scale stand for and s =
 * 1 / (1 + exp(-gate)):
 *   dgate = dh up s (1 + gate (1 - s)),  dup = dh silu(gate)
 *   dh     device, [M] rows of I, UE_F32 or UE_BF16, lddh apart
 *   dgu    device, out, of the same type, [M] rows of 2 I, lddgu apart
 *   h      device, out, of the same type, ldh apart, or NULL: silu(gate) up again
 *          (the rows that the second product's weight gradient takes)
 * I in 1..2^19. dgu must not overlap dh, nor h gu. */
int ue_gated(ue_ctx *ctx, const void *gu, int32_t type, int64_t ldgu, int32_t M,
             int32_t I, void *h, int64_t ldh, int8_t *q, int64_t ldq,
             uint8_t *scale, int64_t lds, void *stream);
int ue_gated_backward(ue_ctx *ctx, const int8_t *q, int64_t ldq,
                      const uint8_t *scale, int64_t lds, const void *dh,
                      int32_t type, int64_t lddh, int32_t M, int32_t I,
                      void *dgu, int64_t lddgu, void *h, int64_t ldh,
                      void *stream);

/* Gradients of the matrices of row groups (a plan's slots):
 *   out[g, n, k] (+)= sum over the rows m of group g of dy[m, n] x[r(m), k]
 * Rows are grouped by `offsets` as in ue_matmul_i8 (entries clamped to 0..M, and
 * should not decrease); without offsets one group holds all rows. r(m) is m, or
 * with `index` index[m] / index_div (a dispatch permutation and its top-k); an
 * entry outside x's rows counts as a row of zeros. Sums are fp32 in a fixed
 * order: results repeat bit for bit.
 *   dy       device, bf16, [M] rows of N, lddy apart
 *   x        device, [x_rows] rows of K, ldx apart: bf16, or with x_scale packed
 *            rows (ue_pack_rows: int8, ldx a multiple of 16, 16-byte aligned)
 *   x_scale  device, bytes, lds apart, or NULL (x is bf16)
 *   out      device, fp32, `groups` matrices of N rows of K, rows ldo apart,
 *            matrices out_stride apart. With `accumulate` the sums are added to
 *            what out holds, else every element is written (0 for an empty
 *            group).
 *   workspace  device, 16-byte aligned, of ue_weight_grad_workspace(ctx, p)
 *            bytes (0 for many shapes), or NULL: few matrices of many rows are
 *            then not split over the device. Calls given the same one must not
 *            overlap.
 * M in 0..2^30, N and K in 0..2^20; rows of dy and x are at most 2^24 apart, and
 * one matrix of out is below 4 GiB. Of packed x, a row's bytes up to K rounded up
 * to 16 must be readable. */
typedef struct ue_weight_grad_product {
    const void *dy;
    const void *x;
    const uint8_t *x_scale;
    const int32_t *offsets;     /* int32 [groups + 1] or NULL */
    const int32_t *index;       /* int32 [M] or NULL          */
    float *out;
    void *workspace;
    int64_t lddy, ldx, lds, ldo, out_stride;
    int32_t x_rows, groups, index_div;
    int32_t M, N, K;
    int32_t accumulate;
} ue_weight_grad_product;

size_t ue_weight_grad_workspace(const ue_ctx *ctx,
                                const ue_weight_grad_product *p);
int ue_weight_grad(ue_ctx *ctx, const ue_weight_grad_product *p, void *stream);

/* Sum of the experts' rows back to their tokens (k is the context's):
 *   out[t] = add[t] + sum_j weights[t, j] y[inv_perm[t, j]]
 * in fp32, j in order, rounded once. Entries of inv_perm outside [0, rows) (an
 * assignment that found no place: -1) add nothing. Without weights they are 1:
 * the gradient of ue_gather_rows.
 *   y         device, [rows] rows of H, UE_F32 or UE_BF16, ldy apart (dispatch
 *             order)
 *   inv_perm  device, int32 [T, k];  weights  device, fp32 [T, k] or NULL
 *   add       device, of y's type, ldadd apart, or NULL (the shared expert's
 *             output, the residual)
 *   out       device, of y's type, [T] rows of H, ldo apart; may be add itself
 * Backward:
 *   dy[inv_perm[t, j]] = weights[t, j] dout[t]  (rows no assignment names are
 *                        left as they are; a row named twice is undefined)
 *   dweights[t, j] = sum_h dout[t, h] y[inv_perm[t, j], h], fp32, in a fixed
 *                    order; 0 where the entry is outside [0, rows)
 * dy or dweights (and then y) may be NULL. T in 0..max_tokens, H in 1..2^20. */
int ue_combine(ue_ctx *ctx, const void *y, int32_t type, int64_t ldy,
               int32_t rows, const int32_t *inv_perm, const float *weights,
               const void *add, int64_t ldadd, int32_t T, int32_t H, void *out,
               int64_t ldo, void *stream);
int ue_combine_backward(ue_ctx *ctx, const void *dout, int32_t type,
                        int64_t lddout, const int32_t *inv_perm,
                        const float *weights, const void *y, int64_t ldy,
                        int32_t rows, int32_t T, int32_t H, void *dy,
                        int64_t lddy, float *dweights, void *stream);
/* The same with the whole gradient: rows of dy that no assignment names are
 * written with zeros. dy may be NULL only if rows is 0.
 *   workspace  device, 16-byte aligned, ue_combine_backward_workspace(ctx, T,
 *              rows) bytes, overwritten; may be NULL where that is 0 (few
 *              assignments). Calls given the same one must not overlap, replays
 *              of captured ones included. */
size_t ue_combine_backward_workspace(const ue_ctx *ctx, int32_t T, int32_t rows);
int ue_combine_backward_all(ue_ctx *ctx, const void *dout, int32_t type,
                            int64_t lddout, const int32_t *inv_perm,
                            const float *weights, const void *y, int64_t ldy,
                            int32_t rows, int32_t T, int32_t H, void *dy,
                            int64_t lddy, float *dweights, void *workspace,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* UE_H */
