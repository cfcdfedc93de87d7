// C ABI of the expert layer's training step: the balance loss, packed rows and
// the gated activation on them, the gradients of the slots' matrices, the sum
// of the experts' rows. As in the other entry points every host-visible
// argument is checked before anything is launched or written.
#include "ue_train.h"

namespace {

using ue::aligned;
using ue::fail;
using ue::hip_fail;
using ue::tbegin;
using ue::tmark;

typedef long long ll;

constexpr int kMaxCols = 1 << 20;
constexpr int kMaxGroups = (1 << 20) - 1;

bool float_type(int t) { return t == UE_F32 || t == UE_BF16; }
size_t type_bytes(int t) { return t == UE_F32 ? 4 : 2; }

bool rows_aligned(const void *p, int64_t ld, size_t esize, size_t bytes) {
    return aligned(p, bytes) && static_cast<size_t>(ld) * esize % bytes == 0;
}
int blocks_of(int K) { return (K + UE_PACK_BLOCK - 1) / UE_PACK_BLOCK; }

int done(ue_ctx *c, hipError_t he, hipStream_t s, const char *what) {
    tmark(c, s);
    return he == hipSuccess ? UE_OK : hip_fail(c, he, what);
}

int check_balance(ue_ctx *c, const char *what, const void *logits, int type,
                  int64_t ld, int T, int score, const int32_t *offsets, int n_seq) {
    if (!float_type(type))
        return fail(c, UE_EINVAL, "%s: logits must be UE_F32 or UE_BF16", what);
    if (score != UE_SCORE_SOFTMAX && score != UE_SCORE_SIGMOID)
        return fail(c, UE_EINVAL, "%s: unknown score %d", what, score);
    if (T < 0 || T > c->cfg.max_tokens)
        return fail(c, UE_ESHAPE, "%s: T=%d outside 0..%d", what, T, c->cfg.max_tokens);
    if (n_seq < 0 || n_seq > (1 << 20) || (!offsets && n_seq != 1))
        return fail(c, UE_ESHAPE, "%s: n_seq=%d%s", what, n_seq,
                    offsets ? " outside 0..2^20" : " without offsets, 1 wanted");
    if (ld < c->E)
        return fail(c, UE_ESHAPE, "%s: rows of %d logits, %lld apart", what, c->E,
                    static_cast<ll>(ld));
    if (T > 0 && !logits) return fail(c, UE_EINVAL, "%s: null logits", what);
    if (!aligned(logits, type_bytes(type)) || !aligned(offsets, 4))
        return fail(c, UE_EINVAL, "%s: unaligned logits or offsets", what);
    return UE_OK;
}

// Packed rows of `cols` columns (each half of them, if gated).
int check_packed(ue_ctx *c, const char *what, const int8_t *q, int64_t ldq,
                 const uint8_t *scale, int64_t lds, int M, int64_t bytes, int64_t blocks) {
    if (ldq < bytes || ldq % 16 || lds < blocks)
        return fail(c, UE_ESHAPE, "%s: ldq=%lld lds=%lld, rows of %lld bytes and %lld scales",
                    what, static_cast<ll>(ldq), static_cast<ll>(lds), static_cast<ll>(bytes),
                    static_cast<ll>(blocks));
    if (M > 0 && (!q || !scale)) return fail(c, UE_EINVAL, "%s: null packed rows", what);
    if (!aligned(q, 16)) return fail(c, UE_EINVAL, "%s: q must be 16-byte aligned", what);
    return UE_OK;
}

int check_rows(ue_ctx *c, const char *what, const char *name, const void *p, int type,
               int64_t ld, int64_t rows, int64_t cols) {
    if (!float_type(type))
        return fail(c, UE_EINVAL, "%s: rows must be UE_F32 or UE_BF16", what);
    if (ld < cols)
        return fail(c, UE_ESHAPE, "%s: rows of %lld in %s, %lld apart", what,
                    static_cast<ll>(cols), name, static_cast<ll>(ld));
    if (rows > 0 && !p) return fail(c, UE_EINVAL, "%s: null %s", what, name);
    if (!aligned(p, type_bytes(type)))
        return fail(c, UE_EINVAL, "%s: %s not aligned to its type", what, name);
    return UE_OK;
}

int check_wgrad(ue_ctx *c, const ue_weight_grad_product *p) {
    const char *what = "ue_weight_grad";
    if (!p) return fail(c, UE_EINVAL, "%s: null product", what);
    if (p->M < 0 || p->M > (1 << 30) || p->N < 0 || p->K < 0 || p->N > kMaxCols ||
        p->K > kMaxCols || p->x_rows < 0)
        return fail(c, UE_ESHAPE, "%s: M=%d N=%d K=%d x_rows=%d", what, p->M, p->N, p->K,
                    p->x_rows);
    if (p->offsets ? p->groups < 0 || p->groups > kMaxGroups : p->groups != 1)
        return fail(c, UE_ESHAPE, "%s: groups=%d, %s", what, p->groups,
                    p->offsets ? "at most 2^20 - 1" : "1 without offsets");
    const int64_t x_bytes = p->x_scale ? (static_cast<int64_t>(p->K) + 15) / 16 * 16 : p->K;
    if (p->lddy < p->N || p->ldx < x_bytes || (p->x_scale && p->ldx % 16) ||
        (p->x_scale && p->lds < blocks_of(p->K)) || p->ldo < p->K)
        return fail(c, UE_ESHAPE, "%s: lddy=%lld ldx=%lld lds=%lld ldo=%lld", what,
                    static_cast<ll>(p->lddy), static_cast<ll>(p->ldx),
                    static_cast<ll>(p->lds), static_cast<ll>(p->ldo));
    // (the kernels address 64 rows of dy and a matrix of out with 32 bits)
    if (p->lddy > (1 << 24) || p->ldx > (1 << 24) || p->lds > (1 << 24) ||
        (p->N > 0 && p->ldo > 0x3FFFFFFFll / p->N))
        return fail(c, UE_ESHAPE, "%s: a matrix of 4 GiB, or rows 2^24 apart", what);
    if (p->groups > 1 &&
        p->out_stride < (p->N > 0 ? (static_cast<int64_t>(p->N) - 1) * p->ldo + p->K : 0))
        return fail(c, UE_ESHAPE, "%s: out_stride=%lld, matrices overlap", what,
                    static_cast<ll>(p->out_stride));
    if (p->index ? p->index_div < 1 : p->x_rows < p->M)
        return fail(c, UE_ESHAPE, "%s: M=%d rows from x_rows=%d, index_div=%d", what, p->M,
                    p->x_rows, p->index_div);
    if (p->M > 0 && p->x_rows == 0) return fail(c, UE_ESHAPE, "%s: no rows of x", what);
    return UE_OK;
}

}  // namespace

extern "C" {

size_t ue_balance_workspace(const ue_ctx *ctx, int32_t T, int32_t n_seq) {
    if (!ctx || T < 0 || n_seq < 0) return 0;
    return static_cast<size_t>(ue::balance_slots(T, n_seq, ctx->E, ctx->num_cu)) *
           ((ctx->E + 3) / 4 * 4) * 8;
}

int ue_balance(ue_ctx *ctx, const void *logits, int32_t type, int64_t ld, int32_t T,
               int32_t score, const int32_t *ids, const int32_t *offsets, int32_t n_seq,
               int32_t *counts, float *prob, float *loss, void *workspace, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (int rc = check_balance(ctx, "ue_balance", logits, type, ld, T, score, offsets, n_seq))
        return rc;
    const int64_t slots = ue::balance_slots(T, n_seq, ctx->E, ctx->num_cu);
    if ((T > 0 && !ids) || (n_seq > 0 && (!counts || !prob || !loss)) ||
        (n_seq > 0 && slots > 0 && !workspace))
        return fail(ctx, UE_EINVAL, "ue_balance: null argument");
    if (!aligned(ids, 4) || !aligned(counts, 4) || !aligned(prob, 4) || !aligned(loss, 4) ||
        !aligned(workspace, 16))
        return fail(ctx, UE_EINVAL, "ue_balance: unaligned argument");
    ue::BalanceArgs g{};
    g.logits = logits;
    g.ld = ld;
    g.bf16 = type == UE_BF16;
    g.sigmoid = score == UE_SCORE_SIGMOID;
    g.E = ctx->E;
    g.k = ctx->k;
    g.T = T;
    g.n_seq = n_seq;
    g.ids = ids;
    g.offsets = offsets;
    g.counts = counts;
    g.prob = prob;
    g.loss = loss;
    if (slots > 0) {
        g.part = static_cast<float *>(workspace);
        g.part_n = reinterpret_cast<int32_t *>(g.part + slots * ((ctx->E + 3) / 4 * 4));
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_balance(*ctx, g, s), s, "k_balance launch");
}

int ue_balance_backward(ue_ctx *ctx, const void *logits, int32_t type, int64_t ld, int32_t T,
                        int32_t score, const int32_t *offsets, int32_t n_seq,
                        const int32_t *counts, const float *dloss, void *dlogits,
                        int64_t ld_out, int32_t accumulate, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (int rc = check_balance(ctx, "ue_balance_backward", logits, type, ld, T, score, offsets,
                               n_seq))
        return rc;
    if (ld_out < ctx->E)
        return fail(ctx, UE_ESHAPE, "ue_balance_backward: gradients %lld apart",
                    static_cast<ll>(ld_out));
    if ((T > 0 && !dlogits) || (n_seq > 0 && (!counts || !dloss)))
        return fail(ctx, UE_EINVAL, "ue_balance_backward: null argument");
    if (!aligned(counts, 4) || !aligned(dloss, 4) || !aligned(dlogits, type_bytes(type)))
        return fail(ctx, UE_EINVAL, "ue_balance_backward: unaligned argument");
    ue::BalanceBackArgs g{};
    g.logits = logits;
    g.ld = ld;
    g.bf16 = type == UE_BF16;
    g.sigmoid = score == UE_SCORE_SIGMOID;
    g.accumulate = accumulate != 0;
    g.E = ctx->E;
    g.k = ctx->k;
    g.T = T;
    g.n_seq = n_seq;
    g.offsets = offsets;
    g.counts = counts;
    g.dloss = dloss;
    g.dlogits = dlogits;
    g.ld_out = ld_out;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_balance_backward(*ctx, g, s), s, "k_balance_backward launch");
}

int ue_pack_rows(ue_ctx *ctx, const void *x, int32_t type, int64_t ldx, int32_t M, int32_t K,
                 int8_t *q, int64_t ldq, uint8_t *scale, int64_t lds, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (M < 0 || K < 1 || K > kMaxCols)
        return fail(ctx, UE_ESHAPE, "ue_pack_rows: M=%d K=%d", M, K);
    if (int rc = check_rows(ctx, "ue_pack_rows", "x", x, type, ldx, M, K)) return rc;
    const int nb = blocks_of(K);
    if (int rc = check_packed(ctx, "ue_pack_rows", q, ldq, scale, lds, M,
                              int64_t(nb) * UE_PACK_BLOCK, nb))
        return rc;
    ue::PackArgs g{};
    g.x = x;
    g.ldx = ldx;
    g.bf16 = type == UE_BF16;
    g.M = M;
    g.K = K;
    g.q = q;
    g.ldq = ldq;
    g.scale = scale;
    g.lds = lds;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_pack(*ctx, g, s), s, "k_pack launch");
}

int ue_unpack_rows(ue_ctx *ctx, const int8_t *q, int64_t ldq, const uint8_t *scale,
                   int64_t lds, int32_t M, int32_t K, void *x, int32_t type, int64_t ldx,
                   void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (M < 0 || K < 1 || K > kMaxCols)
        return fail(ctx, UE_ESHAPE, "ue_unpack_rows: M=%d K=%d", M, K);
    if (int rc = check_rows(ctx, "ue_unpack_rows", "x", x, type, ldx, M, K)) return rc;
    const int nb = blocks_of(K);
    if (int rc = check_packed(ctx, "ue_unpack_rows", q, ldq, scale, lds, M,
                              int64_t(nb) * UE_PACK_BLOCK, nb))
        return rc;
    ue::PackArgs g{};
    g.out = x;
    g.ldx = ldx;
    g.bf16 = type == UE_BF16;
    g.M = M;
    g.K = K;
    g.q_in = q;
    g.ldq = ldq;
    g.scale_in = scale;
    g.lds = lds;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_unpack(*ctx, g, s), s, "k_unpack launch");
}

int ue_gated(ue_ctx *ctx, const void *gu, int32_t type, int64_t ldgu, int32_t M, int32_t I,
             void *h, int64_t ldh, int8_t *q, int64_t ldq, uint8_t *scale, int64_t lds,
             void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (M < 0 || I < 1 || I > kMaxCols / 2)
        return fail(ctx, UE_ESHAPE, "ue_gated: M=%d I=%d", M, I);
    if (int rc = check_rows(ctx, "ue_gated", "gu", gu, type, ldgu, M, 2 * int64_t(I))) return rc;
    if (int rc = check_rows(ctx, "ue_gated", "h", h, type, ldh, M, I)) return rc;
    if (!q != !scale) return fail(ctx, UE_EINVAL, "ue_gated: q and scale belong together");
    const int64_t nb = blocks_of(I);
    if (q)
        if (int rc = check_packed(ctx, "ue_gated", q, ldq, scale, lds, M,
                                  2 * nb * UE_PACK_BLOCK, 2 * nb))
            return rc;
    ue::GatedArgs g{};
    g.gu = gu;
    g.ldin = ldgu;
    g.bf16 = type == UE_BF16;
    g.M = M;
    g.I = I;
    g.h = h;
    g.ldh = ldh;
    g.q = q;
    g.ldq = ldq;
    g.scale = scale;
    g.lds = lds;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_gated(*ctx, g, s), s, "k_gated launch");
}

int ue_gated_backward(ue_ctx *ctx, const int8_t *q, int64_t ldq, const uint8_t *scale,
                      int64_t lds, const void *dh, int32_t type, int64_t lddh, int32_t M,
                      int32_t I, void *dgu, int64_t lddgu, void *h, int64_t ldh, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    const char *what = "ue_gated_backward";
    if (M < 0 || I < 1 || I > kMaxCols / 2)
        return fail(ctx, UE_ESHAPE, "%s: M=%d I=%d", what, M, I);
    if (int rc = check_rows(ctx, what, "dh", dh, type, lddh, M, I)) return rc;
    if (int rc = check_rows(ctx, what, "dgu", dgu, type, lddgu, M, 2 * int64_t(I))) return rc;
    if (h)
        if (int rc = check_rows(ctx, what, "h", h, type, ldh, M, I)) return rc;
    const int64_t nb = blocks_of(I);
    if (int rc = check_packed(ctx, what, q, ldq, scale, lds, M, 2 * nb * UE_PACK_BLOCK, 2 * nb))
        return rc;
    ue::GatedArgs g{};
    g.dh = dh;
    g.ldin = lddh;
    g.bf16 = type == UE_BF16;
    g.M = M;
    g.I = I;
    g.h = h;
    g.ldh = ldh;
    g.dgu = dgu;
    g.lddgu = lddgu;
    g.q_in = q;
    g.ldq = ldq;
    g.scale_in = scale;
    g.lds = lds;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_gated_backward(*ctx, g, s), s, "k_gated_backward launch");
}

size_t ue_weight_grad_workspace(const ue_ctx *ctx, const ue_weight_grad_product *p) {
    if (!ctx || !p || p->M < 0 || p->N < 1 || p->K < 1 || p->groups < 1) return 0;
    const int parts = ue::wgrad_parts(p->M, p->N, p->K, p->groups, ctx->num_cu);
    return parts > 1 ? static_cast<size_t>(parts) * p->groups * p->N * p->K * 4 : 0;
}

int ue_weight_grad(ue_ctx *ctx, const ue_weight_grad_product *p, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (int rc = check_wgrad(ctx, p)) return rc;
    if (p->N == 0 || p->K == 0 || p->groups == 0) return UE_OK;
    if (!p->out || (p->M > 0 && (!p->dy || !p->x)))
        return fail(ctx, UE_EINVAL, "ue_weight_grad: null argument");
    if (!aligned(p->dy, 2) || !aligned(p->x, p->x_scale ? 16 : 2) || !aligned(p->out, 4) ||
        !aligned(p->offsets, 4) || !aligned(p->index, 4) || !aligned(p->workspace, 16))
        return fail(ctx, UE_EINVAL, "ue_weight_grad: unaligned argument");
    ue::WgradArgs g{};
    g.dy = static_cast<const uint16_t *>(p->dy);
    g.lddy = p->lddy;
    g.x = p->x;
    g.ldx = p->ldx;
    g.x_scale = p->x_scale;
    g.lds = p->lds;
    g.x_rows = p->x_rows;
    g.offsets = p->offsets;
    g.G = p->groups;
    g.index = p->index;
    g.index_div = p->index_div;
    g.M = p->M;
    g.N = p->N;
    g.K = p->K;
    g.accumulate = p->accumulate != 0;
    g.vec_dy = rows_aligned(p->dy, p->lddy, 2, 16);
    g.vec_x = p->x_scale || rows_aligned(p->x, p->ldx, 2, 16);
    g.out = p->out;
    g.ldo = p->ldo;
    g.out_stride = p->out_stride;
    g.parts = p->workspace ? ue::wgrad_parts(p->M, p->N, p->K, p->groups, ctx->num_cu)
                           : 1;
    g.part = static_cast<float *>(p->workspace);
    if (ue::wgrad_too_large(g, ctx->num_cu))
        return fail(ctx, UE_ESHAPE, "ue_weight_grad: more tiles than a launch holds");
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_wgrad(*ctx, g, s), s, "k_wgrad launch");
}

int ue_combine(ue_ctx *ctx, const void *y, int32_t type, int64_t ldy, int32_t rows,
               const int32_t *inv_perm, const float *weights, const void *add, int64_t ldadd,
               int32_t T, int32_t H, void *out, int64_t ldo, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (T < 0 || T > ctx->cfg.max_tokens || H < 1 || H > kMaxCols || rows < 0)
        return fail(ctx, UE_ESHAPE, "ue_combine: T=%d (0..%d) H=%d rows=%d", T,
                    ctx->cfg.max_tokens, H, rows);
    if (int rc = check_rows(ctx, "ue_combine", "y", y, type, ldy, T > 0 ? rows : 0, H)) return rc;
    if (int rc = check_rows(ctx, "ue_combine", "out", out, type, ldo, T, H)) return rc;
    if (add)
        if (int rc = check_rows(ctx, "ue_combine", "add", add, type, ldadd, T, H)) return rc;
    if (T > 0 && !inv_perm) return fail(ctx, UE_EINVAL, "ue_combine: null inv_perm");
    if (!aligned(inv_perm, 4) || !aligned(weights, 4))
        return fail(ctx, UE_EINVAL, "ue_combine: unaligned argument");
    ue::CombineArgs g{};
    g.y = y;
    g.ldy = ldy;
    g.rows = rows;
    g.bf16 = type == UE_BF16;
    g.inv = inv_perm;
    g.weights = weights;
    g.T = T;
    g.k = ctx->k;
    g.H = H;
    g.add = add;
    g.ldadd = ldadd;
    g.out = out;
    g.ldo = ldo;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    return done(ctx, ue::launch_combine(*ctx, g, s), s, "k_combine launch");
}

static int combine_backward(ue_ctx *ctx, const char *what, bool every_row, const void *dout,
                            int32_t type, int64_t lddout, const int32_t *inv_perm,
                            const float *weights, const void *y, int64_t ldy, int32_t rows,
                            int32_t T, int32_t H, void *dy, int64_t lddy, float *dweights,
                            void *workspace, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (T < 0 || T > ctx->cfg.max_tokens || H < 1 || H > kMaxCols || rows < 0)
        return fail(ctx, UE_ESHAPE, "%s: T=%d (0..%d) H=%d rows=%d", what, T,
                    ctx->cfg.max_tokens, H, rows);
    if (int rc = check_rows(ctx, what, "dout", dout, type, lddout, T, H)) return rc;
    if (dweights)
        if (int rc = check_rows(ctx, what, "y", y, type, ldy, T > 0 ? rows : 0, H)) return rc;
    const bool notes = every_row && ue::combine_notes(T, ctx->k, rows);
    if (every_row && rows > 0 && (!dy || (notes && !workspace)))
        return fail(ctx, UE_EINVAL, "%s: null dy or workspace", what);
    if (dy)
        if (int rc = check_rows(ctx, what, "dy", dy, type, lddy, T > 0 ? rows : 0, H)) return rc;
    if (T > 0 && !inv_perm) return fail(ctx, UE_EINVAL, "%s: null inv_perm", what);
    if (!aligned(inv_perm, 4) || !aligned(weights, 4) || !aligned(dweights, 4) ||
        !aligned(workspace, 16))
        return fail(ctx, UE_EINVAL, "%s: unaligned argument", what);
    ue::CombineArgs g{};
    g.named_by = notes ? static_cast<uint32_t *>(workspace) : nullptr;
    g.y = y;
    g.ldy = ldy;
    g.rows = rows;
    g.bf16 = type == UE_BF16;
    g.inv = inv_perm;
    g.weights = weights;
    g.T = T;
    g.k = ctx->k;
    g.H = H;
    g.dout = dout;
    g.lddout = lddout;
    g.dy = dy;
    g.lddy = lddy;
    g.dweights = dweights;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    const hipError_t he = dy || dweights ? ue::launch_combine_backward(*ctx, g, every_row, s)
                                         : hipSuccess;
    return done(ctx, he, s, "k_combine_backward launch");
}

int ue_combine_backward(ue_ctx *ctx, const void *dout, int32_t type, int64_t lddout,
                        const int32_t *inv_perm, const float *weights, const void *y,
                        int64_t ldy, int32_t rows, int32_t T, int32_t H, void *dy,
                        int64_t lddy, float *dweights, void *stream) {
    return combine_backward(ctx, "ue_combine_backward", false, dout, type, lddout, inv_perm,
                            weights, y, ldy, rows, T, H, dy, lddy, dweights, nullptr, stream);
}

size_t ue_combine_backward_workspace(const ue_ctx *ctx, int32_t T, int32_t rows) {
    if (!ctx || T < 0 || rows < 0 || !ue::combine_notes(T, ctx->k, rows)) return 0;
    return static_cast<size_t>(rows) * 4;
}

int ue_combine_backward_all(ue_ctx *ctx, const void *dout, int32_t type, int64_t lddout,
                            const int32_t *inv_perm, const float *weights, const void *y,
                            int64_t ldy, int32_t rows, int32_t T, int32_t H, void *dy,
                            int64_t lddy, float *dweights, void *workspace, void *stream) {
    return combine_backward(ctx, "ue_combine_backward_all", true, dout, type, lddout, inv_perm,
                            weights, y, ldy, rows, T, H, dy, lddy, dweights, workspace, stream);
}


}  // extern "C"
