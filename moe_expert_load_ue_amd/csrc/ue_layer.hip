// C ABI of the expert layer's operators: the gate and its gradient, 8-bit
// rows and products, and the whole layer for a few tokens. As in the other
// entry points every host-visible argument is checked before anything is
// launched or written.
#include <new>

#include "ue_internal.h"

namespace {

using ue::aligned;
using ue::fail;
using ue::hip_fail;
using ue::round_up;
using ue::tbegin;
using ue::tmark;

constexpr int kMaxK = 65536;     // int32 sums of 8-bit products stay exact

size_t type_bytes(int type) { return type == UE_F32 ? 4 : type == UE_BF16 ? 2 : 1; }

// Whether rows of `bytes`-sized pieces at p, ld elements apart, are aligned.
bool rows_aligned(const void *p, int64_t ld, size_t esize, size_t bytes) {
    return aligned(p, bytes) && static_cast<size_t>(ld) * esize % bytes == 0;
}

int check_rule(ue_ctx *c, const char *what, int score, const float *bias) {
    if (score != UE_SCORE_SOFTMAX && score != UE_SCORE_SIGMOID)
        return fail(c, UE_EINVAL, "%s: unknown score %d", what, score);
    if (bias && score != UE_SCORE_SIGMOID)
        return fail(c, UE_EINVAL, "%s: a bias needs the sigmoid score", what);
    if (!aligned(bias, 4))
        return fail(c, UE_EINVAL, "%s: bias must be 4-byte aligned", what);
    return UE_OK;
}

int check_logits(ue_ctx *c, const char *what, const void *p, int type,
                 int64_t ld, int T) {
    if (type != UE_F32 && type != UE_BF16)
        return fail(c, UE_EINVAL, "%s: logits must be UE_F32 or UE_BF16", what);
    if (T < 0 || T > c->cfg.max_tokens)
        return fail(c, UE_ESHAPE, "%s: T=%d outside 0..%d", what, T,
                    c->cfg.max_tokens);
    if (ld < c->E)
        return fail(c, UE_ESHAPE, "%s: rows of %d logits, %lld apart", what,
                    c->E, static_cast<long long>(ld));
    if (T > 0 && !p) return fail(c, UE_EINVAL, "%s: null logits", what);
    if (!aligned(p, type_bytes(type)))
        return fail(c, UE_EINVAL, "%s: logits not aligned to their type", what);
    return UE_OK;
}

// Whether a lane may load its logits as one piece (kernels' load_row).
bool lane_loads(const ue_ctx *c, const void *p, int type, int64_t ld) {
    const int v = ue::lane_slots(c->E);
    const size_t es = type_bytes(type);
    const size_t piece = v * es < 16 ? v * es : 16;
    return c->E % v == 0 && rows_aligned(p, ld, es, piece);
}

ue::GateRule rule_of(const ue_ctx *c, int score, int renorm, float scale,
                     const float *bias) {
    return ue::GateRule{c->E, c->k, score == UE_SCORE_SIGMOID, renorm != 0,
                        scale, bias};
}

}  // namespace

extern "C" {

int ue_gate(ue_ctx *ctx, const void *logits, int32_t type, int64_t ld,
            int32_t T, int32_t score, int32_t renorm, float scale,
            const float *bias, int32_t *ids, float *weights, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (int rc = check_logits(ctx, "ue_gate", logits, type, ld, T)) return rc;
    if (int rc = check_rule(ctx, "ue_gate", score, bias)) return rc;
    if (T > 0 && (!ids || !weights))
        return fail(ctx, UE_EINVAL, "ue_gate: null output");
    if (!aligned(ids, 4) || !aligned(weights, 4))
        return fail(ctx, UE_EINVAL, "ue_gate: outputs must be 4-byte aligned");
    ue::GateArgs g{};
    g.logits = logits;
    g.ld = ld;
    g.bf16 = type == UE_BF16;
    g.vec = lane_loads(ctx, logits, type, ld);
    g.vec4 = ctx->E % 4 == 0 && rows_aligned(logits, ld, type_bytes(type), 4 * type_bytes(type));
    g.T = T;
    g.rule = rule_of(ctx, score, renorm, scale, bias);
    g.ids = ids;
    g.weights = weights;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    const hipError_t he = ue::launch_gate(*ctx, g, s);
    tmark(ctx, s);
    return he == hipSuccess ? UE_OK : hip_fail(ctx, he, "k_gate launch");
}

int ue_gate_backward(ue_ctx *ctx, const void *logits, int32_t type, int64_t ld,
                     int32_t T, int32_t score, int32_t renorm, float scale,
                     const int32_t *ids, const float *dweights, void *dlogits,
                     int64_t ld_out, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (int rc = check_logits(ctx, "ue_gate_backward", logits, type, ld, T))
        return rc;
    if (int rc = check_rule(ctx, "ue_gate_backward", score, nullptr)) return rc;
    if (ld_out < ctx->E)
        return fail(ctx, UE_ESHAPE, "ue_gate_backward: gradients %lld apart",
                    static_cast<long long>(ld_out));
    if (T > 0 && (!ids || !dweights || !dlogits))
        return fail(ctx, UE_EINVAL, "ue_gate_backward: null argument");
    if (!aligned(ids, 4) || !aligned(dweights, 4) ||
        !aligned(dlogits, type_bytes(type)))
        return fail(ctx, UE_EINVAL, "ue_gate_backward: unaligned argument");
    ue::GateBackArgs g{};
    g.logits = logits;
    g.ld = ld;
    g.bf16 = type == UE_BF16;
    g.vec = lane_loads(ctx, logits, type, ld);
    const size_t es = type_bytes(type);
    g.vec4 = ctx->E % 4 == 0 && rows_aligned(logits, ld, es, 4 * es) &&
             rows_aligned(dlogits, ld_out, es, 4 * es);
    g.T = T;
    g.rule = rule_of(ctx, score, renorm, scale, nullptr);
    g.ids = ids;
    g.dweights = dweights;
    g.dlogits = dlogits;
    g.ld_out = ld_out;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    const hipError_t he = ue::launch_gate_backward(*ctx, g, s);
    tmark(ctx, s);
    return he == hipSuccess ? UE_OK
                            : hip_fail(ctx, he, "k_gate_backward launch");
}

int ue_quantize_rows(ue_ctx *ctx, const void *x, int32_t type, int64_t ldx,
                     int32_t M, int32_t K, int8_t *q, int64_t ldq,
                     float *scale, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (type != UE_F32 && type != UE_BF16)
        return fail(ctx, UE_EINVAL, "ue_quantize_rows: x must be UE_F32 or UE_BF16");
    if (M < 0 || K < 1 || K > kMaxK)
        return fail(ctx, UE_ESHAPE, "ue_quantize_rows: M=%d K=%d", M, K);
    const int Kpad = (K + 15) / 16 * 16;
    if (ldx < K || ldq < Kpad || ldq % 16 != 0)
        return fail(ctx, UE_ESHAPE, "ue_quantize_rows: ldx=%lld ldq=%lld K=%d",
                    static_cast<long long>(ldx), static_cast<long long>(ldq), K);
    if (M > 0 && (!x || !q || !scale))
        return fail(ctx, UE_EINVAL, "ue_quantize_rows: null argument");
    if (!aligned(x, type_bytes(type)) || !aligned(q, 16) || !aligned(scale, 4))
        return fail(ctx, UE_EINVAL, "ue_quantize_rows: unaligned argument");
    const ue::QuantArgs g{x, ldx, type == UE_BF16,
                          rows_aligned(x, ldx, type_bytes(type), 16),
                          M, K, Kpad, q, ldq, scale};
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    const hipError_t he = ue::launch_quantize(g, s);
    tmark(ctx, s);
    return he == hipSuccess ? UE_OK : hip_fail(ctx, he, "k_quantize launch");
}

int ue_matmul_i8(ue_ctx *ctx, const ue_i8_product *p, void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (!p) return fail(ctx, UE_EINVAL, "ue_matmul_i8: null product");
    if (p->M < 0 || p->N < 0 || p->K < 1 || p->K > kMaxK ||
        p->N > 0x3FFFFFFF || p->a_rows < 0 || p->n_mats < 1)
        return fail(ctx, UE_ESHAPE, "ue_matmul_i8: M=%d N=%d K=%d a_rows=%d n_mats=%d",
                    p->M, p->N, p->K, p->a_rows, p->n_mats);
    const int64_t Kpad = (static_cast<int64_t>(p->K) + 15) / 16 * 16;
    if (p->lda < Kpad || p->lda % 16 || p->ldw < Kpad || p->ldw % 16 ||
        p->w_stride < 0 || p->w_stride % 16 || p->ws_stride < 0 || p->ldo < p->N)
        return fail(ctx, UE_ESHAPE,
                    "ue_matmul_i8: lda=%lld ldw=%lld w_stride=%lld ws_stride=%lld ldo=%lld",
                    static_cast<long long>(p->lda), static_cast<long long>(p->ldw),
                    static_cast<long long>(p->w_stride),
                    static_cast<long long>(p->ws_stride),
                    static_cast<long long>(p->ldo));
    // (the kernels address a matrix, and 256 rows of a, with 32 bits)
    if ((p->gated ? 2 : 1) * static_cast<int64_t>(p->N) > 0xFFFFFFFFll / p->ldw ||
        p->lda > 0xFFFFFF)
        return fail(ctx, UE_ESHAPE, "ue_matmul_i8: a matrix of 4 GiB, or lda=%lld of 16 MiB",
                    static_cast<long long>(p->lda));
    if (p->out_type != UE_F32 && p->out_type != UE_BF16)
        return fail(ctx, UE_EINVAL, "ue_matmul_i8: out must be UE_F32 or UE_BF16");
    if (p->offsets ? p->groups < 0 || p->groups > 0xFFFFF
                   : p->expert_of != nullptr)
        return fail(ctx, UE_ESHAPE, "ue_matmul_i8: groups=%d, %s", p->groups,
                    p->offsets ? "at most 2^20 - 1" : "expert_of needs offsets");
    if (p->index ? p->index_div < 1 : p->a_rows < p->M)
        return fail(ctx, UE_ESHAPE, "ue_matmul_i8: M=%d rows from a_rows=%d, index_div=%d",
                    p->M, p->a_rows, p->index_div);
    if (p->M == 0 || p->N == 0 || (p->offsets && p->groups == 0)) return UE_OK;
    if (!p->w || !p->w_scale || !p->out ||
        (p->a_rows > 0 && (!p->a || !p->a_scale)))
        return fail(ctx, UE_EINVAL, "ue_matmul_i8: null argument");
    if (p->a_rows == 0)
        return fail(ctx, UE_ESHAPE, "ue_matmul_i8: no rows of a");
    const size_t es = type_bytes(p->out_type);
    if (!aligned(p->a, 16) || !aligned(p->w, 16) || !aligned(p->a_scale, 4) ||
        !aligned(p->w_scale, 4) || !aligned(p->offsets, 4) ||
        !aligned(p->expert_of, 4) || !aligned(p->index, 4) || !aligned(p->out, es))
        return fail(ctx, UE_EINVAL, "ue_matmul_i8: unaligned argument");
    ue::I8Args g{};
    g.a = p->a;
    g.lda = p->lda;
    g.a_scale = p->a_scale;
    g.a_rows = p->a_rows;
    g.w = p->w;
    g.ldw = p->ldw;
    g.w_stride = p->w_stride;
    g.w_scale = p->w_scale;
    g.ws_stride = p->ws_stride;
    g.n_mats = p->n_mats;
    g.offsets = p->offsets;
    g.expert_of = p->expert_of;
    g.G = p->offsets ? p->groups : 1;
    g.index = p->index;
    g.index_div = p->index_div;
    g.M = p->M;
    g.N = p->N;
    g.K = p->K;
    g.gated = p->gated != 0;
    g.out_f32 = p->out_type == UE_F32;
    g.vec_out = rows_aligned(p->out, p->ldo, es, 16);
    g.out = p->out;
    g.ldo = p->ldo;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    bool too_large = false;
    const hipError_t he = ue::launch_matmul_i8(*ctx, g, s, too_large);
    tmark(ctx, s);
    if (too_large)
        return fail(ctx, UE_ESHAPE, "ue_matmul_i8: a launch of 2^32 threads or more");
    return he == hipSuccess ? UE_OK : hip_fail(ctx, he, "k_matmul_i8 launch");
}

int ue_register_layer(ue_ctx *ctx, const ue_layer *l) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (!l) return fail(ctx, UE_EINVAL, "ue_register_layer: null layer");
    if (l->weight_type != UE_BF16 && l->weight_type != UE_I8)
        return fail(ctx, UE_EINVAL, "ue_register_layer: weights must be UE_BF16 or UE_I8");
    const bool i8 = l->weight_type == UE_I8;
    const int unit = i8 ? 16 : 8;      // elements of 16 bytes
    if (l->hidden < unit || l->inter < unit || l->hidden % unit ||
        l->inter % unit || l->hidden > (1 << 20) || l->inter > (1 << 20))
        return fail(ctx, UE_ESHAPE, "ue_register_layer: hidden=%d inter=%d, multiples of %d wanted",
                    l->hidden, l->inter, unit);
    const int64_t mat = static_cast<int64_t>(l->hidden) * l->inter;
    if (l->gate_up_stride < 2 * mat || l->down_stride < mat ||
        l->gate_up_stride % unit || l->down_stride % unit)
        return fail(ctx, UE_ESHAPE, "ue_register_layer: strides %lld and %lld",
                    static_cast<long long>(l->gate_up_stride),
                    static_cast<long long>(l->down_stride));
    // the kernels address one expert's matrix, the router and an expert's
    // hidden rows with 32 bits
    if (2 * mat * (i8 ? 1 : 2) > 0xFFFFFFFFll ||
        2ll * ctx->E * l->hidden > 0xFFFFFFFFll)
        return fail(ctx, UE_ESHAPE, "ue_register_layer: a matrix of 4 GiB");
    if (int rc = check_rule(ctx, "ue_register_layer", l->score, l->bias)) return rc;
    if (!l->router || !l->gate_up || !l->down ||
        (i8 && (!l->gate_up_scale || !l->down_scale)))
        return fail(ctx, UE_EINVAL, "ue_register_layer: null matrix or scale");
    // router rows are read 16 bytes at a time whatever the experts' type
    if (!aligned(l->router, 16) || !aligned(l->gate_up, 16) ||
        !aligned(l->down, 16) || !aligned(l->gate_up_scale, 4) ||
        !aligned(l->down_scale, 4))
        return fail(ctx, UE_EINVAL, "ue_register_layer: unaligned matrix or scale");

    const int T = ctx->cfg.max_tokens < ue::kMoeTokens ? ctx->cfg.max_tokens
                                                       : ue::kMoeTokens;
    const size_t rows = static_cast<size_t>(T) * ctx->k;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = round_up(off + bytes, 256);
        return o;
    };
    // (the counter comes first in every layout: no layer's other data may lie
    // over it, since it is zero between calls whichever layer they are of)
    const size_t o_done = take(sizeof(uint32_t));
    const size_t o_logits = take(sizeof(float) * ue::moe_router_parts(l->hidden) * T * ctx->E);
    const size_t o_n = take(sizeof(int32_t));
    const size_t o_part = take(sizeof(float) * l->hidden * T *
                               ue::moe_down_shares(l->hidden, T, ctx->num_cu));
    const size_t o_act = take(sizeof(ue::MoeExpert) * ctx->E);
    const size_t o_w = take(sizeof(float) * rows);
    const size_t o_t = take(sizeof(int32_t) * rows);
    const size_t o_h = take(2 * sizeof(uint16_t) * rows * l->inter);
    if (!ctx->layer_ws || ctx->layer_ws->bytes < off) {
        ue::LayerSpace *w = new (std::nothrow) ue::LayerSpace{nullptr, off, ctx->layer_ws};
        if (!w || hipMalloc(&w->mem, off) != hipSuccess) {
            delete w;
            return fail(ctx, UE_ENOMEM, "ue_register_layer: %zu bytes of workspace", off);
        }
        const hipError_t he = hipMemset(static_cast<char *>(w->mem) + o_done, 0,
                                        sizeof(uint32_t));
        if (he != hipSuccess) {
            (void)hipFree(w->mem);
            delete w;
            return hip_fail(ctx, he, "ue_register_layer: workspace");
        }
        ctx->layer_ws = w;
    }
    // (calls of the layer registered before have ended when this returns, so
    // its matrices may go, and its workspace be used from another stream)
    const hipError_t he = hipDeviceSynchronize();
    if (he != hipSuccess) return hip_fail(ctx, he, "ue_register_layer");
    char *b = static_cast<char *>(ctx->layer_ws->mem);
    ctx->moe_logits = reinterpret_cast<float *>(b + o_logits);
    ctx->moe_done = reinterpret_cast<uint32_t *>(b + o_done);
    ctx->moe_part = reinterpret_cast<float *>(b + o_part);
    ctx->moe_n_active = reinterpret_cast<int32_t *>(b + o_n);
    ctx->moe_active = reinterpret_cast<ue::MoeExpert *>(b + o_act);
    ctx->moe_row_weight = reinterpret_cast<float *>(b + o_w);
    ctx->moe_row_token = reinterpret_cast<int32_t *>(b + o_t);
    ctx->moe_h = reinterpret_cast<uint16_t *>(b + o_h);
    ctx->layer = *l;
    ctx->layer_tokens = T;
    ctx->has_layer = true;
    return UE_OK;
}

int ue_moe_tokens(ue_ctx *ctx, const void *x, int64_t ldx, int32_t T,
                  void *out, int64_t ldo, int32_t *ids, float *weights,
                  void *stream) {
    if (!ctx) return UE_EINVAL;
    ctx->err.clear();
    if (!ctx->has_layer)
        return fail(ctx, UE_ESTATE, "ue_moe_tokens: no layer registered");
    const ue_layer &l = ctx->layer;
    if (T < 0 || T > ctx->layer_tokens)
        return fail(ctx, UE_ESHAPE, "ue_moe_tokens: T=%d outside 0..%d", T,
                    ctx->layer_tokens);
    // (64 rows of x are addressed with 32 bits)
    if (ldx < l.hidden || ldx % 8 || ldx > (1 << 24) || ldo < l.hidden)
        return fail(ctx, UE_ESHAPE, "ue_moe_tokens: ldx=%lld ldo=%lld hidden=%d",
                    static_cast<long long>(ldx), static_cast<long long>(ldo),
                    l.hidden);
    if (T > 0 && (!x || !out || !ids || !weights))
        return fail(ctx, UE_EINVAL, "ue_moe_tokens: null argument");
    if (!aligned(x, 16) || !aligned(out, 2) || !aligned(ids, 4) ||
        !aligned(weights, 4))
        return fail(ctx, UE_EINVAL, "ue_moe_tokens: unaligned argument");
    if (T == 0) return UE_OK;
    ue::MoeArgs g{};
    g.T = T;
    g.H = l.hidden;
    g.I = l.inter;
    g.x = static_cast<const uint16_t *>(x);
    g.ldx = ldx;
    g.router = static_cast<const uint16_t *>(l.router);
    g.rule = rule_of(ctx, l.score, l.renorm, l.scale, l.bias);
    g.i8 = l.weight_type == UE_I8;
    g.gate_up = l.gate_up;
    g.down = l.down;
    g.gate_up_stride = l.gate_up_stride;
    g.down_stride = l.down_stride;
    g.gate_up_scale = l.gate_up_scale;
    g.down_scale = l.down_scale;
    g.logits = ctx->moe_logits;
    g.done = ctx->moe_done;
    g.part = ctx->moe_part;
    g.n_active = ctx->moe_n_active;
    g.active = ctx->moe_active;
    g.row_weight = ctx->moe_row_weight;
    g.row_token = ctx->moe_row_token;
    g.h_hi = ctx->moe_h;
    g.h_lo = ctx->moe_h + static_cast<size_t>(T) * ctx->k * l.inter;
    g.out = static_cast<uint16_t *>(out);
    g.ldo = ldo;
    g.ids = ids;
    g.weights = weights;
    hipStream_t s = static_cast<hipStream_t>(stream);
    tbegin(ctx, s);
    hipError_t he = ue::launch_moe_route(g, s);
    if (he != hipSuccess) return hip_fail(ctx, he, "router launch");
    tmark(ctx, s);
    he = ue::launch_moe_up(g, s);
    if (he != hipSuccess) return hip_fail(ctx, he, "k_moe_up launch");
    tmark(ctx, s);
    he = ue::launch_moe_down(*ctx, g, s);
    tmark(ctx, s);
    return he == hipSuccess ? UE_OK : hip_fail(ctx, he, "k_moe_down launch");
}

}  // extern "C"
