// fp8_api.hip — C ABI of the scored routing and the 8-bit float path (declared
// in include/moe.h): argument validation, workspace layout and dispatch.
#include <math.h>

#include "../../include/moe.h"
#include "fp8.h"

namespace {

constexpr int kFp8MaxDim = 16384;

bool elem_type(int32_t t, moe::ElemType& out) {
    out = t == MOE_F16 ? moe::ElemType::kF16 : (t == MOE_BF16 ? moe::ElemType::kBF16 : moe::ElemType::kF32);
    return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16;
}
int elem_size(moe::ElemType t) { return t == moe::ElemType::kF32 ? 4 : 2; }

moe_status check_route(const float* logits, int T, int E, int k, const moe_route_spec* s, const moe_routing* r) {
    if (!logits) return fail(MOE_ERR_INVALID_ARGUMENT, "logits is NULL");
    if (!aligned(logits, 4)) return fail(MOE_ERR_INVALID_ARGUMENT, "logits must be 4-byte aligned");
    if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T = %d: need at least one token", T);
    if (E < 1 || E > kMaxExperts) return fail(MOE_ERR_INVALID_ARGUMENT, "E = %d: need 1 <= E <= %d", E, kMaxExperts);
    if (k < 1 || k > E || k > kMaxTopK)
        return fail(MOE_ERR_INVALID_ARGUMENT, "k = %d: need 1 <= k <= min(E = %d, %d)", k, E, kMaxTopK);
    if ((int64_t)T * k > (int64_t)1 << 30)
        return fail(MOE_ERR_INVALID_ARGUMENT, "T*k = %lld is too large", (long long)T * k);
    if (!s) return fail(MOE_ERR_INVALID_ARGUMENT, "spec is NULL");
    if (s->score != MOE_SCORE_SOFTMAX && s->score != MOE_SCORE_SIGMOID)
        return fail(MOE_ERR_INVALID_ARGUMENT, "spec.score = %d: use MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID", s->score);
    if (s->n_group < 1 || s->n_group > 64 || E % s->n_group)
        return fail(MOE_ERR_INVALID_ARGUMENT, "spec.n_group = %d: need a divisor of E = %d, at most 64", s->n_group, E);
    const int S = E / s->n_group;
    if (s->topk_group < 1 || s->topk_group > s->n_group)
        return fail(MOE_ERR_INVALID_ARGUMENT, "spec.topk_group = %d: need 1..n_group = %d", s->topk_group, s->n_group);
    if (s->n_group > 1 && k > s->topk_group * S)
        return fail(MOE_ERR_INVALID_ARGUMENT, "k = %d: the topk_group = %d groups of %d hold fewer experts", k,
                    s->topk_group, S);
    if (s->group_top < 1 || s->group_top > 2 || s->group_top > S)
        return fail(MOE_ERR_INVALID_ARGUMENT, "spec.group_top = %d: need 1 or 2, at most E/n_group = %d", s->group_top,
                    S);
    if (!isfinite(s->scale)) return fail(MOE_ERR_INVALID_ARGUMENT, "spec.scale must be finite");
    if (s->bias && !aligned(s->bias, 4)) return fail(MOE_ERR_INVALID_ARGUMENT, "spec.bias must be 4-byte aligned");
    if (!r || !r->idx || !r->w || !r->count || !r->offset || !r->pair || !r->active || !r->n_active)
        return fail(MOE_ERR_INVALID_ARGUMENT, "moe_routing or one of its arrays is NULL");
    return MOE_OK;
}

moe::ScoreRule to_rule(const moe_route_spec& s) {
    return moe::ScoreRule{s.score == MOE_SCORE_SIGMOID, s.n_group, s.topk_group, s.group_top, s.renorm != 0, s.scale,
                          s.bias};
}

// rows, cols < 0: any
moe_status check_fp8(const moe_fp8_matrix& m, const char* name, int rows, int cols, int n_experts) {
    if (!m.data || !m.scale) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: data or scale is NULL", name);
    if (rows >= 0 && (m.rows != rows || m.cols != cols))
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s is %d x %d, expected %d x %d", name, m.rows, m.cols, rows, cols);
    if (m.rows < 1 || m.cols < 16 || m.cols % 16)
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s is %d x %d: need rows >= 1 and cols a positive multiple of 16", name,
                    m.rows, m.cols);
    if (m.row_stride < m.cols || m.row_stride % 16)
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s.row_stride = %lld: need a multiple of 16, at least cols = %d", name,
                    (long long)m.row_stride, m.cols);
    if (m.row_stride > (int64_t)1 << 23)   // 32-bit offsets inside a tile of 256 rows
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s.row_stride = %lld is too large", name, (long long)m.row_stride);
    if (m.expert_stride % 16 ||
        (n_experts > 1 && m.expert_stride < (int64_t)(m.rows - 1) * m.row_stride + m.cols))
        return fail(MOE_ERR_INVALID_ARGUMENT,
                    "%s.expert_stride = %lld: need a multiple of 16 that covers %d rows of row_stride %lld", name,
                    (long long)m.expert_stride, m.rows, (long long)m.row_stride);
    if (!aligned(m.data, 16) || !aligned(m.scale, 4))
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s: data must be 16-byte aligned, scale 4-byte aligned", name);
    return MOE_OK;
}

moe::Fp8Mat to_fp8(const moe_fp8_matrix& m) {
    return moe::Fp8Mat{(const uint8_t*)m.data, m.scale, m.row_stride, m.expert_stride, m.rows, m.cols};
}

moe_status check_fp8_layer(const moe_fp8_layer* L, int T, int k) {
    if (!L) return fail(MOE_ERR_INVALID_ARGUMENT, "layer descriptor is NULL");
    const int E = L->n_experts, H = L->hidden, I = L->inter;
    if (E < 1 || E > kMaxExperts) return fail(MOE_ERR_INVALID_ARGUMENT, "n_experts = %d: need 1..%d", E, kMaxExperts);
    if (H < 128 || H % 128 || I < 128 || I % 128)
        return fail(MOE_ERR_INVALID_ARGUMENT, "hidden = %d, inter = %d: both must be positive multiples of 128", H, I);
    if (H > kFp8MaxDim || I > kFp8MaxDim)
        return fail(MOE_ERR_UNSUPPORTED, "hidden = %d, inter = %d: the fp8 layer supports up to %d", H, I, kFp8MaxDim);
    if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T = %d: need at least one token", T);
    if (k < 1 || k > E || k > kMaxTopK)
        return fail(MOE_ERR_INVALID_ARGUMENT, "k = %d: need 1 <= k <= min(E = %d, %d)", k, E, kMaxTopK);
    if ((int64_t)T * k > (int64_t)1 << 30)
        return fail(MOE_ERR_INVALID_ARGUMENT, "T*k = %lld is too large", (long long)T * k);
    if ((int64_t)T * H >= (int64_t)1 << 32)   // 32-bit offsets of gathered rows
        return fail(MOE_ERR_INVALID_ARGUMENT, "T*hidden = %lld: need less than 2^32", (long long)T * H);
    moe_status st;
    if ((st = check_fp8(L->gate, "gate", I, H, E)) != MOE_OK) return st;
    if ((st = check_fp8(L->up, "up", I, H, E)) != MOE_OK) return st;
    if ((st = check_fp8(L->down, "down", H, I, E)) != MOE_OK) return st;
    if (L->has_shared) {
        if ((st = check_fp8(L->sh_gate, "sh_gate", I, H, 1)) != MOE_OK) return st;
        if ((st = check_fp8(L->sh_up, "sh_up", I, H, 1)) != MOE_OK) return st;
        if ((st = check_fp8(L->sh_down, "sh_down", H, I, 1)) != MOE_OK) return st;
    }
    return MOE_OK;
}

struct Fp8FfnWorkspace {
    size_t hq, hs, tiles, hf, total;
};

Fp8FfnWorkspace fp8_ffn_layout(const moe_fp8_layer* L, int T, int k) {
    const size_t rows = (size_t)T * k + (L->has_shared ? T : 0);
    Fp8FfnWorkspace w{};
    size_t off = 0;
    if (moe::fp8_few_pairs(T, k, L->n_experts)) {
        w.total = align_up(rows * L->inter * sizeof(float), 256);
        return w;
    }
    w.hq = off;
    off += align_up(rows * L->inter, 256);
    w.hs = off;
    off += align_up(rows * (L->inter / MOE_FP8_BLOCK) * sizeof(float), 256);
    w.tiles = off;
    off += align_up(moe::fp8_items_bytes(T, k, L->n_experts, L->has_shared ? 1 : 0), 256);
    w.total = off;
    return w;
}

struct Fp8ForwardWorkspace {
    size_t route, route_bytes, ffn, xq, xs, yp, ysh, ysc, total;
};

Fp8ForwardWorkspace fp8_forward_layout(const moe_fp8_layer* L, int T, int k, bool pair16) {
    Fp8ForwardWorkspace w{};
    size_t off = 0;
    w.route = off;
    w.route_bytes = moe::route_workspace_bytes(T, L->n_experts, k);
    off += align_up(w.route_bytes, 256);
    w.ffn = off;
    off += fp8_ffn_layout(L, T, k).total;
    w.xq = off;
    off += align_up((size_t)T * L->hidden, 256);
    w.xs = off;
    off += align_up((size_t)T * (L->hidden / MOE_FP8_BLOCK) * sizeof(float), 256);
    if (moe::fp8_few_pairs(T, k, L->n_experts)) {   // combined inside the down kernel
        w.total = off;
        return w;
    }
    w.yp = off;
    off += align_up((size_t)T * k * L->hidden * (pair16 ? 2 : 4), 256);
    w.ysh = off;
    if (L->has_shared) off += align_up((size_t)T * L->hidden * (pair16 ? 2 : 4), 256);
    w.ysc = off;
    if (pair16)
        off += align_up(((size_t)T * k + (L->has_shared ? T : 0)) * (L->hidden / moe::kPairBlock) * sizeof(float), 256);
    w.total = off;
    return w;
}

moe::Fp8FfnArgs fp8_ffn_args(const moe_fp8_layer* L, const moe_routing* r, int T, int k, char* ws,
                             const Fp8FfnWorkspace& w) {
    moe::Fp8FfnArgs a{};
    a.gate = to_fp8(L->gate);
    a.up = to_fp8(L->up);
    a.down = to_fp8(L->down);
    a.has_shared = L->has_shared ? 1 : 0;
    if (a.has_shared) {
        a.sgate = to_fp8(L->sh_gate);
        a.sup = to_fp8(L->sh_up);
        a.sdown = to_fp8(L->sh_down);
    }
    a.H = L->hidden;
    a.I = L->inter;
    a.T = T;
    a.k = k;
    a.E = L->n_experts;
    a.r = moe::RoutingPtrs{r->idx, r->w, r->count, r->offset, r->pair, r->active, r->n_active};
    a.hq = (uint8_t*)(ws + w.hq);
    a.hs = (float*)(ws + w.hs);
    a.tiles = ws + w.tiles;
    a.hf = (float*)(ws + w.hf);
    return a;
}

}  // namespace

extern "C" {

moe_status moe_route_scored(const float* logits, int32_t T, int32_t E, int32_t k, const moe_route_spec* spec,
                            const moe_routing* r, void* workspace, size_t ws_bytes, hipStream_t stream) {
    moe_status st = check_route(logits, T, E, k, spec, r);
    if (st != MOE_OK) return st;
    const size_t need = moe::route_workspace_bytes(T, E, k);
    if (need && (!workspace || ws_bytes < need))
        return fail(MOE_ERR_WORKSPACE, "routing workspace: %zu bytes given, %zu needed", ws_bytes, need);
    if (need && !aligned(workspace, 4)) return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be 4-byte aligned");
    const moe::RoutingPtrs rp{r->idx, r->w, r->count, r->offset, r->pair, r->active, r->n_active};
    return finish(from_hip(moe::launch_route_scored(logits, T, E, k, to_rule(*spec), rp, workspace, stream),
                           "moe_route_scored launch"),
                  stream, "moe_route_scored");
}

moe_status moe_quantize_fp8(const void* x, int32_t x_type, int64_t ldx, int32_t T, int32_t H, void* xq, float* xs,
                            hipStream_t stream) {
    moe::ElemType xt;
    if (!x || !xq || !xs) return fail(MOE_ERR_INVALID_ARGUMENT, "x, xq or xs is NULL");
    if (!elem_type(x_type, xt))
        return fail(MOE_ERR_UNSUPPORTED, "x_type = %d: supported are F32 (%d), F16 (%d) and BF16 (%d)", x_type, MOE_F32,
                    MOE_F16, MOE_BF16);
    if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T = %d: need at least one token", T);
    if (H < 16 || H % 16) return fail(MOE_ERR_INVALID_ARGUMENT, "H = %d: must be a positive multiple of 16", H);
    if (ldx < H) return fail(MOE_ERR_INVALID_ARGUMENT, "ldx = %lld: need at least H = %d", (long long)ldx, H);
    if (!aligned(x, 16) || (T > 1 && (ldx % (16 / elem_size(xt))) != 0) || !aligned(xq, 8) || !aligned(xs, 4))
        return fail(MOE_ERR_INVALID_ARGUMENT,
                    "x and its rows (ldx = %lld) must be 16-byte aligned, xq 8-byte, xs 4-byte aligned", (long long)ldx);
    return finish(from_hip(moe::launch_quantize_fp8(x, xt, ldx, T, H, (uint8_t*)xq, xs, stream),
                           "moe_quantize_fp8 launch"),
                  stream, "moe_quantize_fp8");
}

moe_status moe_matmul_fp8(const void* xq, const float* xs, int32_t T, const moe_fp8_matrix* w, void* y, int32_t y_type,
                          int64_t ldy, hipStream_t stream) {
    moe::ElemType yt;
    if (!xq || !xs || !w || !y) return fail(MOE_ERR_INVALID_ARGUMENT, "xq, xs, w or y is NULL");
    if (!elem_type(y_type, yt))
        return fail(MOE_ERR_UNSUPPORTED, "y_type = %d: supported are F32 (%d), F16 (%d) and BF16 (%d)", y_type, MOE_F32,
                    MOE_F16, MOE_BF16);
    if (T < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "T = %d: need at least one token", T);
    moe_status st = check_fp8(*w, "w", -1, -1, 1);
    if (st != MOE_OK) return st;
    if (ldy < w->rows) return fail(MOE_ERR_INVALID_ARGUMENT, "ldy = %lld: need at least N = %d", (long long)ldy, w->rows);
    if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(y, elem_size(yt)))
        return fail(MOE_ERR_INVALID_ARGUMENT, "xq must be 16-byte aligned, xs 4-byte and y element aligned");
    moe::Fp8MatmulArgs a{(const uint8_t*)xq, xs, to_fp8(*w), y, yt, ldy, T};
    return finish(from_hip(moe::launch_matmul_fp8(a, stream), "moe_matmul_fp8 launch"), stream, "moe_matmul_fp8");
}

size_t moe_ffn_fp8_workspace_bytes(const moe_fp8_layer* L, int32_t T, int32_t k) {
    if (!L || T < 1 || k < 1 || L->n_experts < 1) return 0;
    return fp8_ffn_layout(L, T, k).total;
}

moe_status moe_expert_ffn_fp8(const moe_fp8_layer* L, const moe_routing* r, int32_t T, int32_t k, const void* xq,
                              const float* xs, float* y_pair, float* y_shared, void* workspace, size_t ws_bytes,
                              hipStream_t stream) {
    moe_status st = check_fp8_layer(L, T, k);
    if (st != MOE_OK) return st;
    if (!r || !r->idx || !r->count || !r->offset || !r->pair || !r->active || !r->n_active)
        return fail(MOE_ERR_INVALID_ARGUMENT, "moe_routing or one of idx/count/offset/pair/active/n_active is NULL");
    if (!xq || !xs || !y_pair) return fail(MOE_ERR_INVALID_ARGUMENT, "xq, xs or y_pair is NULL");
    if (L->has_shared && !y_shared)
        return fail(MOE_ERR_INVALID_ARGUMENT, "layer has a shared expert but y_shared is NULL");
    if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(y_pair, 16) || (y_shared && !aligned(y_shared, 16)))
        return fail(MOE_ERR_INVALID_ARGUMENT, "xq, y_pair and y_shared must be 16-byte aligned, xs 4-byte aligned");
    const Fp8FfnWorkspace wl = fp8_ffn_layout(L, T, k);
    if (!workspace || ws_bytes < wl.total)
        return fail(MOE_ERR_WORKSPACE, "fp8 FFN workspace: %zu bytes given, %zu needed", ws_bytes, wl.total);
    if (!aligned(workspace, 256)) return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
    moe::Fp8FfnArgs a = fp8_ffn_args(L, r, T, k, (char*)workspace, wl);
    a.xq = (const uint8_t*)xq;
    a.xs = xs;
    a.y_pair = y_pair;
    a.y_shared = y_shared;
    a.exact = 1;
    if (moe::fp8_few_pairs(T, k, L->n_experts))
        return finish(from_hip(moe::launch_skinny_ffn(a, moe::Fp8CombineArgs{}, stream), "moe_expert_ffn_fp8 launch"),
                      stream, "moe_expert_ffn_fp8");
    return finish(from_hip(moe::launch_ffn_fp8(a, false, stream), "moe_expert_ffn_fp8 launch"), stream, "moe_expert_ffn_fp8");
}

size_t moe_forward_fp8_workspace_bytes(const moe_fp8_layer* L, int32_t T, int32_t k, uint32_t ffn_flags) {
    if (!L || T < 1 || k < 1 || L->n_experts < 1 || (ffn_flags & ~(uint32_t)MOE_FFN_PAIR_BF16)) return 0;
    return fp8_forward_layout(L, T, k, ffn_flags != 0).total;
}

moe_status moe_forward_fp8(const moe_fp8_layer* L, const moe_route_spec* spec, const float* logits, const void* x,
                           int32_t x_type, int32_t T, int32_t k, uint32_t ffn_flags, const moe_routing* r,
                           const float* shared_scale, void* out, void* workspace, size_t ws_bytes,
                           hipStream_t stream) {
    moe_status st = check_fp8_layer(L, T, k);
    if (st != MOE_OK) return st;
    if ((st = check_route(logits, T, L->n_experts, k, spec, r)) != MOE_OK) return st;
    moe::ElemType xt;
    if (!x || !out) return fail(MOE_ERR_INVALID_ARGUMENT, "x or out is NULL");
    if (!elem_type(x_type, xt))
        return fail(MOE_ERR_UNSUPPORTED, "x_type = %d: supported are F32 (%d), F16 (%d) and BF16 (%d)", x_type, MOE_F32,
                    MOE_F16, MOE_BF16);
    if (ffn_flags & ~(uint32_t)MOE_FFN_PAIR_BF16)
        return fail(MOE_ERR_INVALID_ARGUMENT, "ffn_flags = 0x%x: use 0 or MOE_FFN_PAIR_BF16", ffn_flags);
    if (shared_scale && !L->has_shared)
        return fail(MOE_ERR_INVALID_ARGUMENT, "shared_scale given for a layer without a shared expert");
    if (!aligned(x, 16) || !aligned(out, 16) || (shared_scale && !aligned(shared_scale, 4)))
        return fail(MOE_ERR_INVALID_ARGUMENT, "x and out must be 16-byte aligned, shared_scale 4-byte aligned");
    const bool pair16 = ffn_flags != 0;
    const Fp8ForwardWorkspace wl = fp8_forward_layout(L, T, k, pair16);
    if (!workspace || ws_bytes < wl.total)
        return fail(MOE_ERR_WORKSPACE, "fp8 forward workspace: %zu bytes given, %zu needed", ws_bytes, wl.total);
    if (!aligned(workspace, 256)) return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
    char* ws = (char*)workspace;
    moe::Fp8FfnArgs a = fp8_ffn_args(L, r, T, k, ws + wl.ffn, fp8_ffn_layout(L, T, k));
    a.xq = (uint8_t*)(ws + wl.xq);
    a.xs = (float*)(ws + wl.xs);
    a.y_pair = ws + wl.yp;
    a.y_shared = L->has_shared ? ws + wl.ysh : nullptr;
    a.y_scale = (float*)(ws + wl.ysc);
    a.pair16 = pair16 ? 1 : 0;
    a.exact = xt == moe::ElemType::kBF16 ? 0 : 1;
    const bool few = moe::fp8_few_pairs(T, k, L->n_experts);
    const moe::Fp8ItemList tl = few ? moe::Fp8ItemList{} : moe::fp8_item_list(a);
    bool list_done = false;
    hipError_t e = moe::launch_route_quantize_fp8(logits, T, L->n_experts, k, to_rule(*spec), a.r, ws + wl.route, tl, x, xt,
                                                  L->hidden, (uint8_t*)(ws + wl.xq), (float*)(ws + wl.xs), stream,
                                                  &list_done);
    if (e != hipSuccess) return from_hip(e, "moe_forward_fp8: routing and quantisation launch");
    const moe::Fp8CombineArgs c{a.y_pair, a.y_shared, a.y_scale, a.pair16, r->w, shared_scale, out, xt, T, k, L->hidden};
    if (few)
        return finish(from_hip(moe::launch_skinny_ffn(a, c, stream), "moe_forward_fp8: expert FFN launch"), stream,
                      "moe_forward_fp8");
    e = moe::launch_ffn_fp8(a, list_done, stream);
    if (e != hipSuccess) return from_hip(e, "moe_forward_fp8: expert FFN launch");
    return finish(from_hip(moe::launch_combine_fp8(c, stream), "moe_forward_fp8: combine launch"), stream,
                  "moe_forward_fp8");
}

}  // extern "C"
