// C ABI of the operators around the expert FFN: scored routing, the norms before
// and after the block, and the 8-bit integer products.  Argument checks on the
// host, then one launch on the caller's stream.
#include "block.h"
#include "kernels.h"
#include "status.h"

using moe::aligned;
using moe::dt_ok;
using moe::fail;
using moe::hip_status;

namespace {

constexpr int32_t ROWS_MAX = 1 << 21;   // rows of a call (one workgroup of at most 1024 threads each)
constexpr int32_t K_MAX = 131056;       // 128 * 128 * K stays below 2^31
constexpr int64_t LD_MAX = 1ll << 22;   // row stride of 8-bit operands: 31-bit offsets inside a tile

// bytes [lo, hi) that a matrix of `rows` rows touches
struct Span {
    uintptr_t lo, hi;
};
Span span(const void* p, int64_t rows, int64_t ld, int64_t cols, int es) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    if (!p || rows < 1) return {0, 0};
    return {b, b + static_cast<uintptr_t>(((rows - 1) * ld + cols) * es)};
}
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
int esize(int32_t dt) { return dt == MOE_F32 ? 4 : 2; }

// Rows of ld elements that no address space holds (2^48 bytes and more): refused, so
// that the byte counts of a span stay inside 64 bits.
bool beyond(int64_t rows, int64_t ld) { return rows > 1 && ld > (1ll << 46) / rows; }

// a row-major matrix read or written in 16-byte pieces
moe_status check_rows(const char* fn, const char* name, const void* p, int32_t rows, int64_t ld, int32_t cols, int es) {
    if (ld < cols) return fail(MOE_E_SHAPE, fn, "row stride %lld of %s is below %d", static_cast<long long>(ld), name, cols);
    if (ld >= (1ll << 40) || beyond(rows, ld)) return fail(MOE_E_SHAPE, fn, "row stride of %s too large", name);
    if (!aligned(p, 16) || ld * es % 16)
        return fail(MOE_E_ARG, fn, "rows of %s must be 16-byte aligned", name);
    return MOE_OK;
}
moe_status check_h(const char* fn, const char* name, int32_t T, int32_t H) {
    if (T < 0 || T > ROWS_MAX) return fail(MOE_E_SHAPE, fn, "T=%d outside [0, %d]", T, ROWS_MAX);
    if (H < 8 || H % 8 || H > moe::NORM_H_MAX)
        return fail(MOE_E_SHAPE, fn, "%s=%d is not a multiple of 8 in [8, %d]", name, H, moe::NORM_H_MAX);
    return MOE_OK;
}
// the outputs of a norm; spans of those that are written go to s[0..2]
moe_status check_norm_out(const char* fn, int32_t T, int32_t H, const moe::NormOut& o, Span* s) {
    moe_status st;
    if (!(o.eps > 0.0f) || !(o.eps < 1e30f)) return fail(MOE_E_ARG, fn, "eps is not a positive number");
    if (o.w_offset != o.w_offset) return fail(MOE_E_ARG, fn, "w_offset is NaN");
    if (o.w && !dt_ok(o.w_dt)) return fail(MOE_E_ARG, fn, "unknown weight dtype %d", o.w_dt);
    if (o.w && !aligned(o.w, 16)) return fail(MOE_E_ARG, fn, "the norm's weight is not 16-byte aligned");
    if (!o.x && !o.xq) return fail(MOE_E_ARG, fn, "neither x nor xq is given");
    if ((o.xq == nullptr) != (o.xq_scale == nullptr)) return fail(MOE_E_ARG, fn, "xq and xq_scale go together");
    if (o.x) {
        if (!dt_ok(o.x_dt)) return fail(MOE_E_ARG, fn, "unknown dtype %d of x", o.x_dt);
        if ((st = check_rows(fn, "x", o.x, T, o.ldx, H, esize(o.x_dt))) != MOE_OK) return st;
    }
    if (o.xq) {
        if (o.ldq < H || o.ldq > LD_MAX)
            return fail(MOE_E_SHAPE, fn, "row stride %lld of xq outside [%d, 2^22]", static_cast<long long>(o.ldq), H);
        if (!aligned(o.xq, 8) || o.ldq % 8) return fail(MOE_E_ARG, fn, "rows of xq must be 8-byte aligned");
        if (!aligned(o.xq_scale, 4)) return fail(MOE_E_ARG, fn, "xq_scale is not 4-byte aligned");
    }
    s[0] = span(o.x, T, o.ldx, H, esize(o.x_dt));
    s[1] = span(o.xq, T, o.ldq, H, 1);
    s[2] = span(o.xq_scale, T, 1, 1, 4);
    return MOE_OK;
}
// no two outputs meet, and no output meets an input
moe_status check_apart(const char* fn, const Span* in, int n_in, const Span* out, int n_out) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return fail(MOE_E_ARG, fn, "two outputs overlap");
        for (int j = 0; j < n_in; ++j)
            if (meet(out[i], in[j])) return fail(MOE_E_ARG, fn, "an output overlaps an input");
    }
    return MOE_OK;
}

}  // namespace

extern "C" {

static moe_status check_score(const char* fn, int32_t T, int32_t E, int32_t k, int32_t score, int32_t n_group,
                              int32_t topk_group, int32_t group_rank, float scale) {
    if (T < 0) return fail(MOE_E_SHAPE, fn, "T=%d < 0", T);
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return fail(MOE_E_ARG, fn, "unknown score %d", score);
    if (group_rank != MOE_GROUP_MAX && group_rank != MOE_GROUP_TOP2)
        return fail(MOE_E_ARG, fn, "unknown group rank %d", group_rank);
    if (E < 1 || E > 512) return fail(MOE_E_SHAPE, fn, "E=%d outside [1, 512]", E);
    if (n_group < 1 || n_group > 64 || E % n_group)
        return fail(MOE_E_SHAPE, fn, "n_group=%d is not a divisor of E=%d in [1, 64]", n_group, E);
    if (topk_group < 1 || topk_group > n_group)
        return fail(MOE_E_SHAPE, fn, "topk_group=%d outside [1, n_group=%d]", topk_group, n_group);
    const int32_t open = E / n_group * topk_group;
    if (k < 1 || k > 32 || k > open)
        return fail(MOE_E_SHAPE, fn, "k=%d outside [1, min(%d experts of the kept groups, 32)]", k, open);
    if (T > (1 << 24) || static_cast<int64_t>(T) * k > (1ll << 30)) return fail(MOE_E_SHAPE, fn, "T=%d or T*k too large", T);
    if (!(scale - scale == 0.0f)) return fail(MOE_E_ARG, fn, "scale is not finite");
    return MOE_OK;
}

static moe::ScoreRouteParams score_params(const float* bias, int32_t T, int32_t E, int32_t k, int32_t score, int32_t n_group,
                                          int32_t topk_group, int32_t group_rank, int32_t renorm, float scale,
                                          int32_t* topk_ids, float* topk_w) {
    moe::ScoreRouteParams p{};
    p.bias = bias;
    p.T = T; p.E = E; p.k = k;
    p.sigmoid = score == MOE_SCORE_SIGMOID;
    p.n_group = n_group;
    p.topk_group = topk_group;
    p.top2 = group_rank == MOE_GROUP_TOP2;
    p.renorm = renorm;
    p.scale = scale;
    p.ids = topk_ids;
    p.w = topk_w;
    return p;
}

moe_status moe_route_score_topk(const void* logits, int32_t logits_dtype, int64_t ld_logits, const float* bias, int32_t T,
                                int32_t E, int32_t k, int32_t score, int32_t n_group, int32_t topk_group,
                                int32_t group_rank, int32_t renorm, float scale, int32_t* topk_ids, float* topk_w,
                                void* stream) {
    const char* fn = "moe_route_score_topk";
    moe_status st = check_score(fn, T, E, k, score, n_group, topk_group, group_rank, scale);
    if (st != MOE_OK) return st;
    if (T > 0 && (!logits || !topk_ids || !topk_w)) return fail(MOE_E_ARG, fn, "null pointer argument");
    if (!dt_ok(logits_dtype)) return fail(MOE_E_ARG, fn, "unknown dtype %d", logits_dtype);
    if (ld_logits < E || ld_logits >= (1ll << 40) || beyond(T, ld_logits))
        return fail(MOE_E_SHAPE, fn, "row stride %lld of logits is below E=%d or too large", static_cast<long long>(ld_logits), E);
    if (!aligned(logits, esize(logits_dtype)) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
        return fail(MOE_E_ARG, fn, "a pointer is not aligned to its elements");
    const Span in[2] = {span(logits, T, ld_logits, E, esize(logits_dtype)), span(bias, 1, E, E, 4)};
    const Span out[2] = {span(topk_ids, T, k, k, 4), span(topk_w, T, k, k, 4)};
    st = check_apart(fn, in, 2, out, 2);
    if (st != MOE_OK || T == 0) return st;
    moe::ScoreRouteParams p = score_params(bias, T, E, k, score, n_group, topk_group, group_rank, renorm, scale, topk_ids, topk_w);
    p.logits = logits;
    p.logits_dt = logits_dtype;
    p.ld = ld_logits;
    return hip_status(fn, moe::launch_route_score(p, static_cast<hipStream_t>(stream)));
}

moe_status moe_router_score_topk(const void* x, int32_t x_dtype, int32_t T, int32_t H, const float* w_router, int32_t E,
                                 int32_t k, const float* bias, int32_t score, int32_t n_group, int32_t topk_group,
                                 int32_t group_rank, int32_t renorm, float scale, float* logits, void* ws, size_t ws_bytes,
                                 int32_t* topk_ids, float* topk_w, void* stream) {
    const char* fn = "moe_router_score_topk";
    moe_status st = check_score(fn, T, E, k, score, n_group, topk_group, group_rank, scale);
    if (st != MOE_OK) return st;
    if (T > 0 && (!x || !w_router || !logits || !ws || !topk_ids || !topk_w))
        return fail(MOE_E_ARG, fn, "null pointer argument");
    if (!dt_ok(x_dtype)) return fail(MOE_E_ARG, fn, "unknown dtype %d", x_dtype);
    if (H < 64 || H % 64) return fail(MOE_E_SHAPE, fn, "H=%d is not a positive multiple of 64", H);
    if (T > moe::ROUTER_T_MAX || static_cast<int64_t>(T) * H >= (1ll << 31) || moe::router_part_floats(T, H, E) >= (1ll << 31))
        return fail(MOE_E_SHAPE, fn, "T=%d too large", T);
    if (T == 0) return MOE_OK;
    if (ws_bytes < moe_router_ws_bytes(T, H, E))
        return fail(MOE_E_WORKSPACE, fn, "ws_bytes=%zu < %zu", ws_bytes, moe_router_ws_bytes(T, H, E));
    if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(ws, 16))
        return fail(MOE_E_ARG, fn, "x, w_router and ws must be 16-byte aligned");
    if (!aligned(bias, 4) || !aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
        return fail(MOE_E_ARG, fn, "a pointer is not aligned to its elements");
    const Span in[3] = {span(x, T, H, H, esize(x_dtype)), span(w_router, E, H, H, 4), span(bias, 1, E, E, 4)};
    const Span out[4] = {span(topk_ids, T, k, k, 4), span(topk_w, T, k, k, 4), span(logits, T, E, E, 4),
                         span(ws, 1, 1, static_cast<int64_t>(moe_router_ws_bytes(T, H, E)), 1)};
    if ((st = check_apart(fn, in, 3, out, 4)) != MOE_OK) return st;
    const moe::ScoreRouteParams p =
        score_params(bias, T, E, k, score, n_group, topk_group, group_rank, renorm, scale, topk_ids, topk_w);
    return hip_status(fn, moe::launch_router_score(x, x_dtype == MOE_F32, w_router, H, logits, static_cast<float*>(ws), p,
                                                   static_cast<hipStream_t>(stream)));
}

moe_status moe_norm_in(const void* h, int32_t h_dtype, int64_t ldh, int32_t T, int32_t H, const void* w, int32_t w_dtype,
                       float w_offset, float eps, void* x, int32_t x_dtype, int64_t ldx, int8_t* xq, int64_t ldq,
                       float* xq_scale, void* stream) {
    const char* fn = "moe_norm_in";
    moe_status st = check_h(fn, "H", T, H);
    if (st != MOE_OK || T == 0) return st;
    if (!h) return fail(MOE_E_ARG, fn, "h is NULL");
    if (!dt_ok(h_dtype)) return fail(MOE_E_ARG, fn, "unknown dtype %d of h", h_dtype);
    if ((st = check_rows(fn, "h", h, T, ldh, H, esize(h_dtype))) != MOE_OK) return st;
    const moe::NormOut o = {w, w_dtype, w_offset, eps, x, x_dtype, ldx, xq, ldq, xq_scale};
    Span out[3];
    if ((st = check_norm_out(fn, T, H, o, out)) != MOE_OK) return st;
    const Span in[2] = {span(h, T, ldh, H, esize(h_dtype)), span(w, 1, H, H, esize(w_dtype))};
    if ((st = check_apart(fn, in, 2, out, 3)) != MOE_OK) return st;
    return hip_status(fn, moe::launch_norm_in(h, h_dtype, ldh, T, H, o, static_cast<hipStream_t>(stream)));
}

moe_status moe_quantize_tokens(const void* x, int32_t x_dtype, int64_t ldx, int32_t T, int32_t K, int8_t* xq, int64_t ldq,
                               float* xq_scale, void* stream) {
    const char* fn = "moe_quantize_tokens";
    moe_status st = check_h(fn, "K", T, K);
    if (st != MOE_OK || T == 0) return st;
    if (!x || !xq || !xq_scale) return fail(MOE_E_ARG, fn, "null pointer argument");
    if (!dt_ok(x_dtype)) return fail(MOE_E_ARG, fn, "unknown dtype %d", x_dtype);
    if ((st = check_rows(fn, "x", x, T, ldx, K, esize(x_dtype))) != MOE_OK) return st;
    const moe::NormOut o = {nullptr, MOE_F32, 0.0f, 1.0f, nullptr, MOE_F32, 0, xq, ldq, xq_scale};
    Span out[3];
    if ((st = check_norm_out(fn, T, K, o, out)) != MOE_OK) return st;
    const Span in[1] = {span(x, T, ldx, K, esize(x_dtype))};
    if ((st = check_apart(fn, in, 1, out, 3)) != MOE_OK) return st;
    return hip_status(fn, moe::launch_quantize_tokens(x, x_dtype, ldx, T, K, xq, ldq, xq_scale,
                                                      static_cast<hipStream_t>(stream)));
}

moe_status moe_norm_out(const void* out_routes, int32_t out_dtype, const float* topk_w, const int32_t* route_pos, int32_t k,
                        const void* y, int32_t y_dtype, int64_t ldy, int32_t T, int32_t H, const void* w_post,
                        int32_t w_dtype, float w_offset, float eps, const void* gate, int32_t gate_dtype,
                        int64_t gate_stride_t, int64_t gate_stride_h, float block_scale, float res_scale, const void* h,
                        int32_t h_dtype, int64_t ldh, void* h_out, int64_t ldho, int32_t next_norm, const void* w_next,
                        void* x, int32_t x_dtype, int64_t ldx, int8_t* xq, int64_t ldq, float* xq_scale, void* stream) {
    const char* fn = "moe_norm_out";
    moe_status st = check_h(fn, "H", T, H);
    if (st != MOE_OK) return st;
    if (k < 0 || k > 32) return fail(MOE_E_SHAPE, fn, "k=%d outside [0, 32]", k);
    if (T == 0) return MOE_OK;
    if (!h || !h_out) return fail(MOE_E_ARG, fn, "h or h_out is NULL");
    if (k > 0 && (!out_routes || !topk_w || !route_pos)) return fail(MOE_E_ARG, fn, "null pointer argument of the routes");
    if (k == 0 && !y) return fail(MOE_E_ARG, fn, "neither routes nor y are given");
    if (!dt_ok(h_dtype) || (k > 0 && !dt_ok(out_dtype)) || (y && !dt_ok(y_dtype)) || (w_post && !dt_ok(w_dtype)) ||
        (gate && !dt_ok(gate_dtype)))
        return fail(MOE_E_ARG, fn, "unknown dtype");
    if (static_cast<int64_t>(T) * k > (1ll << 30)) return fail(MOE_E_SHAPE, fn, "T*k too large");
    if (!(eps > 0.0f) || !(eps < 1e30f)) return fail(MOE_E_ARG, fn, "eps is not a positive number");
    if (w_offset != w_offset || block_scale != block_scale || res_scale != res_scale)
        return fail(MOE_E_ARG, fn, "w_offset or a scale is NaN");
    const int he = esize(h_dtype);
    if ((st = check_rows(fn, "h", h, T, ldh, H, he)) != MOE_OK) return st;
    if ((st = check_rows(fn, "h_out", h_out, T, ldho, H, he)) != MOE_OK) return st;
    if (k > 0 && (!aligned(out_routes, 16) || !aligned(topk_w, 4) || !aligned(route_pos, 4)))
        return fail(MOE_E_ARG, fn, "out_routes must be 16-byte aligned, topk_w and route_pos 4-byte aligned");
    if (y && (st = check_rows(fn, "y", y, T, ldy, H, esize(y_dtype))) != MOE_OK) return st;
    if (w_post && !aligned(w_post, 16)) return fail(MOE_E_ARG, fn, "w_post is not 16-byte aligned");
    Span gs = {0, 0};
    if (gate) {
        if (gate_stride_h != 0 && gate_stride_h != 1)
            return fail(MOE_E_UNSUPPORTED, fn, "gate stride %lld along H is neither 0 nor 1", static_cast<long long>(gate_stride_h));
        if (gate_stride_t < 0 || gate_stride_t >= (1ll << 40) || beyond(T, gate_stride_t))
            return fail(MOE_E_SHAPE, fn, "gate stride along T is negative or too large");
        const int ge = esize(gate_dtype);
        if (!aligned(gate, gate_stride_h ? 16 : ge) || (gate_stride_h && gate_stride_t * ge % 16))
            return fail(MOE_E_ARG, fn, "rows of gate must be 16-byte aligned");
        gs = span(gate, T, gate_stride_t, gate_stride_h ? H : 1, ge);
    }
    moe::NormOutParams p{};
    Span out[4] = {};
    if (next_norm) {
        p.n = moe::NormOut{w_next, w_dtype, w_offset, eps, x, x_dtype, ldx, xq, ldq, xq_scale};
        if ((st = check_norm_out(fn, T, H, p.n, out)) != MOE_OK) return st;
    } else if (x || xq || xq_scale) {
        return fail(MOE_E_ARG, fn, "x, xq and xq_scale are outputs of the next norm (next_norm)");
    }
    out[3] = span(h_out, T, ldho, H, he);
    // h_out may be h itself (a row is read before it is written), and nothing else that is read
    const bool same = h_out == h && ldho == ldh;
    const Span hs = same ? Span{0, 0} : span(h, T, ldh, H, he);
    const int64_t R = static_cast<int64_t>(T) * k;
    const Span in[7] = {hs, gs, span(y, T, ldy, H, esize(y_dtype)), span(w_post, 1, H, H, esize(w_dtype)),
                        span(next_norm ? w_next : nullptr, 1, H, H, esize(w_dtype)), span(k > 0 ? topk_w : nullptr, R, 1, 1, 4),
                        span(k > 0 ? route_pos : nullptr, R, 1, 1, 4)};
    if ((st = check_apart(fn, in, 7, out, 4)) != MOE_OK) return st;
    const Span rt[1] = {span(k > 0 ? out_routes : nullptr, R, H, H, esize(out_dtype))};
    if ((st = check_apart(fn, rt, 1, out, 4)) != MOE_OK) return st;
    p.out_routes = out_routes;
    p.out_dt = k > 0 ? out_dtype : MOE_F32;
    p.topk_w = topk_w;
    p.route_pos = route_pos;
    p.k = k;
    p.y = y;
    p.y_dt = y_dtype;
    p.ldy = ldy;
    p.T = T; p.H = H;
    p.w_post = w_post;
    p.w_dt = w_dtype;
    p.w_offset = w_offset;
    p.eps = eps;
    p.gate = gate;
    p.gate_dt = gate_dtype;
    p.gate_st = gate_stride_t;
    p.gate_sh = gate_stride_h;
    p.block_scale = block_scale;
    p.res_scale = res_scale;
    p.h = h;
    p.h_dt = h_dtype;
    p.ldh = ldh;
    p.h_out = h_out;
    p.ldho = ldho;
    p.next = next_norm != 0;
    return hip_status(fn, moe::launch_norm_out(p, static_cast<hipStream_t>(stream)));
}

static moe_status matmul_entry(const char* fn, bool gated, const int8_t* xq, int64_t ldx, const float* x_scale,
                               const int8_t* wq, int64_t ldw, const float* w_scale, const float* bias, int32_t T, int32_t N,
                               int32_t K, int32_t act, void* out, int32_t out_dtype, int64_t ldo, void* stream) {
    if (T < 0) return fail(MOE_E_SHAPE, fn, "T=%d < 0", T);
    if (N < 1 || N > (1 << 24)) return fail(MOE_E_SHAPE, fn, "N=%d outside [1, 2^24]", N);
    if (K < 16 || K % 16 || K > K_MAX) return fail(MOE_E_SHAPE, fn, "K=%d is not a multiple of 16 in [16, %d]", K, K_MAX);
    if (T == 0) return MOE_OK;
    if (!xq || !x_scale || !wq || !w_scale || !out) return fail(MOE_E_ARG, fn, "null pointer argument");
    if (!dt_ok(out_dtype)) return fail(MOE_E_ARG, fn, "unknown dtype %d", out_dtype);
    if (gated && act != MOE_ACT_GELU_TANH && act != MOE_ACT_SILU) return fail(MOE_E_ARG, fn, "unknown activation %d", act);
    if (ldx < K || ldw < K || ldx > LD_MAX || ldw > LD_MAX)
        return fail(MOE_E_SHAPE, fn, "row strides %lld of xq and %lld of wq must lie in [K=%d, 2^22]",
                    static_cast<long long>(ldx), static_cast<long long>(ldw), K);
    if (ldo < N || ldo >= (1ll << 40) || beyond(T, ldo))
        return fail(MOE_E_SHAPE, fn, "row stride %lld of out is below N=%d or too large", static_cast<long long>(ldo), N);
    if (!aligned(xq, 16) || !aligned(wq, 16) || ldx % 16 || ldw % 16)
        return fail(MOE_E_ARG, fn, "rows of xq and wq must be 16-byte aligned");
    if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(out, esize(out_dtype)))
        return fail(MOE_E_ARG, fn, "a pointer is not aligned to its elements");
    if (T > (1 << 24) || static_cast<int64_t>(T) * N > (1ll << 36))
        return fail(MOE_E_SHAPE, fn, "T=%d N=%d too large (T <= 2^24, T*N <= 2^36)", T, N);
    const int64_t rows = gated ? 2ll * N : N;
    const Span in[5] = {span(xq, T, ldx, K, 1), span(wq, rows, ldw, K, 1), span(x_scale, T, 1, 1, 4),
                        span(w_scale, rows, 1, 1, 4), span(bias, N, 1, 1, 4)};
    const Span o[1] = {span(out, T, ldo, N, esize(out_dtype))};
    const moe_status st = check_apart(fn, in, 5, o, 1);
    if (st != MOE_OK) return st;
    const moe::MatI8Params p = {xq, ldx, x_scale, wq, ldw, w_scale, bias, T, N, K, act, out, out_dtype, ldo};
    return hip_status(fn, moe::launch_matmul_i8(p, gated, static_cast<hipStream_t>(stream)));
}

moe_status moe_matmul_i8(const int8_t* xq, int64_t ldx, const float* x_scale, const int8_t* wq, int64_t ldw,
                         const float* w_scale, const float* bias, int32_t T, int32_t N, int32_t K, void* out,
                         int32_t out_dtype, int64_t ldo, void* stream) {
    return matmul_entry("moe_matmul_i8", false, xq, ldx, x_scale, wq, ldw, w_scale, bias, T, N, K, 0, out, out_dtype, ldo,
                        stream);
}

moe_status moe_gated_matmul_i8(const int8_t* xq, int64_t ldx, const float* x_scale, const int8_t* wq, int64_t ldw,
                               const float* w_scale, int32_t T, int32_t F, int32_t K, int32_t act, void* out,
                               int32_t out_dtype, int64_t ldo, void* stream) {
    return matmul_entry("moe_gated_matmul_i8", true, xq, ldx, x_scale, wq, ldw, w_scale, nullptr, T, F, K, act, out,
                        out_dtype, ldo, stream);
}

}  // extern "C"
