// C ABI of the bfloat16 products, their backward passes and the low-rank adapters
// beside them.  Argument checks on the host, then the launches on the caller's stream.
#include "block.h"
#include "checks.h"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int32_t K_MAX = 1 << 20;
constexpr int64_t LD_MAX = 1ll << 21;   // row stride of a tile's operand: 256 rows below 2 GiB
constexpr int32_t ROWS_MAX = 1 << 24;
constexpr int32_t RANK_MAX = 1024;
constexpr int64_t OUT_MAX = 1ll << 36;  // elements of a result: every launch below 2^32 threads

// an operand of the tiles: bf16 rows in 16-byte pieces
moe_status check_operand(const char* fn, const char* name, const void* p, int64_t ld, int64_t cols) {
    if (ld < cols || ld > LD_MAX)
        return fail(MOE_E_SHAPE, fn, "row stride %lld of %s outside [%lld, 2^21]", static_cast<long long>(ld), name,
                    static_cast<long long>(cols));
    if (!aligned(p, 16) || ld % 8) return fail(MOE_E_ARG, fn, "rows of %s must be 16-byte aligned", name);
    return MOE_OK;
}
// a result, stored at any alignment of its elements
moe_status check_result(const char* fn, const char* name, const void* p, int32_t dt, int64_t rows, int64_t ld, int64_t cols) {
    if (!dt_ok(dt)) return fail(MOE_E_ARG, fn, "unknown dtype %d of %s", dt, name);
    if (ld < cols || ld >= (1ll << 40) || beyond(rows, ld))
        return fail(MOE_E_SHAPE, fn, "row stride %lld of %s is below %lld or too large", static_cast<long long>(ld), name,
                    static_cast<long long>(cols));
    if (!aligned(p, esize(dt))) return fail(MOE_E_ARG, fn, "%s is not aligned to its elements", name);
    return MOE_OK;
}
moe_status check_sizes(const char* fn, const char* name, int32_t T, int32_t N, int32_t K) {
    if (T < 0 || T > ROWS_MAX) return fail(MOE_E_SHAPE, fn, "T=%d outside [0, 2^24]", T);
    if (N < 1 || N > ROWS_MAX) return fail(MOE_E_SHAPE, fn, "%s=%d outside [1, 2^24]", name, N);
    if (K < 8 || K % 8 || K > K_MAX) return fail(MOE_E_SHAPE, fn, "K=%d is not a multiple of 8 in [8, 2^20]", K);
    if (static_cast<int64_t>(T) * N > OUT_MAX) return fail(MOE_E_SHAPE, fn, "T=%d %s=%d too large (T*%s <= 2^36)", T, name, N, name);
    return MOE_OK;
}
bool act_ok(int32_t act) { return act == MOE_ACT_GELU_TANH || act == MOE_ACT_SILU; }

// a pool of n adapters, each `each` contiguous elements
moe_status check_pool(const char* fn, const char* name, const void* p, int64_t stride, int32_t n, int32_t R, int64_t each) {
    if (n < 1 || n > ROWS_MAX) return fail(MOE_E_SHAPE, fn, "n_adapters=%d outside [1, 2^24]", n);
    if (R < 8 || R % 8 || R > RANK_MAX) return fail(MOE_E_SHAPE, fn, "R=%d is not a multiple of 8 in [8, %d]", R, RANK_MAX);
    if (!p) return fail(MOE_E_ARG, fn, "null pointer argument");
    if ((n > 1 && stride < each) || stride < 0 || stride >= (1ll << 40) || beyond(n, stride))
        return fail(MOE_E_SHAPE, fn, "stride %lld of %s is below an adapter's %lld elements or too large",
                    static_cast<long long>(stride), name, static_cast<long long>(each));
    if (!aligned(p, 16) || (n > 1 && stride % 8)) return fail(MOE_E_ARG, fn, "the adapters of %s must be 16-byte aligned", name);
    return MOE_OK;
}

moe_status product_entry(const char* fn, bool gated, const void* x, int64_t ldx, const void* w, int64_t ldw, int32_t T, int32_t N,
                         int32_t K, int32_t act, void* out, int32_t out_dtype, int64_t ldo, void* pre, int64_t ldp, const void* s,
                         int64_t lds, const int32_t* ids, const void* b, int64_t b_stride, const int32_t* ranks, int32_t n,
                         int32_t R, void* stream) {
    moe_status st = check_sizes(fn, gated ? "F" : "N", T, N, K);
    if (st != MOE_OK) return st;
    if (gated && !act_ok(act)) return fail(MOE_E_ARG, fn, "unknown activation %d", act);
    if (T == 0) return MOE_OK;
    if (!x || !w || !out) return fail(MOE_E_ARG, fn, "null pointer argument");
    if ((st = check_operand(fn, "x", x, ldx, K)) != MOE_OK) return st;
    if ((st = check_operand(fn, "w", w, ldw, K)) != MOE_OK) return st;
    if ((st = check_result(fn, "out", out, out_dtype, T, ldo, N)) != MOE_OK) return st;
    if (pre && (st = check_result(fn, "pre", pre, MOE_BF16, T, ldp, 2ll * N)) != MOE_OK) return st;
    const int64_t rows = gated ? 2ll * N : N;
    const int32_t halves = gated ? 2 : 1;
    Span as[4] = {};
    if (s) {
        if (!ids) return fail(MOE_E_ARG, fn, "null pointer argument");
        if ((st = check_pool(fn, "b", b, b_stride, n, R, rows * R)) != MOE_OK) return st;
        if ((st = check_operand(fn, "s", s, lds, static_cast<int64_t>(halves) * R)) != MOE_OK) return st;
        if (!aligned(ids, 4) || !aligned(ranks, 4)) return fail(MOE_E_ARG, fn, "adapter_ids or ranks is not 4-byte aligned");
        as[0] = span(s, T, lds, static_cast<int64_t>(halves) * R, 2);
        as[1] = span(ids, T, 1, 1, 4);
        as[2] = span(b, n, b_stride, rows * R, 2);
        as[3] = span(ranks, n, 1, 1, 4);
    } else if (ids || b || ranks) {
        return fail(MOE_E_ARG, fn, "adapter_ids, b and ranks go with s");
    }
    const Span in[6] = {span(x, T, ldx, K, 2), span(w, rows, ldw, K, 2), as[0], as[1], as[2], as[3]};
    const Span o[2] = {span(out, T, ldo, N, esize(out_dtype)), span(pre, T, ldp, 2ll * N, 2)};
    if ((st = check_apart(fn, in, 6, o, 2)) != MOE_OK) return st;
    MatBf16Params p{};
    p.x = static_cast<const uint16_t*>(x);
    p.ldx = ldx;
    p.w = static_cast<const uint16_t*>(w);
    p.ldw = ldw;
    p.T = T; p.N = N; p.K = K;
    p.act = act;
    p.out = out;
    p.out_dt = out_dtype;
    p.ldo = ldo;
    p.pre = static_cast<uint16_t*>(pre);
    p.ldp = ldp;
    if (s) p.ad = AdapterParams{static_cast<const uint16_t*>(s), lds, ids, static_cast<const uint16_t*>(b), b_stride, ranks, n, R};
    return hip_status(fn, launch_matmul_bf16(p, gated ? MAT_GATED : MAT_NT, static_cast<hipStream_t>(stream)));
}

// What dx and dw are checked for: the operands that they read and where they go.  d: the
// gradient of the sums, [T, M].
struct Gradients {
    const void *x, *w, *d;
    int64_t ldx, ldw, ldd;
    int32_t T, M, K;
    void *dx, *dw;
    int32_t dx_dt, dw_dt;
    int64_t lddx, lddw;
};
moe_status check_gradients(const char* fn, const Gradients& g) {
    moe_status st;
    if (g.dx) {
        if (static_cast<int64_t>(g.T) * g.K > OUT_MAX)
            return fail(MOE_E_SHAPE, fn, "T=%d K=%d of dx too large (T*K <= 2^36)", g.T, g.K);
        if (g.T > 0 && !g.w) return fail(MOE_E_ARG, fn, "null pointer argument");
        if ((st = check_operand(fn, "w", g.w, g.ldw, g.K)) != MOE_OK) return st;
        if ((st = check_result(fn, "dx", g.dx, g.dx_dt, g.T, g.lddx, g.K)) != MOE_OK) return st;
    }
    if (g.dw) {
        if (static_cast<int64_t>(g.M) * g.K > OUT_MAX)
            return fail(MOE_E_SHAPE, fn, "%d rows and K=%d of dw too large (rows * K <= 2^36)", g.M, g.K);
        if (g.T > 0 && !g.x) return fail(MOE_E_ARG, fn, "null pointer argument");
        if ((st = check_operand(fn, "x", g.x, g.ldx, g.K)) != MOE_OK) return st;
        if ((st = check_result(fn, "dw", g.dw, g.dw_dt, g.M, g.lddw, g.K)) != MOE_OK) return st;
    }
    return MOE_OK;
}
hipError_t launch_gradients(const Gradients& g, hipStream_t s) {
    MatBf16Params rows{}, weights{};
    rows.x = weights.x = static_cast<const uint16_t*>(g.d);
    rows.ldx = weights.ldx = g.ldd;
    rows.N = weights.N = g.K;
    rows.T = weights.K = g.T;
    rows.K = weights.T = g.M;
    rows.w = static_cast<const uint16_t*>(g.w);
    rows.ldw = g.ldw;
    rows.out = g.dx;
    rows.out_dt = g.dx_dt;
    rows.ldo = g.lddx;
    weights.w = static_cast<const uint16_t*>(g.x);
    weights.ldw = g.ldx;
    weights.out = g.dw;
    weights.out_dt = g.dw_dt;
    weights.ldo = g.lddw;
    const bool dx = g.dx && g.T > 0;   // (without tokens dw is zeros, and dx has no rows)
    if (dx && g.dw) return launch_matmul_bf16_pair(rows, weights, s);
    if (dx) return launch_matmul_bf16(rows, MAT_NN, s);
    return g.dw ? launch_matmul_bf16(weights, MAT_TN, s) : hipSuccess;
}

}  // namespace

extern "C" {

moe_status moe_matmul_bf16(const void* x, int64_t ldx, const void* w, int64_t ldw, int32_t T, int32_t N, int32_t K, void* out,
                           int32_t out_dtype, int64_t ldo, const void* s, int64_t lds, const int32_t* adapter_ids,
                           const void* b, int64_t b_stride, const int32_t* ranks, int32_t n_adapters, int32_t R, void* stream) {
    return product_entry("moe_matmul_bf16", false, x, ldx, w, ldw, T, N, K, 0, out, out_dtype, ldo, nullptr, 0, s, lds, adapter_ids,
                         b, b_stride, ranks, n_adapters, R, stream);
}

moe_status moe_gated_matmul_bf16(const void* x, int64_t ldx, const void* w, int64_t ldw, int32_t T, int32_t F, int32_t K,
                                 int32_t act, void* out, int32_t out_dtype, int64_t ldo, void* pre, int64_t ldp,
                                 const void* s, int64_t lds, const int32_t* adapter_ids, const void* b, int64_t b_stride,
                                 const int32_t* ranks, int32_t n_adapters, int32_t R, void* stream) {
    return product_entry("moe_gated_matmul_bf16", true, x, ldx, w, ldw, T, F, K, act, out, out_dtype, ldo, pre, ldp, s, lds,
                         adapter_ids, b, b_stride, ranks, n_adapters, R, stream);
}

moe_status moe_adapter_shrink(const void* x, int64_t ldx, int32_t T, int32_t K, const int32_t* adapter_ids,
                              const void* a_pool, int64_t a_stride, int32_t n_adapters, int32_t R, int32_t halves,
                              const float* scale, const int32_t* ranks, void* s, int64_t lds, void* stream) {
    const char* fn = "moe_adapter_shrink";
    moe_status st = check_sizes(fn, "R", T, R, K);
    if (st != MOE_OK) return st;
    if (halves != 1 && halves != 2) return fail(MOE_E_ARG, fn, "halves=%d is neither 1 nor 2", halves);
    if (T == 0) return MOE_OK;
    if (!x || !adapter_ids || !s) return fail(MOE_E_ARG, fn, "null pointer argument");
    const int64_t each = static_cast<int64_t>(halves) * R;
    if ((st = check_pool(fn, "a_pool", a_pool, a_stride, n_adapters, R, each * K)) != MOE_OK) return st;
    if ((st = check_operand(fn, "x", x, ldx, K)) != MOE_OK) return st;
    if ((st = check_operand(fn, "s", s, lds, each)) != MOE_OK) return st;
    if (!aligned(adapter_ids, 4) || !aligned(scale, 4) || !aligned(ranks, 4))
        return fail(MOE_E_ARG, fn, "adapter_ids, scale or ranks is not 4-byte aligned");
    const Span in[5] = {span(x, T, ldx, K, 2), span(adapter_ids, T, 1, 1, 4), span(a_pool, n_adapters, a_stride, each * K, 2),
                        span(scale, n_adapters, 1, 1, 4), span(ranks, n_adapters, 1, 1, 4)};
    const Span o[1] = {span(s, T, lds, each, 2)};
    if ((st = check_apart(fn, in, 5, o, 1)) != MOE_OK) return st;
    const AdapterShrinkParams p = {static_cast<const uint16_t*>(x), ldx, adapter_ids, static_cast<const uint16_t*>(a_pool), a_stride,
                                   scale, ranks, T, K, n_adapters, R, halves, static_cast<uint16_t*>(s), lds};
    return hip_status(fn, launch_adapter_shrink(p, static_cast<hipStream_t>(stream)));
}

moe_status moe_matmul_bf16_backward(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* dout, int64_t ldd,
                                    int32_t T, int32_t N, int32_t K, void* dx, int32_t dx_dtype, int64_t lddx, void* dw,
                                    int32_t dw_dtype, int64_t lddw, void* stream) {
    const char* fn = "moe_matmul_bf16_backward";
    moe_status st = check_sizes(fn, "N", T, N, K);
    if (st != MOE_OK) return st;
    if (N % 8) return fail(MOE_E_SHAPE, fn, "N=%d is not a multiple of 8", N);
    if (!dx && !dw) return fail(MOE_E_ARG, fn, "neither dx nor dw is given");
    if (T > 0 && !dout) return fail(MOE_E_ARG, fn, "null pointer argument");
    if ((st = check_operand(fn, "dout", dout, ldd, N)) != MOE_OK) return st;
    const Gradients g = {x, w, dout, ldx, ldw, ldd, T, N, K, dx, dw, dx_dtype, dw_dtype, lddx, lddw};
    if ((st = check_gradients(fn, g)) != MOE_OK) return st;
    const Span in[3] = {span(dw ? x : nullptr, T, ldx, K, 2), span(dx ? w : nullptr, N, ldw, K, 2), span(dout, T, ldd, N, 2)};
    const Span o[2] = {span(dx, T, lddx, K, esize(dx_dtype)), span(dw, N, lddw, K, esize(dw_dtype))};
    if ((st = check_apart(fn, in, 3, o, 2)) != MOE_OK) return st;
    return hip_status(fn, launch_gradients(g, static_cast<hipStream_t>(stream)));
}

moe_status moe_gated_matmul_bf16_backward(const void* x, int64_t ldx, const void* w, int64_t ldw, int32_t act,
                                          const void* pre, int64_t ldp, const void* dout, int64_t ldd, int32_t T, int32_t F,
                                          int32_t K, void* dpre, int64_t ldg, void* dx, int32_t dx_dtype, int64_t lddx,
                                          void* dw, int32_t dw_dtype, int64_t lddw, void* stream) {
    const char* fn = "moe_gated_matmul_bf16_backward";
    moe_status st = check_sizes(fn, "F", T, F, K);
    if (st != MOE_OK) return st;
    if (F % 8) return fail(MOE_E_SHAPE, fn, "F=%d is not a multiple of 8", F);
    if (!act_ok(act)) return fail(MOE_E_ARG, fn, "unknown activation %d", act);
    if (T > 0 && (!pre || !dout || !dpre)) return fail(MOE_E_ARG, fn, "null pointer argument");
    const int64_t M = 2ll * F;
    if ((st = check_operand(fn, "pre", pre, ldp, M)) != MOE_OK) return st;
    if ((st = check_operand(fn, "dout", dout, ldd, F)) != MOE_OK) return st;
    if ((st = check_operand(fn, "dpre", dpre, ldg, M)) != MOE_OK) return st;
    const Gradients g = {x, w, dpre, ldx, ldw, ldg, T, static_cast<int32_t>(M), K, dx, dw, dx_dtype, dw_dtype, lddx, lddw};
    if ((st = check_gradients(fn, g)) != MOE_OK) return st;
    // dpre may be pre itself: a value is read before its gradient is written there
    const bool same = pre == dpre && ldp == ldg;
    const Span in[4] = {span(dw ? x : nullptr, T, ldx, K, 2), span(dx ? w : nullptr, M, ldw, K, 2), span(dout, T, ldd, F, 2),
                        same ? Span{0, 0} : span(pre, T, ldp, M, 2)};
    const Span o[3] = {span(dx, T, lddx, K, esize(dx_dtype)), span(dw, M, lddw, K, esize(dw_dtype)), span(dpre, T, ldg, M, 2)};
    if ((st = check_apart(fn, in, 4, o, 3)) != MOE_OK) return st;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (T > 0) {
        const GatedGradParams q = {static_cast<const uint16_t*>(pre), ldp, static_cast<const uint16_t*>(dout), ldd,
                                   static_cast<uint16_t*>(dpre), ldg, T, F, act};
        const hipError_t e = launch_gated_grad(q, hs);
        if (e != hipSuccess) return hip_status(fn, e);
    }
    return hip_status(fn, launch_gradients(g, hs));
}

}  // extern "C"
