// Launch functions of the operators around the expert FFN (internal; the C ABI
// is in include/expert_ffn.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// ------------------------------------------------------- scored routing --
struct ScoreRouteParams {
    const void* logits;     // [T, E] fp32 or bf16, rows ld elements apart
    int logits_dt;
    int64_t ld;
    const float* bias;      // [E] or null
    int T, E, k, sigmoid, n_group, topk_group, top2, renorm;
    float scale;
    int* ids;               // [T, k]
    float* w;               // [T, k]
};
hipError_t launch_route_score(const ScoreRouteParams& p, hipStream_t s);
constexpr int ROUTER_T_MAX = 65535 * 64;   // tokens of a router product: a grid row (z) per 64
// the router's product in slices of H: part fp32 [*HS][T][E] (router_part_floats in all), summed in slice order by the reader
hipError_t launch_router_part(const void* x, bool xf32, const float* wr, int T, int H, int E, float* part, int* HS,
                              hipStream_t s);
// the product, then the scored top-k of p (its logits, logits_dt and ld are not read); logits fp32 [T, E] out
hipError_t launch_router_score(const void* x, bool xf32, const float* wr, int H, float* logits, float* part,
                               const ScoreRouteParams& p, hipStream_t s);

// ---------------------------------------------------------------- norms --
// One row's outputs of a norm: x (null: none), 8-bit codes and their scale
// (null: none).  w null: no weight (the norm alone).
struct NormOut {
    const void* w;          // [H] fp32 or bf16
    int w_dt;
    float w_offset, eps;
    void* x;                // [T, H], rows ldx apart
    int x_dt;
    int64_t ldx;
    int8_t* xq;             // [T, H], rows ldq apart
    int64_t ldq;
    float* xq_scale;        // [T]
};
constexpr int NORM_H_MAX = 32768;
hipError_t launch_norm_in(const void* h, int h_dt, int64_t ldh, int T, int H, const NormOut& o, hipStream_t s);
// codes of the rows themselves (no norm)
hipError_t launch_quantize_tokens(const void* x, int x_dt, int64_t ldx, int T, int K, int8_t* q, int64_t ldq,
                                  float* scale, hipStream_t s);

struct NormOutParams {
    const void* out_routes; // [T*k, H] or null
    int out_dt;
    const float* topk_w;    // [T*k]
    const int* route_pos;   // [T*k]
    int k;
    const void* y;          // [T, H] or null
    int y_dt;
    int64_t ldy;
    int T, H;
    const void* w_post;     // [H] or null
    int w_dt;
    float w_offset, eps;
    const void* gate;       // element (t, h) at t * gate_st + h * gate_sh, or null
    int gate_dt;
    int64_t gate_st, gate_sh;
    float block_scale, res_scale;
    const void* h;          // [T, H]
    int h_dt;
    int64_t ldh;
    void* h_out;            // [T, H], may be h
    int64_t ldho;
    int next;               // the next norm is wanted
    NormOut n;
};
hipError_t launch_norm_out(const NormOutParams& p, hipStream_t s);

// ------------------------------------------------------ 8-bit products --
struct MatI8Params {
    const int8_t* x;        // [T, K], rows ldx apart
    int64_t ldx;
    const float* sx;        // [T]
    const int8_t* w;        // [N, K] (gated: [2N, K], gate rows then up rows), rows ldw apart
    int64_t ldw;
    const float* sw;        // [N] (gated: [2N])
    const float* bias;      // [N] or null (not gated)
    int T, N, K, act;
    void* out;              // [T, N], rows ldo apart
    int out_dt;
    int64_t ldo;
};
hipError_t launch_matmul_i8(const MatI8Params& p, bool gated, hipStream_t s);

// ---------------------------------------------------- bfloat16 products --
// out[t][n] = sum over k of (token operand)(t, k) (channel operand)(n, k).  An operand
// is a matrix whose rows run along k, or one whose rows are the k (KIND):
//   NT     x [T, K], w [N, K]: the product of a layer
//   GATED  x [T, K], w [2N, K]: out = act(gate) up; pre [T, 2N] takes the sums
//   NN     x [T, K], w [K, N]: the gradient of the rows
//   TN     x [K, T], w [K, N]: the gradient of the weights
enum MatKind { MAT_NT = 0, MAT_GATED = 1, MAT_NN = 2, MAT_TN = 3 };
// Low-rank adapters of the tokens (NT, GATED): token t adds s[t] b[ids[t]]^T
struct AdapterParams {
    const uint16_t* s;      // [T, halves R], rows lds apart; null: no adapters
    int64_t lds;
    const int* ids;         // [T], outside [0, n): none
    const uint16_t* b;      // [n] of [halves N, R], b_stride apart
    int64_t b_stride;
    const int* ranks;       // [n] or null: R
    int n, R;
};
struct MatBf16Params {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* w;
    int64_t ldw;
    int T, N, K, act;
    void* out;              // [T, N], rows ldo apart
    int out_dt;
    int64_t ldo;
    uint16_t* pre;          // GATED: [T, 2N], rows ldp apart, or null
    int64_t ldp;
    AdapterParams ad;
};
hipError_t launch_matmul_bf16(const MatBf16Params& p, MatKind kind, hipStream_t s);
// both gradients of one product: rows (NN) and weights (TN)
hipError_t launch_matmul_bf16_pair(const MatBf16Params& rows, const MatBf16Params& weights, hipStream_t s);

// dpre = the gradient of pre: dout u act'(g), then dout act(g)
struct GatedGradParams {
    const uint16_t* pre;    // [T, 2F], rows ldp apart
    int64_t ldp;
    const uint16_t* dout;   // [T, F], rows ldd apart
    int64_t ldd;
    uint16_t* dpre;         // [T, 2F], rows ldg apart
    int64_t ldg;
    int T, F, act;
};
hipError_t launch_gated_grad(const GatedGradParams& p, hipStream_t s);

struct AdapterShrinkParams {
    const uint16_t* x;      // [T, K], rows ldx apart
    int64_t ldx;
    const int* ids;         // [T]
    const uint16_t* a;      // [n] of [halves, R, K], a_stride apart
    int64_t a_stride;
    const float* scale;     // [n] or null: 1
    const int* ranks;       // [n] or null: R
    int T, K, n, R, halves;
    uint16_t* s;            // [T, halves R], rows lds apart
    int64_t lds;
};
hipError_t launch_adapter_shrink(const AdapterShrinkParams& p, hipStream_t s);

}  // namespace moe
