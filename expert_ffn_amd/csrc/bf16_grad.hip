// Gradients of the bfloat16 products: the tile kernel on operands whose rows are the k,
// and the gated activation's gradient.
#include <algorithm>

#include "bf16_tile.h"

namespace moe {

hipError_t tiles_nn(const MatBf16Params& p, hipStream_t s) { return bf16_tiles<MAT_NN, false>(p, s); }
hipError_t tiles_tn(const MatBf16Params& p, hipStream_t s) { return bf16_tiles<MAT_TN, false>(p, s); }

template <int BN, int BT, int WN, int WT, int NSTG, int KG>
static hipError_t pair(const MatBf16Params& p, const MatBf16Params& r, hipStream_t s) {
    auto tiles = [](int size, int tile) { return (size + tile - 1) / tile; };
    const int pn = tiles(p.N, BN), pt = tiles(p.T, BT), rn = tiles(r.N, BN), rt = tiles(r.T, BT);
    const int first = (pn * pt + 7) / 8 * 8, second = (rn * rt + 7) / 8 * 8;
    hipLaunchKernelGGL((matmul_bf16_pair_kernel<BN, BT, WN, WT, NSTG, KG>), dim3(first + second), dim3(64 * WN * WT * KG), 0, s, p, pn, pt,
                       r, rn, rt, first);
    return hipGetLastError();
}

// Both gradients in one launch, or one after the other: the smaller estimate.  In one
// launch the workgroups of both fill the CUs together: the sum of their times over the
// CUs, 0.4 of the longer one's for the uneven end, times a factor of the tile, fitted
// to 91 shapes (T 16 to 8192) with six tiles.  The choice is 2.5 % slower than the best of
// eleven tiles and two launches on average, two launches always 36 %.  T = 333, 1408 x
// 1424: 10.5 us in one launch, 14.2 in two; T = 43, 184 x 536: 3.4 and 6.2; T = 858, 5344 x
// 2032: 51.7 and 59.3; T = 2009, 312 x 1976: 20.6 and 19.8.
struct PairTile {
    int tile;   // of Bf16Tiles
    float factor;
};
constexpr PairTile PAIR_TILES[] = {{0, 0.8f}, {1, 0.8f}, {3, 0.9f}, {7, 1.0f}, {8, 1.0f}, {9, 1.0f}};

static int pick_pair(const MatBf16Params& p, const MatBf16Params& r) {
    int best = -1;
    float best_us = bf16_tile_us(Bf16Tiles<MAT_NN>::T[pick_bf16_tile<MAT_NN, false>(p.T, p.N, p.K)], p.T, p.N, p.K) +
                    bf16_tile_us(Bf16Tiles<MAT_TN>::T[pick_bf16_tile<MAT_TN, false>(r.T, r.N, r.K)], r.T, r.N, r.K);
    for (const PairTile& c : PAIR_TILES) {
        float work = 0.0f, alone = 0.0f, longest = 0.0f, fixed = 0.0f;
        int64_t groups = 0;
        auto add = [&](const Bf16Tile& t, const MatBf16Params& q) {
            const int64_t W = ((q.N + t.bn - 1) / t.bn) * ((q.T + t.bt - 1ll) / t.bt);
            const float steps = static_cast<float>((q.K + 63) / 64), full = steps * t.full + t.end;
            groups += W;
            work += static_cast<float>(W) / 256.0f * full;
            alone = std::max(alone, steps * t.alone + t.end);
            longest = std::max(longest, full);
            fixed = std::max(fixed, t.fixed);
        };
        add(Bf16Tiles<MAT_NN>::T[c.tile], p);
        add(Bf16Tiles<MAT_TN>::T[c.tile], r);
        if (groups >= (1 << 22)) continue;   // keeps every launch below 2^32 threads
        const float us = c.factor * (fixed + std::max(alone, work + 0.4f * longest));
        if (us < best_us) {
            best_us = us;
            best = c.tile;
        }
    }
    return best;
}

hipError_t launch_matmul_bf16_pair(const MatBf16Params& p, const MatBf16Params& r, hipStream_t s) {
    switch (pick_pair(p, r)) {
        case 0: return pair<32, 32, 1, 1, 3, 4>(p, r, s);
        case 1: return pair<64, 32, 2, 1, 3, 4>(p, r, s);
        case 3: return pair<64, 64, 2, 2, 3, 1>(p, r, s);
        case 7: return pair<128, 128, 2, 2, 3, 1>(p, r, s);
        case 8: return pair<128, 192, 2, 4, 3, 1>(p, r, s);
        case 9: return pair<192, 192, 2, 2, 3, 1>(p, r, s);
    }
    const hipError_t e = tiles_nn(p, s);
    return e == hipSuccess ? tiles_tn(r, s) : e;
}

// act(g) = g q with q = 1 / (1 + e^z):  act'(g) = q - g q (1 - q) dz/dg
//   silu z = -g;  gelu (tanh form) z = -2 sqrt(2/pi) (g + 0.044715 g^3)
// Where q (1 - q) is 0 in fp32 the second term is left out: its other factor may be
// infinite there.
__device__ __forceinline__ void act_and_slope(int act, float g, float* value, float* slope) {
    const bool silu = act == ACT_SILU;
    const float z = silu ? -g : -1.5957691216057308f * (g + 0.044715f * g * g * g);
    const float dz = silu ? 1.0f : 1.5957691216057308f * (1.0f + 0.134145f * g * g);
    const float q = __builtin_amdgcn_rcpf(1.0f + __expf(z)), t = q * (1.0f - q);
    *value = g * q;
    *slope = t > 0.0f ? q + g * t * dz : q;
}

// One thread takes 8 channels of one row: 16-byte reads of gate, up and the output's
// gradient, 16-byte writes of both gradients.  Bound by memory: 10 bytes a channel, T = 8192,
// F = 4096 53 us (335 MB, 6.3 TB/s: some of it stays in the memory-side cache).
//
// dpre is rounded to bf16, the type in which both products read it (a second bf16 term
// would double their MFMA).  dx and dw differ from 64 bits by 0.0017 of their norm where they
// are fp32, by 0.0023 where they are bf16, of which their own rounding is 0.0017.
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedGradParams p) {
    const int f = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (f >= p.F) return;
    for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y) {
        const u32x4 g = *reinterpret_cast<const u32x4*>(p.pre + t * p.ldp + f);
        const u32x4 u = *reinterpret_cast<const u32x4*>(p.pre + t * p.ldp + p.F + f);
        const u32x4 d = *reinterpret_cast<const u32x4*>(p.dout + t * p.ldd + f);
        u32x4 dg, du;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float vg[2], vu[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                auto of = [&](uint32_t w) { return __uint_as_float(e ? w & 0xFFFF0000u : w << 16); };
                float value, slope;
                act_and_slope(p.act, of(g[i]), &value, &slope);
                vg[e] = of(d[i]) * of(u[i]) * slope;
                vu[e] = of(d[i]) * value;
            }
            dg[i] = pack_bf16x2(vg[0], vg[1]);
            du[i] = pack_bf16x2(vu[0], vu[1]);
        }
        *reinterpret_cast<u32x4*>(p.dpre + t * p.ldg + f) = dg;
        *reinterpret_cast<u32x4*>(p.dpre + t * p.ldg + p.F + f) = du;
    }
}

hipError_t launch_gated_grad(const GatedGradParams& p, hipStream_t s) {
    hipLaunchKernelGGL(gated_grad_kernel, dim3((p.F + 2047) / 2048, p.T < 32768 ? p.T : 32768), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace moe
