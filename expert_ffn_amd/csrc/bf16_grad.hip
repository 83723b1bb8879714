// Gradients of the bfloat16 products: the tile kernel on operands whose rows are the k,
// and the gated activation's gradient.
#include "bf16_tile.h"

namespace moe {

hipError_t tiles_nn(const MatBf16Params& p, hipStream_t s) { return bf16_tiles<MAT_NN, false>(p, s); }
hipError_t tiles_tn(const MatBf16Params& p, hipStream_t s) { return bf16_tiles<MAT_TN, false>(p, s); }

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
// gradient, 16-byte writes of both gradients.  Bound by memory: 10 bytes a channel.
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
