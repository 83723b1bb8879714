// Low-rank adapters of many requests: the first product,
//
//   s[t] = scale[a] (x[t] A[a]^T)      a = ids[t]; zeros where there is none
//
// A workgroup takes 16 TT tokens, 16 RB ranks, and the adapters of these tokens one after
// the other (gridDim.y workgroups share them); its waves share K in steps of 64.  MFMA 16x16x32, A = ranks, B = tokens,
// operands straight from memory: lane l holds row l & 15, k 8 (l >> 4) .. of a step.
// Each adapter's sums are stored for its own tokens only.
#include "block.h"
#include "common.h"

namespace moe {

template <int TT, int RB, int KG>
__global__ __launch_bounds__(64 * KG) void adapter_shrink_kernel(AdapterShrinkParams p) {
    __shared__ __attribute__((aligned(16))) float part[KG][RB][TT][256];
    const int tid = threadIdx.x, lane = tid & 63, kg = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = lane & 15, q = lane >> 4;
    const int t0 = blockIdx.x * 16 * TT;
    const int rblocks = (p.R + 16 * RB - 1) / (16 * RB);   // of a half
    const int h = blockIdx.z / rblocks, r0 = blockIdx.z % rblocks * 16 * RB;
    int aid[TT];
    uint64_t left[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = t0 + 16 * j + row;
        const int a = t < p.T ? p.ids[t] : -1;
        aid[j] = a >= 0 && a < p.n ? a : -1;
        left[j] = __ballot(aid[j] >= 0);
    }
    // tokens without an adapter
    if (blockIdx.y == 0)
        for (int i = tid; i < 16 * TT * 2 * RB; i += 64 * KG) {
            const int t = t0 + i / (2 * RB), r = r0 + i % (2 * RB) * 8;
            if (t >= p.T || r >= p.R) continue;
            const int a = p.ids[t];
            if (a < 0 || a >= p.n) *reinterpret_cast<u32x4*>(p.s + t * p.lds + h * p.R + r) = u32x4{0, 0, 0, 0};
        }
    for (unsigned unit = 0;; ++unit) {
        int a = -1;
#pragma unroll
        for (int j = TT - 1; j >= 0; --j)
            if (left[j]) a = __builtin_amdgcn_readlane(aid[j], __builtin_ctzll(left[j]));
        if (a < 0) return;
#pragma unroll
        for (int j = 0; j < TT; ++j) left[j] &= ~__ballot(aid[j] == a);
        if (unit % gridDim.y != blockIdx.y) continue;
        const int rank = p.ranks ? min(p.ranks[a], p.R) : p.R;
        const uint16_t* pa = p.a + a * p.a_stride + static_cast<int64_t>(h) * p.R * p.K;
        f32x4 acc[RB][TT] = {};
        if (r0 < rank) {
#pragma unroll 2
            for (int k0 = 64 * kg; k0 < p.K; k0 += 64 * KG) {
                u32x4 va[2][RB], vb[2][TT];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = k0 + 32 * s + 8 * q;
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        const int r = r0 + 16 * i + row;
                        va[s][i] = u32x4{0, 0, 0, 0};
                        if (r < rank && k < p.K) va[s][i] = *reinterpret_cast<const u32x4*>(pa + static_cast<int64_t>(r) * p.K + k);
                    }
#pragma unroll
                    for (int j = 0; j < TT; ++j) {
                        vb[s][j] = u32x4{0, 0, 0, 0};
                        if (aid[j] == a && k < p.K)
                            vb[s][j] = *reinterpret_cast<const u32x4*>(p.x + (t0 + 16 * j + row) * p.ldx + k);
                    }
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < RB; ++i)
#pragma unroll
                        for (int j = 0; j < TT; ++j) acc[i][j] = mfma16x16x32(va[s][i], vb[s][j], acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j) *reinterpret_cast<f32x4*>(&part[kg][i][j][lane * 4]) = acc[i][j];
        __syncthreads();
        const float scale = p.scale ? p.scale[a] : 1.0f;
        for (int i = tid; i < RB * TT * 64; i += 64 * KG) {   // 4 ranks of one token
            const int l = i & 63, j = (i >> 6) % TT, b = (i >> 6) / TT;
            const int t = t0 + 16 * j + (l & 15), r = r0 + 16 * b + 4 * (l >> 4);
            if (t >= p.T || r >= p.R || p.ids[t] != a) continue;
            f32x4 v = {0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < KG; ++g) v += *reinterpret_cast<const f32x4*>(&part[g][b][j][l * 4]);
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = r + e < rank ? scale * v[e] : 0.0f;
            *reinterpret_cast<u32x2*>(p.s + t * p.lds + h * p.R + r) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        }
        __syncthreads();
    }
}

hipError_t launch_adapter_shrink(const AdapterShrinkParams& p, hipStream_t s) {
    if (p.T <= 64) {
        hipLaunchKernelGGL((adapter_shrink_kernel<1, 1, 8>), dim3((p.T + 15) / 16, p.T < 16 ? p.T : 16, (p.R + 15) / 16 * p.halves),
                           dim3(512), 0, s, p);
    } else {
        const int blocks = (p.T + 31) / 32;
        hipLaunchKernelGGL((adapter_shrink_kernel<2, 4, 8>), dim3(blocks, 4, (p.R + 63) / 64 * p.halves), dim3(512), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace moe
