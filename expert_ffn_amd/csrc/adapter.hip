// Low-rank adapters of many requests: the first product,
//
//   s[t] = scale[a] (x[t] A[a]^T)      a = ids[t]; zeros where there is none
//
// MFMA 16x16x32, A = ranks, B = tokens, operands straight from memory: lane l holds row
// l & 15, k 8 (l >> 4) .. of a step.  D columns are tokens, and each adapter's sums are
// stored for its own tokens only, so nothing of one request meets another's.
#include "block.h"
#include "common.h"

namespace moe {

// zeros for the tokens of a block that have no adapter: ranks r0 .. r0 + 8 * chunks of half h
__device__ __forceinline__ void clear_others(const AdapterShrinkParams& p, int t0, int tokens, int h, int r0, int chunks, int threads) {
    for (int i = threadIdx.x; i < tokens * chunks; i += threads) {
        const int t = t0 + i / chunks, r = r0 + i % chunks * 8;
        if (t >= p.T || r >= p.R) continue;
        const int a = p.ids[t];
        if (a < 0 || a >= p.n) *reinterpret_cast<u32x4*>(p.s + t * p.lds + h * p.R + r) = u32x4{0, 0, 0, 0};
    }
}

// Few tokens: a workgroup for each token (y) of a block of 16 and each 16 ranks (z),
// which ends if an earlier token of the block has the same adapter.  Its KG waves share K
// in steps of 32, and each requests U steps at once: the time is that of the chain ids,
// operands, sums.  x does not wait for the ids, nor the first 16 ranks for the rank.
template <int KG, int U>
__global__ __launch_bounds__(64 * KG) void adapter_shrink_few_kernel(AdapterShrinkParams p) {
    __shared__ __attribute__((aligned(16))) f32x4 part[KG][64];
    const int tid = threadIdx.x, lane = tid & 63, kg = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = lane & 15, q = lane >> 4;
    const int t0 = blockIdx.x * 16, me = blockIdx.y;
    const int rblocks = (p.R + 15) / 16;   // of a half
    const int h = blockIdx.z / rblocks, r0 = blockIdx.z % rblocks * 16;
    const int id = t0 + row < p.T ? p.ids[t0 + row] : -1;
    u32x4 vb[U];
    auto tokens = [&](int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 32 * KG * u + 8 * q;
            vb[u] = u32x4{0, 0, 0, 0};
            if (t0 + row < p.T && k < p.K) vb[u] = *reinterpret_cast<const u32x4*>(p.x + (t0 + row) * p.ldx + k);
        }
    };
    tokens(32 * kg);
    if (me == 0) clear_others(p, t0, 16, h, r0, 2, 64 * KG);
    const int a = __builtin_amdgcn_readlane(id, me);
    if (t0 + me >= p.T || a < 0 || a >= p.n) return;
    const uint64_t same = __ballot(id == a) & 0xFFFF;
    if (__builtin_ctzll(same) != me) return;
    int rank = p.R;
    if (p.ranks != nullptr) rank = min(p.ranks[a], p.R);
    const uint16_t* pa = p.a + a * p.a_stride + (static_cast<int64_t>(h) * p.R + r0 + row) * p.K;
    f32x4 acc = {0, 0, 0, 0};
    if (r0 == 0 || r0 < rank)
        for (int k0 = 32 * kg;;) {
            u32x4 va[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + 32 * KG * u + 8 * q;
                va[u] = u32x4{0, 0, 0, 0};
                if (r0 + row < p.R && k < p.K) va[u] = *reinterpret_cast<const u32x4*>(pa + k);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) acc = mfma16x16x32(va[u], vb[u], acc);
            k0 += 32 * KG * U;
            if (k0 >= p.K) break;
            tokens(k0);
        }
    part[kg][lane] = acc;
    __syncthreads();
    if (tid >= 64) return;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < KG; ++g) v += part[g][lane];
    const int r = r0 + 4 * q;   // 4 ranks of one token
    if (id != a || r >= p.R) return;
    const float scale = p.scale ? p.scale[a] : 1.0f;
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = r + e < rank ? scale * v[e] : 0.0f;
    *reinterpret_cast<u32x2*>(p.s + (t0 + row) * p.lds + h * p.R + r) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
}

// Many tokens: a workgroup takes 16 TT tokens, 16 RB ranks, and the adapters of these
// tokens one after the other (gridDim.y workgroups share them); its waves share K in
// steps of 64.
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
    if (blockIdx.y == 0) clear_others(p, t0, 16 * TT, h, r0, 2 * RB, 64 * KG);
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
        hipLaunchKernelGGL((adapter_shrink_few_kernel<16, 8>), dim3((p.T + 15) / 16, p.T < 16 ? p.T : 16, (p.R + 15) / 16 * p.halves),
                           dim3(1024), 0, s, p);
    } else {
        const int blocks = (p.T + 31) / 32;
        hipLaunchKernelGGL((adapter_shrink_kernel<2, 4, 8>), dim3(blocks, 4, (p.R + 63) / 64 * p.halves), dim3(512), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace moe
