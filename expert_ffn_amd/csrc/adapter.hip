// Low-rank adapters of many requests: the first product,
//
//   s[t] = scale[a] (x[t] A[a]^T)      a = ids[t]; zeros where there is none
//
// A workgroup takes 16 TT tokens, 16 RB ranks of one half (y), and every gridDim.z-th of
// the adapters that occur among its tokens.  Its KG waves take the K steps of 64 in turn,
// each with a ring of NSTG stages of its own, filled by LDS DMA: 8 rows of 128 bytes a
// copy.  (Fragments straight from memory touch 16 lines an instruction, for which the
// address unit takes about 80 cycles: 9.5 us for 14 adapters of 2 x 16 ranks, K = 2816.)
// Tokens of other adapters are not read.  MFMA 16x16x32, A = ranks, B = tokens: D columns
// are tokens, and each adapter's sums are stored for its own tokens only, so nothing of
// one request meets another's.
//
// s is rounded to bf16, the type in which the second product reads it.  With low-rank parts
// of about 0.4 times the product's size its results differ from 64 bits by 0.0006 to 0.0010 of
// their norm where they are fp32, and by 0.0018 to 0.0020 where they are bf16 (their own
// rounding 0.0017).
#include <algorithm>

#include "bf16_tile.h"

namespace moe {

template <int TT, int RB, int KG, int NSTG>
__global__ __launch_bounds__(64 * KG) void adapter_shrink_kernel(AdapterShrinkParams p) {
    constexpr int BT = 16 * TT, BR = 16 * RB, BK = 64, STAGE = (BT + BR) * 128, CA = 2 * RB, CX = 2 * TT, CPS = CA + CX;
    static_assert(NSTG >= 2 && NSTG <= 3 && CPS * (NSTG - 1) <= 63 && RB * TT * 1024 <= NSTG * STAGE, "copies in flight, sums in the ring");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NSTG * STAGE];
    __shared__ int idl[BT];
    const int tid = threadIdx.x, lane = tid & 63, kg = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int t0 = blockIdx.x * BT;
    const int rblocks = (p.R + BR - 1) / BR;   // of a half
    const int h = blockIdx.y / rblocks, r0 = blockIdx.y % rblocks * BR;
    const int rows = min(BT, p.T - t0), ranks = min(BR, p.R - r0);
    auto id_of = [&](int t) {   // -1: none
        const int a = p.ids[t0 + min(t, rows - 1)];
        return t < rows && a >= 0 && a < p.n ? a : -1;
    };
    int aid[TT], idc[CX];   // of the tokens that this lane computes, and of those it copies
#pragma unroll
    for (int j = 0; j < TT; ++j) aid[j] = id_of(16 * j + l16);
#pragma unroll
    for (int i = 0; i < CX; ++i) idc[i] = id_of(8 * i + lane / 8);
    const rsrc_t xr = make_rsrc(p.x + t0 * p.ldx, static_cast<uint32_t>(((rows - 1) * p.ldx + p.K) * 2));
    uint8_t* ring = lds + kg * NSTG * STAGE;
    const uint32_t kb = 2u * p.K;
    uint32_t chunk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) chunk[i] = ((lane % 8) ^ swz_row(8 * i + lane / 8)) * 16;
    const int nk = ((p.K + BK - 1) / BK + KG - 1) / KG;
    uint64_t left[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) left[j] = __ballot(aid[j] >= 0);
    if (tid < BT) idl[tid] = id_of(tid);
    if (blockIdx.z == 0)   // tokens without an adapter
        for (int i = tid; i < BT * 2 * RB; i += 64 * KG) {
            const int t = i / (2 * RB), r = i % (2 * RB) * 8;
            if (t < rows && r < ranks && id_of(t) < 0)
                *reinterpret_cast<u32x4*>(p.s + (t0 + t) * p.lds + h * p.R + r0 + r) = u32x4{0, 0, 0, 0};
        }
    for (unsigned skip = blockIdx.z;;) {   // adapters of other workgroups before the next one of this
        int a = -1;
#pragma unroll
        for (int j = TT - 1; j >= 0; --j)
            if (left[j]) a = __builtin_amdgcn_readlane(aid[j], __builtin_ctzll(left[j]));
        if (a < 0) return;
#pragma unroll
        for (int j = 0; j < TT; ++j) left[j] &= ~__ballot(aid[j] == a);
        if (skip > 0) {
            --skip;
            continue;
        }
        skip = gridDim.z - 1;
        const rsrc_t ar = make_rsrc(p.a + a * p.a_stride + (static_cast<int64_t>(h) * p.R + r0) * p.K, static_cast<uint32_t>(ranks) * kb);
        uint32_t ao[CA], xo[CX];
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const int row = 8 * i + lane / 8;
            ao[i] = row < ranks ? row * kb + chunk[i & 1] : NO_LANE;
        }
#pragma unroll
        for (int i = 0; i < CX; ++i)
            xo[i] = idc[i] == a ? static_cast<uint32_t>((8 * i + lane / 8) * p.ldx * 2 + chunk[i & 1]) : NO_LANE;
        // what lies past K is zeros; stages past the last are not requested
        auto copy = [&](int c, uint8_t* st) __attribute__((always_inline)) {
            const uint32_t k = 2 * BK * (c * KG + kg);
            const uint32_t so = k < kb ? k : 0;   // inside the resource
#pragma unroll
            for (int i = 0; i < CPS; ++i) {
                const bool in = k + chunk[i & 1] < kb;
                if (i < CA)
                    lds_dma16(ar, st + i * 1024, in ? ao[i] : NO_LANE, so);
                else
                    lds_dma16(xr, st + i * 1024, in ? xo[i - CA] : NO_LANE, so);
            }
        };
        const int rank = p.ranks != nullptr ? min(p.ranks[a], p.R) : p.R;
        const float scale = p.scale != nullptr ? p.scale[a] : 1.0f;
#pragma unroll
        for (int c = 0; c < NSTG; ++c)
            if (c < nk) copy(c, ring + c * STAGE);
        f32x4 acc[RB][TT] = {};
        for (int c = 0, buf = 0; c < nk; ++c) {
            const int behind = min(nk - 1 - c, NSTG - 1);   // the stages behind this one may still be on their way
            if (NSTG > 2 && behind == 2)
                __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * CPS));
            else if (behind == 1)
                __builtin_amdgcn_s_waitcnt(waitcnt_vm(CPS));
            else
                __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
            asm volatile("" ::: "memory");
            uint8_t* st = ring + buf * STAGE;
            u32x4 va[2][RB], vb[2][TT];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int o = l16 * 128 + (((4 * s + q) ^ swz_row(l16)) << 4);
#pragma unroll
                for (int i = 0; i < RB; ++i) va[s][i] = *reinterpret_cast<const u32x4*>(st + i * 2048 + o);
#pragma unroll
                for (int j = 0; j < TT; ++j) vb[s][j] = *reinterpret_cast<const u32x4*>(st + (RB + j) * 2048 + o);
            }
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(63));   // the operands are read, so the buffer may be filled again
            asm volatile("" ::: "memory");
            if (c + NSTG < nk) copy(c + NSTG, st);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int j = 0; j < TT; ++j) acc[i][j] = mfma16x16x32(va[s][i], vb[s][j], acc[i][j]);
            buf = buf + 1 == NSTG ? 0 : buf + 1;
        }
        // the sums of a wave go to its own ring, where nothing is under way any more
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j) *reinterpret_cast<f32x4*>(ring + (i * TT + j) * 1024 + lane * 16) = acc[i][j];
        __syncthreads();
        for (int i = tid; i < RB * TT * 64; i += 64 * KG) {   // 4 ranks of one token
            const int l = i & 63, b = i >> 6;
            const int t = 16 * (b % TT) + (l & 15), r = 16 * (b / TT) + 4 * (l >> 4);
            if (idl[t] != a || r >= ranks) continue;
            f32x4 v = {0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < KG; ++g) v += *reinterpret_cast<const f32x4*>(lds + g * NSTG * STAGE + b * 1024 + l * 16);
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = r0 + r + e < rank ? scale * v[e] : 0.0f;
            *reinterpret_cast<u32x2*>(p.s + (t0 + t) * p.lds + h * p.R + r0 + r) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        }
        __syncthreads();   // the sums are read
    }
}

constexpr int SHRINK_KG = 8, SHRINK_NSTG = 2;

// `most`: the workgroups that the CUs hold at once share the adapters of a block
template <int TT, int RB>
static hipError_t shrink(const AdapterShrinkParams& p, int most, hipStream_t s) {
    const int blocks = (p.T + 16 * TT - 1) / (16 * TT), ranks = (p.R + 16 * RB - 1) / (16 * RB) * p.halves;
    const int share = std::max<int64_t>(1, std::min<int64_t>(std::min(p.T, 16 * TT), most / (static_cast<int64_t>(blocks) * ranks)));
    hipLaunchKernelGGL((adapter_shrink_kernel<TT, RB, SHRINK_KG, SHRINK_NSTG>), dim3(blocks, ranks, share), dim3(64 * SHRINK_KG), 0, s, p);
    return hipGetLastError();
}

// The smallest blocks while they leave CUs idle, larger ones (fewer reads of the same
// rows) behind that.  Runs of 150 tokens, K = 2816: 512 x 64 ranks 16 x 16 5.3 us, 32 x 32
// 7.3; 1024 x 2 x 32 ranks 16 x 16 8.6, 32 x 16 6.4, 32 x 32 7.5; 2048 x 2 x 32 ranks 13.3,
// 10.7, 9.4.  16 waves took 0 to 20 % longer than 8, three stages 0 to 10 %.
hipError_t launch_adapter_shrink(const AdapterShrinkParams& p, hipStream_t s) {
    const int64_t small = static_cast<int64_t>((p.T + 15) / 16) * ((p.R + 15) / 16) * p.halves;
    if (small < 256) return shrink<1, 1>(p, 512, s);
    if (small < 512) return shrink<2, 1>(p, 256, s);
    return shrink<2, 2>(p, 256, s);
}

}  // namespace moe
