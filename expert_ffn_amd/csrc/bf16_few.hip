// bfloat16 products of few tokens (at most 16 TT): workgroups of 16 weight rows (gated:
// 8 gate rows and their up rows), so that all CUs take part, and KG waves that take
// the 64-element K steps in turn.  Each wave has a ring of its own, so none waits for
// another before the sums are added.  MFMA 16x16x32: lane l holds row l & 15, chunk
// 4 s + (l >> 4) of both operands; swz16 spreads the rows that are read together over
// all banks.
#include "bf16_tile.h"

namespace moe {

__device__ __forceinline__ int swz16(int r) { return (r & 15) >> 1; }

constexpr int FEW_KG = 4, FEW_NSTG = 2;

template <int TT, bool GATED, bool AD>
__global__ __launch_bounds__(64 * FEW_KG) void matmul_bf16_few_kernel(MatBf16Params p) {
    constexpr int KG = FEW_KG, NSTG = FEW_NSTG, BK = 64, STAGE = (16 + 16 * TT) * 128, CH = GATED ? 8 : 16, CPS = 2 + 2 * TT;
    static_assert(KG >= 4 && NSTG == 2 && CPS <= 63, "256 threads for the results, copies in flight");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NSTG * STAGE];
    __shared__ __attribute__((aligned(16))) float part[KG][TT][256];
    const int tid = threadIdx.x, lane = tid & 63, kg = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * CH, nch = min(CH, p.N - n0);
    const uint32_t kb = 2u * p.K;
    auto rows_of = [&](const uint16_t* base, int64_t ld, int r0, int rows) {
        return make_rsrc(base + static_cast<int64_t>(r0) * ld, static_cast<uint32_t>(((rows - 1) * ld + p.K) * 2));
    };
    const rsrc_t wr0 = rows_of(p.w, p.ldw, n0, nch);
    const rsrc_t wr1 = rows_of(p.w, p.ldw, GATED ? p.N + n0 : n0, nch);
    const rsrc_t xr = rows_of(p.x, p.ldx, 0, p.T);
    // copies: 8 rows each, lane l row l / 8, chunk (l % 8) ^ swz16(row)
    uint8_t* ring = lds + kg * NSTG * STAGE;
    uint32_t chunk[2], wo[2], xo[2 * TT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + lane / 8, c = GATED ? row & 7 : row;
        chunk[i] = ((lane % 8) ^ swz16(row)) * 16;
        wo[i] = c < nch ? static_cast<uint32_t>(c * p.ldw * 2 + chunk[i]) : NO_LANE;
    }
#pragma unroll
    for (int i = 0; i < 2 * TT; ++i) {
        const int row = 8 * i + lane / 8;
        xo[i] = row < p.T ? static_cast<uint32_t>(row * p.ldx * 2 + chunk[i & 1]) : NO_LANE;
    }
    const int nk = ((p.K + BK - 1) / BK + KG - 1) / KG;
    // chunks past K are zeros; stages past the last are not requested
    auto copy = [&](int c, uint8_t* st) {
        const uint32_t k = 2 * BK * (c * KG + kg);
        const uint32_t so = k < kb ? k : 0;   // inside the resource
#pragma unroll
        for (int i = 0; i < CPS; ++i) {
            const bool in = k + chunk[i & 1] < kb;
            if (i < 2)
                lds_dma16(i == 0 ? wr0 : wr1, st + i * 1024, in ? wo[i] : NO_LANE, so);
            else
                lds_dma16(xr, st + i * 1024, in ? xo[i - 2] : NO_LANE, so);
        }
    };
    const int row = lane & 15, q = lane >> 4;
    int aid[TT];   // the adapters of this lane's tokens
    if (AD) {
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int a = row + 16 * j < p.T ? p.ad.ids[row + 16 * j] : -1;
            aid[j] = a >= 0 && a < p.ad.n ? a : -1;
        }
    }
#pragma unroll
    for (int c = 0; c < NSTG; ++c)
        if (c < nk) copy(c, ring + c * STAGE);
    f32x4 acc[TT] = {};
    for (int c = 0, buf = 0; c < nk; ++c) {
        if (c + 1 < nk)
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(CPS));   // the next stage may still be on its way
        else
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        asm volatile("" ::: "memory");
        uint8_t* st = ring + buf * STAGE;
        u32x4 a[2], b[2][TT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int o = row * 128 + (((4 * s + q) ^ swz16(row)) << 4);
            a[s] = *reinterpret_cast<const u32x4*>(st + o);
#pragma unroll
            for (int j = 0; j < TT; ++j) b[s][j] = *reinterpret_cast<const u32x4*>(st + (16 + 16 * j) * 128 + o);
        }
        __builtin_amdgcn_s_waitcnt(wait_vm_lds(63));   // read, so the buffer may be filled again
        asm volatile("" ::: "memory");
        if (c + NSTG < nk) copy(c + NSTG, st);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[j] = mfma16x16x32(a[s], b[s][j], acc[j]);
        buf = buf + 1 == NSTG ? 0 : buf + 1;
    }
    if (AD) {
        // The low-rank part as in the tile kernel: adapter by adapter, each from zero and
        // added in the lanes of its own tokens; the waves take the adapters in turn.
        uint64_t left[TT];
#pragma unroll
        for (int j = 0; j < TT; ++j) left[j] = __ballot(aid[j] >= 0);
        for (int unit = 0;; ++unit) {
            int a = -1;
#pragma unroll
            for (int j = TT - 1; j >= 0; --j)
                if (left[j]) a = __builtin_amdgcn_readlane(aid[j], __builtin_ctzll(left[j]));
            if (a < 0) break;
#pragma unroll
            for (int j = 0; j < TT; ++j) left[j] &= ~__ballot(aid[j] == a);
            if (unit % KG != kg) continue;
            const int rank = p.ad.ranks ? min(p.ad.ranks[a], p.ad.R) : p.ad.R;
            const uint16_t* pb = p.ad.b + a * p.ad.b_stride;
            f32x4 low[TT] = {};
            for (int h = 0; h < (GATED ? 2 : 1); ++h)
                for (int k0 = 0; k0 < rank; k0 += 32) {
                    const int k = k0 + 8 * q, n = GATED ? row & 7 : row;
                    u32x4 va = {0, 0, 0, 0};
                    if (k < rank && n < nch && (!GATED || (row >> 3) == h))
                        va = low_ranks(*reinterpret_cast<const u32x4*>(pb + (static_cast<int64_t>(h) * p.N + n0 + n) * p.ad.R + k), rank - k);
#pragma unroll
                    for (int j = 0; j < TT; ++j) {
                        u32x4 vb = {0, 0, 0, 0};
                        if (k < rank && aid[j] == a)
                            vb = *reinterpret_cast<const u32x4*>(p.ad.s + (row + 16 * j) * p.ad.lds + h * p.ad.R + k);
                        low[j] = mfma16x16x32(va, vb, low[j]);
                    }
                }
#pragma unroll
            for (int j = 0; j < TT; ++j)
                if (aid[j] == a) acc[j] += low[j];
        }
    }
    // lane l: token l & 15 of tile j, tile rows 4 (l >> 4) ..
#pragma unroll
    for (int j = 0; j < TT; ++j) *reinterpret_cast<f32x4*>(&part[kg][j][lane * 4]) = acc[j];
    __syncthreads();
    const int tok = tid / CH, ch = tid % CH;
    if (tid >= 16 * CH || ch >= nch) return;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = tok + 16 * j;
        if (t >= p.T) return;
        auto total = [&](int r) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < KG; ++g) s += part[g][j][(tok + 16 * (r >> 2)) * 4 + (r & 3)];
            return s;
        };
        float v = total(ch);
        if (GATED) {
            const float u = total(8 + ch);
            if (p.pre != nullptr) {
                p.pre[t * p.ldp + n0 + ch] = static_cast<uint16_t>(pack_bf16x2(v, v));
                p.pre[t * p.ldp + p.N + n0 + ch] = static_cast<uint16_t>(pack_bf16x2(u, u));
            }
            v = act_fn(p.act, v) * u;
        }
        const int64_t o = t * p.ldo + n0 + ch;
        if (p.out_dt == F32)
            static_cast<float*>(p.out)[o] = v;
        else
            static_cast<uint16_t*>(p.out)[o] = static_cast<uint16_t>(pack_bf16x2(v, v));
    }
}

template <int TT, bool GATED>
static hipError_t few(const MatBf16Params& p, hipStream_t s) {
    constexpr int CH = GATED ? 8 : 16;
    auto kn = p.ad.s ? matmul_bf16_few_kernel<TT, GATED, true> : matmul_bf16_few_kernel<TT, GATED, false>;
    hipLaunchKernelGGL(kn, dim3((p.N + CH - 1) / CH), dim3(64 * FEW_KG), 0, s, p);
    return hipGetLastError();
}

hipError_t tiles_nt(const MatBf16Params& p, hipStream_t s);
hipError_t tiles_gated(const MatBf16Params& p, hipStream_t s);
hipError_t tiles_nn(const MatBf16Params& p, hipStream_t s);
hipError_t tiles_tn(const MatBf16Params& p, hipStream_t s);

// Which kernel.
template <bool GATED>
static hipError_t forward(const MatBf16Params& p, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.N) * (GATED ? 2 : 1);
    if (p.T <= 16) return few<1, GATED>(p, s);
    if (rows <= 256 * 16) {
        if (p.T <= 32) return few<2, GATED>(p, s);
        if (p.T <= 48) return few<3, GATED>(p, s);
    }
    return GATED ? tiles_gated(p, s) : tiles_nt(p, s);
}

hipError_t launch_matmul_bf16(const MatBf16Params& p, MatKind kind, hipStream_t s) {
    switch (kind) {
        case MAT_NT: return forward<false>(p, s);
        case MAT_GATED: return forward<true>(p, s);
        case MAT_NN: return tiles_nn(p, s);
        default: return tiles_tn(p, s);
    }
}

}  // namespace moe
