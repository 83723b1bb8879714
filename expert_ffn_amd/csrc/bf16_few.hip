// bfloat16 products of few tokens (at most 16 TT): workgroups of 16 weight rows (gated:
// 8 gate rows and their up rows), so that all CUs take part, and KG waves that take
// the 64-element K steps in turn.  Each wave has a ring of its own, so none waits for
// another before the sums are added.  MFMA 16x16x32: lane l holds row l & 15, chunk
// 4 s + (l >> 4) of both operands; swz16 spreads the rows that are read together over
// all banks.
//
// Bound by memory: T = 1, 2 x 2112 x 2816 reads 23.8 MB in 5.6 to 6.3 us (3.8 to 4.2 TB/s), of
// which an empty launch is 1.6; T = 16 7.0 us, with an adapter of 2 x 16 ranks for each
// token (of 32) 9.0.
#include "bf16_tile.h"

namespace moe {

__device__ __forceinline__ int swz16(int r) { return (r & 15) >> 1; }

template <int TT, int KG, int NSTG, bool GATED, bool AD>
__global__ __launch_bounds__(64 * KG) void matmul_bf16_few_kernel(MatBf16Params p) {
    constexpr int BK = 64, STAGE = (16 + 16 * TT) * 128, CH = GATED ? 8 : 16, CPS = 2 + 2 * TT;
    static_assert(KG >= 4 && NSTG >= 2 && NSTG <= 3, "256 threads for the results, copies in flight");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NSTG * STAGE];
    __shared__ __attribute__((aligned(16))) float part[KG][TT][256];
    __shared__ __attribute__((aligned(16))) int ids_of[AD ? KG : 1][64];
    __shared__ uint64_t lists[AD ? KG : 1][64];
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
    int id_l = -1;   // of token `lane`
    if (AD) id_l = p.ad.ids[min(lane, p.T - 1)];
#pragma unroll
    for (int c = 0; c < NSTG; ++c)
        if (c < nk) copy(c, ring + c * STAGE);
    // The low-rank part, 32 ranks at a time: the tokens' s, and NI adapters' rows at once,
    // straight from memory; the waves take the adapters in turn, one that several tokens
    // have once.  The first ones are requested here, behind the first copies.  Each
    // adapter's product is taken from zero and added in the lanes of its own tokens only,
    // so that no value of one adapter, an infinity or NaN included, meets another
    // request's row, and none of one half the other's sums.
    constexpr int H = GATED ? 2 : 1, NI = 8, LOADS = H * (TT + NI);
    static_assert(CPS * (NSTG - 1) + LOADS <= 63, "loads in flight");
    int rank_l = p.ad.R, aid[TT];              // the token's rank; the adapters of this lane's columns
    int count = 0, at = 0, ia[NI], k0 = 0;     // adapters with these ranks, the wave's next; the first rank
    bool leader = false;
    u32x4 va[NI][H], vb[TT][H];
    const rsrc_t sr = AD ? make_rsrc(p.ad.s, static_cast<uint32_t>(((p.T - 1) * p.ad.lds + H * p.ad.R) * 2)) : rsrc_t();
    auto tokens = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int h = 0; h < H; ++h)
                vb[j][h] = bload16(sr, aid[j] >= 0 && k0 + 8 * q < p.ad.R
                                           ? static_cast<uint32_t>((row + 16 * j) * p.ad.lds + h * p.ad.R + k0 + 8 * q) * 2 : NO_LANE);
        at = kg;
    };
    auto adapters = [&]() __attribute__((always_inline)) {   // the next NI of this wave
        const int ch = GATED ? row & 7 : row;
        const uint32_t bytes = static_cast<uint32_t>(nch) * p.ad.R * 2u;
        const uint32_t off = ch < nch && k0 + 8 * q < p.ad.R ? static_cast<uint32_t>(ch * p.ad.R + k0 + 8 * q) * 2 : NO_LANE;
        uint64_t of[NI];
#pragma unroll
        for (int n = 0; n < NI; ++n) of[n] = lists[kg][min(at + n * KG, 63)];
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const bool in = at + n * KG < count;
            ia[n] = in ? __builtin_amdgcn_readfirstlane(static_cast<int>(of[n])) : -1;
            const uint16_t* pb = p.ad.b + max(ia[n], 0) * p.ad.b_stride + static_cast<int64_t>(n0) * p.ad.R;
#pragma unroll
            for (int h = 0; h < H; ++h)   // gate's rows and up's, the lanes of the other half zeros
                va[n][h] = bload16(make_rsrc(pb + static_cast<int64_t>(h) * p.N * p.ad.R, bytes),
                                   in && (!GATED || (row >> 3) == h) ? off : NO_LANE);
        }
        at += NI * KG;
    };
    if (AD) {
        if (lane >= p.T || id_l < 0 || id_l >= p.ad.n) id_l = -1;
        leader = is_leader(id_l, 16 * TT, ids_of[kg]);
#pragma unroll
        for (int j = 0; j < TT; ++j) aid[j] = ids_of[kg][16 * j + row];
        if (p.ad.ranks != nullptr) rank_l = p.ad.ranks[max(id_l, 0)];
        count = list_adapters(leader, id_l, 1, 0, lists[kg]);   // all: their ranks are not waited for here
        tokens();
        adapters();
        // the waits below count these loads: they stay in front of them
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    f32x4 acc[TT] = {};
    for (int c = 0, buf = 0; c < nk; ++c) {
        // the stages behind this one, and behind the first ones the items, may still be on
        // their way
        const int behind = min(nk - 1 - c, NSTG - 1);
        if (AD && c < NSTG) {
            if (NSTG > 2 && behind == 2)
                __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * CPS + LOADS));
            else if (behind == 1)
                __builtin_amdgcn_s_waitcnt(waitcnt_vm(CPS + LOADS));
            else
                __builtin_amdgcn_s_waitcnt(waitcnt_vm(LOADS));
        } else if (NSTG > 2 && behind == 2) {
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * CPS));
        } else if (behind == 1) {
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(CPS));
        } else {
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        }
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
        __builtin_amdgcn_s_waitcnt(wait_vm_lds(63));   // the operands are read, so the buffer may be filled again
        asm volatile("" ::: "memory");
        if (c + NSTG < nk) copy(c + NSTG, st);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[j] = mfma16x16x32(a[s], b[s][j], acc[j]);
        buf = buf + 1 == NSTG ? 0 : buf + 1;
    }
    if (AD) {
        for (;;) {
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                if (ia[n] < 0) continue;
                // (at least 0, so that the lanes' differences stay inside 32 bits)
                const int rank = max(__builtin_amdgcn_readlane(rank_l, __builtin_ctzll(__ballot(id_l == ia[n]))), 0);
                if (rank < k0 + 32) {   // some lane holds less than 8 ranks
#pragma unroll
                    for (int h = 0; h < H; ++h) va[n][h] = low_ranks(va[n][h], rank - k0 - 8 * q);
                }
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    f32x4 low[H];
#pragma unroll
                    for (int h = 0; h < H; ++h) low[h] = mfma16x16x32(va[n][h], vb[j][h], f32x4{0, 0, 0, 0});
                    // gated: D rows 0 .. 7 are gate's, 8 .. 15 up's; zeros in the other half's
                    // rows of A do not keep its infinities out, so each half has its own product
                    if (aid[j] == ia[n]) acc[j] += q < 2 ? low[0] : low[H - 1];
                }
            }
            if (at >= count) {   // the next 32 ranks, of the adapters that have them
                k0 += 32;
                if (k0 >= p.ad.R) break;
                count = list_adapters(leader, id_l, rank_l, k0, lists[kg]);
                tokens();
            }
            adapters();
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

template <int TT, bool GATED, int KG, int NSTG>
static hipError_t few(const MatBf16Params& p, hipStream_t s) {
    constexpr int CH = GATED ? 8 : 16;
    auto kn = p.ad.s ? matmul_bf16_few_kernel<TT, KG, NSTG, GATED, true> : matmul_bf16_few_kernel<TT, KG, NSTG, GATED, false>;
    hipLaunchKernelGGL(kn, dim3((p.N + CH - 1) / CH), dim3(64 * KG), 0, s, p);
    return hipGetLastError();
}

hipError_t tiles_nt(const MatBf16Params& p, hipStream_t s);
hipError_t tiles_gated(const MatBf16Params& p, hipStream_t s);
hipError_t tiles_nn(const MatBf16Params& p, hipStream_t s);
hipError_t tiles_tn(const MatBf16Params& p, hipStream_t s);

// Up to 16 tokens the kernel for few tokens (T = 1 and 16: 1.1 to 1.8 times as fast as the
// best tile from 64 to 8192 weight rows, K 136 to 4096: N = 2816, K = 2112 3.6 and 3.8 us).
// Further as long as every workgroup has a CU of its own: to 32 tokens 1.2 to 1.6 times as
// fast (more workgroups: 5 to 10 % slower), to 48 1.0 to 1.3 times, to 64 as fast with K =
// 1424, 1.1 to 1.2 times with K up to 1024.  Three stages against two: 4 to 9 % less
// time up to 32 tokens, equal or slower for more.
template <bool GATED>
static hipError_t forward(const MatBf16Params& p, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.N) * (GATED ? 2 : 1);
    if (p.T <= 16) return few<1, GATED, 4, 3>(p, s);
    if (rows <= 256 * 16) {
        if (p.T <= 32) return few<2, GATED, 4, 3>(p, s);
        if (p.T <= 48) return few<3, GATED, 4, 2>(p, s);
        if (p.T <= 64 && p.K <= 1024) return few<4, GATED, 4, 2>(p, s);
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
