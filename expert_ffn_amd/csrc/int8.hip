// 8-bit integer products with a scale per token and per channel (W8A8):
//
//   out[t][n] = (sum_k x[t][k] w[n][k]) sx[t] sw[n] (+ bias[n])
//   gated:      act(out gate channel n) * (out up channel n), w = gate rows then up rows
//
// The sums are int32 and exact for K <= 131056 (128^2 K < 2^31), so neither the
// split of K over waves nor any order changes a result.  The epilogue is fp32
// and rounds once to the output type.
//
// MFMA operands: A = channels (weight rows), B = tokens, D column = token, so a
// lane holds 4 consecutive channels of one token.  A and B take their K bytes in
// the same order, so any fixed order of K inside an instruction is right.
#include "block.h"
#include "common.h"

namespace moe {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

__device__ __forceinline__ i32x4 mfma16_i8(const u32x4& a, const u32x4& b, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
__device__ __forceinline__ i32x16 mfma32_i8(const u32x4& a, const u32x4& b, const i32x16& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// resource over rows [r0, r0 + rows) of a K-byte-row matrix (at most 2 GiB apart)
__device__ __forceinline__ rsrc_t rows_rsrc(const int8_t* base, int64_t ld, int r0, int rows, int K) {
    return make_rsrc(base + static_cast<int64_t>(r0) * ld, static_cast<uint32_t>((rows - 1) * ld + K));
}

// LDS DMA: 64 lanes x 16 bytes to dst + 16 * lane (dst uniform); a lane past the
// resource writes zeros.  Completion is the wave's vmcnt, waited for by the caller.
__device__ __forceinline__ void lds_copy16(rsrc_t r, uint8_t* dst, uint32_t off, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(dst)), 16, off, soff, 0, 0);
}

__device__ __forceinline__ void store_out(const MatI8Params& p, int t, int n, float v) {
    const int64_t i = static_cast<int64_t>(t) * p.ldo + n;
    if (p.out_dt == F32)
        static_cast<float*>(p.out)[i] = v;
    else
        static_cast<uint16_t*>(p.out)[i] = f32_to_bf16(v);
}

// ------------------------------------------------------------ few tokens --
// Weight streaming for T <= 64: a workgroup takes 16 RT channels (gated: those
// gate rows and the matching up rows) and all tokens (TT tiles of 16); its NW
// waves take the 64-byte pieces of K in turn and their int32 sums meet in LDS.
// Weights go from memory to registers, U pieces requested at a time; the tokens'
// codes come from L2.
template <int RT, int TT, int NW, int U, bool GATED>
__global__ __launch_bounds__(64 * NW) void matmul_i8_stream_kernel(MatI8Params p) {
    constexpr int R = GATED ? 2 * RT : RT;   // weight row tiles
    __shared__ i32x4 red[NW][R * TT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16 * RT, l16 = lane & 15, kq = (lane >> 4) * 16;
    const int nrow = min(16 * RT, p.N - n0);
    const rsrc_t wr0 = rows_rsrc(p.w, p.ldw, n0, nrow, p.K);
    const rsrc_t wr1 = rows_rsrc(p.w, p.ldw, GATED ? p.N + n0 : n0, nrow, p.K);
    const rsrc_t xr = rows_rsrc(p.x, p.ldx, 0, p.T, p.K);
    uint32_t wo[RT], xo[TT];
#pragma unroll
    for (int r = 0; r < RT; ++r) wo[r] = 16 * r + l16 < nrow ? static_cast<uint32_t>((16 * r + l16) * p.ldw + kq) : NO_LANE;
#pragma unroll
    for (int i = 0; i < TT; ++i) xo[i] = 16 * i + l16 < p.T ? static_cast<uint32_t>((16 * i + l16) * p.ldx + kq) : NO_LANE;
    i32x4 acc[R][TT] = {};
    for (int k0 = 64 * wave; k0 < p.K; k0 += 64 * NW * U) {
        u32x4 a[U][R], b[U][TT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 64 * NW * u;
            const bool ok = k + kq < p.K;   // K is a multiple of 16
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                a[u][r] = bload16s(wr0, ok ? wo[r] : NO_LANE, k);
                if (GATED) a[u][RT + r] = bload16s(wr1, ok ? wo[r] : NO_LANE, k);
            }
#pragma unroll
            for (int i = 0; i < TT; ++i) b[u][i] = bload16s(xr, ok ? xo[i] : NO_LANE, k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < TT; ++i) acc[r][i] = mfma16_i8(a[u][r], b[u][i], acc[r][i]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < TT; ++i) red[wave][r * TT + i][lane] = acc[r][i];
    __syncthreads();
    // item = (row tile, token tile, lane): 4 consecutive channels of one token
    for (int it = tid; it < RT * TT * 64; it += 64 * NW) {
        const int tile = it >> 6, l = it & 63;
        i32x4 s = red[0][tile][l], s2 = {};
#pragma unroll
        for (int v = 1; v < NW; ++v) s += red[v][tile][l];
        if (GATED) {
            s2 = red[0][RT * TT + tile][l];
#pragma unroll
            for (int v = 1; v < NW; ++v) s2 += red[v][RT * TT + tile][l];
        }
        const int t = 16 * (tile % TT) + (l & 15), n = n0 + 16 * (tile / TT) + 4 * (l >> 4);
        if (t >= p.T) continue;
        const float sx = p.sx[t];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n + j >= p.N) continue;
            float v = static_cast<float>(s[j]) * sx * p.sw[n + j];
            if (GATED)
                v = act_fn(p.act, v) * (static_cast<float>(s2[j]) * sx * p.sw[p.N + n + j]);
            else if (p.bias != nullptr)
                v += p.bias[n + j];
            store_out(p, t, n + j, v);
        }
    }
}

// ----------------------------------------------------------- many tokens --
// Tiles of BN weight rows x BT tokens, WN x WT waves, each wave a block of
// 32-row by 32-token MFMA tiles.  128-byte K steps of both operands are copied by
// LDS DMA into two stages in turn: a step's copies are requested right after the
// barrier that ends the reads of the stage they overwrite, and waited for one
// step later.  A copy writes 8 rows of 128 bytes in lane order; the 16-byte
// chunk q of row r is stored at position q ^ (r & 7), so that the 8 rows that
// are read together fall into different banks.  Gated: the tile's first BN / 2
// rows are gate rows and the others the matching up rows; a wave owns both rows
// of its channels.
template <int BN, int BT, int WN, int WT, bool GATED>
__global__ __launch_bounds__(64 * WN * WT, 1) void matmul_i8_tile_kernel(MatI8Params p, int nt_n, int nt_t) {
    constexpr int NW = WN * WT, NB = BN / WN / 32, TB = BT / WT / 32;
    constexpr int STAGE = (BN + BT) * 128, DA = BN / 8 / NW, DB = BT / 8 / NW;
    constexpr int CH = GATED ? BN / 2 : BN;   // output channels per tile
    static_assert(DA * 8 * NW == BN && DB * 8 * NW == BT && (!GATED || (NB % 2 == 0 && DA % 2 == 0)), "tile shape");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
    __shared__ float sws[BN], sxs[BT], bs[BN];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wt = wave / WN;
    // XCD-aware order: workgroups go to the 8 XCDs in turn, so XCD x takes one
    // contiguous range of the tile list, which runs down 8 token tiles before it
    // goes to the next channel tile
    const int ntile = nt_n * nt_t, per = (ntile + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (id >= ntile || (blockIdx.x >> 3) >= per) return;
    constexpr int GRP = 8;
    const int g0 = id / (GRP * nt_n) * GRP, gh = min(GRP, nt_t - g0), r = id - g0 * nt_n;
    const int t0 = (g0 + r % gh) * BT, n0 = r / gh * CH;
    const int nch = min(CH, p.N - n0), ntok = min(BT, p.T - t0);
    const rsrc_t wr0 = rows_rsrc(p.w, p.ldw, n0, nch, p.K);
    const rsrc_t wr1 = rows_rsrc(p.w, p.ldw, GATED ? p.N + n0 : n0, nch, p.K);
    const rsrc_t xr = rows_rsrc(p.x, p.ldx, t0, ntok, p.K);
    for (int i = tid; i < BN; i += 64 * NW) {
        const int c = GATED && i >= CH ? i - CH : i;
        sws[i] = c < nch ? p.sw[(GATED && i >= CH ? p.N : 0) + n0 + c] : 0.0f;
        bs[i] = !GATED && p.bias != nullptr && c < nch ? p.bias[n0 + c] : 0.0f;
    }
    for (int i = tid; i < BT; i += 64 * NW) sxs[i] = i < ntok ? p.sx[t0 + i] : 0.0f;
    // copies: this wave's rows 8 (wave + NW i) .. + 7 of each operand
    const int sub = lane >> 3, chunk = ((lane & 7) ^ sub) * 16;
    uint32_t ao[DA], bo[DB];
#pragma unroll
    for (int i = 0; i < DA; ++i) {
        const int row = 8 * (wave + NW * i) + sub, c = GATED && row >= CH ? row - CH : row;
        ao[i] = c < nch ? static_cast<uint32_t>(c * p.ldw + chunk) : NO_LANE;
    }
#pragma unroll
    for (int i = 0; i < DB; ++i) {
        const int row = 8 * (wave + NW * i) + sub;
        bo[i] = row < ntok ? static_cast<uint32_t>(row * p.ldx + chunk) : NO_LANE;
    }
    const int nk = (p.K + 127) / 128;
    auto dma = [&](int c, int buf) {
        const int k = 128 * c;
        const bool in = k + chunk < p.K;   // the last step may end inside (K is a multiple of 16)
#pragma unroll
        for (int i = 0; i < DA; ++i) {
            // copies i >= DA / 2 are the up rows of a gated tile
            uint8_t* dst = lds + buf * STAGE + 8 * (wave + NW * i) * 128;
            if (GATED && i >= DA / 2)
                lds_copy16(wr1, dst, in ? ao[i] : NO_LANE, k);
            else
                lds_copy16(wr0, dst, in ? ao[i] : NO_LANE, k);
        }
#pragma unroll
        for (int i = 0; i < DB; ++i)
            lds_copy16(xr, lds + buf * STAGE + (BN + 8 * (wave + NW * i)) * 128, in ? bo[i] : NO_LANE, k);
    };
    // fragments: row l & 31 of a 32-row block, chunk 2 s + (l >> 5)
    const int l32 = lane & 31, hh = lane >> 5;
    int arow[NB], brow[TB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (GATED)   // first half of the blocks: gate rows, second half: up rows
            arow[b] = (b < NB / 2 ? 0 : CH) + wn * (CH / WN) + 32 * (b % (NB / 2 > 0 ? NB / 2 : 1)) + l32;
        else
            arow[b] = wn * (BN / WN) + 32 * b + l32;
    }
#pragma unroll
    for (int b = 0; b < TB; ++b) brow[b] = BN + wt * (BT / WT) + 32 * b + l32;
    i32x16 acc[NB][TB] = {};
    dma(0, 0);
    for (int c = 0; c < nk; ++c) {
        // stage c has landed (for every wave after the barrier), and the reads of
        // stage c - 1 are over: its buffer takes stage c + 1
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        __syncthreads();
        if (c + 1 < nk) dma(c + 1, (c + 1) & 1);
        const uint8_t* st = lds + (c & 1) * STAGE;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int co = ((2 * s + hh) ^ (l32 & 7)) * 16;
            u32x4 a[NB], b[TB];
#pragma unroll
            for (int i = 0; i < NB; ++i) a[i] = *reinterpret_cast<const u32x4*>(st + arow[i] * 128 + co);
#pragma unroll
            for (int i = 0; i < TB; ++i) b[i] = *reinterpret_cast<const u32x4*>(st + brow[i] * 128 + co);
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j) acc[i][j] = mfma32_i8(a[i], b[j], acc[i][j]);
        }
    }
    __syncthreads();   // the stages are free: each wave transposes through its own part
    // Epilogue, 32 tokens at a time: the wave's [32 tokens][CW channels] go through
    // LDS (16-byte chunks at position c ^ token) and leave as row pieces.
    constexpr int CW = CH / WN, NBO = CW / 32, REG = 2 * STAGE / NW;
    static_assert(32 * CW * 4 <= REG, "epilogue region");
    uint8_t* my = lds + wave * REG;
    const bool f32 = p.out_dt == F32;
    const int es = f32 ? 4 : 2, cpr = CW * es / 16;   // 16-byte chunks per row (a power of two)
    const bool vec = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ldo * es % 16 == 0;
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
        const int tl = wt * (BT / WT) + 32 * tb;   // first token of the block in the tile
        const float sx = sxs[tl + l32];
#pragma unroll
        for (int b = 0; b < NBO; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // channels 32 b + 8 q + 4 hh .. + 3
                const int cl = 32 * b + 8 * q + 4 * hh, cw = wn * CW + cl;
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = static_cast<float>(acc[b][tb][4 * q + j]) * sx * sws[cw + j];
                    if (GATED)
                        v[j] = act_fn(p.act, v[j]) *
                               (static_cast<float>(acc[NB / 2 + b < NB ? NB / 2 + b : 0][tb][4 * q + j]) * sx * sws[CH + cw + j]);
                    else
                        v[j] += bs[cw + j];
                }
                if (f32) {
                    *reinterpret_cast<f32x4*>(my + l32 * CW * 4 + (((cl >> 2) ^ (l32 & (cpr - 1))) << 4)) =
                        f32x4{v[0], v[1], v[2], v[3]};
                } else {
                    *reinterpret_cast<u32x2*>(my + l32 * CW * 2 + (((cl >> 3) ^ (l32 & (cpr - 1))) << 4) + 8 * hh) =
                        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                }
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        for (int it = lane; it < 32 * cpr; it += 64) {
            const int tok = it / cpr, c = it & (cpr - 1);
            const u32x4 v = *reinterpret_cast<const u32x4*>(my + tok * CW * es + ((c ^ (tok & (cpr - 1))) << 4));
            const int t = tl + tok, ch = wn * CW + c * (16 / es);
            if (t >= ntok || ch >= nch) continue;
            const int64_t o = static_cast<int64_t>(t0 + t) * p.ldo + n0 + ch;
            if (f32) {
                float* d = static_cast<float*>(p.out) + o;
                if (vec && ch + 4 <= nch) {
                    *reinterpret_cast<u32x4*>(d) = v;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (ch + j < nch) d[j] = __uint_as_float(v[j]);
                }
            } else {
                uint16_t* d = static_cast<uint16_t*>(p.out) + o;
                if (vec && ch + 8 <= nch) {
                    *reinterpret_cast<u32x4*>(d) = v;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (ch + j < nch) d[j] = static_cast<uint16_t>(v[j >> 1] >> (16 * (j & 1)));
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <int RT, int TT, int NW, int U, bool GATED>
static hipError_t stream(const MatI8Params& p, hipStream_t s) {
    hipLaunchKernelGGL((matmul_i8_stream_kernel<RT, TT, NW, U, GATED>), dim3((p.N + 16 * RT - 1) / (16 * RT)),
                       dim3(64 * NW), 0, s, p);
    return hipGetLastError();
}

template <int BN, int BT, int WN, int WT, bool GATED>
static hipError_t tile(const MatI8Params& p, hipStream_t s) {
    constexpr int CH = GATED ? BN / 2 : BN;
    const int nt_n = (p.N + CH - 1) / CH, nt_t = (p.T + BT - 1) / BT;
    const int per = (nt_n * nt_t + 7) / 8;
    hipLaunchKernelGGL((matmul_i8_tile_kernel<BN, BT, WN, WT, GATED>), dim3(8 * per), dim3(64 * WN * WT), 0, s, p, nt_n,
                       nt_t);
    return hipGetLastError();
}

template <bool GATED>
static hipError_t dispatch(const MatI8Params& p, hipStream_t s) {
    if (p.T <= 16) return stream<1, 1, 8, 6, GATED>(p, s);
    if (p.T <= 32) return stream<1, 2, 8, 4, GATED>(p, s);
    if (p.T <= 64) return stream<1, 4, 8, 3, GATED>(p, s);
    const int64_t rows = static_cast<int64_t>(p.N) * (GATED ? 2 : 1);
    const int64_t big = ((rows + 255) / 256) * ((p.T + 255) / 256);
    if (big >= 200) return tile<256, 256, 2, 4, GATED>(p, s);
    return tile<128, 128, 2, 2, GATED>(p, s);
}

hipError_t launch_matmul_i8(const MatI8Params& p, bool gated, hipStream_t s) {
    return gated ? dispatch<true>(p, s) : dispatch<false>(p, s);
}

}  // namespace moe
