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
#include <algorithm>

#include "block.h"
#include "common.h"

namespace moe {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

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

// Tiles of BN weight rows x BT tokens, WN x WT waves, each wave a block of
// 32-row by 32-token MFMA tiles.  K steps of 128 bytes of both operands are copied
// by LDS DMA into a ring of NSTG stages (64-byte steps with twice the stages took
// 6 to 20 % longer: each copy then touches 16 half lines of L2).  A copy writes 8
// rows in lane order; the 16-byte chunk q of row r is stored at position q ^
// swz(r).  A 16-byte read is served 16 lanes at a time, lanes 0-3, 12-15, 20-27
// (and 4-11, 16-19, 28-31) together: swz makes their 16 rows fall into all 64 banks.
//
// Within a step the operands of MFMA round s + 1 are read while round s runs.
// The step's last round runs after the barrier: at the barrier every wave holds
// the last operands of stage c in registers and its copies of stage c + 1 have
// landed, so the reads of stage c + 1 begin, and the copies of stage c + NSTG go
// to the buffer of stage c, while that round is computed.
//
// KG > 1: KG groups of WN x WT waves, each with a ring of its own, take the K
// steps in turn and their int32 tiles are added through LDS.
//
// Gated: each 32-row block holds 16 gate rows, then the up rows of the same 16
// channels, so a lane holds both products of its channels.
__host__ __device__ constexpr int waitcnt_vm_lds(int n) { return waitcnt_vm(n) & ~0x0F00; }   // and LDS reads to 0

// the rows of out are 16-byte aligned
__host__ __device__ __forceinline__ bool rows_in_pieces(const MatI8Params& p) {
    return reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ldo * (p.out_dt == F32 ? 4 : 2) % 16 == 0;
}

// 16-byte chunk q of row r is stored at position q ^ swz(r)
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 3); }

template <int BN, int BT, int WN, int WT, int NSTG, int KG, bool GATED, int OT, bool PIECES>
__global__ __launch_bounds__(64 * WN * WT * KG, 1) void matmul_i8_tile_kernel(MatI8Params p, int nt_n, int nt_t) {
    constexpr int NW = WN * WT, NB = BN / WN / 32, TB = BT / WT / 32;
    constexpr int BK = 128, RPC = 1024 / BK, CPR = BK / 16;   // K bytes of a step, rows of a copy, chunks of a row
    constexpr int STAGE = (BN + BT) * BK, DA = BN / RPC / NW, DB = BT / RPC / NW, CPS = DA + DB;
    constexpr int CH = GATED ? BN / 2 : BN;   // output channels per tile
    constexpr int CW = CH / WN;               // of a wave
    constexpr int RING = NSTG * STAGE, NTH = 64 * NW * KG;
    static_assert(DA * RPC * NW == BN && DB * RPC * NW == BT && BN % 32 == 0, "tile shape");
    static_assert(NSTG >= 2 && NSTG <= 4 && CPS * (NSTG - 1) <= 63, "copies in flight");
    static_assert((KG - 1) * BN * BT * 4 <= KG * RING, "epilogue regions");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * RING];
    __shared__ float sws[BN], sxs[BT], bs[BN];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wid / NW, wave = wid % NW, wn = wave % WN, wt = wave / WN;
    // XCD-aware order: workgroups go to the 8 XCDs in turn, so XCD x takes one
    // contiguous range of the tile list, which runs down 8 token tiles before it
    // goes to the next channel tile
    const int ntile = nt_n * nt_t, per = (ntile + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (id >= ntile) return;
    constexpr int GRP = 8;
    const int g0 = id / (GRP * nt_n) * GRP, gh = min(GRP, nt_t - g0), r = id - g0 * nt_n;
    const int t0 = (g0 + r % gh) * BT, n0 = r / gh * CH;
    const int nch = min(CH, p.N - n0), ntok = min(BT, p.T - t0);
    const rsrc_t wr0 = rows_rsrc(p.w, p.ldw, n0, nch, p.K);
    const rsrc_t wr1 = rows_rsrc(p.w, p.ldw, GATED ? p.N + n0 : n0, nch, p.K);
    const rsrc_t xr = rows_rsrc(p.x, p.ldx, t0, ntok, p.K);
    uint8_t* ring = lds + kg * RING;
    // copies: this wave's rows RPC (wave + NW i) .. of each operand, lane l row l / CPR
    auto crow = [&](int i) { return RPC * (wave + NW * i) + lane / CPR; };
    auto chunk = [&](int i) { return ((lane % CPR) ^ swz(crow(i))) * 16; };
    auto channel = [](int row) { return GATED ? (row >> 5) * 16 + (row & 15) : row; };   // of a tile row
    auto is_up = [](int row) { return GATED && (row & 16); };
    uint32_t ao[DA], bo[DB];
#pragma unroll
    for (int i = 0; i < DA; ++i) {
        const int c = channel(crow(i));
        ao[i] = c < nch ? static_cast<uint32_t>(c * p.ldw + chunk(i)) : NO_LANE;
    }
#pragma unroll
    for (int i = 0; i < DB; ++i) {
        const int row = crow(i);
        bo[i] = row < ntok ? static_cast<uint32_t>(row * p.ldx + chunk(i)) : NO_LANE;
    }
    const int nk = ((p.K + BK - 1) / BK + KG - 1) / KG;   // steps of each group, the same for all
    // copy i of stage c: weight rows (RPC of them lie on one side of a gated
    // block), then tokens.  Chunks past K are zeros: nothing is read for them.
    // Stages past the last are not requested either, by a copy of the loop's body
    // without copies (32 to 128 tokens: 3 to 4 % less time).  The largest tile requests them as zeros: its body is 10 KB, and
    // twice that took 1 to 7 % longer.
    constexpr bool TAIL = NSTG > 2;
    auto copy = [&](int c, uint8_t* st, int i) {
        const int k = BK * (c * KG + kg);
        // the scalar offset stays inside the resource: the range check subtracts it
        // from the resource's size
        const uint32_t so = k < p.K ? k : 0;
        if (i < DA) {
            const uint32_t o = k + chunk(i) < p.K ? ao[i] : NO_LANE;
            uint8_t* dst = st + RPC * (wave + NW * i) * BK;
            if (is_up(RPC * (wave + NW * i)))
                lds_copy16(wr1, dst, o, so);
            else
                lds_copy16(wr0, dst, o, so);
        } else {
            const int j = i - DA;
            lds_copy16(xr, st + (BN + RPC * (wave + NW * j)) * BK, k + chunk(j) < p.K ? bo[j] : NO_LANE, so);
        }
    };
    // fragments: row l & 31 of a 32-row block (blocks start at multiples of 32), chunk 2 s + (l >> 5)
    const int l32 = lane & 31, hh = lane >> 5;
    int arow[NB], brow[TB];
#pragma unroll
    for (int b = 0; b < NB; ++b) arow[b] = wn * (BN / WN) + 32 * b + l32;
#pragma unroll
    for (int b = 0; b < TB; ++b) brow[b] = BN + wt * (BT / WT) + 32 * b + l32;
    u32x4 fa[2][NB], fb[2][TB];
    auto read = [&](const uint8_t* st, int s, int set) {
        const int co = ((2 * s + hh) ^ swz(l32)) * 16;
#pragma unroll
        for (int i = 0; i < NB; ++i) fa[set][i] = *reinterpret_cast<const u32x4*>(st + arow[i] * BK + co);
#pragma unroll
        for (int i = 0; i < TB; ++i) fb[set][i] = *reinterpret_cast<const u32x4*>(st + brow[i] * BK + co);
    };
    i32x16 acc[NB][TB] = {};
    // Round s of a step, with its share of the copies of stage c between its MFMAs
    // (c < 0: none).  A stage is requested over M MFMAs, from the last round of one
    // step into the next, so that the address unit (16 cycles a copy, for all waves
    // of the CU) works beside the MFMAs: a wave that issues its copies in one go
    // waits for it with its MFMAs behind them (T = 512, N = 5632, K = 2816: 16.6 us,
    // spread 14.0).  With two stages the copies are wanted a step later and start
    // within two rounds.
    constexpr int S = BK / 32;   // rounds of a step (even: a step starts with set 0)
    constexpr int M = (NSTG > 2 ? S : 2) * NB * TB;
    auto round = [&](int s, int c, uint8_t* to) {
#pragma unroll
        for (int m = 0; m < NB * TB; ++m) {
            const int i = m / TB, j = m % TB, slot = (s + 1) % S * NB * TB + m;
            acc[i][j] = mfma32_i8(fa[s & 1][i], fb[s & 1][j], acc[i][j]);
            if (c >= 0) {
#pragma unroll
                for (int q = slot * CPS / M; q < (slot + 1) * CPS / M && q < CPS; ++q) copy(c, to, q);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto most = [&](const uint8_t* st, int c, uint8_t* to) {   // rounds 0 .. S - 2, each reading the next one's operands first
#pragma unroll
        for (int s = 0; s + 1 < S; ++s) {
            read(st, s + 1, (s + 1) & 1);
            __builtin_amdgcn_sched_barrier(0);
            round(s, c, to);
        }
    };
#pragma unroll
    for (int c = 0; c < NSTG; ++c) {
        if (TAIL && c >= nk) break;
#pragma unroll
        for (int q = 0; q < CPS; ++q) copy(c, ring + c * STAGE, q);
    }
    // per-row factors, behind the first copies
    for (int i = tid; i < BN; i += NTH) {
        const int c = channel(i);
        sws[i] = c < nch ? p.sw[(is_up(i) ? p.N : 0) + n0 + c] : 0.0f;
        bs[i] = !GATED && p.bias != nullptr && c < nch ? p.bias[n0 + c] : 0.0f;
    }
    for (int i = tid; i < BT; i += NTH) sxs[i] = i < ntok ? p.sx[t0 + i] : 0.0f;
    // (those loads were issued after the copies, so their wait covered every copy)
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(0));
    __syncthreads();
    read(ring, 0, 0);
    most(ring, -1, ring);
    int buf = 0;
    // from step c to step c + 1: `left` of the stages behind that one may still be on their way
    auto step = [&](int left, int next) {
        if (NSTG > 3 && left >= 2)
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(CPS * 2));
        else if (NSTG > 2 && left >= 1)
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(CPS));
        else
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(0));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        uint8_t* done = ring + buf * STAGE;
        buf = buf + 1 == NSTG ? 0 : buf + 1;
        const uint8_t* st = ring + buf * STAGE;
        read(st, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        round(S - 1, next, done);
        most(st, next, done);
    };
    int c = 0;
    for (; c + (TAIL ? NSTG : 1) < nk; ++c) step(NSTG - 2, c + NSTG);
    if (TAIL)
        for (; c + 1 < nk; ++c) step(nk - 2 - c, -1);
    round(S - 1, -1, ring);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(0));   // zero stages have landed too
    __syncthreads();   // the rings are free
    if (KG > 1) {
        int* part = reinterpret_cast<int*>(lds);
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<i32x4*>(part + (((((kg - 1) * NW + wave) * NB + i) * TB + j) * 4 + v) * 256 + lane * 4) =
                            i32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int q = 1; q < KG; ++q)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const i32x4 o = *reinterpret_cast<const i32x4*>(
                            part + (((((q - 1) * NW + wave) * NB + i) * TB + j) * 4 + v) * 256 + lane * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * v + e] += o[e];
                    }
    }
    // Epilogue, 32 tokens at a time: the wave's [32 tokens][CW channels] go through
    // LDS (16-byte chunks at position c ^ token) and leave as row pieces.  With
    // groups, the partial sums may lie where another wave of group 0 still reads:
    // the waves' regions start behind them.
    constexpr int PART = KG > 1 ? (KG - 1) * BN * BT * 4 : 0;
    constexpr bool f32 = OT == F32;
    constexpr int es = f32 ? 4 : 2, cpr = CW * es / 16;   // 16-byte chunks per row
    constexpr bool p2 = (cpr & (cpr - 1)) == 0;           // else the rows are 16 bytes apart instead
    constexpr int RS = CW * es + (p2 ? 0 : 16);
    static_assert(PART + 32 * RS * NW <= KG * RING, "epilogue regions");
    uint8_t* my = lds + PART + wave * 32 * RS;
    auto at = [&](int tok, int c) { return my + tok * RS + ((p2 ? c ^ (tok & (cpr - 1)) : c) << 4); };
    const bool vec = KG == 1 || rows_in_pieces(p);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
        const int tl = wt * (BT / WT) + 32 * tb;   // first token of the block in the tile
        const float sx = sxs[tl + l32];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int q = 0; q < (GATED ? 2 : 4); ++q) {   // 4 channels: tile rows rw .. rw + 3 (and up rows 16 further)
                const int cl = (GATED ? 16 : 32) * b + 8 * q + 4 * hh, rw = wn * (BN / WN) + 32 * b + 8 * q + 4 * hh;
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = static_cast<float>(acc[b][tb][4 * q + j]) * sx * sws[rw + j];
                    if (GATED)
                        v[j] = act_fn(p.act, v[j]) *
                               (static_cast<float>(acc[b][tb][GATED ? 8 + 4 * q + j : 0]) * sx * sws[rw + 16 + j]);
                    else
                        v[j] += bs[rw + j];
                }
                if (f32) {
                    *reinterpret_cast<f32x4*>(at(l32, cl >> 2)) = f32x4{v[0], v[1], v[2], v[3]};
                } else {
                    *reinterpret_cast<u32x2*>(at(l32, cl >> 3) + 8 * hh) =
                        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                }
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (PIECES) {
#pragma unroll 4
            for (int i0 = 0; i0 < 32 * cpr; i0 += 64) {
                const int it = i0 + lane;
                const int tok = it / cpr, c = it % cpr;
                const u32x4 v = *reinterpret_cast<const u32x4*>(at(tok, c));
                const int t = tl + tok, ch = wn * CW + c * (16 / es);
                if (t >= ntok || ch >= nch) continue;
                uint8_t* d = static_cast<uint8_t*>(p.out) + (static_cast<int64_t>(t0 + t) * p.ldo + n0 + ch) * es;
                if (vec && ch + 16 / es <= nch) {
                    *reinterpret_cast<u32x4*>(d) = v;
                } else if (f32) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (ch + j < nch) reinterpret_cast<uint32_t*>(d)[j] = v[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (ch + j < nch) reinterpret_cast<uint16_t*>(d)[j] = static_cast<uint16_t>(v[j >> 1] >> (16 * (j & 1)));
                }
            }
        } else {
            // Rows that are not 16-byte aligned (!PIECES): neighbouring lanes store neighbouring
            // elements (T = 4096, N = 5633, K = 704: 40 us, the chunks' elements lane by
            // lane 63).  The small tiles with K groups have one or two waves here, and
            // the fewer reads of the chunks serve them (N = 703: 4.0 us against 4.4).
#pragma unroll 4
            for (int i0 = 0; i0 < 32 * CW; i0 += 64) {
                const int it = i0 + lane;
                const int tok = it / CW, e = it % CW;
                const uint8_t* s = at(tok, e * es / 16) + e * es % 16;
                const int t = tl + tok, ch = wn * CW + e;
                if (t >= ntok || ch >= nch) continue;
                const int64_t o = static_cast<int64_t>(t0 + t) * p.ldo + n0 + ch;
                if (f32)
                    static_cast<uint32_t*>(p.out)[o] = *reinterpret_cast<const uint32_t*>(s);
                else
                    static_cast<uint16_t*>(p.out)[o] = *reinterpret_cast<const uint16_t*>(s);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Few tokens (at most 16 TT): workgroups of 16 weight rows (gated: 8 gate rows and
// their up rows), so that all CUs take part, and FEW_KG waves that take the 128-byte K
// steps in turn.  Each wave has a ring of its own, so none waits for another before
// the sums are added.  MFMA 16x16x64: lane l holds row l & 15, chunk 4 s + (l >> 4) of
// both operands; swz16 spreads the rows that are read together over all banks.
//
// What is left are the launch, about 2 us of the kernel's time, and the memory's rate
// (16 MB of weights, N = 5632, K = 2816, 16 tokens: 4.9 us; 6 MB: 2.9 us).  Three stages took 0 to 8 %
// longer, 8 waves 2 to 30 %: more LDS per workgroup leaves fewer of them on a CU.
__device__ __forceinline__ int swz16(int r) { return (r & 15) >> 1; }

constexpr int FEW_KG = 4, FEW_NSTG = 2;

template <int TT, bool GATED, int OT>
__global__ __launch_bounds__(64 * FEW_KG) void matmul_i8_few_kernel(MatI8Params p) {
    constexpr int KG = FEW_KG, NSTG = FEW_NSTG, BK = 128, STAGE = (16 + 16 * TT) * BK, CH = GATED ? 8 : 16, CPS = 2 + 2 * TT;
    static_assert(KG >= 4 && NSTG == 2 && CPS <= 63, "256 threads for the results, copies in flight");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NSTG * STAGE];
    __shared__ __attribute__((aligned(16))) int part[KG][TT][256];
    const int tid = threadIdx.x, lane = tid & 63, kg = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * CH, nch = min(CH, p.N - n0);
    const rsrc_t wr0 = rows_rsrc(p.w, p.ldw, n0, nch, p.K);
    const rsrc_t wr1 = rows_rsrc(p.w, p.ldw, GATED ? p.N + n0 : n0, nch, p.K);
    const rsrc_t xr = rows_rsrc(p.x, p.ldx, 0, p.T, p.K);
    // this thread's results: channel ch of tokens tok, tok + 16 ..
    const int tok = tid / CH, ch = tid % CH;
    const bool mine = tid < 16 * CH && ch < nch;
    float sx[TT] = {}, sg = 0.0f, su = 0.0f, bias = 0.0f;
    if (mine) {
#pragma unroll
        for (int j = 0; j < TT; ++j) sx[j] = p.sx[min(tok + 16 * j, p.T - 1)];
        sg = p.sw[n0 + ch];
        if (GATED) su = p.sw[p.N + n0 + ch];
        if (!GATED && p.bias != nullptr) bias = p.bias[n0 + ch];
    }
    // copies: 8 rows each, lane l row l / 8, chunk (l % 8) ^ swz16(row)
    uint8_t* ring = lds + kg * NSTG * STAGE;
    uint32_t chunk[2], wo[2], xo[2 * TT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + lane / 8, c = GATED ? row & 7 : row;
        chunk[i] = ((lane % 8) ^ swz16(row)) * 16;
        wo[i] = c < nch ? static_cast<uint32_t>(c * p.ldw + chunk[i]) : NO_LANE;
    }
#pragma unroll
    for (int i = 0; i < 2 * TT; ++i) {
        const int row = 8 * i + lane / 8;
        xo[i] = row < p.T ? static_cast<uint32_t>(row * p.ldx + chunk[i & 1]) : NO_LANE;
    }
    const int nk = ((p.K + BK - 1) / BK + KG - 1) / KG;
    // chunks past K are zeros; stages past the last are not requested (T = 16, N = 5632,
    // K = 704: 3.0 -> 2.7 us)
    auto copy = [&](int c, uint8_t* st) {
        const uint32_t k = BK * (c * KG + kg);
        const uint32_t so = k < static_cast<uint32_t>(p.K) ? k : 0;   // inside the resource
#pragma unroll
        for (int i = 0; i < CPS; ++i) {
            const bool in = k + chunk[i & 1] < static_cast<uint32_t>(p.K);
            if (i < 2)
                lds_copy16(i == 0 ? wr0 : wr1, st + i * 8 * BK, in ? wo[i] : NO_LANE, so);
            else
                lds_copy16(xr, st + i * 8 * BK, in ? xo[i - 2] : NO_LANE, so);
        }
    };
#pragma unroll
    for (int c = 0; c < NSTG; ++c)
        if (c < nk) copy(c, ring + c * STAGE);
    i32x4 acc[TT] = {};
    const int row = lane & 15, q = lane >> 4;
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
            const int o = row * BK + (((4 * s + q) ^ swz16(row)) << 4);
            a[s] = *reinterpret_cast<const u32x4*>(st + o);
#pragma unroll
            for (int j = 0; j < TT; ++j) b[s][j] = *reinterpret_cast<const u32x4*>(st + (16 + 16 * j) * BK + o);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(63));   // read, so the buffer may be filled again
        asm volatile("" ::: "memory");
        if (c + NSTG < nk) copy(c + NSTG, st);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < TT; ++j)
                acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a[s]), __builtin_bit_cast(i32x4, b[s][j]),
                                                               acc[j], 0, 0, 0);
        buf = buf + 1 == NSTG ? 0 : buf + 1;
    }
    // lane l: token l & 15 of tile j, tile rows 4 (l >> 4) ..
#pragma unroll
    for (int j = 0; j < TT; ++j) *reinterpret_cast<i32x4*>(&part[kg][j][lane * 4]) = acc[j];
    __syncthreads();
    if (!mine) return;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = tok + 16 * j;
        if (t >= p.T) return;
        auto total = [&](int r) {
            int s = 0;
#pragma unroll
            for (int g = 0; g < KG; ++g) s += part[g][j][(tok + 16 * (r >> 2)) * 4 + (r & 3)];
            return static_cast<float>(s);
        };
        float v = total(ch) * sx[j] * sg;
        if (GATED)
            v = act_fn(p.act, v) * (total(8 + ch) * sx[j] * su);
        else
            v += bias;
        const int64_t o = static_cast<int64_t>(t) * p.ldo + n0 + ch;
        if (OT == F32)
            static_cast<float*>(p.out)[o] = v;
        else
            static_cast<uint16_t*>(p.out)[o] = static_cast<uint16_t>(pack_bf16x2(v, v));
    }
}

template <int TT, bool GATED>
static hipError_t few(const MatI8Params& p, hipStream_t s) {
    constexpr int CH = GATED ? 8 : 16;
    auto kn = p.out_dt == F32 ? matmul_i8_few_kernel<TT, GATED, F32> : matmul_i8_few_kernel<TT, GATED, BF16>;
    hipLaunchKernelGGL(kn, dim3((p.N + CH - 1) / CH), dim3(64 * FEW_KG), 0, s, p);
    return hipGetLastError();
}

template <int BN, int BT, int WN, int WT, int NSTG, int KG, bool GATED>
static hipError_t tile(const MatI8Params& p, hipStream_t s) {
    constexpr int CH = GATED ? BN / 2 : BN;
    const int nt_n = (p.N + CH - 1) / CH, nt_t = (p.T + BT - 1) / BT;
    const int per = (nt_n * nt_t + 7) / 8;
    // (PIECES of the tiles with K groups is a choice inside)
    constexpr bool ELEMENTS = KG > 1;
    auto kn = KG > 1 || rows_in_pieces(p)
                  ? (p.out_dt == F32 ? matmul_i8_tile_kernel<BN, BT, WN, WT, NSTG, KG, GATED, F32, true>
                                     : matmul_i8_tile_kernel<BN, BT, WN, WT, NSTG, KG, GATED, BF16, true>)
                  : (p.out_dt == F32 ? matmul_i8_tile_kernel<BN, BT, WN, WT, NSTG, KG, GATED, F32, ELEMENTS>
                                     : matmul_i8_tile_kernel<BN, BT, WN, WT, NSTG, KG, GATED, BF16, ELEMENTS>);
    hipLaunchKernelGGL(kn, dim3(8 * per), dim3(64 * WN * WT * KG), 0, s, p, nt_n, nt_t);
    return hipGetLastError();
}

// Which tile: the one with the smallest estimated time.  A launch of W workgroups
// over 256 CUs takes ceil(W / 256) of them after each other, so with `steps`
// 128-byte K steps about steps * max(alone, ceil(W / 256) * full) + fixed: `full` is
// the time of a step, `alone` that of a workgroup that has its CU for itself where it
// is longer (several of the 64 x 64 ones fit on a CU).  The figures (us) are fitted to
// times of every tile at 274 shapes (T 20 to 16384, N 704 to 16384, K 704 to 8192, both
// kinds); the choice is then within 0.2 % of the best tile on average, 11 % at worst.
// The ends of the range: T = 64, N = 2819, K = 1424: 32 x 32 5.0 us, 64 x 64 6.6; T =
// 4096, N = 8192, K = 4096: 32 x 32 over 400 us, 256 x 128 143, 256 x 256 123.  The two
// that are no powers of two fill the CUs where their neighbours leave many of them idle
// or need a second round (T = 1024, gated, N = 2112, K = 2816: 192 x 128 17.7 us, 256 x
// 128 20.1, 128 x 128 26.3; T = 2048: 256 x 192 31.0 us, 256 x 256 36.3, 256 x 128 41.1);
// without them the choice is 2 % slower on average, 18 % at worst.
struct Tile {
    int bn, bt;
    float alone, full, fixed;
};
constexpr Tile TILES[] = {
    {32, 32, 0.12f, 0.12f, 1.3f},   {32, 64, 0.14f, 0.14f, 1.7f},   {64, 64, 0.18f, 0.18f, 1.9f},   {64, 64, 0.32f, 0.20f, 0.2f},
    {128, 64, 0.32f, 0.32f, 1.2f},  {128, 128, 0.52f, 0.52f, 0.4f}, {192, 128, 0.66f, 0.66f, 0.7f}, {256, 128, 0.79f, 0.79f, 1.1f},
    {256, 192, 1.08f, 1.08f, 1.1f}, {256, 256, 1.32f, 1.32f, 0.3f},
};
constexpr int N_TILES = sizeof(TILES) / sizeof(TILES[0]);

static int pick_tile(int64_t T, int64_t rows, int K) {
    int best = N_TILES - 1;
    float best_us = 1e30f;
    for (int i = 0; i < N_TILES; ++i) {
        const Tile& c = TILES[i];
        const int64_t W = ((rows + c.bn - 1) / c.bn) * ((T + c.bt - 1) / c.bt);
        if (W >= (1 << 22)) continue;   // keeps every launch below 2^32 threads
        const float us = static_cast<float>((K + 127) / 128) * std::max(c.alone, static_cast<float>((W + 255) / 256) * c.full) + c.fixed;
        if (us < best_us) {
            best_us = us;
            best = i;
        }
    }
    return best;
}

// Up to 16 tokens the kernel for few (210 shapes, T 1 to 16, N 704 to 8192, K 704 to
// 8192: 1.37 times as fast as the best tile on average, T = 16, N = 2112, K = 2816 2.85
// and 4.9 us, 8 of them slower, N = 8192, K = 4096 10.5 and 8.8).  Further as long as
// every workgroup has a CU of its own: up to 32 tokens 1.36 times as fast (N = 2112, K =
// 2816 3.9 and 5.0 us; with more workgroups 5 % slower), to 48 1.14 to 1.24 times, to 80 as
// fast, to 96 slower.  To 64 tokens the length of a row counts (30 shapes at each of 22
// lengths): 1.11 times as fast at 12 steps, 1.05 at 22; past that, rows of whole 128-byte
// lines keep 1.03 to 1.06 up to 36 steps, others fall to 1.00 to 1.01 at 23, 0.99 at 25, 0.98
// at 28 and 0.95 at 32: the limit is where those cross.
template <bool GATED>
static hipError_t dispatch(const MatI8Params& p, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.N) * (GATED ? 2 : 1);
    if (p.T <= 16) return few<1, GATED>(p, s);
    if (rows <= 256 * 16) {
        if (p.T <= 32) return few<2, GATED>(p, s);
        if (p.T <= 48) return few<3, GATED>(p, s);
        if (p.T <= 64 && p.K <= 23 * 128) return few<4, GATED>(p, s);
    }
    switch (pick_tile(p.T, rows, p.K)) {
        case 0: return tile<32, 32, 1, 1, 3, 4, GATED>(p, s);
        case 1: return tile<32, 64, 1, 2, 3, 4, GATED>(p, s);
        case 2: return tile<64, 64, 2, 2, 4, 2, GATED>(p, s);
        case 3: return tile<64, 64, 2, 2, 3, 1, GATED>(p, s);
        case 4: return tile<128, 64, 2, 2, 3, 1, GATED>(p, s);
        case 5: return tile<128, 128, 2, 4, 4, 1, GATED>(p, s);
        case 6: return tile<192, 128, 2, 4, 3, 1, GATED>(p, s);
        case 7: return tile<256, 128, 4, 2, 3, 1, GATED>(p, s);
        case 8: return tile<256, 192, 4, 2, 2, 1, GATED>(p, s);
        default: return tile<256, 256, 4, 2, 2, 1, GATED>(p, s);
    }
}

hipError_t launch_matmul_i8(const MatI8Params& p, bool gated, hipStream_t s) {
    return gated ? dispatch<true>(p, s) : dispatch<false>(p, s);
}

}  // namespace moe
