// Tile kernel of the bfloat16 products (block.h: MatKind), included by the files
// that instantiate it:
//
//   out[t][n] = sum over k of (token operand)(t, k) (channel operand)(n, k)
//   gated:      act(sum of gate channel n) * (sum of up channel n)
//
// Sums are fp32 in the MFMA's accumulators, in a fixed order; the epilogue is fp32
// and rounds once to the output type.  Operands are bf16, the MFMA's type: that is why
// the adapters' s and the gradient of pre, fp32 where they are made, are rounded to it
// (what that costs: adapter.hip, bf16_grad.hip).
//
// MFMA 16x16x32, A = channels, B = tokens, D column = token, so a lane holds 4
// consecutive channels of one token.  Long products run at the power limit, where
// this form gives 2.08 PFLOP/s and 32x32x16 1.85 (back to back on random values; on
// zeros both 2.4): it moves half the accumulators per product.
//
// What bounds it: long products the power limit (T = 8192, 4096 x 8192: 404 us, 1.36 PFLOP/s,
// MFMA busy 64 to 68 % of the cycles; on zeros 360 to 373 us), products of one or two turns of
// the CUs the steps' waits and the last turn (T = 4096, 2 x 2112 x 2816 with pre: 89 to 94 us,
// 49 %), short ones launch, first copies and epilogue (T = 77, 2 x 1411 x 1424: 7.5 us).
#pragma once

#include <type_traits>

#include "block.h"
#include "common.h"

namespace moe {

typedef __attribute__((ext_vector_type(4))) short s16x4;

// LDS DMA: 64 lanes x 16 bytes to dst + 16 * lane (dst uniform); a lane past the
// resource writes zeros.  Completion is the wave's vmcnt, waited for by the caller.
__device__ __forceinline__ void lds_dma16(rsrc_t r, uint8_t* dst, uint32_t off, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(dst)), 16, off, soff, 0, 0);
}

// 4 x 16 block of 16-bit values, its rows in memory, read by columns: the 16 lanes of
// a group give the addresses of its 8-byte pieces (lane i: row i / 4, columns 4 (i % 4)
// ..), and lane i receives column i, rows 0 .. 3.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ u32x2 lds_read_columns(lds_s16x4* __restrict__ p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}
__device__ __forceinline__ u32x2 lds_read_columns(const uint8_t* p) {
    return lds_read_columns(reinterpret_cast<lds_s16x4*>(reinterpret_cast<uintptr_t>(p)));
}

// the first n of 8 ranks (16-bit values), zeros behind them
__device__ __forceinline__ u32x4 low_ranks(const u32x4& v, int n) {
    if (n >= 8) return v;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = n >= 2 * i + 2 ? v[i] : n > 2 * i ? v[i] & 0xFFFFu : 0u;
    return r;
}

// The adapters that occur among up to 64 tokens, lane t's id (-1: none), once each: the
// first token of an adapter is its leader.  ids: 64 words of LDS of this wave's own.
__device__ __forceinline__ bool is_leader(int id, int count, int* ids) {
    const int lane = threadIdx.x & 63;
    ids[lane] = id;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    int first = 64;
    for (int t = (count + 3) / 4 * 4 - 4; t >= 0; t -= 4) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(ids + t);
#pragma unroll
        for (int e = 3; e >= 0; --e) first = static_cast<int>(v[e]) == id ? t + e : first;
    }
    return id >= 0 && first == lane;
}
// their ids and ranks, those with more than `past` ranks, into list (64 pairs of words of LDS); how many
__device__ __forceinline__ int list_adapters(bool leader, int id, int rank, int past, uint64_t* list) {
    const uint64_t m = __ballot(leader && rank > past);
    if (leader && rank > past)
        list[__builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0))] =
            static_cast<uint64_t>(static_cast<uint32_t>(rank)) << 32 | static_cast<uint32_t>(id);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return __builtin_popcountll(m);
}

__host__ __device__ constexpr int wait_vm_lds(int n) { return waitcnt_vm(n) & ~0x0F00; }   // and LDS reads to 0

// 16-byte chunk q of row r (128 bytes) is stored at position q ^ swz_row(r)
__device__ __forceinline__ int swz_row(int r) { return (r & 15) >> 1; }

// One operand of a tile: ROWS channels or tokens, 64 k in a stage of ROWS * 128 bytes.
//
// Rows along k (!TR): [ROWS][128 bytes]; a copy writes 8 rows.  A 16-byte read of a
// fragment (16 rows, 4 chunks) is served 16 lanes at a time, lanes 0-3, 12-15, 20-27
// (and 4-11, 16-19, 28-31) together: swz_row makes their 16 rows fall into all 64 banks.
//
// Rows are the k (TR): [64][ROWS * 2 bytes].  A fragment is read by columns: half a wave
// reads 16 columns (32 bytes) of k 0 .. 3 and 8 .. 11 (of 4 .. 7 and 12 .. 15, and so on)
// at once.  swz_k exchanges 32-byte pieces inside a row so that these eight cover all 64
// banks.
template <int ROWS, bool TR>
struct Operand {
    static constexpr bool COLUMNS = TR;
    static constexpr int PITCH = TR ? ROWS * 2 : 128, CPR = PITCH / 16;
    static_assert(!TR || PITCH % 64 == 0, "banks of a row");
    __device__ static int swz_k(int k) {
        const int far = (k >> 3) & 1;
        return PITCH % 256 == 0 ? ((k & 3) | far << 2) << 1 : PITCH % 256 == 128 ? (((k >> 1) & 1) | far << 1) << 1 : far << 1;
    }
    // copy number c (1024 bytes each), lane l: row of the stage, and the 16-byte chunk of the source row
    __device__ static int row(int c, int lane) { return (c * 64 + lane) / CPR; }
    __device__ static int chunk(int c, int lane) {
        const int r = row(c, lane), q = (c * 64 + lane) % CPR;
        return q ^ (TR ? swz_k(r) : swz_row(r));
    }
};

// One tile: number `id` of nt_n x nt_t (see the order below).  lds: KG * NSTG * (BN + BT) * 128 bytes.
template <int BN, int BT, int WN, int WT, int NSTG, int KG, int KIND, bool AD>
__device__ __forceinline__ void matmul_bf16_tile(const MatBf16Params& p, int nt_n, int nt_t, int block, uint8_t* lds, int (*ids_of)[64],
                                                 uint64_t (*lists)[64]) {
    constexpr bool GATED = KIND == MAT_GATED, TRA = KIND == MAT_NN || KIND == MAT_TN, TRB = KIND == MAT_TN;
    using OA = Operand<BN, TRA>;
    using OB = Operand<BT, TRB>;
    constexpr int NW = WN * WT, NB = BN / WN / 16, TB = BT / WT / 16;   // blocks of 16 channels, of 16 tokens
    constexpr int BK = 64;                                  // k of a step
    constexpr int STAGE = (BN + BT) * 128, DA = BN / 8 / NW, DB = BT / 8 / NW, CPS = DA + DB;
    constexpr int CH = GATED ? BN / 2 : BN;   // output channels per tile
    constexpr int CW = CH / WN;               // of a wave
    constexpr int RING = NSTG * STAGE;
    static_assert(DA * 8 * NW == BN && DB * 8 * NW == BT && NB * 16 * WN == BN && TB * 16 * WT == BT && (!GATED || NB % 2 == 0), "tile shape");
    static_assert(NSTG >= 2 && NSTG <= 4 && CPS * (NSTG - 1) <= 63, "copies in flight");
    static_assert((KG - 1) * BN * BT * 4 <= KG * RING, "epilogue regions");
    static_assert(!AD || BT / WT <= 64, "tokens of a wave");
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wid / NW, wave = wid % NW, wn = wave % WN, wt = wave / WN;
    // XCD-aware order: workgroups go to the 8 XCDs in turn, so XCD x takes one
    // contiguous range of the tile list, which runs down 8 token tiles before it
    // goes to the next channel tile
    const int ntile = nt_n * nt_t, per = (ntile + 7) / 8;
    const int id = (block & 7) * per + (block >> 3);
    if (id >= ntile) return;
    constexpr int GRP = 8;
    const int g0 = id / (GRP * nt_n) * GRP, gh = min(GRP, nt_t - g0), r = id - g0 * nt_n;
    const int t0 = (g0 + r % gh) * BT, n0 = r / gh * CH;
    const int nch = min(CH, p.N - n0), ntok = min(BT, p.T - t0);
    const uint32_t kb = 2u * p.K;             // bytes of a row along k
    // resources of operands along k: their rows of the tile (at most 2 GiB apart)
    auto rows_of = [&](const uint16_t* base, int64_t ld, int r0, int rows) {
        return make_rsrc(base + static_cast<int64_t>(r0) * ld, static_cast<uint32_t>(((rows - 1) * ld + p.K) * 2));
    };
    // of operands whose rows are the k: those of one step, the columns of the tile
    auto step_of = [&](const uint16_t* base, int64_t ld, int col0, int cols, int k) {
        const int left = min(BK, p.K - k);
        return make_rsrc(base + static_cast<int64_t>(left > 0 ? k : 0) * ld + col0,
                         left > 0 ? static_cast<uint32_t>(((left - 1) * ld + cols) * 2) : 0u);
    };
    const rsrc_t wr0 = TRA ? rsrc_t() : rows_of(p.w, p.ldw, n0, nch);
    const rsrc_t wr1 = GATED ? rows_of(p.w, p.ldw, p.N + n0, nch) : wr0;
    const rsrc_t xr = TRB ? rsrc_t() : rows_of(p.x, p.ldx, t0, ntok);
    uint8_t* ring = lds + kg * RING;
    // Gated: each 32-row block holds 16 gate rows, then the up rows of the same 16 channels
    auto channel = [](int row) { return GATED ? (row >> 5) * 16 + (row & 15) : row; };   // of a tile row
    auto is_up = [](int row) { return GATED && (row & 16); };
    uint32_t ao[DA], bo[DB];
#pragma unroll
    for (int i = 0; i < DA; ++i) {
        const int c = wave + NW * i, row = OA::row(c, lane), q = OA::chunk(c, lane);
        if (TRA)
            ao[i] = 8 * q < nch ? static_cast<uint32_t>(row * p.ldw + 8 * q) * 2 : NO_LANE;
        else
            ao[i] = channel(row) < nch ? static_cast<uint32_t>(channel(row) * p.ldw + 8 * q) * 2 : NO_LANE;
    }
#pragma unroll
    for (int i = 0; i < DB; ++i) {
        const int c = wave + NW * i, row = OB::row(c, lane), q = OB::chunk(c, lane);
        if (TRB)
            bo[i] = 8 * q < ntok ? static_cast<uint32_t>(row * p.ldx + 8 * q) * 2 : NO_LANE;
        else
            bo[i] = row < ntok ? static_cast<uint32_t>(row * p.ldx + 8 * q) * 2 : NO_LANE;
    }
    const int nk = max(1, ((p.K + BK - 1) / BK + KG - 1) / KG);   // steps of each group, the same for all; K = 0: one of zeros
    // Copy i of stage c: channels, then tokens.  What lies past K is zeros.  Stages
    // past the last are not requested, by a copy of the loop's body without copies; the
    // largest tiles (two stages) request them as zeros, which keeps their body short.
    constexpr bool TAIL = NSTG > 2;
    rsrc_t wk = rsrc_t(), xk = rsrc_t();   // operands whose rows are the k: of the stage that is requested
    auto stage = [&](int c) __attribute__((always_inline)) {
        const int k = BK * (c * KG + kg);
        if (TRA) wk = step_of(p.w, p.ldw, n0, nch, k);
        if (TRB) xk = step_of(p.x, p.ldx, t0, ntok, k);
    };
    auto copy = [&](int c, uint8_t* st, int i) __attribute__((always_inline)) {
        const int k = BK * (c * KG + kg);
        // the scalar offset stays inside the resource: the range check subtracts it
        // from the resource's size
        const uint32_t b = 2u * k, so = b < kb ? b : 0;
        if (i < DA) {
            uint8_t* dst = st + (wave + NW * i) * 1024;
            if (TRA) {
                lds_dma16(wk, dst, ao[i], 0);
            } else {
                const uint32_t o = b + 16 * OA::chunk(wave + NW * i, lane) < kb ? ao[i] : NO_LANE;
                if (is_up(8 * (wave + NW * i)))   // 8 rows lie on one side of a gated block
                    lds_dma16(wr1, dst, o, so);
                else
                    lds_dma16(wr0, dst, o, so);
            }
        } else {
            const int j = i - DA;
            uint8_t* dst = st + BN * 128 + (wave + NW * j) * 1024;
            if (TRB) {
                lds_dma16(xk, dst, bo[j], 0);
            } else {
                lds_dma16(xr, dst, b + 16 * OB::chunk(wave + NW * j, lane) < kb ? bo[j] : NO_LANE, so);
            }
        }
    };
    // Fragments: row (channel, token) l & 15 of a block, k 32 s + 8 (l >> 4) .. + 7
    const int l16 = lane & 15, q4 = lane >> 4;
    auto base_of = [&](auto o, int first) {   // lane's part of the address
        using O = decltype(o);
        if (!O::COLUMNS) return (first + l16) * 128;
        const int k = 8 * q4 + l16 / 4, q = first / 8 + ((lane >> 1) & 1);
        return k * O::PITCH + ((q ^ O::swz_k(k)) << 4) + 8 * (lane & 1);
    };
    int abase[NB], bbase[TB];
#pragma unroll
    for (int b = 0; b < NB; ++b) abase[b] = base_of(OA(), wn * (BN / WN) + 16 * b);
#pragma unroll
    for (int b = 0; b < TB; ++b) bbase[b] = BN * 128 + base_of(OB(), wt * (BT / WT) + 16 * b);
    u32x4 fa[2][NB], fb[2][TB];
    auto fragment = [&](bool tr, int pitch, const uint8_t* at, int s) __attribute__((always_inline)) {
        if (!tr) return *reinterpret_cast<const u32x4*>(at + ((4 * s + q4) ^ swz_row(l16)) * 16);
        const u32x2 lo = lds_read_columns(at + 32 * s * pitch), hi = lds_read_columns(at + (32 * s + 4) * pitch);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    // operand q of round s: the channels' fragments, then the tokens'
    auto read = [&](const uint8_t* st, int s, int q) __attribute__((always_inline)) {
        if (q < NB)
            fa[s & 1][q] = fragment(TRA, OA::PITCH, st + abase[q], s);
        else
            fb[s & 1][q - NB] = fragment(TRB, OB::PITCH, st + bbase[q - NB], s);
    };
    f32x4 acc[NB][TB] = {};
    // Rounds of 32 k, S to a step.  While round s runs, token block by token block, the
    // operands of the next round are read, about as many with each block and the last
    // with the last block but one: a token fragment then takes the registers of one
    // that is used up.  The step's last round runs after the barrier: at the barrier
    // every wave holds the last operands of stage c in registers and its copies of stage
    // c + 1 have landed, so the reads of stage c + 1 begin, and the copies of stage c +
    // NSTG go to the buffer of stage c, while that round is computed.  The copies of a
    // stage are spread between the MFMAs, so that the address unit (16 cycles a copy,
    // for all waves of the CU) works beside them.
    constexpr int S = BK / 32;
    constexpr int NR = NB + TB, RG = TB > 1 ? TB - 1 : 1;   // operands of a round, the blocks they are read with
    constexpr int M = (NSTG > 2 ? S : 1) * NB * TB;
    // round s; reads round rs of stage st, where that is wanted
    auto round = [&](int s, auto reads, const uint8_t* st, int rs, int c, uint8_t* to) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < TB; ++j) {
            if (decltype(reads)::value) {
#pragma unroll
                for (int q = 0; q < NR; ++q)
                    if (q * RG / NR == j) read(st, rs, q);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int slot = (s + 1) % S * NB * TB + j * NB + i;
                acc[i][j] = mfma16x16x32(fa[s & 1][i], fb[s & 1][j], acc[i][j]);
                if (c >= 0) {
#pragma unroll
                    for (int q = slot * CPS / M; q < (slot + 1) * CPS / M && q < CPS; ++q) copy(c, to, q);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    auto most = [&](const uint8_t* st, int c, uint8_t* to) __attribute__((always_inline)) {   // rounds 0 .. S - 2
#pragma unroll
        for (int s = 0; s + 1 < S; ++s) round(s, std::true_type(), st, s + 1, c, to);
    };
    const int tw = wt * (BT / WT);   // the wave's first token of the tile
    int id_l = -1;                   // of the wave's token `lane`
    if (AD) id_l = p.ad.ids[t0 + min(tw + lane, ntok - 1)];
#pragma unroll
    for (int c = 0; c < NSTG; ++c) {
        if (TAIL && c >= nk) break;
        stage(c);
#pragma unroll
        for (int q = 0; q < CPS; ++q) copy(c, ring + c * STAGE, q);
    }
    int rank_l = p.ad.R, aid[TB];    // its rank; the adapters of this lane's columns
    bool leader = false;
    if (AD) {
        if (lane >= BT / WT || tw + lane >= ntok || id_l < 0 || id_l >= p.ad.n) id_l = -1;
        if (p.ad.ranks != nullptr) rank_l = p.ad.ranks[max(id_l, 0)];
        leader = is_leader(id_l, BT / WT, ids_of[wid]);
#pragma unroll
        for (int j = 0; j < TB; ++j) aid[j] = ids_of[wid][16 * j + l16];
    }
    // The low-rank part, one half (gated) and 32 ranks at a time: the tokens' s, and the
    // rows of NI of the adapters of this wave's tokens at once, straight from memory; the K
    // groups take the adapters in turn.  Each adapter's product is taken from zero and
    // added in the columns (lanes) of its own tokens only, so that no value of one adapter,
    // an infinity or NaN included, meets another request's row.
    // The first ones are requested at the start by the small tiles, else before the steps
    // that request no more copies; LOADS loads, masked lanes among them.
    constexpr bool AHEAD = NB + TB <= 4;
    constexpr int NI = NB + TB <= 4 ? 8 : NB + TB <= 9 ? 3 : 1, NH = GATED ? NB / 2 : NB;
    constexpr int LOADS = AD && !AHEAD && TAIL ? TB + NI * NH : 0;
    static_assert(CPS * (NSTG - 2) + LOADS <= 63, "loads in flight");
    int count = 0, at = 0, h = 0, k0 = 0;   // adapters of this phase, the group's next; half, first rank
    u32x4 va[NI][NH], vb[TB];
    int ia[NI], rank_of[NI];
    const rsrc_t sr = AD ? make_rsrc(p.ad.s + t0 * p.ad.lds, static_cast<uint32_t>(((ntok - 1) * p.ad.lds + (GATED ? 2 : 1) * p.ad.R) * 2))
                         : rsrc_t();
    auto tokens = [&]() __attribute__((always_inline)) {
        count = list_adapters(leader, id_l, min(rank_l, p.ad.R), k0, lists[wid]);
        at = kg;
#pragma unroll
        for (int j = 0; j < TB; ++j)
            vb[j] = bload16(sr, aid[j] >= 0 && k0 + 8 * q4 < p.ad.R
                                    ? static_cast<uint32_t>((tw + 16 * j + l16) * p.ad.lds + h * p.ad.R + k0 + 8 * q4) * 2 : NO_LANE);
    };
    auto adapters = [&]() __attribute__((always_inline)) {   // the next NI of this group
        uint64_t of[NI];
#pragma unroll
        for (int n = 0; n < NI; ++n) of[n] = lists[wid][min(at + n * KG, 63)];
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const bool in = at + n * KG < count;
            ia[n] = in ? __builtin_amdgcn_readfirstlane(static_cast<int>(of[n])) : -1;
            rank_of[n] = __builtin_amdgcn_readfirstlane(static_cast<int>(of[n] >> 32));
            const bool ranks = in && k0 + 8 * q4 < rank_of[n];   // the lane has some
            const rsrc_t br = make_rsrc(p.ad.b + max(ia[n], 0) * p.ad.b_stride + (static_cast<int64_t>(h) * p.N + n0) * p.ad.R,
                                        static_cast<uint32_t>(nch) * p.ad.R * 2u);
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                const int c = wn * CW + 16 * i + l16;
                va[n][i] = bload16(br, ranks && c < nch ? static_cast<uint32_t>(c * p.ad.R + k0 + 8 * q4) * 2 : NO_LANE);
            }
        }
        at += NI * KG;
    };
    auto first_adapters = [&]() __attribute__((always_inline)) {
        tokens();
        adapters();
        // the waits that follow count these loads: they stay in front of them
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));
    __syncthreads();
    if (AD && AHEAD) first_adapters();
#pragma unroll
    for (int q = 0; q < NR; ++q) read(ring, 0, q);
    most(ring, -1, ring);
    int buf = 0;
    // from step c to step c + 1: `left` of the stages behind that one, and `more` later
    // loads, may still be on their way (the first stages have landed: no wait for the items
    // that were requested after them)
    auto step = [&](int c, int left, auto more, int next) __attribute__((always_inline)) {
        constexpr int MORE = decltype(more)::value;
        if (AD && AHEAD && c + 1 < NSTG)
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(63));
        else if (NSTG > 3 && left >= 2)
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(CPS * 2 + MORE));
        else if (NSTG > 2 && left >= 1)
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(CPS + MORE));
        else
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(MORE));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        uint8_t* done = ring + buf * STAGE;
        buf = buf + 1 == NSTG ? 0 : buf + 1;
        const uint8_t* st = ring + buf * STAGE;
        if (next >= 0) stage(next);
        round(S - 1, std::true_type(), st, 0, next, done);
        most(st, next, done);
    };
    int c = 0;
    for (; c + (TAIL ? NSTG : 1) < nk; ++c) step(c, NSTG - 2, std::integral_constant<int, 0>(), c + NSTG);
    if (AD && !AHEAD) first_adapters();
    if (TAIL)
        for (; c + 1 < nk; ++c) step(c, nk - 2 - c, std::integral_constant<int, LOADS>(), -1);
    round(S - 1, std::false_type(), ring, 0, -1, ring);
    if (AD) {
        for (;;) {
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                if (ia[n] < 0) continue;
                if (rank_of[n] & 7) {   // some lane holds less than 8 ranks
#pragma unroll
                    for (int i = 0; i < NH; ++i) va[n][i] = low_ranks(va[n][i], rank_of[n] - k0 - 8 * q4);
                }
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    f32x4 low[NH];
#pragma unroll
                    for (int i = 0; i < NH; ++i) low[i] = mfma16x16x32(va[n][i], vb[j], f32x4{0, 0, 0, 0});
                    if (aid[j] == ia[n]) {
#pragma unroll
                        for (int i = 0; i < NB; ++i)
                            if (!GATED || (i & 1) == h) acc[i][j] += low[GATED ? i / 2 : i];
                    }
                }
            }
            if (at >= count) {   // the other half, then the next 32 ranks, of the adapters that have them
                if (GATED && h == 0) {
                    h = 1;
                } else {
                    h = 0;
                    k0 += 32;
                    if (k0 >= p.ad.R) break;
                }
                tokens();
            }
            adapters();
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));   // zero stages have landed too
    __syncthreads();   // the rings are free
    if (KG > 1) {
        f32x4* part = reinterpret_cast<f32x4*>(lds);
        auto at = [&](int g, int i, int j) { return part + ((((g - 1) * NW + wave) * NB + i) * TB + j) * 64 + lane; };
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j) *at(kg, i, j) = acc[i][j];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int g = 1; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j) acc[i][j] += *at(g, i, j);
    }
    // Epilogue, TK tokens at a time: the wave's [TK tokens][CW channels] go through
    // LDS (16-byte chunks at position c ^ token) and leave as row pieces; rows that are
    // not 16-byte aligned leave by elements, neighbouring lanes storing neighbouring
    // ones.  With groups, the partial sums may lie where another wave of group 0 still
    // reads: the waves' regions start behind them.
    constexpr int PART = KG > 1 ? (KG - 1) * BN * BT * 4 : 0, TK = TB % 2 ? 16 : 32;
    auto leave = [&](auto type, int tb, void* out, int64_t ldo, int col0, auto value) {
        constexpr int es = decltype(type)::value == F32 ? 4 : 2, cpr = CW * es / 16;   // 16-byte chunks per row
        constexpr bool p2 = (cpr & (cpr - 1)) == 0;           // else the rows are 16 bytes apart instead
        constexpr int RS = CW * es + (p2 ? 0 : 16);
        constexpr int REGION = TK * (CW * 4 + 16);   // of a wave, the same for both types: they may follow each other
        static_assert(RS * TK <= REGION && PART + REGION * NW <= KG * RING, "epilogue regions");
        uint8_t* my = lds + PART + wave * REGION;
        auto at = [&](int tok, int c) { return my + tok * RS + ((p2 ? c ^ (tok & (cpr - 1)) : c) << 4); };
        const int tl = wt * (BT / WT) + TK * tb;   // first token of these in the tile
#pragma unroll
        for (int j = 0; j < TK / 16; ++j)
#pragma unroll
            for (int b = 0; b < (GATED ? NB / 2 : NB); ++b) {   // 4 channels
                const int cl = 16 * b + 4 * q4, tok = 16 * j + l16;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = value(b, TK / 16 * tb + j, e);
                if (es == 4)
                    *reinterpret_cast<f32x4*>(at(tok, cl >> 2)) = f32x4{v[0], v[1], v[2], v[3]};
                else
                    *reinterpret_cast<u32x2*>(at(tok, cl >> 3) + 8 * (q4 & 1)) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint8_t* base = static_cast<uint8_t*>(out) + ((t0 + tl) * ldo + n0 + col0) * es;
        if (reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo * es % 16 == 0 && col0 * es % 16 == 0) {
#pragma unroll 4
            for (int i0 = 0; i0 < TK * cpr; i0 += 64) {
                const int it = i0 + lane;
                if (TK * cpr % 64 && it >= TK * cpr) continue;
                const int tok = it / cpr, c = it % cpr;
                const u32x4 v = *reinterpret_cast<const u32x4*>(at(tok, c));
                const int ch = wn * CW + c * (16 / es);
                if (tl + tok >= ntok || ch >= nch) continue;
                uint8_t* d = base + (tok * ldo + ch) * es;
                if (ch + 16 / es <= nch) {
                    *reinterpret_cast<u32x4*>(d) = v;
                } else if (es == 4) {
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
#pragma unroll 4
            for (int i0 = 0; i0 < TK * CW; i0 += 64) {
                const int it = i0 + lane;
                const int tok = it / CW, e = it % CW;
                const uint8_t* s = at(tok, e * es / 16) + e * es % 16;
                const int ch = wn * CW + e;
                if (tl + tok >= ntok || ch >= nch) continue;
                uint8_t* d = base + (tok * ldo + ch) * es;
                if (es == 4)
                    *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(s);
                else
                    *reinterpret_cast<uint16_t*>(d) = *reinterpret_cast<const uint16_t*>(s);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    using is_f32 = std::integral_constant<int, F32>;
    using is_bf16 = std::integral_constant<int, BF16>;
#pragma unroll
    for (int tb = 0; tb < TB * 16 / TK; ++tb) {
        auto gate = [&](int b, int j, int e) { return acc[GATED ? 2 * b : b][j][e]; };
        auto up = [&](int b, int j, int e) { return acc[GATED ? 2 * b + 1 : b][j][e]; };
        auto result = [&](int b, int j, int e) { return GATED ? act_fn(p.act, gate(b, j, e)) * up(b, j, e) : gate(b, j, e); };
        if (p.out_dt == F32)
            leave(is_f32(), tb, p.out, p.ldo, 0, result);
        else
            leave(is_bf16(), tb, p.out, p.ldo, 0, result);
        if (GATED && p.pre != nullptr) {
            leave(is_bf16(), tb, p.pre, p.ldp, 0, gate);
            leave(is_bf16(), tb, p.pre, p.ldp, p.N, up);
        }
    }
}

template <int BN, int BT, int WN, int WT, int NSTG, int KG, int KIND, bool AD>
__global__ __launch_bounds__(64 * WN * WT * KG, 1) void matmul_bf16_tile_kernel(MatBf16Params p, int nt_n, int nt_t) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NSTG * (BN + BT) * 128];
    __shared__ __attribute__((aligned(16))) int ids_of[AD ? WN * WT * KG : 1][64];
    __shared__ uint64_t lists[AD ? WN * WT * KG : 1][64];
    matmul_bf16_tile<BN, BT, WN, WT, NSTG, KG, KIND, AD>(p, nt_n, nt_t, blockIdx.x, lds, ids_of, lists);
}

// Both gradients of a product in one launch: the workgroups of the rows' (NN), then those
// of the weights' (TN).
template <int BN, int BT, int WN, int WT, int NSTG, int KG>
__global__ __launch_bounds__(64 * WN * WT * KG, 1) void matmul_bf16_pair_kernel(MatBf16Params p, int np_n, int np_t, MatBf16Params r,
                                                                               int nr_n, int nr_t, int first) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NSTG * (BN + BT) * 128];
    const int block = blockIdx.x;
    if (block < first)
        matmul_bf16_tile<BN, BT, WN, WT, NSTG, KG, MAT_NN, false>(p, np_n, np_t, block, lds, nullptr, nullptr);
    else
        matmul_bf16_tile<BN, BT, WN, WT, NSTG, KG, MAT_TN, false>(r, nr_n, nr_t, block - first, lds, nullptr, nullptr);
}

template <int KIND, bool AD, int BN, int BT, int WN, int WT, int NSTG, int KG>
static hipError_t bf16_tile(const MatBf16Params& p, hipStream_t s) {
    constexpr int CH = KIND == MAT_GATED ? BN / 2 : BN;
    const int nt_n = (p.N + CH - 1) / CH, nt_t = (p.T + BT - 1) / BT;
    const int per = (nt_n * nt_t + 7) / 8;
    hipLaunchKernelGGL((matmul_bf16_tile_kernel<BN, BT, WN, WT, NSTG, KG, KIND, AD>), dim3(8 * per), dim3(64 * WN * WT * KG), 0, s,
                       p, nt_n, nt_t);
    return hipGetLastError();
}

// Which tile: the one with the smallest estimated time.  A launch of W workgroups
// over 256 CUs takes ceil(W / 256) of them after each other, so with `steps` 64-element
// K steps about fixed + max(steps * alone + end, ceil(W / 256) * (steps * full + end)):
// `full` is the time of a step, `alone` that of a workgroup that has its CU for itself
// (several of the small ones fit on a CU), `end` that of prologue and epilogue.  The
// figures (us) are fitted to times at 102 to 107 shapes of each kind, without adapters (T
// 16 to 8192, the other sizes 64 to 8192).  There these twelve lose 0.1 to 0.6 % on average
// against the best of 18 tiles (the ends of the range: T = 752, N = 960, K = 536, TN: 64 x 64
// 4.8 us, 256 x 256 15.5; T = 8192, N = 4096, K = 8192, NN: 32 x 32 2229 us, 256 x 256 411),
// and the choice by the estimate 0.3 to 0.9 % against the best of the twelve, for TN 1.7 %.
// A product with adapters takes the tile of the same product without: what that loses is
// not fitted (the adapters' part depends on how many of them a tile's tokens have).
// A tile's LDS reads a step, (BN / 16 * WT + BT / 16 * WN) KB at 128 bytes a cycle, take longer
// than its MFMA where the waves' parts are small: 128 x 128 in four waves of 64 x 64 takes 33
// us at T = 1024, N = 2816, K = 4224, NN, in eight 40.  192 x 192 is there for three stages of
// copies under 160 KB (gated T = 2048, 2 x 2112 x 2816: 42 us, 256 x 192 48, 128 x 192 54);
// where operands are read by columns it has four waves (T = N = K = 4096, NN: 120 us, in
// eight 126).
struct Bf16Tile {
    int bn, bt;
    float alone, full, fixed, end;
};
template <int KIND>
struct Bf16Tiles;
template <>
struct Bf16Tiles<MAT_NT> {
    static constexpr Bf16Tile T[] = {
        {32, 32, 0.074f, 0.087f, 1.25f, 2.10f},  {64, 32, 0.142f, 0.145f, 0.99f, 2.45f},  {64, 64, 0.205f, 0.213f, 0.70f, 2.84f},
        {64, 64, 0.236f, 0.220f, 2.47f, 0.51f},  {64, 96, 0.231f, 0.252f, 1.06f, 3.42f},  {96, 96, 0.209f, 0.240f, 3.74f, 4.88f},
        {128, 64, 0.111f, 0.263f, 1.87f, 4.45f}, {128, 128, 0.401f, 0.441f, 1.57f, 4.32f}, {128, 192, 0.586f, 0.587f, 0.00f, 5.31f},
        {192, 192, 0.691f, 0.691f, 4.04f, 4.53f}, {256, 192, 0.994f, 1.014f, 0.00f, 7.44f}, {256, 256, 1.060f, 1.100f, 0.00f, 10.20f},
    };
};
template <>
struct Bf16Tiles<MAT_GATED> {
    static constexpr Bf16Tile T[] = {
        {32, 32, 0.111f, 0.097f, 1.24f, 2.00f},  {64, 32, 0.183f, 0.157f, 0.83f, 2.31f},  {64, 64, 0.248f, 0.235f, 0.68f, 2.50f},
        {64, 64, 0.270f, 0.211f, 1.97f, 0.64f},  {64, 96, 0.298f, 0.267f, 0.40f, 3.39f},  {96, 96, 0.297f, 0.271f, 0.21f, 6.76f},
        {128, 64, 0.306f, 0.295f, 0.37f, 5.07f}, {128, 128, 0.487f, 0.467f, 0.00f, 5.09f}, {128, 192, 0.609f, 0.611f, 0.00f, 5.05f},
        {192, 192, 0.751f, 0.763f, 0.00f, 7.31f}, {256, 192, 1.100f, 1.069f, 0.00f, 6.19f}, {256, 256, 1.252f, 1.255f, 0.00f, 8.23f},
    };
};
template <>
struct Bf16Tiles<MAT_NN> {
    static constexpr Bf16Tile T[] = {
        {32, 32, 0.052f, 0.143f, 1.22f, 1.53f},  {64, 32, 0.135f, 0.186f, 0.88f, 1.88f},  {64, 64, 0.239f, 0.242f, 0.49f, 2.29f},
        {64, 64, 0.269f, 0.220f, 1.97f, 0.54f},  {64, 96, 0.046f, 0.296f, 0.26f, 2.84f},  {96, 96, 0.235f, 0.321f, 0.04f, 4.28f},
        {128, 64, 0.296f, 0.305f, 0.27f, 3.70f}, {128, 128, 0.300f, 0.463f, 0.00f, 3.59f}, {128, 192, 0.499f, 0.609f, 0.00f, 3.88f},
        {192, 192, 0.751f, 0.751f, 0.00f, 5.61f}, {256, 192, 0.926f, 1.026f, 0.00f, 4.04f}, {256, 256, 1.065f, 1.181f, 0.00f, 4.97f},
    };
};
template <>
struct Bf16Tiles<MAT_TN> {
    // (64 x 64 with two K groups is never the fastest here: not built)
    static constexpr Bf16Tile T[] = {
        {32, 32, 0.153f, 0.176f, 1.25f, 1.43f},  {64, 32, 0.205f, 0.209f, 1.08f, 1.88f},  {64, 64, 9.0f, 9.0f, 9.0f, 9.0f},
        {64, 64, 0.253f, 0.223f, 2.22f, 0.42f},  {64, 96, 0.101f, 0.307f, 1.03f, 2.37f},  {96, 96, 0.242f, 0.347f, 0.77f, 3.53f},
        {128, 64, 0.008f, 0.324f, 0.95f, 3.08f}, {128, 128, 0.440f, 0.465f, 0.16f, 3.32f}, {128, 192, 0.614f, 0.663f, 0.00f, 3.55f},
        {192, 192, 0.671f, 0.776f, 0.00f, 5.51f}, {256, 192, 1.014f, 1.015f, 0.00f, 4.43f}, {256, 256, 1.096f, 1.158f, 0.00f, 5.09f},
    };
};

static float bf16_tile_us(const Bf16Tile& c, int64_t T, int64_t rows, int K) {
    const int64_t W = ((rows + c.bn - 1) / c.bn) * ((T + c.bt - 1) / c.bt);
    if (W >= (1 << 22)) return 1e30f;   // keeps every launch below 2^32 threads
    const float steps = static_cast<float>((K + 63) / 64);
    const float alone = steps * c.alone + c.end, turns = static_cast<float>((W + 255) / 256) * (steps * c.full + c.end);
    return c.fixed + (alone > turns ? alone : turns);
}

template <int KIND, bool AD>
static int pick_bf16_tile(int64_t T, int64_t rows, int K) {
    // (256 x 256 with adapters does not fit the registers)
    constexpr int n = sizeof(Bf16Tiles<KIND>::T) / sizeof(Bf16Tile) - AD;
    int best = n - 1;
    float best_us = 1e30f;
    for (int i = 0; i < n; ++i) {
        const float us = bf16_tile_us(Bf16Tiles<KIND>::T[i], T, rows, K);
        if (us < best_us) {
            best_us = us;
            best = i;
        }
    }
    return best;
}

template <int KIND, bool AD>
static hipError_t bf16_tiles(const MatBf16Params& p, hipStream_t s) {
    switch (pick_bf16_tile<KIND, AD>(p.T, static_cast<int64_t>(p.N) * (KIND == MAT_GATED ? 2 : 1), p.K)) {
        case 0: return bf16_tile<KIND, AD, 32, 32, 1, 1, 3, 4>(p, s);
        case 1: return bf16_tile<KIND, AD, 64, 32, 2, 1, 3, 4>(p, s);
        case 2:
            if constexpr (KIND != MAT_TN) return bf16_tile<KIND, AD, 64, 64, 2, 2, 4, 2>(p, s);
            break;
        case 3: return bf16_tile<KIND, AD, 64, 64, 2, 2, 3, 1>(p, s);
        case 4: return bf16_tile<KIND, AD, 64, 96, 2, 2, 3, 2>(p, s);
        case 5: return bf16_tile<KIND, AD, 96, 96, 1, 2, 3, 2>(p, s);
        case 6: return bf16_tile<KIND, AD, 128, 64, 2, 1, 3, 2>(p, s);
        case 7: return bf16_tile<KIND, AD, 128, 128, 2, 2, 3, 1>(p, s);
        case 8: return bf16_tile<KIND, AD, 128, 192, 2, 4, 3, 1>(p, s);
        case 9: return bf16_tile<KIND, AD, 192, 192, 2, KIND == MAT_NN || KIND == MAT_TN ? 2 : 4, 3, 1>(p, s);
        case 10: return bf16_tile<KIND, AD, 256, 192, AD ? 2 : 4, AD ? 4 : 2, 2, 1>(p, s);   // (64 tokens of a wave at most)
    }
    if constexpr (!AD) return bf16_tile<KIND, AD, 256, 256, 4, 2, 2, 1>(p, s);
    return hipErrorInvalidValue;   // not reached
}

}  // namespace moe
