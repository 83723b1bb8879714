// Tile kernel of the bfloat16 products (block.h: MatKind), included by the files
// that instantiate it:
//
//   out[t][n] = sum over k of (token operand)(t, k) (channel operand)(n, k)
//   gated:      act(sum of gate channel n) * (sum of up channel n)
//
// Sums are fp32 in the MFMA's accumulators, in a fixed order; the epilogue is fp32
// and rounds once to the output type.
//
// MFMA operands: A = channels, B = tokens, D column = token, so a lane holds 4
// consecutive channels of one token.
#pragma once

#include <type_traits>

#include "block.h"
#include "common.h"

namespace moe {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;

__device__ __forceinline__ f32x16 mfma32_bf16(const u32x4& a, const u32x4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// LDS DMA: 64 lanes x 16 bytes to dst + 16 * lane (dst uniform); a lane past the
// resource writes zeros.  Completion is the wave's vmcnt, waited for by the caller.
__device__ __forceinline__ void lds_dma16(rsrc_t r, uint8_t* dst, uint32_t off, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(dst)), 16, off, soff, 0, 0);
}

// 4 x 16 block of 16-bit values, its rows in memory, read by columns: the 16 lanes of
// a group give the addresses of its 8-byte pieces (lane i: row i / 4, columns 4 (i % 4)
// ..), and lane i receives column i, rows 0 .. 3.
__device__ __forceinline__ u32x2 lds_read_columns(const uint8_t* p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) s16x4*>(
                                         reinterpret_cast<uintptr_t>(p))));
}

// the first n of 8 ranks (16-bit values), zeros behind them
__device__ __forceinline__ u32x4 low_ranks(const u32x4& v, int n) {
    if (n >= 8) return v;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = n >= 2 * i + 2 ? v[i] : n > 2 * i ? v[i] & 0xFFFFu : 0u;
    return r;
}

__host__ __device__ constexpr int wait_vm_lds(int n) { return waitcnt_vm(n) & ~0x0F00; }   // and LDS reads to 0

// 16-byte chunk q of row r (128 bytes) is stored at position q ^ swz_row(r)
__device__ __forceinline__ int swz_row(int r) { return (r & 7) ^ ((r >> 3) & 3); }

// One operand of a tile: ROWS channels or tokens, 64 k in a stage of ROWS * 128 bytes.
//
// Rows along k (!TR): [ROWS][128 bytes]; a copy writes 8 rows.  A 16-byte read of a
// fragment is served 16 lanes at a time, lanes 0-3, 12-15, 20-27 (and 4-11, 16-19,
// 28-31) together: swz_row makes their 16 rows fall into all 64 banks.
//
// Rows are the k (TR): [64][ROWS * 2 bytes].  A fragment is read by columns, four k of
// 32 columns (64 bytes each) by half a wave at once: 64-byte pieces of rows that would
// meet in the same banks are exchanged inside their row (swz_k), so that the four
// pieces cover all 64 banks.
template <int ROWS, bool TR>
struct Operand {
    static constexpr bool COLUMNS = TR;
    static constexpr int PITCH = TR ? ROWS * 2 : 128, CPR = PITCH / 16;
    __device__ static int swz_k(int k) {
        return PITCH % 256 == 0 ? (k & 3) << 2 : PITCH % 256 == 128 ? ((k >> 1) & 1) << 2 : 0;
    }
    // copy number c (1024 bytes each), lane l: row of the stage, and the 16-byte chunk of the source row
    __device__ static int row(int c, int lane) { return (c * 64 + lane) / CPR; }
    __device__ static int chunk(int c, int lane) {
        const int r = row(c, lane), q = (c * 64 + lane) % CPR;
        return q ^ (TR ? swz_k(r) : swz_row(r));
    }
};

template <int BN, int BT, int WN, int WT, int NSTG, int KG, int KIND, bool AD>
__global__ __launch_bounds__(64 * WN * WT * KG, 1) void matmul_bf16_tile_kernel(MatBf16Params p, int nt_n, int nt_t) {
    constexpr bool GATED = KIND == MAT_GATED, TRA = KIND == MAT_NN || KIND == MAT_TN, TRB = KIND == MAT_TN;
    using OA = Operand<BN, TRA>;
    using OB = Operand<BT, TRB>;
    constexpr int NW = WN * WT, NB = BN / WN / 32, TB = BT / WT / 32;
    constexpr int BK = 64;                                  // k of a step
    constexpr int STAGE = (BN + BT) * 128, DA = BN / 8 / NW, DB = BT / 8 / NW, CPS = DA + DB;
    constexpr int CH = GATED ? BN / 2 : BN;   // output channels per tile
    constexpr int CW = CH / WN;               // of a wave
    constexpr int RING = NSTG * STAGE;
    static_assert(DA * 8 * NW == BN && DB * 8 * NW == BT && BN % 32 == 0, "tile shape");
    static_assert(NSTG >= 2 && NSTG <= 4 && CPS * (NSTG - 1) <= 63, "copies in flight");
    static_assert((KG - 1) * BN * BT * 4 <= KG * RING, "epilogue regions");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * RING];
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
    auto copy = [&](int c, uint8_t* st, int i) {
        const int k = BK * (c * KG + kg);
        // the scalar offset stays inside the resource: the range check subtracts it
        // from the resource's size
        const uint32_t b = 2u * k, so = b < kb ? b : 0;
        if (i < DA) {
            uint8_t* dst = st + (wave + NW * i) * 1024;
            if (TRA) {
                lds_dma16(step_of(p.w, p.ldw, n0, nch, k), dst, ao[i], 0);
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
                lds_dma16(step_of(p.x, p.ldx, t0, ntok, k), dst, bo[j], 0);
            } else {
                lds_dma16(xr, dst, b + 16 * OB::chunk(wave + NW * j, lane) < kb ? bo[j] : NO_LANE, so);
            }
        }
    };
    // Fragments: row (channel, token) l & 31 of a 32-row block, k 16 s + 8 (l >> 5) .. + 7
    const int l32 = lane & 31, hh = lane >> 5;
    auto base_of = [&](auto o, int first) {   // lane's part of the address
        using O = decltype(o);
        if (!O::COLUMNS) return (first + l32) * 128;
        const int k = 8 * hh + (lane & 15) / 4;
        const int q = first / 8 + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
        return k * O::PITCH + ((q ^ O::swz_k(k)) << 4) + 8 * (lane & 1);
    };
    int abase[NB], bbase[TB];
#pragma unroll
    for (int b = 0; b < NB; ++b) abase[b] = base_of(OA(), wn * (BN / WN) + 32 * b);
#pragma unroll
    for (int b = 0; b < TB; ++b) bbase[b] = BN * 128 + base_of(OB(), wt * (BT / WT) + 32 * b);
    u32x4 fa[2][NB], fb[2][TB];
    auto fragment = [&](bool tr, int pitch, const uint8_t* at, int s) {
        if (!tr) return *reinterpret_cast<const u32x4*>(at + ((2 * s + hh) ^ swz_row(l32)) * 16);
        const u32x2 lo = lds_read_columns(at + 16 * s * pitch), hi = lds_read_columns(at + (16 * s + 4) * pitch);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    auto read = [&](const uint8_t* st, int s, int set) {
#pragma unroll
        for (int i = 0; i < NB; ++i) fa[set][i] = fragment(TRA, OA::PITCH, st + abase[i], s);
#pragma unroll
        for (int i = 0; i < TB; ++i) fb[set][i] = fragment(TRB, OB::PITCH, st + bbase[i], s);
    };
    f32x16 acc[NB][TB] = {};
    // Within a step the operands of MFMA round s + 1 are read while round s runs.  The
    // step's last round runs after the barrier: at the barrier every wave holds the
    // last operands of stage c in registers and its copies of stage c + 1 have landed,
    // so the reads of stage c + 1 begin, and the copies of stage c + NSTG go to the
    // buffer of stage c, while that round is computed.  The copies of a stage are
    // spread between the MFMAs of its rounds, so that the address unit (16 cycles a
    // copy, for all waves of the CU) works beside them.
    constexpr int S = BK / 16;   // rounds of a step (even: a step starts with set 0)
    constexpr int M = (NSTG > 2 ? S : 2) * NB * TB;
    auto round = [&](int s, int c, uint8_t* to) {
#pragma unroll
        for (int m = 0; m < NB * TB; ++m) {
            const int i = m / TB, j = m % TB, slot = (s + 1) % S * NB * TB + m;
            acc[i][j] = mfma32_bf16(fa[s & 1][i], fb[s & 1][j], acc[i][j]);
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
    // the adapters of this lane's tokens
    int aid[TB];
    if (AD) {
#pragma unroll
        for (int j = 0; j < TB; ++j) {
            const int t = wt * (BT / WT) + 32 * j + l32;
            const int a = t < ntok ? p.ad.ids[t0 + t] : -1;
            aid[j] = a >= 0 && a < p.ad.n ? a : -1;
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));
    __syncthreads();
    read(ring, 0, 0);
    most(ring, -1, ring);
    int buf = 0;
    // from step c to step c + 1: `left` of the stages behind that one may still be on their way
    auto step = [&](int left, int next) {
        if (NSTG > 3 && left >= 2)
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(CPS * 2));
        else if (NSTG > 2 && left >= 1)
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(CPS));
        else
            __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));
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
    if (AD) {
        // The low-rank part, adapter by adapter of this wave's tokens: 16 ranks are one
        // MFMA, the operands straight from memory.  Each adapter's product is taken from
        // zero and added in the columns (lanes) of its own tokens only, so that no value
        // of one adapter, an infinity or NaN included, meets another request's row.
        uint64_t left[TB];
#pragma unroll
        for (int j = 0; j < TB; ++j) left[j] = __ballot(aid[j] >= 0);
        int unit = 0;
        for (;;) {
            int a = -1;
#pragma unroll
            for (int j = TB - 1; j >= 0; --j)
                if (left[j]) a = __builtin_amdgcn_readlane(aid[j], __builtin_ctzll(left[j]));
            if (a < 0) break;
            bool has[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                const uint64_t same = __ballot(aid[j] == a);
                has[j] = same != 0;
                left[j] &= ~same;
            }
            if (KG > 1 && unit++ % KG != kg) continue;
            const int rank = p.ad.ranks ? min(p.ad.ranks[a], p.ad.R) : p.ad.R;
            const uint16_t* pb = p.ad.b + a * p.ad.b_stride;
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                if (!has[j]) continue;
                const int t = t0 + wt * (BT / WT) + 32 * j + l32;
                f32x16 low[NB] = {};
                for (int h = 0; h < (GATED ? 2 : 1); ++h)
                    for (int k = 8 * hh; k < rank + 8 * hh; k += 16) {
                        u32x4 vb = {0, 0, 0, 0}, va[NB] = {};
                        if (k < rank) {
                            if (aid[j] == a) vb = *reinterpret_cast<const u32x4*>(p.ad.s + t * p.ad.lds + h * p.ad.R + k);
#pragma unroll
                            for (int i = 0; i < NB; ++i) {
                                const int row = wn * (BN / WN) + 32 * i + l32, n = channel(row);
                                if (n < nch && is_up(row) == (h == 1))
                                    va[i] = low_ranks(*reinterpret_cast<const u32x4*>(pb + (static_cast<int64_t>(h) * p.N + n0 + n) * p.ad.R + k),
                                                      rank - k);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < NB; ++i) low[i] = mfma32_bf16(va[i], vb, low[i]);
                    }
                if (aid[j] == a) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) acc[i][j] += low[i];
                }
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));   // zero stages have landed too
    __syncthreads();   // the rings are free
    if (KG > 1) {
        float* part = reinterpret_cast<float*>(lds);
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<f32x4*>(part + (((((kg - 1) * NW + wave) * NB + i) * TB + j) * 4 + v) * 256 + lane * 4) =
                            f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
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
                        const f32x4 o = *reinterpret_cast<const f32x4*>(
                            part + (((((q - 1) * NW + wave) * NB + i) * TB + j) * 4 + v) * 256 + lane * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * v + e] += o[e];
                    }
    }
    // Epilogue, 32 tokens at a time: the wave's [32 tokens][CW channels] go through
    // LDS (16-byte chunks at position c ^ token) and leave as row pieces; rows that are
    // not 16-byte aligned leave by elements, neighbouring lanes storing neighbouring
    // ones.  With groups, the partial sums may lie where another wave of group 0 still
    // reads: the waves' regions start behind them.
    constexpr int PART = KG > 1 ? (KG - 1) * BN * BT * 4 : 0;
    auto leave = [&](auto type, int tb, void* out, int64_t ldo, int col0, auto value) {
        constexpr int es = decltype(type)::value == F32 ? 4 : 2, cpr = CW * es / 16;   // 16-byte chunks per row
        constexpr bool p2 = (cpr & (cpr - 1)) == 0;           // else the rows are 16 bytes apart instead
        constexpr int RS = CW * es + (p2 ? 0 : 16);
        static_assert(PART + 32 * RS * NW <= KG * RING, "epilogue regions");
        uint8_t* my = lds + PART + wave * 32 * RS;
        auto at = [&](int tok, int c) { return my + tok * RS + ((p2 ? c ^ (tok & (cpr - 1)) : c) << 4); };
        const int tl = wt * (BT / WT) + 32 * tb;   // first token of the block in the tile
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int q = 0; q < (GATED ? 2 : 4); ++q) {   // 4 channels
                const int cl = (GATED ? 16 : 32) * b + 8 * q + 4 * hh;
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = value(b, 4 * q + j);
                if (es == 4)
                    *reinterpret_cast<f32x4*>(at(l32, cl >> 2)) = f32x4{v[0], v[1], v[2], v[3]};
                else
                    *reinterpret_cast<u32x2*>(at(l32, cl >> 3) + 8 * hh) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint8_t* base = static_cast<uint8_t*>(out) + ((t0 + tl) * ldo + n0 + col0) * es;
        if (reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo * es % 16 == 0 && col0 * es % 16 == 0) {
#pragma unroll 4
            for (int i0 = 0; i0 < 32 * cpr; i0 += 64) {
                const int it = i0 + lane;
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
            for (int i0 = 0; i0 < 32 * CW; i0 += 64) {
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
    for (int tb = 0; tb < TB; ++tb) {
        auto result = [&](int b, int v) {
            return GATED ? act_fn(p.act, acc[b][tb][v]) * acc[b][tb][GATED ? v + 8 : v] : acc[b][tb][v];
        };
        if (p.out_dt == F32)
            leave(is_f32(), tb, p.out, p.ldo, 0, result);
        else
            leave(is_bf16(), tb, p.out, p.ldo, 0, result);
        if (GATED && p.pre != nullptr) {
            leave(is_bf16(), tb, p.pre, p.ldp, 0, [&](int b, int v) { return acc[b][tb][v]; });
            leave(is_bf16(), tb, p.pre, p.ldp, p.N, [&](int b, int v) { return acc[b][tb][GATED ? v + 8 : v]; });
        }
    }
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
// over 256 CUs takes ceil(W / 256) of them after each other, so with `steps` K steps
// about steps * max(alone, ceil(W / 256) * full) + fixed: `full` is the time of a step,
// `alone` that of a workgroup that has its CU for itself where it is longer.
struct Bf16Tile {
    int bn, bt;
    float alone, full, fixed;
};
constexpr int N_BF16_TILES = 10;

static int pick_bf16_tile(const Bf16Tile* tiles, int64_t T, int64_t rows, int K) {
    int best = N_BF16_TILES - 1;
    float best_us = 1e30f;
    for (int i = 0; i < N_BF16_TILES; ++i) {
        const Bf16Tile& c = tiles[i];
        const int64_t W = ((rows + c.bn - 1) / c.bn) * ((T + c.bt - 1) / c.bt);
        if (W >= (1 << 22)) continue;   // keeps every launch below 2^32 threads
        const float turns = static_cast<float>((W + 255) / 256) * c.full;
        const float us = static_cast<float>((K + 63) / 64) * (turns > c.alone ? turns : c.alone) + c.fixed;
        if (us < best_us) {
            best_us = us;
            best = i;
        }
    }
    return best;
}

template <int KIND, bool AD>
static hipError_t bf16_tiles(const Bf16Tile* tiles, const MatBf16Params& p, hipStream_t s) {
    switch (pick_bf16_tile(tiles, p.T, static_cast<int64_t>(p.N) * (KIND == MAT_GATED ? 2 : 1), p.K)) {
        case 0: return bf16_tile<KIND, AD, 32, 32, 1, 1, 3, 4>(p, s);
        case 1: return bf16_tile<KIND, AD, 32, 64, 1, 2, 3, 4>(p, s);
        case 2: return bf16_tile<KIND, AD, 64, 64, 2, 2, 4, 2>(p, s);
        case 3: return bf16_tile<KIND, AD, 64, 64, 2, 2, 3, 1>(p, s);
        case 4: return bf16_tile<KIND, AD, 128, 64, 2, 2, 3, 1>(p, s);
        case 5: return bf16_tile<KIND, AD, 128, 128, 2, 4, 4, 1>(p, s);
        case 6: return bf16_tile<KIND, AD, 192, 128, 2, 4, 3, 1>(p, s);
        case 7: return bf16_tile<KIND, AD, 256, 128, 4, 2, 3, 1>(p, s);
        case 8: return bf16_tile<KIND, AD, 256, 192, 4, 2, 2, 1>(p, s);
        default: return bf16_tile<KIND, AD, 256, 256, 4, 2, 2, 1>(p, s);
    }
}

constexpr Bf16Tile BF16_TILES[N_BF16_TILES] = {
    {32, 32, 0.12f, 0.12f, 1.3f},   {32, 64, 0.14f, 0.14f, 1.7f},   {64, 64, 0.18f, 0.18f, 1.9f},   {64, 64, 0.32f, 0.20f, 0.2f},
    {128, 64, 0.32f, 0.32f, 1.2f},  {128, 128, 0.52f, 0.52f, 0.4f}, {192, 128, 0.66f, 0.66f, 0.7f}, {256, 128, 0.79f, 0.79f, 1.1f},
    {256, 192, 1.08f, 1.08f, 1.1f}, {256, 256, 1.32f, 1.32f, 0.3f},
};

}  // namespace moe
