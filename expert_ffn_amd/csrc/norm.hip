// RMS norms before and after the block, fused with what stands next to them:
// the 8-bit codes of the integer products before, and after the block the
// combine, the dense expert's rows, the gate, the residual and the next norm.
//
//   norm:   r = 1 / sqrt(mean h^2 + eps),  x = (h r) (off + w)
//   codes:  u = h (off + w),  a = max |u|,  s = a fl(1 / 127),  q = rint(u / s),
//           scale = s r: r cancels in the codes of the normed row, so they
//           depend on no order of summation, and one pass over the row gives
//           the sum of squares and the maximum together.
//   after:  b = sum_j w_j o_pos(j) + y,  n = norm(b),
//           h' = res h + block gate n,  x = norm(h' as stored)
//
// Memory bound: every input is read once and every output written once.  One
// workgroup takes one row and keeps it in registers between the reduction and
// the write; a thread holds C chunks of 8 elements, chunk i at
// threadIdx + i * blockDim.  Before the block, rows of up to 512 elements share
// workgroups, 16, 32 or 64 lanes a row: with a workgroup of 64 threads each their
// dispatch decides (16384 bf16 rows of 64: 5.6 us, shared 3.0; codes 6.7 and 3.2).
// After it that gained nothing (12.1 and 11.8).  Sums and statistics are fp32, in a
// fixed order (chunks in a thread, lanes, waves), so results are reproducible.
#include "block.h"
#include "common.h"
#include "route.h"

#pragma clang fp contract(off)

namespace moe {

struct Raw8 {
    u32x4 a, b;   // 8 elements: bf16 in a, fp32 in a and b
};

__device__ __forceinline__ Raw8 load_raw8(const void* p, int dt, int64_t i) {
    Raw8 r;
    if (dt == F32) {
        const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
        r.a = s[0];
        r.b = s[1];
    } else {
        r.a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
        r.b = u32x4{0u, 0u, 0u, 0u};
    }
    return r;
}
__device__ __forceinline__ void widen8(const Raw8& r, int dt, float (&v)[8]) {
    if (dt == F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(r.a[j]);
            v[4 + j] = __uint_as_float(r.b[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(r.a[j] << 16);
            v[2 * j + 1] = __uint_as_float(r.a[j] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ u32x4 narrow8(const float (&v)[8]) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    return o;
}
__device__ __forceinline__ void store8(void* p, int dt, int64_t i, const float (&v)[8]) {
    if (dt == F32) {
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
        d[0] = f32x4{v[0], v[1], v[2], v[3]};
        d[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = narrow8(v);
    }
}

// off + w of 8 channels (1 without a weight)
__device__ __forceinline__ void weight8(const Raw8& r, const void* w, int dt, float off, float (&v)[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
        return;
    }
    widen8(r, dt, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = off + v[j];
}

// |v| as bits: ordered like |v|, infinities above every number and NaN above them
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// step of the codes of a row whose largest |u| has the bits `top`: one product with
// 1 / 127 rounded to fp32, as a division by a constant is usually computed
__device__ __forceinline__ float code_step(uint32_t top) { return __uint_as_float(top) * (1.0f / 127.0f); }

// 8 codes of u at scale s (all 0 when s is 0, infinite or NaN)
__device__ __forceinline__ u32x2 codes8(const float (&u)[8], float s) {
    u32x2 o = {0u, 0u};
    if (s > 0.0f && s < __builtin_inff()) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = fminf(fmaxf(rintf(u[j] / s), -127.0f), 127.0f);
            o[j >> 2] |= (static_cast<uint32_t>(static_cast<int>(c)) & 0xFFu) << (8 * (j & 3));
        }
    }
    return o;
}

struct RowStat {
    float sum;
    uint32_t top;
};
constexpr int MAX_WAVES = 16;

// Sum and maximum over the workgroup; red has MAX_WAVES entries of its own for
// each use in a kernel, so one barrier is enough.
__device__ __forceinline__ RowStat block_stat(RowStat s, RowStat* red, bool top) {
    s.sum = wave_sum_f32(s.sum);
    if (top) s.top = wave_max_u32(s.top);
    const int nw = blockDim.x >> 6;
    if (nw == 1) return s;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    RowStat r = red[0];
    for (int i = 1; i < nw; ++i) {
        r.sum += red[i].sum;
        r.top = max(r.top, red[i].top);
    }
    return r;
}

// Sum and maximum over LPR lanes, 16, 32 or 64: the sums of block_stat where the
// lanes past LPR hold zeros.
template <int LPR>
__device__ __forceinline__ RowStat lanes_stat(RowStat s, bool top) {
    s.sum += __uint_as_float(dpp_u32<DPP_QUAD_1032>(__float_as_uint(s.sum)));
    s.sum += __uint_as_float(dpp_u32<DPP_QUAD_2301>(__float_as_uint(s.sum)));
    s.sum += __uint_as_float(dpp_u32<DPP_ROW_HALF_MIRROR>(__float_as_uint(s.sum)));
    s.sum += __uint_as_float(dpp_u32<DPP_ROW_MIRROR>(__float_as_uint(s.sum)));
    if (LPR >= 32) s.sum = sum16(s.sum);
    if (LPR >= 64) s.sum = sum32(s.sum);
    if (top) {
        s.top = max(s.top, dpp_u32<DPP_QUAD_1032>(s.top));
        s.top = max(s.top, dpp_u32<DPP_QUAD_2301>(s.top));
        s.top = max(s.top, dpp_u32<DPP_ROW_HALF_MIRROR>(s.top));
        s.top = max(s.top, dpp_u32<DPP_ROW_MIRROR>(s.top));
        if (LPR >= 32) s.top = max16(s.top);
        if (LPR >= 64) s.top = max32(s.top);
    }
    return s;
}

constexpr int SHARED_THREADS = 256;   // of a workgroup that several rows share

// LPR = 0: a row per workgroup.  Else LPR lanes a row, C = 1.
template <int HT, int C, bool NORM, int LPR>
__global__ __launch_bounds__(LPR ? SHARED_THREADS : 1024) void norm_in_kernel(const void* __restrict__ h, int64_t ldh, int T, int H,
                                                                              NormOut o) {
    static_assert(LPR == 0 || C == 1, "a short row has one chunk per lane");
    __shared__ RowStat red[MAX_WAVES];
    constexpr int D = LPR ? LPR : 1;
    const int row = LPR ? static_cast<int>(blockIdx.x) * (SHARED_THREADS / D) + static_cast<int>(threadIdx.x) / D : blockIdx.x;
    const int t = LPR ? min(row, T - 1) : row, tid = LPR ? threadIdx.x % D : threadIdx.x, nt = LPR ? LPR : blockDim.x;
    const int nchunk = LPR && row >= T ? 0 : H >> 3;
    const int64_t hb = static_cast<int64_t>(t) * ldh;
    Raw8 hr[C], wr[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = tid + i * nt;
        if (c < nchunk) {
            hr[i] = load_raw8(h, HT, hb + 8 * c);
            if (NORM && o.w != nullptr) wr[i] = load_raw8(o.w, o.w_dt, 8 * c);
        }
    }
    RowStat st = {0.0f, 0u};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (tid + i * nt >= nchunk) continue;
        float v[8], w[8];
        widen8(hr[i], HT, v);
        if (NORM) {
#pragma unroll
            for (int j = 0; j < 8; ++j) st.sum = fmaf(v[j], v[j], st.sum);
            weight8(wr[i], o.w, o.w_dt, o.w_offset, w);
        }
        if (o.xq != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) st.top = max(st.top, abs_bits(NORM ? v[j] * w[j] : v[j]));
        }
    }
    st = LPR ? lanes_stat<LPR>(st, o.xq != nullptr) : block_stat(st, red, o.xq != nullptr);
    const float r = NORM ? 1.0f / sqrtf(st.sum / static_cast<float>(H) + o.eps) : 1.0f;
    const float s = code_step(st.top);
    if (o.xq != nullptr && tid == 0 && nchunk > 0) o.xq_scale[t] = s * r;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = tid + i * nt;
        if (c >= nchunk) continue;
        float v[8], w[8], x[8];
        widen8(hr[i], HT, v);
        if (NORM) weight8(wr[i], o.w, o.w_dt, o.w_offset, w);
        if (NORM && o.x != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = v[j] * r * w[j];
            store8(o.x, o.x_dt, static_cast<int64_t>(t) * o.ldx + 8 * c, x);
        }
        if (o.xq != nullptr) {
            if (NORM) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * w[j];
            }
            *reinterpret_cast<u32x2*>(o.xq + static_cast<int64_t>(t) * o.ldq + 8 * c) = codes8(v, s);
        }
    }
}

// Threads and chunks per thread of a row of nchunk chunks: one chunk each while
// at most `cap` threads take part, then 2 or 4 (at most 1024 threads then:
// NORM_H_MAX = 1024 * 4 * 8).
static int row_threads(int nchunk, int cap, int* C) {
    int c = 1;
    while (c < 4 && (nchunk + c - 1) / c > cap) c *= 2;
    *C = c;
    return ((nchunk + c - 1) / c + 63) / 64 * 64;
}
// Many rows: at most 256 threads to a row, so that a CU holds several rows and one's
// reads run behind another's reductions (8191 bf16 rows of 2816 17.3 us, with up to
// 1024 threads 20.2; of 8192 48.3 and 52.3).  Few rows: a thread has one chunk if it
// can (256 rows of 8192 3.8 us, in 256 threads 4.3).
constexpr int NORM_MANY_ROWS = 1024;

template <int HT, bool NORM>
static hipError_t norm_in_by_chunks(const void* h, int64_t ldh, int T, int H, const NormOut& o, hipStream_t s) {
    const int nchunk = H / 8;
    if (nchunk <= 64) {
        const int lpr = nchunk <= 16 ? 16 : nchunk <= 32 ? 32 : 64, rows = SHARED_THREADS / lpr;
        auto kn = lpr == 16 ? norm_in_kernel<HT, 1, NORM, 16>
                            : lpr == 32 ? norm_in_kernel<HT, 1, NORM, 32> : norm_in_kernel<HT, 1, NORM, 64>;
        hipLaunchKernelGGL(kn, dim3((T + rows - 1) / rows), dim3(SHARED_THREADS), 0, s, h, ldh, T, H, o);
        return hipGetLastError();
    }
    int C;
    const int nt = row_threads(nchunk, T >= NORM_MANY_ROWS ? 256 : 1024, &C);
    const dim3 grid(T), block(nt);
    auto kn = C == 1 ? norm_in_kernel<HT, 1, NORM, 0>
                     : C == 2 ? norm_in_kernel<HT, 2, NORM, 0> : norm_in_kernel<HT, 4, NORM, 0>;
    hipLaunchKernelGGL(kn, grid, block, 0, s, h, ldh, T, H, o);
    return hipGetLastError();
}

hipError_t launch_norm_in(const void* h, int h_dt, int64_t ldh, int T, int H, const NormOut& o, hipStream_t s) {
    return h_dt == F32 ? norm_in_by_chunks<F32, true>(h, ldh, T, H, o, s)
                       : norm_in_by_chunks<BF16, true>(h, ldh, T, H, o, s);
}

hipError_t launch_quantize_tokens(const void* x, int x_dt, int64_t ldx, int T, int K, int8_t* q, int64_t ldq,
                                  float* scale, hipStream_t s) {
    NormOut o{};
    o.xq = q;
    o.ldq = ldq;
    o.xq_scale = scale;
    return x_dt == F32 ? norm_in_by_chunks<F32, false>(x, ldx, T, K, o, s)
                       : norm_in_by_chunks<BF16, false>(x, ldx, T, K, o, s);
}

// After the block.  The routes of a row are requested four at a time, all loads
// before the first addition; the sums run in ascending j, then y, fp32.  (Eight at a
// time, with the weights and the gate requested at the start, took 3 to 9 % less for
// 16 to 256 rows of 2816 and 5 to 18 % more for rows of 7168 and for many rows.)
//
// The loads go through buffer resources of one row each, sized 0 where there is
// nothing to read (no y, an absent route, the upper half of a bf16 chunk, chunks past
// H): such a load gives zeros without a branch.  With branches the compiler waits for
// every load in flight before the next one (16 rows of 2816 with 8 fp32 routes: 6.0 us,
// without 5.2; 1024 rows 25.0 and 23.4, 113 MB).
struct RowSrc {
    rsrc_t a, b;   // elements 0-3 (fp32) or 0-7 (bf16) of a chunk, elements 4-7
    uint32_t es;
};
__device__ __forceinline__ RowSrc row_src(const void* p, int dt, int64_t i, int H, bool on) {
    RowSrc r;
    r.es = dt == F32 ? 4 : 2;
    const uint8_t* q = static_cast<const uint8_t*>(p) + (on ? i * r.es : 0);
    const uint32_t n = on ? H * r.es : 0;
    r.a = make_rsrc(q, n);
    r.b = make_rsrc(q, dt == F32 ? n : 0);
    return r;
}
__device__ __forceinline__ Raw8 load_src(const RowSrc& r, int c) {
    const uint32_t o = static_cast<uint32_t>(c) * 8 * r.es;
    return Raw8{bload16(r.a, o), bload16(r.b, o + 16)};
}

// FAR: out_routes of 2 GiB or more, a resource per route; else one, and 32-bit offsets
// (a resource takes 25 scalar instructions, an offset 4: 16 rows of 2816 with 8 routes
// 5.24 us, 5.04 with offsets; 16 of 7168 7.06 and 6.71).
template <int OT, int C, bool FAR>
__global__ __launch_bounds__(1024) void norm_out_kernel(NormOutParams p) {
    constexpr int CH = C == 4 ? 2 : 4;   // (within 128 registers)
    __shared__ RowStat red[2][MAX_WAVES];
    const int t = blockIdx.x, nt = blockDim.x, H = p.H, nchunk = H >> 3;
    const bool codes = p.next && p.n.xq != nullptr;
    const RowSrc hs = row_src(p.h, p.h_dt, t * p.ldh, H, true), ys = row_src(p.y, p.y_dt, t * p.ldy, H, p.y != nullptr);
    const RowSrc wps = row_src(p.w_post, p.w_dt, 0, H, p.w_post != nullptr);
    const RowSrc wns = row_src(p.n.w, p.w_dt, 0, H, p.next && p.n.w != nullptr);
    // the gate's row, or its one element
    const RowSrc gs = row_src(p.gate, p.gate_dt, t * p.gate_st, H, p.gate != nullptr && p.gate_sh != 0);
    const RowSrc g1 = row_src(p.gate, p.gate_dt, t * p.gate_st, 1, p.gate != nullptr && p.gate_sh == 0);
    auto load_gate = [&](int c) {
        Raw8 r = load_src(gs, c);
        // (g1.b has size 0 for bf16)
        const uint32_t e = __builtin_amdgcn_raw_buffer_load_b32(g1.b, 0, 0, 0), h = bload_u16(g1.a, 0, 0) << 16;
        if (p.gate_sh == 0) r.a[0] = p.gate_dt == F32 ? e : h;
        return r;
    };
    auto gate8 = [&](const Raw8& r, float (&g)[8]) {
        if (p.gate_sh != 0) {
            widen8(r, p.gate_dt, g);
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __uint_as_float(r.a[0]);
    };
    const uint32_t rowb = static_cast<uint32_t>(H) * (OT == F32 ? 4 : 2);
    const rsrc_t routes = make_rsrc(p.out_routes, FAR ? 0 : static_cast<uint32_t>(p.T * p.k) * rowb);
    auto load_route = [&](int pj, bool on, int c) {
        if (FAR) return load_src(row_src(p.out_routes, OT, static_cast<int64_t>(pj) * H, H, on), c);
        const uint32_t o = on && c < nchunk ? static_cast<uint32_t>(pj) * rowb + static_cast<uint32_t>(c) * (OT == F32 ? 32 : 16) : NO_LANE;
        return Raw8{bload16(routes, o), OT == F32 ? bload16(routes, o + 16) : u32x4{0u, 0u, 0u, 0u}};
    };
    float b[C][8];
    Raw8 hr[C], yr[C];
    RowStat st = {0.0f, 0u};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * nt;
        hr[i] = load_src(hs, c);
        yr[i] = load_src(ys, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[i][j] = 0.0f;
        for (int j0 = 0; j0 < p.k; j0 += CH) {
            int pj[CH];
            float wj[CH];
            Raw8 rows[CH];
#pragma unroll
            for (int q = 0; q < CH; ++q) {
                const int64_t j = static_cast<int64_t>(t) * p.k + min(j0 + q, p.k - 1);
                pj[q] = p.route_pos[j];
                wj[q] = p.topk_w[j];
            }
            __builtin_amdgcn_sched_barrier(0);   // all of them before the first wait
#pragma unroll
            for (int q = 0; q < CH; ++q) {
                const bool on = j0 + q < p.k && pj[q] >= 0 && pj[q] < p.T * p.k;
                wj[q] = on ? wj[q] : 0.0f;
                rows[q] = load_route(pj[q], on, c);
            }
#pragma unroll
            for (int q = 0; q < CH; ++q) {
                float v[8];
                widen8(rows[q], OT, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[i][j] = fmaf(wj[q], v[j], b[i][j]);
            }
        }
        float v[8];
        widen8(yr[i], p.y_dt, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            b[i][j] += v[j];
            st.sum = fmaf(b[i][j], b[i][j], st.sum);
        }
    }
    float r = 1.0f;
    if (p.w_post != nullptr) {
        st = block_stat(st, red[0], false);
        r = 1.0f / sqrtf(st.sum / static_cast<float>(H) + p.eps);
    }
    st = {0.0f, 0u};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= nchunk) continue;
        float v[8], g[8];
        if (p.w_post != nullptr) {
            weight8(load_src(wps, c), p.w_post, p.w_dt, p.w_offset, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[i][j] = b[i][j] * r * v[j];
        }
        if (p.gate != nullptr) {
            gate8(load_gate(c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[i][j] = b[i][j] * g[j];
        }
        widen8(hr[i], p.h_dt, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p.res_scale * v[j] + p.block_scale * b[i][j];
        store8(p.h_out, p.h_dt, static_cast<int64_t>(t) * p.ldho + 8 * c, v);
        if (!p.next) continue;
        if (p.h_dt == BF16) {   // the next norm is that of the row as it is stored
            Raw8 s;
            s.a = narrow8(v);
            widen8(s, BF16, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) st.sum = fmaf(v[j], v[j], st.sum);
        if (codes) {
            weight8(load_src(wns, c), p.n.w, p.w_dt, p.w_offset, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) st.top = max(st.top, abs_bits(v[j] * g[j]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) b[i][j] = v[j];
    }
    if (!p.next) return;
    st = block_stat(st, red[1], codes);
    r = 1.0f / sqrtf(st.sum / static_cast<float>(H) + p.n.eps);
    const float s = code_step(st.top);
    if (codes && threadIdx.x == 0) p.n.xq_scale[t] = s * r;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= nchunk) continue;
        float w[8], x[8];
        weight8(load_src(wns, c), p.n.w, p.w_dt, p.w_offset, w);
        if (p.n.x != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = b[i][j] * r * w[j];
            store8(p.n.x, p.n.x_dt, static_cast<int64_t>(t) * p.n.ldx + 8 * c, x);
        }
        if (codes) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = b[i][j] * w[j];
            *reinterpret_cast<u32x2*>(p.n.xq + static_cast<int64_t>(t) * p.n.ldq + 8 * c) = codes8(x, s);
        }
    }
}

template <int OT>
static hipError_t norm_out_by_chunks(const NormOutParams& p, hipStream_t s) {
    int C;
    const int nt = row_threads(p.H / 8, 1024, &C);
    const bool far = static_cast<int64_t>(p.T) * p.k * p.H * (OT == F32 ? 4 : 2) >= (1ll << 31);
    auto kn = far ? (C == 1 ? norm_out_kernel<OT, 1, true> : C == 2 ? norm_out_kernel<OT, 2, true> : norm_out_kernel<OT, 4, true>)
                  : (C == 1 ? norm_out_kernel<OT, 1, false> : C == 2 ? norm_out_kernel<OT, 2, false> : norm_out_kernel<OT, 4, false>);
    hipLaunchKernelGGL(kn, dim3(p.T), dim3(nt), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_norm_out(const NormOutParams& p, hipStream_t s) {
    return p.out_dt == F32 ? norm_out_by_chunks<F32>(p, s) : norm_out_by_chunks<BF16>(p, s);
}

}  // namespace moe
