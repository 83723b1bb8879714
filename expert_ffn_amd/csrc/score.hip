// Router top-k over scores (moe_route_score_topk), one wavefront per token.
//
//   s = softmax(l) or 1 / (1 + exp(-l));  c = s + bias;  the topk_group best of
//   the n_group groups by their largest c or the sum of their two largest; the k
//   largest c among those groups, equal ones by the lower expert id;
//   w = s of the chosen, over their sum when asked, times a scale.
//
// The choice is taken in 64 bits: a sum with a bias rounds away differences of
// the scores that decide, and two programs that round differently in 32 bits
// choose different experts.  Lane l holds experts l + 64 s (s < NPL).
#include "block.h"
#include "common.h"
#include "route.h"

namespace moe {

// Order-preserving image of a double: NaN -> 1 (below -inf), 0 is left for
// experts that cannot be chosen.
__device__ __forceinline__ uint64_t score_key(double c) {
    if (c != c) return 1ull;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(c + 0.0));
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    return (static_cast<uint64_t>(dpp_u32<CTRL>(static_cast<uint32_t>(v >> 32))) << 32) |
           dpp_u32<CTRL>(static_cast<uint32_t>(v));
}
__device__ __forceinline__ uint64_t swap16_max(uint64_t v) {
    const auto lo = __builtin_amdgcn_permlane16_swap(static_cast<uint32_t>(v), static_cast<uint32_t>(v), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(static_cast<uint32_t>(v >> 32), static_cast<uint32_t>(v >> 32),
                                                     false, false);
    return max((static_cast<uint64_t>(hi[0]) << 32) | lo[0], (static_cast<uint64_t>(hi[1]) << 32) | lo[1]);
}
__device__ __forceinline__ uint64_t swap32_max(uint64_t v) {
    const auto lo = __builtin_amdgcn_permlane32_swap(static_cast<uint32_t>(v), static_cast<uint32_t>(v), false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(static_cast<uint32_t>(v >> 32), static_cast<uint32_t>(v >> 32),
                                                     false, false);
    return max((static_cast<uint64_t>(hi[0]) << 32) | lo[0], (static_cast<uint64_t>(hi[1]) << 32) | lo[1]);
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
    v = max(v, dpp_u64<DPP_QUAD_1032>(v));
    v = max(v, dpp_u64<DPP_QUAD_2301>(v));
    v = max(v, dpp_u64<DPP_ROW_HALF_MIRROR>(v));
    v = max(v, dpp_u64<DPP_ROW_MIRROR>(v));
    return swap32_max(swap16_max(v));
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    return v;
}
__device__ __forceinline__ double lane_f64(double v, int ln) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), ln);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), ln);
    return __longlong_as_double(static_cast<long long>((static_cast<uint64_t>(hi) << 32) | lo));
}

// LDS written by some lanes of the wave and read by others of the same wave
__device__ __forceinline__ void lds_wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

constexpr int SCORE_MAX_GROUPS = 64;

template <int NPL>
__global__ __launch_bounds__(256) void route_score_kernel(ScoreRouteParams p) {
    __shared__ double cs[4][64 * NPL];
    __shared__ uint64_t gk[4][SCORE_MAX_GROUPS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * 4 + wave;
    if (t >= p.T) return;   // wave-uniform; the kernel has no workgroup barrier
    const int E = p.E;
    float val[NPL];
    double sc[NPL], c[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) {
        const int e = lane + 64 * s;
        const int64_t i = static_cast<int64_t>(t) * p.ld + e;
        val[s] = __builtin_nanf("");
        if (e < E)
            val[s] = p.logits_dt == F32 ? static_cast<const float*>(p.logits)[i]
                                        : bf16_to_f32(static_cast<const uint16_t*>(p.logits)[i]);
    }
    // scores; a NaN logit (and a lane past E) scores 0
    if (p.sigmoid) {
#pragma unroll
        for (int s = 0; s < NPL; ++s)
            sc[s] = val[s] == val[s] ? 1.0 / (1.0 + exp(-static_cast<double>(val[s]))) : 0.0;
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < NPL; ++s) top = max(top, logit_ord(val[s]));
        top = wave_max_u32(top);
        // the largest logit (NaN when there is none): equal ones score alike also when infinite
        const float m = top <= 1u ? __builtin_nanf("")
                                  : __uint_as_float((top & 0x80000000u) ? (top & 0x7FFFFFFFu) : ~top);
        double sum = 0.0;
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            sc[s] = val[s] == m ? 1.0
                                : (val[s] == val[s] ? exp(static_cast<double>(val[s]) - static_cast<double>(m)) : 0.0);
            if (m == -__builtin_inff()) sc[s] = 0.0;   // every logit masked
            sum += sc[s];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int s = 0; s < NPL; ++s) sc[s] = sum > 0.0 ? sc[s] / sum : 0.0;
    }
    uint64_t key[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) {
        const int e = lane + 64 * s;
        c[s] = sc[s];
        if (p.bias != nullptr && e < E) c[s] += static_cast<double>(p.bias[e]);
        if (val[s] != val[s]) c[s] = __builtin_nan("");
        key[s] = e < E ? score_key(c[s]) : 0ull;
    }
    if (p.topk_group < p.n_group) {
        // group ranks through LDS, P lanes per group (a power of two)
        const int G = p.n_group, size = E / G;
#pragma unroll
        for (int s = 0; s < NPL; ++s) cs[wave][lane + 64 * s] = c[s] == c[s] ? c[s] : -__builtin_inf();
        lds_wave_sync();
        int lg = 0;   // log2 P
        while ((2 << lg) * G <= 64) ++lg;
        const int P = 1 << lg, g = lane >> lg, sub = lane & (P - 1);
        double m1 = -__builtin_inf(), m2 = -__builtin_inf();
        if (g < G)
            for (int i = sub; i < size; i += P) {
                const double v = cs[wave][g * size + i];
                m2 = fmax(m2, fmin(m1, v));
                m1 = fmax(m1, v);
            }
        for (int d = 1; d < P; d <<= 1) {
            const double o1 = __shfl_xor(m1, d, 64), o2 = __shfl_xor(m2, d, 64);
            m2 = fmax(fmin(m1, o1), fmax(m2, o2));
            m1 = fmax(m1, o1);
        }
        if (g < G && sub == 0) gk[wave][g] = score_key(p.top2 && size > 1 ? m1 + m2 : m1);
        lds_wave_sync();
        // lane g keeps its group when fewer than topk_group groups precede it
        int before = 0;
        const uint64_t mine = lane < G ? gk[wave][lane] : 0ull;
        for (int q = 0; q < G; ++q) {
            const uint64_t o = gk[wave][q];
            before += (o > mine || (o == mine && q < lane)) ? 1 : 0;
        }
        const uint64_t kept = __ballot(lane < G && before < p.topk_group);
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            const int e = lane + 64 * s;
            if (e < E && !((kept >> (e / size)) & 1ull)) key[s] = 0ull;
        }
    }
    int my_id = 0;
    double my_s = 0.0;
    for (int j = 0; j < p.k; ++j) {
        uint64_t best = key[0];
#pragma unroll
        for (int s = 1; s < NPL; ++s) best = max(best, key[s]);
        best = wave_max_u64(best);
        int e = 0;
        double se = 0.0;
#pragma unroll
        for (int s = NPL - 1; s >= 0; --s) {   // ends at the lowest s holding the maximum
            const uint64_t b = __ballot(key[s] == best);
            if (b != 0ull) {
                const int ln = __ffsll(static_cast<unsigned long long>(b)) - 1;
                e = ln + 64 * s;
                se = lane_f64(sc[s], ln);
            }
        }
#pragma unroll
        for (int s = 0; s < NPL; ++s)
            if (lane + 64 * s == e) key[s] = 0ull;
        if (lane == j) {
            my_id = e;
            my_s = se;
        }
    }
    const double sum = wave_sum_f64(lane < p.k ? my_s : 0.0);
    if (lane < p.k) {
        const double w = p.renorm ? (sum > 0.0 ? my_s / sum : 0.0) : my_s;
        p.ids[static_cast<int64_t>(t) * p.k + lane] = my_id;
        p.w[static_cast<int64_t>(t) * p.k + lane] = static_cast<float>(w * static_cast<double>(p.scale));
    }
}

hipError_t launch_route_score(const ScoreRouteParams& p, hipStream_t s) {
    const dim3 grid((p.T + 3) / 4), block(256);
    auto kn = p.E <= 64 ? route_score_kernel<1>
                        : p.E <= 128 ? route_score_kernel<2>
                                     : p.E <= 256 ? route_score_kernel<4> : route_score_kernel<8>;
    hipLaunchKernelGGL(kn, grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace moe
