// Router top-k over scores (moe_route_score_topk), one wavefront per token.
//
//   s = softmax(l) or 1 / (1 + exp(-l));  c = s + bias;  the topk_group best of
//   the n_group groups by their largest c or the sum of their two largest; the k
//   largest c among those groups, equal ones by the lower expert id;
//   w = s of the chosen, over their sum when asked, times a scale.
//
// The choice is that of 64-bit scores: 32-bit rounding loses differences that
// decide, and two programs that round differently choose different experts.  But
// 64-bit exponentials and keys of every expert cost three times the instructions,
// and a wave is bound by instructions here (T = 16383, E = 160: 30 us, 6 MB).  So:
//   - without a bias the scores order like the logits, and the logits are compared;
//   - else the scores are taken in 32 bits with a bound on their error.  Where
//     every gap that decides (between groups, between consecutive choices and the
//     first one left out) exceeds twice the bound, the 64-bit choice is the same;
//   - where one does not, the token is chosen again in 64 bits.
// The weights of the k chosen are 64-bit always.
// Lane l holds experts l + 64 s (s < NPL).
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
// LDS written by some lanes of the wave and read by others of the same wave
__device__ __forceinline__ void lds_wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

constexpr int SCORE_MAX_GROUPS = 64;

// score of one logit in 64 bits (softmax: before the division); NaN scores 0
__device__ __forceinline__ double score64(float v, float m, int sigmoid) {
    if (v != v) return 0.0;
    if (sigmoid) return 1.0 / (1.0 + exp(-static_cast<double>(v)));
    if (m == -__builtin_inff()) return 0.0;   // every logit masked
    return v == m ? 1.0 : exp(static_cast<double>(v) - static_cast<double>(m));
}

// Ranks of the groups: lane g < G gets group g's first and second largest value
// (m1, m2) of c [E] in LDS, scanned by P lanes per group (a power of two).
template <typename F>
__device__ __forceinline__ void group_top2(const F* c, int G, int size, F lowest, F* rank, bool top2) {
    const int lane = threadIdx.x & 63;
    int lg = 0;   // log2 P
    while ((2 << lg) * G <= 64) ++lg;
    const int P = 1 << lg, g = lane >> lg, sub = lane & (P - 1);
    F m1 = lowest, m2 = lowest;
    if (g < G)
        for (int i = sub; i < size; i += P) {
            const F v = c[g * size + i];
            m2 = max(m2, min(m1, v));
            m1 = max(m1, v);
        }
    for (int d = 1; d < P; d <<= 1) {
        const F o1 = __shfl_xor(m1, d, 64), o2 = __shfl_xor(m2, d, 64);
        m2 = max(min(m1, o1), max(m2, o2));
        m1 = max(m1, o1);
    }
    if (g < G && sub == 0) rank[g] = top2 && size > 1 ? m1 + m2 : m1;
}

// Bit g: group g (rank key in lane g) is among the keep best, equal keys by the lower group.
template <typename K>
__device__ __forceinline__ uint64_t best_groups(const K* key, int G, int keep) {
    const int lane = threadIdx.x & 63;
    const K mine = key[lane < G ? lane : 0];
    int before = 0;
    for (int q = 0; q < G; ++q) {
        const K o = key[q];
        before += (o > mine || (o == mine && q < lane)) ? 1 : 0;
    }
    return __ballot(lane < G && before < keep);
}

// e / size for 0 <= e < 512, inv = 1 / size: (e + 1/2) / size is at least 1 / 1024 from
// an integer, far more than its rounding
__device__ __forceinline__ int group_of(int e, float inv) { return static_cast<int>((static_cast<float>(e) + 0.5f) * inv); }

template <int NPL>
__global__ __launch_bounds__(256) void route_score_kernel(ScoreRouteParams p) {
    __shared__ double cs[4][64 * NPL];   // c of the token (fp32 or fp64)
    __shared__ uint64_t gk[4][SCORE_MAX_GROUPS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * 4 + wave;
    if (t >= p.T) return;   // wave-uniform; the kernel has no workgroup barrier
    const int E = p.E, G = p.n_group, size = E / G;
    const bool grouped = p.topk_group < G;
    const float inv_size = 1.0f / static_cast<float>(size);
    float val[NPL], bias[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) {
        const int e = lane + 64 * s;
        const int64_t i = static_cast<int64_t>(t) * p.ld + e;
        val[s] = __builtin_nanf("");
        bias[s] = 0.0f;
        if (e < E) {
            val[s] = p.logits_dt == F32 ? static_cast<const float*>(p.logits)[i]
                                        : bf16_to_f32(static_cast<const uint16_t*>(p.logits)[i]);
            if (p.bias != nullptr) bias[s] = p.bias[e];
        }
    }
    // the largest logit (NaN when there is none): equal ones score alike also when infinite
    float m = 0.0f;
    if (!p.sigmoid) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < NPL; ++s) top = max(top, logit_ord(val[s]));
        top = __builtin_amdgcn_readfirstlane(wave_max_u32(top));
        m = top <= 1u ? __builtin_nanf("") : __uint_as_float((top & 0x80000000u) ? (top & 0x7FFFFFFFu) : ~top);
    }
    const bool by_logit = p.bias == nullptr && !(grouped && p.top2);
    float* cf = reinterpret_cast<float*>(cs[wave]);
    uint32_t* gu = reinterpret_cast<uint32_t*>(gk[wave]);

    // --- 32 bits.  U = 2^-24.  A score errs by less than 32 U: an exponential by
    // the rounding of its argument (|x| U, times e^-|x| at most 0.4 U) and 3 U, a
    // softmax sum of up to 512 terms by (8 + 6 additions) U more, the division by
    // 2 U; the sum with the bias rounds once more, by U of the result.
    float c[NPL];
    if (by_logit) {
#pragma unroll
        for (int s = 0; s < NPL; ++s) c[s] = val[s];
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            const float v = val[s];
            c[s] = p.sigmoid ? 1.0f / (1.0f + __expf(-v)) : (v == m ? 1.0f : __expf(v - m));
            if (!(v == v) || m == -__builtin_inff()) c[s] = 0.0f;
            sum += c[s];
        }
        if (!p.sigmoid) {
            sum = wave_sum_f32(sum);
            sum = sum > 0.0f ? 1.0f / sum : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            c[s] = (p.sigmoid ? c[s] : c[s] * sum) + bias[s];
            if (!(val[s] == val[s])) c[s] = __builtin_nanf("");
        }
    }
    constexpr float U = 5.9604645e-8f;
    bool sure = true;
    uint32_t key[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) key[s] = lane + 64 * s < E ? logit_ord(c[s]) : 0u;
    if (grouped) {
#pragma unroll
        for (int s = 0; s < NPL; ++s) cf[lane + 64 * s] = c[s] == c[s] ? c[s] : -__builtin_inff();
        lds_wave_sync();
        float* gf = reinterpret_cast<float*>(gk[wave]) + SCORE_MAX_GROUPS;
        group_top2<float>(cf, G, size, -__builtin_inff(), gf, p.top2);
        lds_wave_sync();
        const float mine = gf[lane < G ? lane : 0];
        if (lane < G) gu[lane] = logit_ord(mine);
        lds_wave_sync();
        const uint64_t kept = best_groups(gu, G, p.topk_group);
        if (!by_logit) {
            const bool in = lane < G && ((kept >> lane) & 1ull), out = lane < G && !((kept >> lane) & 1ull);
            // lowest kept and highest dropped rank, as order images
            const uint32_t im = logit_ord(mine);
            const uint32_t lo = ~wave_max_u32(in ? ~im : 0u), hi = wave_max_u32(out ? im : 0u);
            const float fl = __uint_as_float((lo & 0x80000000u) ? (lo & 0x7FFFFFFFu) : ~lo);
            const float fh = __uint_as_float((hi & 0x80000000u) ? (hi & 0x7FFFFFFFu) : ~hi);
            sure = fl - fh > 2.0f * (66.0f * U + 4.0f * U * fmaxf(fabsf(fl), fabsf(fh)));   // two scores each; false for NaN
        }
#pragma unroll
        for (int s = 0; s < NPL; ++s)
            if (!((kept >> (group_of(lane + 64 * s, inv_size) & 63)) & 1ull)) key[s] = 0u;
    }
    int my_id = 0;
    float my_logit = 0.0f;
    uint32_t my_key = 0;
    const int rounds = by_logit ? p.k : p.k + 1;   // one more: the first one left out (key 0 if there is none)
    for (int j = 0; j < rounds; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int s = 1; s < NPL; ++s) best = max(best, key[s]);
        best = __builtin_amdgcn_readfirstlane(wave_max_u32(best));
        int e = 0;
        float ve = 0.0f;
#pragma unroll
        for (int s = NPL - 1; s >= 0; --s) {   // ends at the lowest s holding the maximum
            const uint64_t b = __ballot(key[s] == best);
            if (b != 0ull) {
                const int ln = __ffsll(static_cast<unsigned long long>(b)) - 1;
                e = ln + 64 * s;
                ve = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(val[s]), ln));
            }
        }
#pragma unroll
        for (int s = 0; s < NPL; ++s)
            if (lane + 64 * s == e) key[s] = 0u;
        if (lane == j) {
            my_id = e;
            my_logit = ve;
            my_key = best;
        }
    }
    if (!by_logit) {
        // lane j < k: the gap to the next one (lane k holds the first left out)
        const uint32_t next = __shfl_down(my_key, 1, 64);
        const float a = __uint_as_float((my_key & 0x80000000u) ? (my_key & 0x7FFFFFFFu) : ~my_key);
        const float b = __uint_as_float((next & 0x80000000u) ? (next & 0x7FFFFFFFu) : ~next);
        const bool ok = lane >= p.k || next == 0u || a - b > 2.0f * (32.0f * U + 2.0f * U * fmaxf(fabsf(a), fabsf(b)));
        sure = sure && __ballot(!ok) == 0ull;
    }

    double sum64 = 0.0;   // softmax: the 64-bit sum over all experts, where it is wanted
    const bool full = !p.sigmoid && (!sure || !p.renorm);
    double sc[NPL];
    if (full || !sure) {
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            sc[s] = score64(val[s], m, p.sigmoid);
            sum64 += sc[s];
        }
        if (full) sum64 = wave_sum_f64(sum64);
    }
    if (!sure) {
        // --- 64 bits
        uint64_t key64[NPL];
        double* cd = cs[wave];
        lds_wave_sync();   // the 32-bit values have been read
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            double x = sc[s];
            if (!p.sigmoid) x = sum64 > 0.0 ? x / sum64 : 0.0;
            x += static_cast<double>(bias[s]);
            if (!(val[s] == val[s])) x = __builtin_nan("");
            key64[s] = lane + 64 * s < E ? score_key(x) : 0ull;
            cd[lane + 64 * s] = x == x ? x : -__builtin_inf();
        }
        if (grouped) {
            lds_wave_sync();
            double* gd = reinterpret_cast<double*>(gk[wave]);
            group_top2<double>(cd, G, size, -__builtin_inf(), gd, p.top2);
            lds_wave_sync();
            const double mine = gd[lane < G ? lane : 0];
            lds_wave_sync();
            if (lane < G) gk[wave][lane] = score_key(mine);
            lds_wave_sync();
            const uint64_t kept = best_groups(gk[wave], G, p.topk_group);
#pragma unroll
            for (int s = 0; s < NPL; ++s)
                if (!((kept >> (group_of(lane + 64 * s, inv_size) & 63)) & 1ull)) key64[s] = 0ull;
        }
        for (int j = 0; j < p.k; ++j) {
            uint64_t best = key64[0];
#pragma unroll
            for (int s = 1; s < NPL; ++s) best = max(best, key64[s]);
            best = wave_max_u64(best);
            int e = 0;
            float ve = 0.0f;
#pragma unroll
            for (int s = NPL - 1; s >= 0; --s) {
                const uint64_t b = __ballot(key64[s] == best);
                if (b != 0ull) {
                    const int ln = __ffsll(static_cast<unsigned long long>(b)) - 1;
                    e = ln + 64 * s;
                    ve = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(val[s]), ln));
                }
            }
#pragma unroll
            for (int s = 0; s < NPL; ++s)
                if (lane + 64 * s == e) key64[s] = 0ull;
            if (lane == j) {
                my_id = e;
                my_logit = ve;
            }
        }
    }
    // weights, lane j
    double w = lane < p.k ? score64(my_logit, m, p.sigmoid) : 0.0;
    if (p.renorm) {
        const double sum = wave_sum_f64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    } else if (!p.sigmoid) {
        w = sum64 > 0.0 ? w / sum64 : 0.0;
    }
    if (lane < p.k) {
        p.ids[static_cast<int64_t>(t) * p.k + lane] = my_id;
        p.w[static_cast<int64_t>(t) * p.k + lane] = static_cast<float>(w * static_cast<double>(p.scale));
    }
}

hipError_t launch_route_score(const ScoreRouteParams& p, hipStream_t s) {
    const dim3 grid((p.T + 3) / 4), block(256);
    auto kn = p.E <= 64 ? route_score_kernel<1>
                        : p.E <= 128 ? route_score_kernel<2>
                                     : p.E <= 192 ? route_score_kernel<3>
                                                  : p.E <= 256 ? route_score_kernel<4> : route_score_kernel<8>;
    hipLaunchKernelGGL(kn, grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace moe
