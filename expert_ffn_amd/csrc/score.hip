// Router top-k over scores (moe_route_score_topk).
//
//   s = softmax(l) or 1 / (1 + exp(-l));  c = s + bias;  the topk_group best of
//   the n_group groups by their largest c or the sum of their two largest; the k
//   largest c among those groups, equal ones by the lower expert id;
//   w = s of the chosen, over their sum when asked, times a scale.
//
// The choice is that of 64-bit scores: 32-bit rounding loses differences that
// decide, and two programs that round differently choose different experts.  But
// 64-bit exponentials and keys of every expert cost three times the instructions, and
// the time follows (T = 16383, E = 160, 6 MB of logits: 30 us in 64 bits, 8.5 as below,
// where the VALU issues in 34 % of the cycles and a wave waits 18 % of its time: the
// rest is the latency of dependent lane steps, with four waves to a SIMD).  So:
//   - without a bias the scores order like the logits, and the logits are compared
//     (all but sums of two scores that rank groups; logits that differ decide also
//     where their scores are equal in 64 bits);
//   - else the scores are taken in 32 bits with a bound on their error.  Where
//     every gap that decides (between groups, between consecutive choices and the
//     first one left out) exceeds twice the bound, the 64-bit choice is the same;
//   - where one does not, the token is chosen again in 64 bits.
// The weights of the k chosen are 64-bit always.
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
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    return __longlong_as_double(static_cast<long long>(dpp_u64<CTRL>(static_cast<uint64_t>(__double_as_longlong(v)))));
}
// sum over the 16 lanes of a row (every lane gets it)
__device__ __forceinline__ double row_sum(double v) {
    v += dpp_f64<DPP_QUAD_1032>(v);
    v += dpp_f64<DPP_QUAD_2301>(v);
    v += dpp_f64<DPP_ROW_HALF_MIRROR>(v);
    return v + dpp_f64<DPP_ROW_MIRROR>(v);
}
__device__ __forceinline__ double two_halves(uint32_t lo0, uint32_t hi0, uint32_t lo1, uint32_t hi1) {
    return __hiloint2double(static_cast<int>(hi0), static_cast<int>(lo0)) +
           __hiloint2double(static_cast<int>(hi1), static_cast<int>(lo1));
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v = row_sum(v);
    uint32_t l = static_cast<uint32_t>(__double2loint(v)), h = static_cast<uint32_t>(__double2hiint(v));
    const auto l16 = __builtin_amdgcn_permlane16_swap(l, l, false, false);
    const auto h16 = __builtin_amdgcn_permlane16_swap(h, h, false, false);
    v = two_halves(l16[0], h16[0], l16[1], h16[1]);
    l = static_cast<uint32_t>(__double2loint(v)), h = static_cast<uint32_t>(__double2hiint(v));
    const auto l32 = __builtin_amdgcn_permlane32_swap(l, l, false, false);
    const auto h32 = __builtin_amdgcn_permlane32_swap(h, h, false, false);
    return two_halves(l32[0], h32[0], l32[1], h32[1]);
}
// LDS written by some lanes of the wave and read by others of the same wave
__device__ __forceinline__ void lds_wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// score of one logit in 64 bits (softmax: before the division); NaN scores 0
__device__ __forceinline__ double score64(float v, float m, int sigmoid) {
    if (v != v) return 0.0;
    if (sigmoid) return 1.0 / (1.0 + exp(-static_cast<double>(v)));
    if (m == -__builtin_inff()) return 0.0;   // every logit masked
    return v == m ? 1.0 : exp(static_cast<double>(v) - static_cast<double>(m));
}

// The rank of group g in lane g < G: the largest value of c [E] in LDS in the group,
// or the sum of its two largest.  P lanes scan a group (a power of two).
template <typename F>
__device__ __forceinline__ F group_rank(const F* c, int G, int size, F lowest, bool top2) {
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
    return __shfl(top2 && size > 1 ? m1 + m2 : m1, (lane << lg) & 63, 64);
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int l) {
    return (static_cast<uint64_t>(lane_value(static_cast<uint32_t>(v >> 32), l)) << 32) | lane_value(static_cast<uint32_t>(v), l);
}
// Bit g: group g (rank key in lane g) is among the keep best, equal keys by the lower group.
template <typename K>
__device__ __forceinline__ uint64_t best_groups(K key, int G, int keep) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int q = 0; q < G; ++q) {
        const K o = lane_value(key, q);
        before += (o > key || (o == key && q < lane)) ? 1 : 0;
    }
    return __ballot(lane < G && before < keep);
}

// e / size for 0 <= e < 512, inv = 1 / size: (e + 1/2) / size is at least 1 / 1024 from
// an integer, far more than its rounding
__device__ __forceinline__ int group_of(int e, float inv) { return static_cast<int>((static_cast<float>(e) + 0.5f) * inv); }

// LDS of one wave
template <int NPL>
struct ScoreLds {
    double c[64 * NPL];   // c of the token (fp32 or fp64)
    float v[64 * NPL];    // logits
};

__device__ __forceinline__ float ord_value(uint32_t o) {   // the number of an order image of a number
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// Errors of the 32-bit scores, U = 2^-24.  An exponential e^-x has its argument off
// by 1.23 x U (the product with log2 e and that constant's own 0.23 U; a softmax's
// x = m - v by x U more) and errs by 2 U itself.  Sigmoid s = 1 / (1 + e): s (1 - s)
// (1.23 x + 2) U <= 0.8 U, the sum and the division U each: below 3 U.  Softmax s = e /
// sum: the score's own exponential errs by s (2.23 x + 2) U, and s x = s ln(q / s) <=
// 0.37 q with q the largest score.  The sum errs by the mean of that under the weights
// and U per addition, 13 of them with a token to a wave (8 experts a lane, 6 lane
// steps), 19 with four tokens to a wave (16 and 4, E <= 256).  The mean of x is largest
// where all the others are equal: (1 - q) ln(q (E - 1) / (1 - q)), at most 3.34 for E =
// 256 and 3.89 for 512, over all q.  The division and the product add U each.  Together s
// times 0.8 + 2.23 * 3.34 + 6 + 19 = 33.3 U (E = 512: 28.5 U): below (1 + 34 q) U.  A sum
// with a bias rounds by U of the result.
constexpr float SU = 5.9604645e-8f;
__device__ __forceinline__ float score_err(int sigmoid, float smax) { return sigmoid ? 3.0f * SU : (1.0f + 34.0f * smax) * SU; }
// Whether a > b in 32 bits settles the order in 64, each off by at most err and U of
// its size.  False for NaN.
__device__ __forceinline__ bool settled(float a, float b, float err) {
    return a - b > 2.01f * (err + SU * fmaxf(fabsf(a), fabsf(b)));
}
// |c| of a finite c (an infinite one is exact)
__device__ __forceinline__ float finite_size(float c) { return fabsf(c) < __builtin_inff() ? fabsf(c) : 0.0f; }
// nothing adds scores up: without a bias they order like the logits, and groups need
// them only for sums of two
__host__ __device__ __forceinline__ bool by_logits(const ScoreRouteParams& p) {
    return p.bias == nullptr && !(p.topk_group < p.n_group && p.top2 && p.n_group < p.E);
}
__device__ __forceinline__ float load_logit(const ScoreRouteParams& p, int t, int e) {
    const int64_t i = static_cast<int64_t>(t) * p.ld + e;
    return p.logits_dt == F32 ? static_cast<const float*>(p.logits)[i]
                              : bf16_to_f32(static_cast<const uint16_t*>(p.logits)[i]);
}
// score in 32 bits before a softmax's division; NaN scores 0
__device__ __forceinline__ float score32(float v, float m, int sigmoid) {
    const float s = sigmoid ? 1.0f / (1.0f + __expf(-v)) : (v == m ? 1.0f : __expf(v - m));
    return v == v && !(m == -__builtin_inff()) ? s : 0.0f;
}

// One token on one wave; lane l holds experts l + 64 s (s < NPL), val their logits
// (NaN past E).
template <int NPL>
__device__ __forceinline__ void score_token(const ScoreRouteParams& p, int t, const float (&val)[NPL], ScoreLds<NPL>& L) {
    const int lane = threadIdx.x & 63;
    const int E = p.E, G = p.n_group, size = E / G;
    const bool grouped = p.topk_group < G;
    const float inv_size = 1.0f / static_cast<float>(size);
    float bias[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) bias[s] = p.bias != nullptr && lane + 64 * s < E ? p.bias[lane + 64 * s] : 0.0f;
    // the largest logit (NaN when there is none): equal ones score alike also when infinite
    float m = 0.0f;
    if (!p.sigmoid) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < NPL; ++s) top = max(top, logit_ord(val[s]));
        top = __builtin_amdgcn_readfirstlane(wave_max_u32(top));
        m = top <= 1u ? __builtin_nanf("") : ord_value(top);
    }
    const bool by_logit = by_logits(p);
    float* cf = reinterpret_cast<float*>(L.c);

    // --- 32 bits
    float c[NPL], err = 0.0f;
    if (by_logit) {
#pragma unroll
        for (int s = 0; s < NPL; ++s) c[s] = val[s];
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            c[s] = score32(val[s], m, p.sigmoid);
            sum += c[s];
        }
        if (!p.sigmoid) {
            sum = wave_sum_f32(sum);
            sum = sum > 0.0f ? 1.0f / sum : 0.0f;   // the largest score too
        }
        err = score_err(p.sigmoid, sum);
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            c[s] = (p.sigmoid ? c[s] : c[s] * sum) + bias[s];
            if (!(val[s] == val[s])) c[s] = __builtin_nanf("");
        }
    }
    // --- 64 bits, where they are wanted: scores (softmax: before the division) and their sum
    double sc[NPL], sum64 = 0.0;
    auto scores64 = [&]() {
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            sc[s] = score64(val[s], m, p.sigmoid);
            sum64 += sc[s];
        }
        if (!p.sigmoid) sum64 = wave_sum_f64(sum64);
    };
    // sc becomes c (NaN where the logit is), returns the kept groups
    auto kept64 = [&]() -> uint64_t {
        double* cd = L.c;
        lds_wave_sync();   // the 32-bit values have been read
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            double x = sc[s];
            if (!p.sigmoid) x = sum64 > 0.0 ? x / sum64 : 0.0;
            x += static_cast<double>(bias[s]);
            if (!(val[s] == val[s])) x = __builtin_nan("");
            cd[lane + 64 * s] = x == x ? x : -__builtin_inf();
            sc[s] = x;
        }
        if (!grouped) return ~0ull;
        lds_wave_sync();
        return best_groups(score_key(group_rank<double>(cd, G, size, -__builtin_inf(), p.top2)), G, p.topk_group);
    };

    bool sure = true, have64 = false;
    const bool plain = p.bias == nullptr;
    uint32_t key[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) key[s] = lane + 64 * s < E ? logit_ord(plain ? val[s] : c[s]) : 0u;
    if (grouped) {
#pragma unroll
        for (int s = 0; s < NPL; ++s) cf[lane + 64 * s] = c[s] == c[s] ? c[s] : -__builtin_inff();
        lds_wave_sync();
        // of a lane past the groups: never looked at
        const uint32_t im = logit_ord(group_rank<float>(cf, G, size, -__builtin_inff(), p.top2));
        uint64_t kept = best_groups(im, G, p.topk_group);
        if (!by_logit) {
            const bool in = lane < G && ((kept >> lane) & 1ull), out = lane < G && !((kept >> lane) & 1ull);
            // lowest kept and highest dropped rank, as order images
            const uint32_t lo = ~wave_max_u32(in ? ~im : 0u), hi = wave_max_u32(out ? im : 0u);
            float two = err;   // of a group's rank: one c, or two and their sum
            if (p.top2) {
                float cmax = 0.0f;
#pragma unroll
                for (int s = 0; s < NPL; ++s) cmax = fmaxf(cmax, finite_size(c[s]));
                two = 2.0f * err + 4.0f * SU * __uint_as_float(wave_max_u32(__float_as_uint(cmax)));
            }
            sure = settled(ord_value(lo), ord_value(hi), two);
            if (plain && !sure) {
                scores64();
                kept = kept64();
                sure = have64 = true;
            }
        }
#pragma unroll
        for (int s = 0; s < NPL; ++s)
            if (!((kept >> (group_of(lane + 64 * s, inv_size) & 63)) & 1ull)) key[s] = 0u;
    }
#pragma unroll
    for (int s = 0; s < NPL; ++s) L.v[lane + 64 * s] = val[s];
    int my_id = 0;
    uint32_t my_key = 0;
    const int rounds = plain ? p.k : p.k + 1;   // one more: the first one left out (key 0 if there is none)
    for (int j = 0; j < rounds; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int s = 1; s < NPL; ++s) best = max(best, key[s]);
        best = __builtin_amdgcn_readfirstlane(wave_max_u32(best));
        int e = 0;
#pragma unroll
        for (int s = NPL - 1; s >= 0; --s) {   // ends at the lowest s holding the maximum
            const uint64_t b = __ballot(key[s] == best);
            e = b != 0ull ? __builtin_ctzll(b) + 64 * s : e;
        }
#pragma unroll
        for (int s = 0; s < NPL; ++s)
            if (lane + 64 * s == e) key[s] = 0u;
        if (lane == j) {
            my_id = e;
            my_key = best;
        }
    }
    if (!plain) {
        // lane j < k: the gap to the next one (lane k holds the first left out)
        const uint32_t next = __shfl_down(my_key, 1, 64);
        const bool ok = lane >= p.k || next == 0u || settled(ord_value(my_key), ord_value(next), err);
        sure = sure && __ballot(!ok) == 0ull;
    }

    if (!have64 && (!sure || (!p.sigmoid && !p.renorm))) scores64();
    if (!sure) {
        const uint64_t kept = kept64();
        uint64_t key64[NPL];
#pragma unroll
        for (int s = 0; s < NPL; ++s) {
            key64[s] = lane + 64 * s < E ? score_key(sc[s]) : 0ull;
            if (grouped && !((kept >> (group_of(lane + 64 * s, inv_size) & 63)) & 1ull)) key64[s] = 0ull;
        }
        for (int j = 0; j < p.k; ++j) {
            uint64_t best = key64[0];
#pragma unroll
            for (int s = 1; s < NPL; ++s) best = max(best, key64[s]);
            best = wave_max_u64(best);
            int e = 0;
#pragma unroll
            for (int s = NPL - 1; s >= 0; --s) {
                const uint64_t b = __ballot(key64[s] == best);
                e = b != 0ull ? __builtin_ctzll(b) + 64 * s : e;
            }
#pragma unroll
            for (int s = 0; s < NPL; ++s)
                if (lane + 64 * s == e) key64[s] = 0ull;
            if (lane == j) my_id = e;
        }
    }
    // weights, lane j
    lds_wave_sync();
    double w = lane < p.k ? score64(L.v[my_id], m, p.sigmoid) : 0.0;
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

template <int NPL>
__device__ __forceinline__ void score_token(const ScoreRouteParams& p, int t, ScoreLds<NPL>& L) {
    const int lane = threadIdx.x & 63;
    float val[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) val[s] = lane + 64 * s < p.E ? load_logit(p, t, lane + 64 * s) : __builtin_nanf("");
    score_token<NPL>(p, t, val, L);
}

template <int NPL>
__global__ __launch_bounds__(256) void route_score_kernel(ScoreRouteParams p) {
    __shared__ ScoreLds<NPL> lds[4];
    const int wave = threadIdx.x >> 6, t = blockIdx.x * 4 + wave;
    if (t >= p.T) return;   // wave-uniform; the kernel has no workgroup barrier
    score_token<NPL>(p, t, lds[wave]);
}

// The same behind the router's product: the logits are the sums of its HS slices
// (part [HS][T][E]) in slice order, and are written (p.logits [T, E]).
template <int NPL>
__global__ __launch_bounds__(256) void route_score_part_kernel(ScoreRouteParams p, const float* __restrict__ part, int HS,
                                                               float* __restrict__ logits) {
    __shared__ ScoreLds<NPL> lds[4];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, t = blockIdx.x * 4 + wave;
    if (t >= p.T) return;
    const int64_t stride = static_cast<int64_t>(p.T) * p.E;
    float val[NPL];
#pragma unroll
    for (int s = 0; s < NPL; ++s) {
        const int e = lane + 64 * s;
        val[s] = __builtin_nanf("");
        if (e >= p.E) continue;
        const float* q = part + static_cast<int64_t>(t) * p.E + e;
        float v = 0.0f;
        for (int s0 = 0; s0 < HS; s0 += 8) {   // eight slices' loads in flight at a time
            float b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = s0 + j < HS ? q[(s0 + j) * stride] : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s0 + j < HS) v = s0 + j == 0 ? b[j] : v + b[j];
        }
        logits[static_cast<int64_t>(t) * p.E + e] = v;
        val[s] = v;
    }
    score_token<NPL>(p, t, val, lds[wave]);
}

// Reductions over the 16 lanes of a row (every lane gets the result).
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, dpp_u32<DPP_QUAD_1032>(v));
    v = max(v, dpp_u32<DPP_QUAD_2301>(v));
    v = max(v, dpp_u32<DPP_ROW_HALF_MIRROR>(v));
    return max(v, dpp_u32<DPP_ROW_MIRROR>(v));
}
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(dpp_u32<DPP_QUAD_1032>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<DPP_QUAD_2301>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<DPP_ROW_HALF_MIRROR>(__float_as_uint(v)));
    return v + __uint_as_float(dpp_u32<DPP_ROW_MIRROR>(__float_as_uint(v)));
}

// Many tokens: four to a wave, 16 lanes each, lane r with experts r + 16 s.  The
// same steps on rows; one instruction serves four tokens, at the price of longer
// rounds (a lane looks through 4 times the experts), so it is for launches that
// fill the chip: by logits from 4096 tokens on (E = 128, k = 8: 4096 tokens 5.1 us
// either way, 8192 7.4 -> 5.7, 65536 39.4 -> 22.0), with 32-bit scores from 6144
// + 48 E on (E = 64: 8192 8.2 and 8.0, 12288 10.4 -> 8.4; E = 128: 8192 9.1 against
// 11.3, 16384 15.3 -> 13.2, 65536 49.1 -> 31.5; E = 256: 16384 25.4 against 26.1,
// 32768 44.1 -> 37.6).
// A token that is not settled in 32 bits is left to score_token.
// E <= 256, at most 16 groups, k <= 15.
template <int VPL>
struct RowLds {
    float c[4][16 * VPL];
    uint32_t g[4][16];
};
constexpr int ROW_T_LOGITS = 4096, ROW_T_SCORES = 6144, ROW_T_SCORES_E = 48;
constexpr int ROW_E_MAX = 256, ROW_G_MAX = 16, ROW_K_MAX = 15;

// PACKED, for bf16 logits whose order decides: the 16 bits of an order image and the
// complement of the expert's id make one key, so a round has no ids to look for (T =
// 16383, E = 160: 10.5 -> 8.7 us; T = 16384, E = 256 15.7 -> 12.4).
template <int VPL, bool PACKED>
__global__ __launch_bounds__(256) void route_score_row_kernel(ScoreRouteParams p) {
    constexpr int NPL = (VPL + 3) / 4;
    __shared__ union Lds {
        RowLds<VPL> row;
        ScoreLds<NPL> one;
    } lds[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane >> 4, r = lane & 15;
    const int t0 = (blockIdx.x * 4 + wave) * 4;
    if (t0 >= p.T) return;   // wave-uniform; the kernel has no workgroup barrier
    const bool live = t0 + row < p.T;
    const int t = live ? t0 + row : p.T - 1;
    const int E = p.E, G = p.n_group, size = E / G, k = p.k;
    const bool grouped = p.topk_group < G, by_logit = PACKED || by_logits(p);
    const float inv_size = 1.0f / static_cast<float>(size);
    RowLds<VPL>& L = lds[wave].row;
    float val[VPL], c[VPL], err = 0.0f;
#pragma unroll
    for (int s = 0; s < VPL; ++s) val[s] = r + 16 * s < E ? load_logit(p, t, r + 16 * s) : __builtin_nanf("");
    float m = 0.0f;
    if (!p.sigmoid) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < VPL; ++s) top = max(top, logit_ord(val[s]));
        top = row_max(top);
        m = top <= 1u ? __builtin_nanf("") : ord_value(top);
    }
    if (by_logit) {
#pragma unroll
        for (int s = 0; s < VPL; ++s) c[s] = val[s];
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int s = 0; s < VPL; ++s) {
            c[s] = score32(val[s], m, p.sigmoid);
            sum += c[s];
        }
        sum = row_sum(sum);
        const float inv = p.sigmoid ? 1.0f : (sum > 0.0f ? 1.0f / sum : 0.0f);
        err = score_err(p.sigmoid, inv);
#pragma unroll
        for (int s = 0; s < VPL; ++s) {
            c[s] *= inv;
            if (p.bias != nullptr && r + 16 * s < E) c[s] += p.bias[r + 16 * s];
            if (!(val[s] == val[s])) c[s] = __builtin_nanf("");
        }
    }
    bool sure = true;
    const bool plain = PACKED || p.bias == nullptr;
    uint32_t key[VPL];
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
        key[s] = logit_ord(plain ? val[s] : c[s]);
        if (PACKED) key[s] = (key[s] & 0xFFFF0000u) | (0xFFFFu - (r + 16 * s));   // (a NaN keeps its id: above 0, below every number)
        if (r + 16 * s >= E) key[s] = 0u;
    }
    if (grouped) {
#pragma unroll
        for (int s = 0; s < VPL; ++s) L.c[row][r + 16 * s] = c[s] == c[s] ? c[s] : -__builtin_inff();
        lds_wave_sync();
        int lg = 0;   // log2 of the lanes per group
        while ((2 << lg) * G <= 16) ++lg;
        const int P = 1 << lg, g = r >> lg, sub = r & (P - 1);
        float m1 = -__builtin_inff(), m2 = -__builtin_inff();
        if (g < G)
            for (int i = sub; i < size; i += P) {
                const float v = L.c[row][g * size + i];
                m2 = fmaxf(m2, fminf(m1, v));
                m1 = fmaxf(m1, v);
            }
        for (int d = 1; d < P; d <<= 1) {
            const float o1 = __shfl_xor(m1, d, 64), o2 = __shfl_xor(m2, d, 64);
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        }
        if (g < G && sub == 0) L.g[row][g] = logit_ord(p.top2 && size > 1 ? m1 + m2 : m1);
        lds_wave_sync();
        const uint32_t mine = L.g[row][r < G ? r : 0];
        int before = 0;
        for (int q = 0; q < G; ++q) {
            const uint32_t o = L.g[row][q];
            before += (o > mine || (o == mine && q < r)) ? 1 : 0;
        }
        const bool in = r < G && before < p.topk_group;
        const uint32_t kept = static_cast<uint32_t>(__ballot(in) >> (16 * row)) & 0xFFFFu;
        if (!by_logit) {
            const uint32_t lo = ~row_max(in ? ~mine : 0u), hi = row_max(r < G && !in ? mine : 0u);
            float two = err;
            if (p.top2) {
                float cmax = 0.0f;
#pragma unroll
                for (int s = 0; s < VPL; ++s) cmax = fmaxf(cmax, finite_size(c[s]));
                two = 2.0f * err + 4.0f * SU * __uint_as_float(row_max(__float_as_uint(cmax)));
            }
            sure = settled(ord_value(lo), ord_value(hi), two);
        }
#pragma unroll
        for (int s = 0; s < VPL; ++s)
            if (!((kept >> (group_of(r + 16 * s, inv_size) & 31)) & 1u)) key[s] = 0u;
    }
    int my_id = 0;
    uint32_t my_key = 0;
    const int rounds = plain ? k : k + 1;
    for (int j = 0; j < rounds; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int s = 1; s < VPL; ++s) best = max(best, key[s]);
        best = row_max(best);
        uint32_t e;
        if (PACKED) {
            e = 0xFFFFu - (best & 0xFFFFu);
#pragma unroll
            for (int s = 0; s < VPL; ++s) key[s] = key[s] == best ? 0u : key[s];
        } else {
            e = 0xFFFFu;
#pragma unroll
            for (int s = VPL - 1; s >= 0; --s) e = key[s] == best ? static_cast<uint32_t>(r + 16 * s) : e;
            e = ~row_max(~e);   // the lowest id of the row that holds the maximum
            const int d = static_cast<int>(e) - r;
#pragma unroll
            for (int s = 0; s < VPL; ++s)
                if (d == 16 * s) key[s] = 0u;
        }
        if (r == j) {
            my_id = static_cast<int>(e);
            my_key = best;
        }
    }
    if (!plain) {
        const uint32_t next = __shfl_down(my_key, 1, 64);
        if (r < k && next != 0u) sure = sure && settled(ord_value(my_key), ord_value(next), err);
    }
    const uint64_t unsure = __ballot(live && !sure);
    // weights, lane r < k
    const float ml = r < k ? load_logit(p, t, my_id) : 0.0f;
    double w = r < k ? score64(ml, m, p.sigmoid) : 0.0;
    double sum = 1.0;
    if (p.renorm) {
        sum = row_sum(w);
    } else if (!p.sigmoid) {
        sum = 0.0;
#pragma unroll
        for (int s = 0; s < VPL; ++s) sum += score64(val[s], m, 0);
        sum = row_sum(sum);
    }
    w = sum > 0.0 ? w / sum : 0.0;
    if (live && r < k && ((unsure >> (16 * row)) & 0xFFFFull) == 0ull) {
        p.ids[static_cast<int64_t>(t) * k + r] = my_id;
        p.w[static_cast<int64_t>(t) * k + r] = static_cast<float>(w * static_cast<double>(p.scale));
    }
    for (int q = 0; q < 4; ++q) {
        if (((unsure >> (16 * q)) & 0xFFFFull) == 0ull) continue;   // wave-uniform
        lds_wave_sync();
        score_token<NPL>(p, t0 + q, lds[wave].one);
    }
}

template <bool PACKED>
static auto row_kernel(int E) {
    return E <= 64 ? route_score_row_kernel<4, PACKED>
                   : E <= 96 ? route_score_row_kernel<6, PACKED>
                   : E <= 128 ? route_score_row_kernel<8, PACKED>
                   : E <= 160 ? route_score_row_kernel<10, PACKED>
                   : E <= 192 ? route_score_row_kernel<12, PACKED>
                   : E <= 224 ? route_score_row_kernel<14, PACKED> : route_score_row_kernel<16, PACKED>;
}

hipError_t launch_route_score(const ScoreRouteParams& p, hipStream_t s) {
    const dim3 block(256);
    if (p.T >= (by_logits(p) ? ROW_T_LOGITS : ROW_T_SCORES + ROW_T_SCORES_E * p.E) && p.E <= ROW_E_MAX && p.n_group <= ROW_G_MAX && p.k <= ROW_K_MAX) {
        const dim3 grid((p.T + 15) / 16);
        const bool packed = by_logits(p) && p.logits_dt == BF16;
        // a width for every 32 experts: two idle experts a lane cost 5 to 13 %
        // (T = 65536: E = 96 in 8 a lane 15.3, in 6 13.5 us; 160 in 12 21.0, in 10 19.3;
        // 224 in 16 28.0, in 14 25.0; T = 16384: 5.5 and 5.0, 6.9 and 6.4, 9.3 and 8.8)
        auto kn = packed ? row_kernel<true>(p.E) : row_kernel<false>(p.E);
        hipLaunchKernelGGL(kn, grid, block, 0, s, p);
        return hipGetLastError();
    }
    const dim3 grid((p.T + 3) / 4);
    auto kn = p.E <= 64 ? route_score_kernel<1>
                        : p.E <= 128 ? route_score_kernel<2>
                                     : p.E <= 192 ? route_score_kernel<3>
                                                  : p.E <= 256 ? route_score_kernel<4>
                                                               : p.E <= 384 ? route_score_kernel<6> : route_score_kernel<8>;
    hipLaunchKernelGGL(kn, grid, block, 0, s, p);
    return hipGetLastError();
}

hipError_t launch_router_score(const void* x, bool xf32, const float* wr, int H, float* logits, float* part,
                               const ScoreRouteParams& p, hipStream_t s) {
    int HS = 0;
    const hipError_t e = launch_router_part(x, xf32, wr, p.T, H, p.E, part, &HS, s);
    if (e != hipSuccess) return e;
    auto kn = p.E <= 64 ? route_score_part_kernel<1>
                        : p.E <= 128 ? route_score_part_kernel<2>
                                     : p.E <= 192 ? route_score_part_kernel<3>
                                                  : p.E <= 256 ? route_score_part_kernel<4>
                                                               : p.E <= 384 ? route_score_part_kernel<6> : route_score_part_kernel<8>;
    hipLaunchKernelGGL(kn, dim3((p.T + 3) / 4), dim3(256), 0, s, p, part, HS, logits);
    return hipGetLastError();
}

}  // namespace moe
