// Scored router: expert choice by softmax or sigmoid scores, a selection bias,
// expert groups and top-k, and the grouping of its pairs by expert.
//
// For token t, with x the logits and b the bias:
//   p_e = 1 / (1 + exp(-x_e)) or softmax(x)_e;  c_e = p_e + b_e (the order of
//   x without a bias);  group g = E / n_group consecutive experts, G_g = the
//   sum of its group_top (1 or 2) largest c;  candidates: the topk_group
//   groups with the largest G;  ids: the k largest c among them, descending,
//   ties to the lower index;  w_j = p_j (/ sum p) * scale.
// Masked experts (logit NaN or at most its type's lowest value, bias NaN or at
// most -FLT_MAX) rank after every other, by index, and get weight 0.
//
// One warp per token, lane l holding experts l + 32 i.  Bound: integer and
// compare instructions (8192 x 256 logits are 8 MB, 1.3 us of HBM), so the
// selection avoids a warp-wide argmax per winner: the k-th largest of the 32
// lane maxima bounds the k-th largest value from below, few more than k values
// reach that bound (9 for k = 8), and those, one per lane, find their rank by
// comparing with one another.
//
// The choice is that of 64-bit values at 32-bit speed: c is computed in fp32
// with a bounded error (score_tol).  Where two of the candidates lie closer
// than the bound, the candidates' scores are computed again in 64 bits, where the
// border between chosen and dropped groups is that close, the groups'; where
// there are more candidates than places (many equal values) or fewer unmasked
// experts than k, the whole token is decided in 64 bits.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "ptx_cluster.cuh"

namespace moe {

namespace {

constexpr float kFltMax = 3.402823466e38f;
constexpr float kBf16Lowest = -3.38953138925153547590e38f;
constexpr int kNone = 0x7fffffff;

__device__ __forceinline__ float ld_logit(const float* l, int e) { return l[e]; }
__device__ __forceinline__ float ld_logit(const __nv_bfloat16* l, int e) {
    return __bfloat162float(l[e]);
}
__device__ __forceinline__ bool logit_masked(const float*, float x) { return !(x > -kFltMax); }
__device__ __forceinline__ bool logit_masked(const __nv_bfloat16*, float x) {
    return !(x > kBf16Lowest);
}

// Order-preserving map of floats to unsigned integers above 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// Bound on |difference of two fp32 selection values - the exact difference|,
// v being one of them.  __expf is off by (2 + 1.173 |z|) ulps at argument z,
// rcp.approx by one.
//  sigmoid + b: p (1 - p) (2 + 1.173 |x|) + 1.5 ulps <= 1.1 * 2^-22 a score and
//    one rounding of the sum; group values hold two scores: 2^-19 + 2^-21 |v|.
//  softmax + b: p (2 + 1.7 d) e^-d ulps of the exponential, 24 ulps of a 37-term
//    sum of such terms, and all p together are 1: 2^-17, the same relative part.
//  no bias (group values, sums of scores): relative, with arguments up to 88
//    (2 + 1.7 * 88) 2^-23 a side, 2^-14; below 1e-36 scores lose bits to
//    underflow.
// Half of it bounds one value's own error.  A group's value t1 + t2 is off by
// its terms' roundings, so v is |t1| + |t2| there: with biases of 1e4 and -1e4
// that is 2e4, and the sum about 1.
__device__ __forceinline__ float score_tol(const ScoreArgs& a, float v) {
    const float m = fabsf(v);
    if (!a.bias) return 6.103515625e-05f * m + 1e-36f;
    return (a.sigmoid ? 1.9073486328125e-06f : 7.62939453125e-06f) + 4.76837158203125e-07f * m;
}

__device__ __forceinline__ bool bias_masked(const ScoreArgs& a, int e) {
    return a.bias && !(a.bias[e] > -kFltMax);
}

// exp(x - big) (softmax), or sigmoid(x) / exp(big) (big <= 0, and 0 where x > 0).
__device__ __forceinline__ float score_over(const ScoreArgs& a, float x, float big) {
    if (!a.sigmoid) return expf(x - big);
    return (x > 0.0f ? 1.0f : expf(x - big)) * rcp_approx(1.0f + expf(-fabsf(x)));
}

// Largest unmasked logit and sum of exp(x - largest) in 64 bits, for softmax.
template <typename LT>
__device__ __forceinline__ void softmax_f64(const ScoreArgs& a, const LT* l, double& mx, double& z) {
    mx = -__longlong_as_double(0x7ff0000000000000ll);
    z = 0.0;
    const int lane = threadIdx.x & 31;
    for (int e = lane; e < a.E; e += 32) {
        const float x = ld_logit(l, e);
        if (!logit_masked(l, x) && !bias_masked(a, e)) mx = fmax(mx, static_cast<double>(fminf(x, kFltMax)));
    }
    for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    for (int e = lane; e < a.E; e += 32) {
        const float x = ld_logit(l, e);
        if (!logit_masked(l, x) && !bias_masked(a, e)) z += exp(static_cast<double>(fminf(x, kFltMax)) - mx);
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
}

__device__ __forceinline__ double score_f64(const ScoreArgs& a, double x, double mx, double z) {
    return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - mx) / z;
}

// The whole choice with 64-bit scores; lane j < k returns the j-th expert.
template <int PER, typename LT>
__device__ __noinline__ int choose_f64(const ScoreArgs& a, const LT* l) {
    const int lane = threadIdx.x & 31;
    const int gs = a.E / a.n_group;
    const double none = -__longlong_as_double(0x7ff0000000000000ll);
    double mx = 0.0, z = 1.0;
    if (!a.sigmoid) softmax_f64(a, l, mx, z);
    // c: value the experts are ordered by; p: value that group sums add up
    double c[PER], p[PER];
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        c[i] = p[i] = none;
        if (e >= a.E) continue;
        float x = ld_logit(l, e);
        if (logit_masked(l, x) || bias_masked(a, e)) continue;
        x = fminf(x, kFltMax);
        const double s = score_f64(a, x, mx, z);
        c[i] = a.bias ? s + static_cast<double>(fminf(a.bias[e], kFltMax)) : static_cast<double>(x);
        p[i] = a.bias || a.group_top == 1 ? c[i] : s;
    }
    uint32_t groups = 1u;
    if (a.n_group > 1) {
        double mine = none;  // lane g: group g's value
        for (int g = 0; g < a.n_group; ++g) {
            double t1 = none, t2 = none;
            for (int i = 0; i < PER; ++i) {
                const int e = lane + 32 * i;
                if (e < g * gs || e >= (g + 1) * gs) continue;
                t2 = fmax(t2, fmin(t1, p[i]));
                t1 = fmax(t1, p[i]);
            }
            for (int o = 16; o > 0; o >>= 1) {
                const double u1 = __shfl_xor_sync(0xffffffffu, t1, o);
                const double u2 = __shfl_xor_sync(0xffffffffu, t2, o);
                t2 = fmax(fmin(t1, u1), fmax(t2, u2));
                t1 = fmax(t1, u1);
            }
            const double v = a.group_top == 2 && t2 != none ? t1 + t2 : t1;
            if (lane == g) mine = v;
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const double v = __shfl_sync(0xffffffffu, mine, g);
            rank += v > mine || (v == mine && g < lane) ? 1 : 0;
        }
        groups = __ballot_sync(0xffffffffu, lane < a.n_group && rank < a.topk_group);
    }
    uint32_t gone = 0;
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.E || !((groups >> (e / gs)) & 1u)) gone |= 1u << i;
    }
    int chosen = 0;
    for (int j = 0; j < a.k; ++j) {
        double bv = none;
        int be = kNone;
        for (int i = 0; i < PER; ++i) {
            if ((gone >> i) & 1u) continue;
            if (be == kNone || c[i] > bv) {
                bv = c[i];
                be = lane + 32 * i;
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (oe != kNone && (be == kNone || ov > bv || (ov == bv && oe < be))) {
                bv = ov;
                be = oe;
            }
        }
        if (lane == (be & 31)) gone |= 1u << (be >> 5);
        if (lane == j) chosen = be;
    }
    return chosen;
}

// Log2 of the lanes that scan a group together.
__device__ __forceinline__ int group_lanes_log2(int n_group) {
    return n_group > 16 ? 0 : n_group > 8 ? 1 : n_group > 4 ? 2 : n_group > 2 ? 3 : 4;
}

// Group values and ranks from the E selection values in scratch (-inf where
// masked): lane's group is lane >> lp; gv its value, size the sum of its terms'
// magnitudes (-1 where every expert is masked), returns its rank.
template <typename T>
__device__ __forceinline__ int rank_groups(const ScoreArgs& a, const T* scratch, T& gv, T& size) {
    const int lane = threadIdx.x & 31;
    const int lp = group_lanes_log2(a.n_group), gs = a.E / a.n_group;
    const int grp = lane >> lp;
    const T ninf = -static_cast<T>(INFINITY);
    T t1 = ninf, t2 = ninf;
    if (grp < a.n_group)
        for (int i = lane & ((1 << lp) - 1); i < gs; i += 1 << lp) {
            const T f = scratch[grp * gs + i];
            t2 = max(t2, min(t1, f));
            t1 = max(t1, f);
        }
    for (int o = (1 << lp) >> 1; o > 0; o >>= 1) {
        const T u1 = __shfl_xor_sync(0xffffffffu, t1, o);
        const T u2 = __shfl_xor_sync(0xffffffffu, t2, o);
        t2 = max(min(t1, u1), max(t2, u2));
        t1 = max(t1, u1);
    }
    const bool two = a.group_top == 2 && t2 > ninf;
    gv = two ? t1 + t2 : t1;
    size = !(t1 > ninf) ? static_cast<T>(-1) : two ? abs(t1) + abs(t2) : abs(t1);
    int rank = 0;
    for (int o = 0; o < a.n_group; ++o) {
        const T ov = __shfl_sync(0xffffffffu, gv, o << lp);
        rank += ov > gv || (ov == gv && o < grp) ? 1 : 0;
    }
    return rank;
}

// Lanes whose group is chosen, by 64-bit values; scratch: E doubles.
template <typename LT>
__device__ __noinline__ uint32_t choose_groups_f64(const ScoreArgs& a, const LT* l, double* scratch) {
    const int lane = threadIdx.x & 31;
    double mx = 0.0, z = 1.0;
    if (!a.sigmoid) softmax_f64(a, l, mx, z);
    __syncwarp();
    for (int e = lane; e < a.E; e += 32) {
        const float x = ld_logit(l, e);
        double s = -static_cast<double>(INFINITY);
        if (!logit_masked(l, x) && !bias_masked(a, e)) {
            s = score_f64(a, fminf(x, kFltMax), mx, z);
            if (a.bias) s += static_cast<double>(fminf(a.bias[e], kFltMax));
        }
        scratch[e] = s;
    }
    __syncwarp();
    double gv, size;
    const int rank = rank_groups(a, scratch, gv, size);
    const int grp = lane >> group_lanes_log2(a.n_group);
    return __ballot_sync(0xffffffffu, grp < a.n_group && rank < a.topk_group);
}

// Ranks of the m candidates in scratch (their experts ascending at ids[]) by
// 64-bit values, lane l's candidates being l and l + 32.
template <int CPL, typename LT>
__device__ __noinline__ void rank_f64(const ScoreArgs& a, const LT* l, const int* ids, int m, double* c,
                                      int (&rank)[CPL]) {
    const int lane = threadIdx.x & 31;
    double mx = 0.0, z = 1.0;
    if (!a.sigmoid) softmax_f64(a, l, mx, z);
    for (int q = 0; q < CPL; ++q)
        if (lane + 32 * q < m) {
            const int e = ids[lane + 32 * q];
            const float x = fminf(ld_logit(l, e), kFltMax);
            c[lane + 32 * q] =
                score_f64(a, x, mx, z) + static_cast<double>(fminf(a.bias[e], kFltMax));
        }
    __syncwarp();
    for (int q = 0; q < CPL; ++q) {
        rank[q] = 0;
        const int i = lane + 32 * q;
        const double mine = i < m ? c[i] : 0.0;
        for (int j = 0; j < m; ++j) rank[q] += c[j] > mine || (c[j] == mine && j < i) ? 1 : 0;
    }
}

// Scratch of a warp: the group scan's E values (fp32, or 64-bit where they are
// close), then the candidates' values, experts and 64-bit values.
template <int CPL>
__host__ __device__ constexpr int scratch_floats(int E, bool groups) {
    return groups && 2 * E > 4 * 32 * CPL ? (2 * E + 3) & ~3 : 4 * 32 * CPL;   // 16-byte aligned
}

// One token by one warp.  CPL: places for candidates a lane, and lane maxima
// that bound them.  The candidates are as many as it takes to meet k of the 32
// CPL maxima: 15 of 32 places for k = 12, 22 for 16 (one token in 200 has more
// than 32 and is decided in 64 bits: 4096 x 1024 top-16 took 49 us, with two
// places a lane 18), 44 of 64 for k = 32.
template <int PER, int CPL, typename LT>
__device__ __forceinline__ void score_token(const ScoreArgs& a, int t, float* scratch) {
    const int lane = threadIdx.x & 31;
    const LT* l = static_cast<const LT*>(a.logits) + static_cast<long long>(t) * a.E;
    const bool sums = a.n_group > 1 && a.group_top == 2;   // group values add scores up
    const bool need_score = a.bias != nullptr || sums;
    const bool need_z = !a.sigmoid && (need_score || !a.renorm);
    const float ninf = -INFINITY;
    // v: logits, then selection values; -inf where masked or no expert
    float v[PER], g[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < a.E ? ld_logit(l, e) : ninf;
        g[i] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool m = logit_masked(l, v[i]) || !(g[i] > -kFltMax);
        v[i] = m ? ninf : fminf(v[i], kFltMax);
    }
    float mx = 0.0f, zinv = 0.0f;
    if (need_z) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = fmaxf(m, v[i]);
        mx = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
        if (mx == ninf) mx = 0.0f;   // nothing unmasked: every term below is 0
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) z += __expf(v[i] - mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        zinv = z > 0.0f ? __frcp_rn(z) : 0.0f;
    }
    if (need_score) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool live = v[i] > ninf;
            const float s = a.sigmoid ? rcp_approx(1.0f + __expf(-v[i])) : __expf(v[i] - mx) * zinv;
            if (a.bias) {
                v[i] = live ? s + fminf(g[i], kFltMax) : ninf;
                g[i] = v[i];
            } else {
                g[i] = live ? s : ninf;
            }
        }
    }
    if (a.n_group > 1) {
        const int gs = a.E / a.n_group;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < a.E) scratch[lane + 32 * i] = need_score ? g[i] : v[i];
        __syncwarp();
        // the lanes of a group (2^lp of them, 2^lp * n_group <= 32) scan it together
        const int lp = group_lanes_log2(a.n_group), grp = lane >> lp;
        float gv, size;
        const int rank = rank_groups(a, scratch, gv, size);
        const bool in = grp < a.n_group && rank < a.topk_group;
        uint32_t lanes_in = __ballot_sync(0xffffffffu, in);
        if (need_score && a.topk_group < a.n_group) {
            // every chosen group's least possible value above every other's largest?
            // (two biases near -FLT_MAX add up to -infinity: such a group is none of
            // masked experts, and only its 64-bit value tells its place)
            const bool live = grp < a.n_group && size >= 0.0f;
            const bool finite = size <= kFltMax;
            const float err = 0.5f * score_tol(a, size);
            const float least = finite ? gv - err : ninf, most = finite ? gv + err : -ninf;
            const uint32_t lo = __reduce_min_sync(0xffffffffu, in && live ? order_key(least) : 0xffffffffu);
            const uint32_t hi = __reduce_max_sync(0xffffffffu, !in && live ? order_key(most) : 0u);
            if (hi != 0u && (lo == 0xffffffffu || !(key_value(lo) > key_value(hi))))
                lanes_in = choose_groups_f64(a, l, reinterpret_cast<double*>(scratch));
        }
        // e / gs = e * inv_gs >> 20 for e, gs <= 1024
        const uint32_t inv_gs = ((1u << 20) + gs - 1) / gs;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((lanes_in >> (((e * inv_gs) >> 20) << lp)) & 1u)) v[i] = ninf;
        }
        __syncwarp();
    }
    // the k-th largest of the lanes' maxima (CPL of each lane)
    float top[CPL];
#pragma unroll
    for (int q = 0; q < CPL; ++q) {
        top[q] = v[q * (PER / CPL)];
#pragma unroll
        for (int i = 1; i < PER / CPL; ++i) top[q] = fmaxf(top[q], v[q * (PER / CPL) + i]);
    }
    uint32_t cur[CPL], kth;
#pragma unroll
    for (int q = 0; q < CPL; ++q) cur[q] = top[q] > ninf ? order_key(top[q]) : 0u;
    int seen = 0;
    do {
        uint32_t m = cur[0];
        if constexpr (CPL == 2) m = max(m, cur[1]);
        kth = __reduce_max_sync(0xffffffffu, m);
#pragma unroll
        for (int q = 0; q < CPL; ++q) {
            const bool eq = cur[q] == kth;
            seen += __popc(__ballot_sync(0xffffffffu, eq));
            if (eq) cur[q] = 0u;
        }
    } while (seen < a.k && kth != 0u);
    float bound = kth != 0u ? key_value(kth) : ninf;
    if (a.bias && kth != 0u) bound -= score_tol(a, bound);
    // candidates, in ascending expert order
    float* cv = scratch;
    int* ce = reinterpret_cast<int*>(scratch) + 32 * CPL;
    int m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool pass = v[i] >= bound && v[i] > ninf;
        const uint32_t who = __ballot_sync(0xffffffffu, pass);
        if (who) {
            const int at = m + __popc(who & ((1u << lane) - 1u));
            if (pass && at < 32 * CPL) {
                cv[at] = v[i];
                ce[at] = lane + 32 * i;
            }
            m += __popc(who);
        }
    }
    // more candidates than places; or fewer unmasked experts than k (the lanes
    // then run out before k are seen, and every unmasked expert is a candidate)
    const bool whole = m > 32 * CPL || m < a.k;   // decide the whole token in 64 bits
    int expert[CPL], rank[CPL];
    if (!whole) {
#pragma unroll
        for (int q = 0; q < CPL; ++q)
            if (lane + 32 * q >= m) cv[lane + 32 * q] = ninf;
        __syncwarp();
        float mine[CPL];
#pragma unroll
        for (int q = 0; q < CPL; ++q) {
            const int i = lane + 32 * q;
            mine[q] = cv[i];
            expert[q] = i < m ? ce[i] : 0;
            rank[q] = 0;
        }
        for (int j = 0; j < m; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(cv + j);
#pragma unroll
            for (int q = 0; q < CPL; ++q)
                rank[q] += (f.x > mine[q] ? 1 : 0) + (f.y > mine[q] ? 1 : 0) + (f.z > mine[q] ? 1 : 0) +
                           (f.w > mine[q] ? 1 : 0);
        }
        // neighbours in the order: equal values share a rank and leave a hole
        // (NaN) behind it
        float* sorted = scratch + 2 * 32 * CPL;
#pragma unroll
        for (int q = 0; q < CPL; ++q) sorted[lane + 32 * q] = __int_as_float(0x7fffffff);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < CPL; ++q)
            if (lane + 32 * q < m) sorted[rank[q]] = mine[q];
        __syncwarp();
        bool close = false;
#pragma unroll
        for (int q = 0; q < CPL; ++q)
            if (lane + 32 * q < m && rank[q] + 1 < m)
                close |= !(mine[q] - sorted[rank[q] + 1] > (a.bias ? score_tol(a, mine[q]) : 0.0f));
        if (__any_sync(0xffffffffu, close)) {
            if (a.bias) {
                rank_f64<CPL, LT>(a, l, ce, m, reinterpret_cast<double*>(sorted), rank);
            } else {
                // equal logits: by position, which is expert order
                for (int j = 0; j < m; ++j) {
                    const float o = cv[j];
#pragma unroll
                    for (int q = 0; q < CPL; ++q) rank[q] += o == mine[q] && j < lane + 32 * q ? 1 : 0;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < CPL; ++q)
            if (lane + 32 * q >= m) rank[q] = kNone;
    } else {
        expert[0] = choose_f64<PER, LT>(a, l);
        rank[0] = lane;
        if constexpr (CPL == 2) rank[1] = kNone;
    }
    __syncwarp();   // the scratch is free for the warp's next token
    // weights of the k winners
    float x[CPL], u[CPL];
    bool on[CPL];
#pragma unroll
    for (int q = 0; q < CPL; ++q) {
        on[q] = false;
        x[q] = 0.0f;
        if (rank[q] < a.k) {
            x[q] = ld_logit(l, expert[q]);
            on[q] = !logit_masked(l, x[q]) && !bias_masked(a, expert[q]);
            x[q] = fminf(x[q], kFltMax);
        }
    }
    if (a.renorm) {
        // scaled by the largest so that no row of small scores underflows
        uint32_t xk = 0u;
#pragma unroll
        for (int q = 0; q < CPL; ++q) xk = max(xk, on[q] ? order_key(x[q]) : 0u);
        xk = __reduce_max_sync(0xffffffffu, xk);
        float big = xk ? key_value(xk) : 0.0f;
        if (a.sigmoid) big = fminf(big, 0.0f);
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < CPL; ++q) {
            u[q] = on[q] ? score_over(a, x[q], big) : 0.0f;
            sum += u[q];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum > 0.0f ? __frcp_rn(sum) : 0.0f;
#pragma unroll
        for (int q = 0; q < CPL; ++q) u[q] *= inv;
    } else {
#pragma unroll
        for (int q = 0; q < CPL; ++q)
            u[q] = !on[q] ? 0.0f : a.sigmoid ? score_over(a, x[q], 0.0f) : expf(x[q] - mx) * zinv;
    }
#pragma unroll
    for (int q = 0; q < CPL; ++q)
        if (rank[q] < a.k) {
            const long long at = static_cast<long long>(t) * a.k + rank[q];
            a.ids[at] = expert[q];
            a.w[at] = u[q] * a.scale;
        }
}

constexpr int kScoreWarps = 4;

template <int PER, int CPL, typename LT>
__global__ void __launch_bounds__(32 * kScoreWarps, PER <= 16 ? 7 : 6) score_kernel(const ScoreArgs a) {
    extern __shared__ __align__(16) float scratch[];
    const int warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kScoreWarps + warp;
    pdl_launch();
    pdl_wait();
    if (t >= a.T) return;
    score_token<PER, CPL, LT>(a, t, scratch + warp * scratch_floats<CPL>(a.E, a.n_group > 1));
}

// ------------------------------------------------------------ grouping
// Stable grouping of n consecutive pairs by expert in one CTA of NW warps.
// Each warp owns a segment of the pairs and ranks each pair among the earlier
// ones of its segment (one ballot per expert-id bit gives the lanes with the
// same expert); a thread per expert then scans the segments' counts.
//   cnt   shared [NW][E], zeroed
//   base  shared [E]: first output row of each expert
template <int NW, int STEPS>   // warps, most 32-pair steps of a segment
struct Segment {
    int p0, n;                 // this warp's pairs: p0 + [0, n)
    int e[STEPS], r[STEPS];    // each pair's expert and its rank in the segment
};

template <int NW, int kSteps>
__device__ __forceinline__ void count_pairs(Segment<NW, kSteps>& s, const int32_t* ids, int first, int n, int E,
                                            int nbits, int* cnt) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = ((n + NW - 1) / NW + 31) & ~31;
    s.p0 = first + min(n, warp * per);
    s.n = min(per, n - min(n, warp * per));
    int* c = cnt + warp * E;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int p = i * 32 + lane;
        s.e[i] = p < s.n ? __ldcg(ids + s.p0 + p) : -1;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (i * 32 >= s.n) break;
        const bool ok = s.e[i] >= 0;
        unsigned peers = __ballot_sync(0xffffffffu, ok);
        for (int b = 0; b < nbits; ++b) {
            const bool bit = (s.e[i] >> b) & 1;
            const unsigned bb = __ballot_sync(0xffffffffu, bit);
            peers &= bit ? bb : ~bb;
        }
        const int before = ok ? c[s.e[i]] : 0;
        s.r[i] = before + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (ok && (peers & ((1u << lane) - 1u)) == 0) c[s.e[i]] = before + __popc(peers);
        __syncwarp();
    }
}

template <int NW, int kSteps>
__device__ __forceinline__ void place_pairs(const Segment<NW, kSteps>& s, int E, const int* cnt, const int* base,
                                            int32_t* perm, int32_t* inv_perm) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int p = i * 32 + lane;
        if (p < s.n) {
            const int row = base[s.e[i]] + cnt[warp * E + s.e[i]] + s.r[i];
            perm[row] = s.p0 + p;
            if (inv_perm) inv_perm[s.p0 + p] = row;
        }
    }
}

// Exclusive scan over the CTA's threads (NW warps) of one value each.
template <int NW>
__device__ __forceinline__ int cta_exclusive(int v, int* warp_tot) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < NW; ++w) before += w < warp ? warp_tot[w] : 0;
    return before + incl - v;
}

__host__ __device__ inline int bits_of(int E) {
    int n = 0;
    while ((1 << n) < E) ++n;
    return n;
}

// Few tokens: the scored router over a cluster of 8 CTAs (a warp per token for
// up to 128 tokens), then the grouping in the cluster's first CTA.  One launch;
// one CTA alone would issue 64 tokens' selection in ~6 us.
constexpr int kSmallWarps = 16;
constexpr int kSmallCluster = 8;
constexpr int kSmallTokens = 128;
constexpr int kSmallSteps = kSmallTokens * 32 / (kSmallWarps * 32);   // steps of 32 pairs a warp, k <= 32

template <int PER, int CPL, typename LT>
__global__ void __launch_bounds__(32 * kSmallWarps)
    score_route_small(const ScoreArgs a, int32_t* m_indptr, int32_t* perm, int32_t* inv_perm,
                      int* status, int nbits) {
    extern __shared__ __align__(16) float scratch[];
    __shared__ int warp_tot[kSmallWarps];
    const int warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_ctarank();
    const int sf = scratch_floats<CPL>(a.E, a.n_group > 1);
    int* cnt = reinterpret_cast<int*>(scratch + kSmallWarps * sf);   // [warps][E]
    int* base = cnt + kSmallWarps * a.E;                             // [E]
    pdl_launch();
    pdl_wait();
    if (rank == 0) {
        for (int i = threadIdx.x; i < kSmallWarps * a.E; i += 32 * kSmallWarps) cnt[i] = 0;
        if (threadIdx.x < kStatusInts) status[threadIdx.x] = 0;
    }
    for (int t = rank + kSmallCluster * warp; t < a.T; t += kSmallCluster * kSmallWarps)
        score_token<PER, CPL, LT>(a, t, scratch + warp * sf);
    __syncwarp();
    cluster_sync_all();      // every CTA's ids are visible
    if (rank != 0) return;
    const int R = a.T * a.k;
    Segment<kSmallWarps, kSmallSteps> seg;
    count_pairs(seg, a.ids, 0, R, a.E, nbits, cnt);
    __syncthreads();
    // experts [e0, e1) of this thread: counts of the segments before, totals
    const int ept = (a.E + 32 * kSmallWarps - 1) / (32 * kSmallWarps);
    const int e0 = min(a.E, static_cast<int>(threadIdx.x) * ept), e1 = min(a.E, e0 + ept);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int run = 0, c[kSmallWarps];
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) c[w] = cnt[w * a.E + e];
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) {
            cnt[w * a.E + e] = run;
            run += c[w];
        }
        base[e] = run;
        sum += run;
    }
    int first = cta_exclusive<kSmallWarps>(sum, warp_tot);
    for (int e = e0; e < e1; ++e) {
        const int n = base[e];
        base[e] = first;
        m_indptr[e] = first;
        first += n;
    }
    if (threadIdx.x == 0) m_indptr[a.E] = R;
    __syncthreads();
    place_pairs(seg, a.E, cnt, base, perm, inv_perm);
}

// More tokens: the router alone, then a CTA per chunk of 1024 pairs counts the
// chunk's experts, then one places its pairs.  Up to 16 chunks the placing CTAs
// count all ids themselves, one launch less (T = 1024, k = 8: 4.0 us behind the
// router against 5.8).  From 32768 counts on, a launch between them adds up the
// chunks' counts, since every placing CTA would read them all (E = 256, k = 8,
// launches behind the router: 128 chunks 8.5 us without it, 10.2 with; 256 chunks
// 18.1 against 11.4; 512 chunks 50 against 18).
constexpr int kCountChunks = 16;
constexpr int kSumCounts = 32768;   // counts (chunks x experts, as a power of two) that a placing CTA adds up

__global__ void __launch_bounds__(256) count_kernel(const int32_t* ids, int R, int E, int32_t* chunk_hist,
                                                    int* status) {
    __shared__ int hist[kMaxRouteExperts];
    for (int e = threadIdx.x; e < E; e += 256) hist[e] = 0;
    __syncthreads();
    pdl_launch();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x < kStatusInts) status[threadIdx.x] = 0;
    const int p0 = blockIdx.x * kRouteChunk + threadIdx.x;
    int id[kRouteChunk / 256];
#pragma unroll
    for (int i = 0; i < kRouteChunk / 256; ++i) id[i] = p0 + 256 * i < R ? __ldcg(ids + p0 + 256 * i) : -1;
#pragma unroll
    for (int i = 0; i < kRouteChunk / 256; ++i)
        if (id[i] >= 0) atomicAdd(&hist[id[i]], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256)
        chunk_hist[static_cast<long long>(blockIdx.x) * E + e] = hist[e];
}

// Many chunks: the counts of a chunk become the sums up to and with it.  A CTA per
// 32 experts; its 32 warps take a 32nd of the chunks each, in two passes.
__global__ void __launch_bounds__(1024) scan_kernel(int32_t* chunk_hist, int E, int nchunks) {
    __shared__ int sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = 32 * blockIdx.x + lane;
    const int per = (nchunks + 31) / 32, c0 = min(nchunks, warp * per), c1 = min(nchunks, c0 + per);
    pdl_launch();
    pdl_wait();
    int sum = 0;
    if (e < E)
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += __ldcg(chunk_hist + static_cast<long long>(c) * E + e);
    sums[warp][lane] = sum;
    __syncthreads();
    int run = 0;
    for (int w = 0; w < warp; ++w) run += sums[w][lane];
    if (e >= E) return;
    for (int c = c0; c < c1; c += 8) {
        int h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = c + i < c1 ? __ldcg(chunk_hist + static_cast<long long>(c + i) * E + e) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            run += h[i];
            if (c + i < c1) chunk_hist[static_cast<long long>(c + i) * E + e] = run;
        }
    }
}

// One CTA per chunk adds up the counts of the chunks before it (every CTA for
// itself out of L2, where there are at most kSumCounts in all) and places its
// pairs.  Thread (g, e) of the 1024 reads every G-th row of counts at expert e, so
// that 64 chunks of 256 experts are one round of 16 loads a thread; 32 warps have
// one step of 32 pairs each.
constexpr int kPlaceWarps = 32;

// kCount: without a counting launch before it (few chunks), every CTA counts all R
// ids itself, 8 a thread; the first clears status.  kPrefix: behind scan_kernel,
// two rows hold what is needed.
enum Place { kCount, kSum, kPrefix };
template <Place MODE>
__global__ void __launch_bounds__(32 * kPlaceWarps)
    place_kernel(const int32_t* ids, int R, int E, int nbits, const int32_t* chunk_hist, int32_t* m_indptr,
                 int32_t* perm, int32_t* inv_perm, int* status) {
    extern __shared__ __align__(16) int smem[];
    __shared__ int warp_tot[kPlaceWarps];
    __shared__ int part_total[32 * kPlaceWarps], part_before[32 * kPlaceWarps];
    int* cnt = smem;                       // [warps][E]
    int* base = cnt + kPlaceWarps * E;     // [E]
    const int nchunks = gridDim.x, chunk = blockIdx.x;
    const int e = threadIdx.x & ((1 << nbits) - 1), g = threadIdx.x >> nbits;   // E <= 2^nbits <= 1024
    const int G = MODE != kSum ? 1 : (32 * kPlaceWarps) >> nbits;
    const int first = chunk * kRouteChunk;
    if constexpr (MODE == kCount) {
        part_total[threadIdx.x] = part_before[threadIdx.x] = 0;
        __syncthreads();
    }
    pdl_wait();
    int total = 0, before = 0;
    if constexpr (MODE == kCount) {
        if (chunk == 0 && threadIdx.x < kStatusInts) status[threadIdx.x] = 0;
        for (int p0 = threadIdx.x; p0 < R; p0 += 8 * 32 * kPlaceWarps) {
            int id[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = p0 + i * 32 * kPlaceWarps;
                id[i] = p < R ? __ldcg(ids + p) : -1;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (id[i] >= 0) {
                    atomicAdd(&part_total[id[i]], 1);
                    if (p0 + i * 32 * kPlaceWarps < first) atomicAdd(&part_before[id[i]], 1);
                }
        }
    } else if constexpr (MODE == kPrefix) {
        if (threadIdx.x < E) {
            total = __ldcg(chunk_hist + static_cast<long long>(nchunks - 1) * E + e);
            before = chunk ? __ldcg(chunk_hist + static_cast<long long>(chunk - 1) * E + e) : 0;
        }
        part_total[threadIdx.x] = total;
        part_before[threadIdx.x] = before;
    } else {
        for (int c0 = g; c0 < nchunks; c0 += 16 * G) {
            int h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int c = c0 + i * G;
                h[i] = c < nchunks && e < E ? __ldcg(chunk_hist + static_cast<long long>(c) * E + e) : 0;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (c0 + i * G < chunk) before += h[i];
                total += h[i];
            }
        }
        part_total[threadIdx.x] = total;
        part_before[threadIdx.x] = before;
    }
    for (int i = threadIdx.x; i < kPlaceWarps * E; i += 32 * kPlaceWarps) cnt[i] = 0;
    __syncthreads();
    Segment<kPlaceWarps, kRouteChunk / 32 / kPlaceWarps> seg;
    count_pairs(seg, ids, first, min(kRouteChunk, R - first), E, nbits, cnt);
    const bool mine = threadIdx.x < E;     // one thread an expert from here
    total = before = 0;
    if (mine)
        for (int i = 0; i < G; ++i) {
            total += part_total[(i << nbits) + e];
            before += part_before[(i << nbits) + e];
        }
    const int row = cta_exclusive<kPlaceWarps>(total, warp_tot);   // a barrier: cnt is complete
    if (mine) {
        base[e] = row + before;
        if (chunk == 0) m_indptr[e] = row;
        int run = 0;
#pragma unroll 16
        for (int w = 0; w < kPlaceWarps; ++w) {
            const int n = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += n;
        }
    }
    if (chunk == 0 && threadIdx.x == 0) m_indptr[E] = R;
    __syncthreads();
    place_pairs(seg, E, cnt, base, perm, inv_perm);
}

// ------------------------------------------------------------ launches
// Opt-in of a kernel to `bytes` of dynamic shared memory, once per device and
// kernel; `ready_dev` is the kernel's own (alternating devices set it again).
template <typename Kern>
bool smem_ready(Kern kern, size_t bytes, std::atomic<int>& ready_dev) {
    if (bytes <= 32 * 1024) return true;   // with the static part below the 48 KB that need none
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (ready_dev.load() == dev) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess)
        return false;
    ready_dev.store(dev);
    return true;
}

template <Place MODE>
int launch_place(const RouteArgs& r, int nchunks, cudaStream_t s) {
    static std::atomic<int> ready{-1};
    const size_t smem = (kPlaceWarps + 1ull) * r.E * sizeof(int);
    if (!smem_ready(place_kernel<MODE>, smem, ready)) return ST_CUDA;
    return launch_dependent(place_kernel<MODE>, dim3(nchunks), dim3(32 * kPlaceWarps), 0, smem, s, r.topk_ids,
                            r.T * r.k, r.E, bits_of(r.E), static_cast<const int32_t*>(r.chunk_hist), r.m_indptr,
                            r.perm, r.inv_perm, r.status) == cudaSuccess ? ST_OK : ST_CUDA;
}

template <int PER, int CPL, typename LT>
int launch_inst(const ScoreArgs& a, const RouteArgs* r, cudaStream_t s) {
    const size_t sf = scratch_floats<CPL>(a.E, a.n_group > 1) * sizeof(float);
    const int R = a.T * a.k;
    if (r && a.T <= kSmallTokens) {
        static std::atomic<int> ready{-1};
        const size_t smem = kSmallWarps * sf + (kSmallWarps + 1ull) * a.E * sizeof(int);
        auto kern = score_route_small<PER, CPL, LT>;
        if (!smem_ready(kern, smem, ready)) return ST_CUDA;
        return launch_dependent(kern, dim3(kSmallCluster), dim3(32 * kSmallWarps), kSmallCluster, smem, s, a,
                                r->m_indptr, r->perm, r->inv_perm, r->status, bits_of(a.E)) == cudaSuccess
                   ? ST_OK : ST_CUDA;
    }
    static std::atomic<int> ready{-1};
    auto kern = score_kernel<PER, CPL, LT>;
    if (!smem_ready(kern, kScoreWarps * sf, ready)) return ST_CUDA;
    const unsigned grid = static_cast<unsigned>((a.T + kScoreWarps - 1) / kScoreWarps);
    if (launch_dependent(kern, dim3(grid), dim3(32 * kScoreWarps), 0, kScoreWarps * sf, s, a) != cudaSuccess)
        return ST_CUDA;
    if (!r) return ST_OK;
    const int nchunks = (R + kRouteChunk - 1) / kRouteChunk;
    if (nchunks <= kCountChunks) return launch_place<kCount>(*r, nchunks, s);
    if (launch_dependent(count_kernel, dim3(nchunks), dim3(256), 0, 0, s, static_cast<const int32_t*>(r->topk_ids),
                         R, r->E, r->chunk_hist, r->status) != cudaSuccess)
        return ST_CUDA;
    if (static_cast<long long>(nchunks) << bits_of(r->E) <= kSumCounts) return launch_place<kSum>(*r, nchunks, s);
    if (launch_dependent(scan_kernel, dim3((r->E + 31) / 32), dim3(1024), 0, 0, s, r->chunk_hist, r->E, nchunks) !=
        cudaSuccess)
        return ST_CUDA;
    return launch_place<kPrefix>(*r, nchunks, s);
}

template <int PER, typename LT>
int launch_k(const ScoreArgs& a, const RouteArgs* r, cudaStream_t s) {
    return a.k <= 12 ? launch_inst<PER, 1, LT>(a, r, s) : launch_inst<PER, 2, LT>(a, r, s);
}

template <typename LT>
int launch_e(const ScoreArgs& a, const RouteArgs* r, cudaStream_t s) {
    if (a.E <= 128) return launch_k<4, LT>(a, r, s);
    if (a.E <= 256) return launch_k<8, LT>(a, r, s);
    if (a.E <= 512) return launch_k<16, LT>(a, r, s);
    return launch_k<32, LT>(a, r, s);
}

}  // namespace

int launch_router_score(const ScoreArgs& a, cudaStream_t s) {
    if (a.T == 0) return ST_OK;
    return a.bf16 ? launch_e<__nv_bfloat16>(a, nullptr, s) : launch_e<float>(a, nullptr, s);
}

int launch_router_score_route(const ScoreArgs& a, const RouteArgs& r, cudaStream_t s) {
    return a.bf16 ? launch_e<__nv_bfloat16>(a, &r, s) : launch_e<float>(a, &r, s);
}

}  // namespace moe
