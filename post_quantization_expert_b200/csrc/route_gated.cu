// Routing with gate weights: scores, a balance bias, expert groups, top-k and renormalised weights.
//
// With logits l of one token, s = softmax(l) or sigmoid(l) and the choice c = s + bias. Where the experts
// come in groups of E / G, the groups are ranked by their largest choice or by the sum of their two
// largest, and only the first G' groups stay. The k largest choices are taken in descending order, ties
// to the lower expert (and the lower group). The weights are the scores s (without the bias) of the
// chosen experts, divided by their sum where asked, times a constant.
//
// HBM-bound in principle (E logits in, 8 k bytes out), issue-bound in fact: k rounds of an arg-max. So a
// token takes only as many lanes as give each 8 experts or more (4 lanes for 32 experts, 8 for 64, ... all 32
// from 256 on; the lanes of a token hold consecutive experts), and a round is a float maximum over the
// lane, log2(lanes) exchanges, a vote for the first lane that has it, and a scan of the winner's 8 values.
// A group that is a power of two of whole lanes is ranked by its own lanes, others (up to 32 of them) one after
// the other by all. More than 512 experts, more groups, and k above twice the lanes take the general kernel (a
// warp a token, lane i holds experts i, i + 32, ...).
// 32768 tokens x 64 experts, top 6: general kernel 44 us, this one 13 us; 9973 x 256 in 8 groups, top 8, with a
// bias: general 87 us, this one 31 us (22 us in float32 alone).
//
// The order of the choices is that of exact arithmetic to float64's precision, although they are float32
// here: two choices nearer than the float32 error bound (see `choice_slack`) make a warp repeat the token's
// selection in float64, so that a rounding never picks the expert. Without a bias, unless groups are
// ranked by sums, the logits themselves are compared (both scores increase with them), which is exact at
// once.
#include "clha_internal.h"

namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

struct GateArgs {
    const void* logits;
    int64_t n;
    int E, k, sigmoid, n_groups, top_groups, top2, renorm;
    int group_lanes;         // lanes kernel: whole lanes of a group, a power of two; 0: groups cut through lanes
    float scale;
    const float* bias;
    int32_t* ids;
    float* weights;
    int32_t* counts;
    int* err;
};

template <typename T>
__device__ __forceinline__ float load_logit(const void* p, int64_t i);
template <>
__device__ __forceinline__ float load_logit<float>(const void* p, int64_t i) { return __ldg((const float*)p + i); }
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const void* p, int64_t i) {
    return __bfloat162float(((const __nv_bfloat16*)p)[i]);
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_max(F v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const F u = __shfl_xor_sync(kAll, v, o);
        v = u > v ? u : v;
    }
    return v;
}

// Largest (value, lowest index) over the warp; index 0x7fffffff: none.
template <typename F>
__device__ __forceinline__ void warp_best(F& v, int& i) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const F ov = __shfl_xor_sync(kAll, v, o);
        const int oi = __shfl_xor_sync(kAll, i, o);
        if (oi != 0x7fffffff && (i == 0x7fffffff || ov > v || (ov == v && oi < i))) { v = ov; i = oi; }
    }
}

// Bound on the difference of two float32 choices whose exact order it leaves open. A sigmoid, 1 / (1 + e) or, for l < 0,
// e / (1 + e) with e = e^-|l| (1 + e^-l passes 2^126 at l = -87.4, and the fast division by more than that gives 0), is off by
// less than 2^-24 through e (two steps, 2^-22 of it, times s (1 - s) <= 1/4), 2^-24 through the sum and 2^-22 through
// the fast division (two steps): 1.5 2^-22. A softmax is off by less than 2^-18 of the largest score: 2^-22 and the
// rounded argument's 0.37 2^-24 through the exponential, as much through the sum, whose up to 37 roundings add
// 37 2^-24, and 2^-23 through the division and the product. Twice that, or more, for the two.
__device__ __forceinline__ float choice_slack(bool sigmoid, float top_score) {
    return sigmoid ? 0x1p-20f : 0x1p-17f * top_score;
}
// A biased choice adds 2^-24 of its own size. That of the lower one counts: the upper exceeds it by their distance at
// most. (So a bias of float32's lowest value, which shuts an expert out, leaves the others' order alone. The first round
// compares with +inf, the round behind the last expert with -inf: not near.)
__device__ __forceinline__ bool too_near(float above, float below, float slack) {
    return above - below < fmaf(0x1p-22f, fabsf(below), slack);
}
// Half-width of the interval of a group's rank, a choice or the sum of two whose larger size is `size`: a sum is off by
// twice a choice's error, half the slack each, and by a rounding of its own of 2^-24 of up to twice the size.
__device__ __forceinline__ float rank_error(float slack, float size) { return fmaf(0x1p-21f, size, 2 * slack); }

// One token's selection by a warp, in float32. Lane j < k (and j + 32, ...) writes the j-th expert and its
// weight. Returns false, with nothing written, where a decision was nearer than the error bound.
template <int VPL>
__device__ __forceinline__ bool select_token(const GateArgs& p, const float (&l)[VPL], int64_t t, int lane, int* hist) {
    const bool by_logit = !p.bias && (p.n_groups == 1 || !p.top2);
    float s[VPL], c[VPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < p.E) m = l[i] > m ? l[i] : m;
    float top_score = 1;
    if (!p.sigmoid) {
        m = warp_max(m);
        float sum = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            s[i] = lane + 32 * i < p.E ? expf(l[i] - m) : 0;
            sum += s[i];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = s[i] / sum;
        top_score = 1 / sum;
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const float e = expf(-fabsf(l[i]));
            s[i] = lane + 32 * i < p.E ? (l[i] < 0 ? e : 1) / (1 + e) : 0;
        }
    }
    unsigned live = 0;   // bit i: expert lane + 32 i may be chosen
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        c[i] = by_logit ? l[i] : s[i];
        if (e < p.E) {
            live |= 1u << i;
            if (p.bias) {
                const float b = __ldg(p.bias + e);
                if (isfinite(b))
                    c[i] += b;
                else                                          // recorded; taken as 0
                    clha_record_error(p.err, CLHA_ERR_NONFINITE, (int)(t & 0x7fffffff), e, KID_GATE);
            }
        }
    }
    const float slack = choice_slack(p.sigmoid != 0, top_score);

    if (p.n_groups > 1) {
        // rank every group (all lanes hold it), then keep the first top_groups
        const int size = p.E / p.n_groups;
        float rank[VPL], off[VPL];   // lane holds groups lane, lane + 32, ...; half-widths of the ranks' intervals
        unsigned open = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            rank[i] = off[i] = 0;
            if (lane + 32 * i < p.n_groups) open |= 1u << i;
        }
        for (int g = 0; g < p.n_groups; ++g) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = lane + 32 * i;
                if (e >= g * size && e < (g + 1) * size) {
                    if (c[i] > a) { b = a; a = c[i]; } else if (c[i] > b) b = c[i];
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {   // the two largest of two pairs
                const float oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
                const float lo = a < oa ? a : oa;
                a = a < oa ? oa : a;
                b = b < ob ? ob : b;
                b = b < lo ? lo : b;
            }
            const bool two = p.top2 && size > 1;
            const float r = two ? a + b : a, o = rank_error(slack, two ? fmaxf(fabsf(a), fabsf(b)) : fabsf(a));
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (g == lane + 32 * i) { rank[i] = r; off[i] = o; }
        }
        unsigned kept = 0;
        float above = INFINITY, below = -INFINITY;            // the kept ranks' lowest, the others' highest bound
        for (int r = 0; r < p.top_groups; ++r) {
            float bv = 0;
            int bi = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if ((open >> i & 1) && (bi == 0x7fffffff || rank[i] > bv)) { bv = rank[i]; bi = lane + 32 * i; }
            warp_best(bv, bi);
            if ((bi & 31) == lane) { open &= ~(1u << (bi >> 5)); kept |= 1u << (bi >> 5); }
        }
        if (!by_logit && p.top_groups < p.n_groups) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (kept >> i & 1) above = fminf(above, rank[i] - off[i]);
                if (open >> i & 1) below = fmaxf(below, rank[i] + off[i]);
            }
            if (!(-warp_max(-above) > warp_max(below))) return false;   // (sums that overflow: -inf on both sides)
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i, g = e < p.E ? e / size : 0;
            const unsigned who = __shfl_sync(kAll, kept, g & 31);
            if (e < p.E && !(who >> (g >> 5) & 1)) live &= ~(1u << i);
        }
    }

    float sum = 0, last = 0;
    int my_id[VPL];
    float my_s[VPL];
    bool open_order = false;
    for (int r = 0; r <= p.k; ++r) {
        float bv = 0;
        int bi = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if ((live >> i & 1) && (bi == 0x7fffffff || c[i] > bv)) { bv = c[i]; bi = lane + 32 * i; }
        warp_best(bv, bi);
        if (bi == 0x7fffffff) break;
        if (!by_logit && r > 0 && too_near(last, bv, slack)) open_order = true;
        if (r == p.k || open_order) break;
        last = bv;
        float sv = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i == bi >> 5) sv = s[i];
        sv = __shfl_sync(kAll, sv, bi & 31);
        if ((bi & 31) == lane) live &= ~(1u << (bi >> 5));
        sum += sv;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (r == lane + 32 * i) { my_id[i] = bi; my_s[i] = sv; }
    }
    if (open_order) return false;
    if (p.renorm && !(sum > 1e-30f)) return false;   // float32 scores that underflow
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int j = lane + 32 * i;
        if (j < p.k) {
            float w = my_s[i];
            if (p.renorm) w /= sum;                           // (above 1e-30)
            p.ids[t * p.k + j] = my_id[i];
            p.weights[t * p.k + j] = (float)(w * p.scale);
            atomicAdd(&hist[my_id[i]], 1);
        }
    }
    return true;
}

template <typename T>
__device__ __forceinline__ float finite_logit(const T* row, int e) {
    const float l = load_logit<T>(row, e);
    return isfinite(l) ? l : 0.f;
}

// ------------------------------------------------------------------ the selection in float64
// Taken by a warp for a token whose float32 choices leave a decision open (0 to 9 of 9973 tokens x 256 experts), but its
// latency is the kernel's tail, so the doubles are compared as ordered 64-bit integers, whose warp-wide
// maximum is two integer reductions (9973 x 256 experts with one such token: 24 us more as a selection by
// exchanged doubles, 9 us more this way).
__device__ __forceinline__ uint64_t to_key(double v) {        // larger value, larger key; never 0
    const int64_t b = __double_as_longlong(v + 0.0);          // one zero
    return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}
__device__ __forceinline__ double from_key(uint64_t k) {
    return __longlong_as_double(k >> 63 ? (int64_t)(k & 0x7fffffffffffffffull) : ~(int64_t)k);
}
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}
// The largest key over the warp and the lowest index 32 i + lane that holds it, among those that `in` admits.
template <int N, typename In>
__device__ __forceinline__ uint64_t best_key(const uint64_t (&key)[N], int lane, In in, int& index) {
    uint64_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (in(i) && key[i] > m) m = key[i];
    m = warp_max_key(m);
    unsigned at = 0xffffffffu;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
        if (in(i) && key[i] == m) at = 32 * i + lane;
    index = (int)__reduce_min_sync(kAll, at);
    return m;
}

// VPL experts and GPL groups a lane.
template <typename T, int VPL, int GPL>
__device__ __noinline__ void exact_token(const GateArgs& p, int64_t t, int lane, int* hist) {
    const T* row = reinterpret_cast<const T*>(p.logits) + t * p.E;
    double s[VPL];
    uint64_t key[VPL];
    float l[VPL], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        l[i] = lane + 32 * i < p.E ? finite_logit<T>(row, lane + 32 * i) : -INFINITY;
        m = fmaxf(m, l[i]);
    }
    m = warp_max(m);
    double total = 1;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = exp(p.sigmoid ? -(double)l[i] : (double)l[i] - (double)m);
    if (!p.sigmoid) {
        total = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) total += s[i];
        total = warp_sum(total);
    }
    const bool by_logit = !p.bias && (p.n_groups == 1 || !p.top2);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        s[i] = p.sigmoid ? 1 / (1 + s[i]) : s[i] / total;
        key[i] = 0;
        if (e < p.E) {
            const float b = p.bias ? __ldg(p.bias + e) : 0.f;
            key[i] = to_key(by_logit ? (double)l[i] : isfinite(b) ? s[i] + (double)b : s[i]);
        }
    }
    if (p.n_groups > 1) {
        const int size = p.E / p.n_groups;
        uint64_t rank[GPL];                                   // of groups lane, lane + 32, ...
#pragma unroll
        for (int i = 0; i < GPL; ++i) rank[i] = 0;
        for (int g = 0; g < p.n_groups; ++g) {
            int first, second;
            const auto inside = [&](int i) { return (unsigned)(lane + 32 * i - g * size) < (unsigned)size; };
            uint64_t r = best_key(key, lane, inside, first);
            if (p.top2 && size > 1) {
                const uint64_t r2 =
                    best_key(key, lane, [&](int i) { return inside(i) && lane + 32 * i != first; }, second);
                r = to_key(from_key(r) + from_key(r2));
            }
#pragma unroll
            for (int i = 0; i < GPL; ++i)
                if (g == lane + 32 * i) rank[i] = r;
        }
        unsigned kept = 0;
        for (int r = 0; r < p.top_groups; ++r) {
            int g;
            best_key(rank, lane, [](int) { return true; }, g);
#pragma unroll
            for (int i = 0; i < GPL; ++i)
                if (g == lane + 32 * i) { rank[i] = 0; kept |= 1u << i; }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i, g = e < p.E ? e / size : 0;
            const unsigned who = __shfl_sync(kAll, kept, g & 31);
            if (!(who >> (g >> 5) & 1)) key[i] = 0;
        }
    }
    const double scale = p.scale;
    double sum = 0, mine = 0;                                 // the score of this lane's last choice
    for (int r = 0; r < p.k; ++r) {
        int e;
        best_key(key, lane, [](int) { return true; }, e);
        double sv = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e == lane + 32 * i) { key[i] = 0; sv = s[i]; }
        sv = __shfl_sync(kAll, sv, e & 31);
        sum += sv;
        if (lane == (r & 31)) {
            p.ids[t * p.k + r] = e;
            atomicAdd(&hist[e], 1);
            mine = sv;
            if (!p.renorm) p.weights[t * p.k + r] = (float)(sv * scale);
        }
    }
    if (!p.renorm) return;
    for (int j = lane; j < p.k; j += 32) {
        double w = mine;
        if (j + 32 < p.k) {                                   // more than 32 choices: an earlier one's score again
            const float l = finite_logit<T>(row, p.ids[t * p.k + j]);
            w = p.sigmoid ? 1 / (1 + exp(-(double)l)) : exp((double)l - (double)m) / total;
        }
        p.weights[t * p.k + j] = (float)((sum > 0 ? w / sum : 1.0 / p.k) * scale);
    }
}

template <typename T, int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_gated_kernel(GateArgs p, int one_block) {
    clha_allow_next();
    clha_wait_inputs();
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < p.n; t += (int64_t)gridDim.x * kWarps) {
        float l[VPL];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < p.E ? load_logit<T>(p.logits, t * p.E + e) : 0.f;
            if (!isfinite(l[i])) { bad = true; l[i] = 0.f; }     // recorded; the ids stay in range
        }
        if (__any_sync(kAll, bad) && lane == 0)
            clha_record_error(p.err, CLHA_ERR_NONFINITE, (int)(t & 0x7fffffff), 0, KID_GATE);
        if (!select_token<VPL>(p, l, t, lane, hist)) exact_token<T, VPL, VPL>(p, t, lane, hist);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        if (one_block)
            p.counts[e] = hist[e];
        else if (hist[e])
            atomicAdd(&p.counts[e], hist[e]);
    }
}

// ------------------------------------------------------------------ LPT lanes a token, VPL experts a lane
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
    if (LPT == 32) {
        asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
    } else {
#pragma unroll
        for (int o = LPT / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

template <typename T, int VPL>
__device__ __forceinline__ void load_run(const T* p, float (&l)[VPL]) {   // 16-byte aligned, VPL a multiple of 8
#pragma unroll
    for (int i = 0; i < VPL; i += 8) {
        if (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
            const float4 b = __ldg(reinterpret_cast<const float4*>(p + i) + 1);
            l[i] = a.x; l[i + 1] = a.y; l[i + 2] = a.z; l[i + 3] = a.w;
            l[i + 4] = b.x; l[i + 5] = b.y; l[i + 6] = b.z; l[i + 7] = b.w;
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(p + i));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                l[i + 2 * j] = __uint_as_float(w[j] << 16);
                l[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
}

template <typename T, int LPT, int VPL>
__global__ void __launch_bounds__(kWarps * 32, VPL == 8 ? 4 : 2) route_lanes_kernel(GateArgs p, int one_block, int vec) {
    constexpr int TPW = 32 / LPT;                            // tokens a warp
    clha_allow_next();
    clha_wait_inputs();
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, sub = lane & (LPT - 1), first = lane & ~(LPT - 1);
    const unsigned mine = LPT == 32 ? kAll : ((1u << LPT) - 1) << first;     // the token's lanes
    const int e0 = sub * VPL;
    const bool by_logit = !p.bias && (p.n_groups == 1 || !p.top2);
    const int64_t per_block = kWarps * TPW;
    float bias[VPL];
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            bias[i] = e0 + i < p.E ? __ldg(p.bias + e0 + i) : 0.f;
            if (!isfinite(bias[i])) {                        // recorded; taken as 0
                clha_record_error(p.err, CLHA_ERR_NONFINITE, 0, e0 + i, KID_GATE);
                bias[i] = 0.f;
            }
        }
    }
    for (int64_t tb = (int64_t)blockIdx.x * per_block + (threadIdx.x >> 5) * TPW; tb < p.n;
         tb += (int64_t)gridDim.x * per_block) {
        const int64_t t = tb + lane / LPT;
        const bool real = t < p.n;
        float c[VPL];
        const T* row = reinterpret_cast<const T*>(p.logits) + (real ? t : 0) * p.E;
        if (vec && e0 + VPL <= p.E) {
            load_run<T, VPL>(row + e0, c);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) c[i] = e0 + i < p.E ? load_logit<T>(row, e0 + i) : -INFINITY;
        }
        float m = 0.f, top_score = 1.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e0 + i < p.E && !isfinite(c[i])) { bad = true; c[i] = 0.f; }   // recorded; the ids stay in range
        if (bad && real) clha_record_error(p.err, CLHA_ERR_NONFINITE, (int)(t & 0x7fffffff), 0, KID_GATE);
        if (!p.sigmoid) {
            m = c[0];
            float sum = 0.f;
#pragma unroll
            for (int i = 1; i < VPL; ++i) m = fmaxf(m, c[i]);
            m = lanes_max<LPT>(m);
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum += expf(c[i] - m);   // past E: exp(-inf) = 0
            top_score = 1.f / lanes_sum<LPT>(sum);
        }
        const auto score = [&](float l) {
            if (!p.sigmoid) return expf(l - m) * top_score;
            const float e = expf(-fabsf(l));
            return __fdividef(l < 0.f ? e : 1.f, 1.f + e);
        };
        const float slack = choice_slack(p.sigmoid != 0, top_score);
        if (!by_logit) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (e0 + i < p.E) c[i] = score(c[i]) + (p.bias ? bias[i] : 0.f);
        }
        bool open = false;                                   // a decision inside the error bound
        if (p.n_groups > 1) {
            const int size = p.E / p.n_groups;
            const int q = p.group_lanes ? p.group_lanes : 1; // lanes a group, a power of two; or lane h has group h's rank
            float rank = -INFINITY, off = 0.f;               // and the half-width of its interval
            const auto set_rank = [&](float a, float b, bool two) {
                rank = two ? a + b : a;
                off = rank_error(slack, two ? fmaxf(fabsf(a), fabsf(b)) : fabsf(a));
            };
            if (p.group_lanes) {
                float a = -INFINITY, b = -INFINITY;          // the two largest choices of the group
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    b = fmaxf(b, fminf(a, c[i]));
                    a = fmaxf(a, c[i]);
                }
                for (int o = 1; o < q; o <<= 1) {
                    const float oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
                    b = fmaxf(fmaxf(b, ob), fminf(a, oa));
                    a = fmaxf(a, oa);
                }
                if (e0 < p.E) set_rank(a, b, p.top2);
            } else {
                for (int h = 0; h < p.n_groups; ++h) {
                    const unsigned from = h * size - e0;     // the group's first expert among this lane's
                    float a = -INFINITY, b = -INFINITY;
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
                        if (i - from < (unsigned)size) {
                            b = fmaxf(b, fminf(a, c[i]));
                            a = fmaxf(a, c[i]);
                        }
#pragma unroll
                    for (int o = LPT / 2; o; o >>= 1) {
                        const float oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
                        b = fmaxf(fmaxf(b, ob), fminf(a, oa));
                        a = fmaxf(a, oa);
                    }
                    if (sub == h) set_rank(a, b, p.top2 && size > 1);
                }
            }
            const int g = sub / q;
            const bool in = g < p.n_groups;
            int ahead = 0;
            for (int h = 0; h < p.n_groups; ++h) {
                const float r = __shfl_sync(kAll, rank, first + h * q);
                ahead += r > rank || (r == rank && h < g);
            }
            const bool kept = in && ahead < p.top_groups;
            if (!by_logit && p.top_groups < p.n_groups) {    // the kept ranks' lowest, the others' highest bound
                const float above = -lanes_max<LPT>(kept ? off - rank : -INFINITY);
                const float below = lanes_max<LPT>(in && !kept ? rank + off : -INFINITY);
                open = !(above > below);                     // (sums that overflow: -inf on both sides)
            }
            const unsigned stay = __ballot_sync(kAll, kept) >> first;   // by lanes
            if (p.group_lanes) {
                if (!kept) {
#pragma unroll
                    for (int i = 0; i < VPL; ++i) c[i] = -INFINITY;
                }
            } else {
                int h = e0 / size, left = (h + 1) * size - e0;          // the expert's group; experts left in it
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    if (!(stay >> h & 1)) c[i] = -INFINITY;
                    if (--left == 0) { ++h; left = size; }
                }
            }
        }
        float last = INFINITY;
        int id0 = 0, id1 = 0;                                // this lane's choices: the sub-th and the (sub + LPT)-th
        const int rounds = by_logit ? p.k : p.k + 1;         // one more, to see how near the first loser is
        for (int r = 0; r < rounds; ++r) {
            float mx = c[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) mx = fmaxf(mx, c[i]);
            const float best = lanes_max<LPT>(mx);
            if (too_near(last, best, slack) && !by_logit) open = true;
            last = best;
            const int owner = __ffs(__ballot_sync(kAll, mx == best) & mine) - 1;
            int idx = 0;
#pragma unroll
            for (int i = VPL - 1; i >= 0; --i) idx = c[i] == best ? i : idx;   // the first that is the largest
            const int gone = owner == lane ? idx : -1;
#pragma unroll
            for (int i = 0; i < VPL; ++i) c[i] = i == gone ? -INFINITY : c[i];
            const int e = __shfl_sync(kAll, e0 + idx, owner);
            id0 = r == sub ? e : id0;
            id1 = r == sub + LPT ? e : id1;
        }
        const bool has0 = sub < p.k, has1 = sub + LPT < p.k;
        const float s0 = has0 ? score(finite_logit<T>(row, id0)) : 0.f, s1 = has1 ? score(finite_logit<T>(row, id1)) : 0.f;
        float f = p.scale;
        if (p.renorm) {
            const float sum = lanes_sum<LPT>(s0 + s1);
            f = p.scale / sum;
            if (!(sum > 1e-30f && fabsf(f) < INFINITY)) open = true;   // float32 scores that underflow
        }
        if (real && !open) {
            if (has0) {
                p.ids[t * p.k + sub] = id0;
                p.weights[t * p.k + sub] = s0 * f;
                atomicAdd(&hist[id0], 1);
            }
            if (has1) {
                p.ids[t * p.k + sub + LPT] = id1;
                p.weights[t * p.k + sub + LPT] = s1 * f;
                atomicAdd(&hist[id1], 1);
            }
        }
        unsigned again = __ballot_sync(kAll, real && open && sub == 0);
        while (again) {
            const int w = __ffs(again) - 1;
            again &= again - 1;
            exact_token<T, LPT * VPL / 32 ? LPT * VPL / 32 : 1, 1>(p, tb + w / LPT, lane, hist);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        if (one_block)
            p.counts[e] = hist[e];
        else if (hist[e])
            atomicAdd(&p.counts[e], hist[e]);
    }
}

// The counts' clearing, as a kernel so that the routing's set-up overlaps it (after a memset, which nothing overlaps,
// 32768 tokens x 64 experts took 16.4 us, after this 13.1).
__global__ void __launch_bounds__(1024) clear_counts_kernel(int32_t* counts, int E) {
    clha_allow_next();
    clha_wait_inputs();
    if ((int)threadIdx.x < E) counts[threadIdx.x] = 0;
}

template <typename T>
cudaError_t launch_t(cudaStream_t s, int num_sms, GateArgs p) {
    const int vpl = p.E <= 256 ? 8 : 16, size = p.E / p.n_groups, q = size / vpl;
    int lpt = p.E <= 32 ? 4 : p.E <= 64 ? 8 : p.E <= 128 ? 16 : 32;
    p.group_lanes = size % vpl == 0 && (q & (q - 1)) == 0 ? q : 0;
    if (!p.group_lanes)
        while (lpt < 32 && lpt < p.n_groups) lpt *= 2;       // a lane for each group's rank
    const bool lanes = p.E <= 512 && p.k <= 2 * lpt && (p.n_groups == 1 || p.group_lanes || p.n_groups <= lpt);
    const int tokens = kWarps * (lanes ? 32 / lpt : 1);      // a block's tokens at a time
    int64_t blocks = (p.n + tokens - 1) / tokens;
    // up to two rounds of one block: it overwrites the counts, and the clearing launch is saved
    const int one = blocks <= 2;
    cudaError_t e = cudaSuccess;
    if (one) {
        blocks = 1;
    } else {
        e = clha_launch_overlapped(clear_counts_kernel, 1, 1024, 0, s, 1, p.counts, p.E);
        clha_note_launches(1);
    }
    if (e != cudaSuccess) return e;
    // one wave: a block's histogram and bias serve all of its tokens
    const int64_t wave = (int64_t)num_sms * (lanes ? 4 : 8);
    if (blocks > wave) blocks = wave;
    const size_t smem = p.E * sizeof(int);
    if (lanes) {
        const int vec = p.E % 8 == 0 && ((uintptr_t)p.logits & 15) == 0;
#define CLHA_GATE(L, V) \
    e = clha_launch_overlapped(route_lanes_kernel<T, L, V>, (unsigned)blocks, kWarps * 32, smem, s, 1, p, one, vec)
        if (vpl == 16) CLHA_GATE(32, 16);
        else if (lpt == 4) CLHA_GATE(4, 8);
        else if (lpt == 8) CLHA_GATE(8, 8);
        else if (lpt == 16) CLHA_GATE(16, 8);
        else CLHA_GATE(32, 8);
#undef CLHA_GATE
    } else {
#define CLHA_GATE(V) \
    e = clha_launch_overlapped(route_gated_kernel<T, V>, (unsigned)blocks, kWarps * 32, smem, s, 1, p, one)
        if (p.E <= 32) CLHA_GATE(1);
        else if (p.E <= 64) CLHA_GATE(2);
        else if (p.E <= 128) CLHA_GATE(4);
        else if (p.E <= 256) CLHA_GATE(8);
        else if (p.E <= 512) CLHA_GATE(16);
        else CLHA_GATE(32);
#undef CLHA_GATE
    }
    if (e != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_gated(cudaStream_t s, int num_sms, const void* logits, int is_f32, int64_t n,
                               const clha_route_params& rp, const float* bias, int32_t* ids, float* weights,
                               int32_t* counts, int* err) {
    GateArgs p{logits, n, rp.E, rp.k, rp.score == CLHA_SCORE_SIGMOID, rp.n_groups, rp.top_groups,
               rp.group_rank == CLHA_GROUP_TOP2, rp.renormalise != 0, 0, rp.scale, bias, ids, weights, counts, err};
    return is_f32 ? launch_t<float>(s, num_sms, p) : launch_t<__nv_bfloat16>(s, num_sms, p);
}
