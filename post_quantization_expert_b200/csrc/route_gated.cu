// Routing with gate weights: scores, a balance bias, expert groups, top-k and renormalised weights.
//
// With logits l of one token, s = softmax(l) or sigmoid(l) and the choice c = s + bias. Where the experts
// come in groups of E / G, the groups are ranked by their largest choice or by the sum of their two
// largest, and only the first G' groups stay. The k largest choices are taken in descending order, ties
// to the lower expert (and the lower group). The weights are the scores s (without the bias) of the
// chosen experts, divided by their sum where asked, times a constant.
//
// One warp a token, the values in registers (lane i holds experts i, i + 32, ...): HBM-bound for many
// tokens (4 E bytes a token), latency-bound for few. The order of the choices is that of exact
// arithmetic to float64's precision, although they are float32 here: two choices nearer than the float32
// error bound (see `slack`) make the token repeat the selection in float64, so that a rounding never picks
// the expert. Without a bias, unless groups are ranked by sums, the logits themselves are compared
// (both scores increase with them), which is exact at once.
#include "clha_internal.h"

namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

struct GateArgs {
    const void* logits;
    int64_t n;
    int E, k, sigmoid, n_groups, top_groups, top2, renorm;
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
__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

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

// One token's selection in the arithmetic of F. Lane j < k (and j + 32, ...) writes the j-th expert and its
// weight. Returns false, with nothing written, where a decision was nearer than the error bound.
template <typename F, int VPL>
__device__ __forceinline__ bool select_token(const GateArgs& p, const float (&l)[VPL], int64_t t, int lane, int* hist) {
    constexpr bool kExact = sizeof(F) == 8;
    const bool by_logit = !p.bias && (p.n_groups == 1 || !p.top2);
    F s[VPL], c[VPL];
    F m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < p.E) m = l[i] > m ? (F)l[i] : m;
    F top_score = 1;
    if (!p.sigmoid) {
        m = warp_max(m);
        F sum = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            s[i] = lane + 32 * i < p.E ? exp_of((F)l[i] - m) : (F)0;
            sum += s[i];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = s[i] / sum;
        top_score = (F)1 / sum;
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = lane + 32 * i < p.E ? (F)1 / ((F)1 + exp_of(-(F)l[i])) : (F)0;
    }
    unsigned live = 0;   // bit i: expert lane + 32 i may be chosen
    F big = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        c[i] = by_logit ? (F)l[i] : s[i];
        if (e < p.E) {
            live |= 1u << i;
            if (p.bias) {
                const float b = __ldg(p.bias + e);
                if (isfinite(b))
                    c[i] += (F)b;
                else                                          // recorded; taken as 0
                    clha_record_error(p.err, CLHA_ERR_NONFINITE, (int)(t & 0x7fffffff), e, KID_GATE);
                big = fabs(c[i]) > big ? (F)fabs(c[i]) : big;
            }
        }
    }
    // Bound on the difference of two float32 choices whose exact order it leaves open: a score is off by
    // less than 2^-18 of the largest (exponential, a sum of up to 1024 terms, a division), a biased one by
    // another 2^-24 of its size; doubled, and doubled again for sums of two.
    F slack = 0;
    if (!kExact && !by_logit) slack = (F)0x1p-16f * top_score + (F)0x1p-21f * warp_max(big);

    if (p.n_groups > 1) {
        // rank every group (all lanes hold it), then keep the first top_groups
        const int size = p.E / p.n_groups;
        F rank[VPL];     // lane holds groups lane, lane + 32, ...
        unsigned open = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            rank[i] = 0;
            if (lane + 32 * i < p.n_groups) open |= 1u << i;
        }
        for (int g = 0; g < p.n_groups; ++g) {
            F a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = lane + 32 * i;
                if (e >= g * size && e < (g + 1) * size) {
                    if (c[i] > a) { b = a; a = c[i]; } else if (c[i] > b) b = c[i];
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {   // the two largest of two pairs
                const F oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
                const F lo = a < oa ? a : oa;
                a = a < oa ? oa : a;
                b = b < ob ? ob : b;
                b = b < lo ? lo : b;
            }
            const F r = p.top2 && size > 1 ? a + b : a;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (g == lane + 32 * i) rank[i] = r;
        }
        unsigned kept = 0;
        F last = 0;
        for (int r = 0; r <= p.top_groups && r < p.n_groups; ++r) {
            F bv = 0;
            int bi = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if ((open >> i & 1) && (bi == 0x7fffffff || rank[i] > bv)) { bv = rank[i]; bi = lane + 32 * i; }
            warp_best(bv, bi);
            if (r == p.top_groups) {
                if (!kExact && !by_logit && last - bv <= 2 * slack) return false;
                break;
            }
            last = bv;
            if ((bi & 31) == lane) { open &= ~(1u << (bi >> 5)); kept |= 1u << (bi >> 5); }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i, g = e < p.E ? e / size : 0;
            const unsigned who = __shfl_sync(kAll, kept, g & 31);
            if (e < p.E && !(who >> (g >> 5) & 1)) live &= ~(1u << i);
        }
    }

    F sum = 0, last = 0;
    int my_id[VPL];
    F my_s[VPL];
    bool open_order = false;
    for (int r = 0; r <= p.k; ++r) {
        F bv = 0;
        int bi = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if ((live >> i & 1) && (bi == 0x7fffffff || c[i] > bv)) { bv = c[i]; bi = lane + 32 * i; }
        warp_best(bv, bi);
        if (bi == 0x7fffffff) break;
        if (!kExact && !by_logit && r > 0 && last - bv <= slack) open_order = true;
        if (r == p.k || open_order) break;
        last = bv;
        F sv = 0;
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
    if (!kExact && p.renorm && !(sum > (F)1e-30f)) return false;   // float32 scores that underflow
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int j = lane + 32 * i;
        if (j < p.k) {
            F w = my_s[i];
            if (p.renorm) w = sum > 0 ? w / sum : (F)1 / p.k;
            p.ids[t * p.k + j] = my_id[i];
            p.weights[t * p.k + j] = (float)(w * (F)p.scale);
            atomicAdd(&hist[my_id[i]], 1);
        }
    }
    return true;
}

template <typename T, int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_gated_kernel(GateArgs p, int one_block) {
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
        if (!select_token<float, VPL>(p, l, t, lane, hist)) select_token<double, VPL>(p, l, t, lane, hist);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        if (one_block)
            p.counts[e] = hist[e];
        else if (hist[e])
            atomicAdd(&p.counts[e], hist[e]);
    }
}

template <typename T>
cudaError_t launch_t(cudaStream_t s, int num_sms, const GateArgs& p) {
    int64_t blocks = (p.n + kWarps - 1) / kWarps;
    // up to two tokens a warp in one block: it overwrites the counts, and the clearing launch is saved
    const int one = p.n <= 2 * kWarps;
    if (one) blocks = 1;
    if (!one) {
        cudaError_t e = cudaMemsetAsync(p.counts, 0, p.E * sizeof(int32_t), s);
        if (e != cudaSuccess) return e;
    }
    if (blocks > (int64_t)num_sms * 16) blocks = (int64_t)num_sms * 16;
    const size_t smem = p.E * sizeof(int);
#define CLHA_GATE(V) route_gated_kernel<T, V><<<(unsigned)blocks, kWarps * 32, smem, s>>>(p, one)
    if (p.E <= 32) CLHA_GATE(1);
    else if (p.E <= 64) CLHA_GATE(2);
    else if (p.E <= 128) CLHA_GATE(4);
    else if (p.E <= 256) CLHA_GATE(8);
    else if (p.E <= 512) CLHA_GATE(16);
    else CLHA_GATE(32);
#undef CLHA_GATE
    clha_note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_gated(cudaStream_t s, int num_sms, const void* logits, int is_f32, int64_t n,
                               const clha_route_params& rp, const float* bias, int32_t* ids, float* weights,
                               int32_t* counts, int* err) {
    GateArgs p{logits, n, rp.E, rp.k, rp.score == CLHA_SCORE_SIGMOID, rp.n_groups, rp.top_groups,
               rp.group_rank == CLHA_GROUP_TOP2, rp.renormalise != 0, rp.scale, bias, ids, weights, counts, err};
    return is_f32 ? launch_t<float>(s, num_sms, p) : launch_t<__nv_bfloat16>(s, num_sms, p);
}
