// Combination of the experts' outputs: y[t] = add[t] + sum_j w[t][j] z[row(t, j)], j ascending, in float32.
//
// The packed row of a token's slot is found where clha_gather put it: the expert's segment lists its
// tokens in ascending order, so a binary search of perm gives the row, and no inverse permutation is
// stored or written. HBM-bound: each z row is read once. A block takes one token and 256 * 8 columns at a
// time; its first k threads search (for few tokens a search is a step or two; for many the other blocks of the
// SM hide it). 32768 tokens x 2048, six float32 rows each and an addend: 321 us, 89 % of the measured copy bandwidth.
#include "clha_internal.h"

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[2 * i])) |
               (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * i + 1])) << 16;
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(o[0], o[1], o[2], o[3]));
}

template <typename TZ, typename TY, typename TA>
__global__ void __launch_bounds__(kThreads) combine_kernel(const TZ* __restrict__ Z, int64_t rows, int d,
                                                           const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                           int64_t n, int k, int E, const int64_t* __restrict__ seg,
                                                           const int32_t* __restrict__ perm, const TA* add, TY* Y,
                                                           int* err) {
    clha_allow_next();
    clha_wait_inputs();
    extern __shared__ int64_t row_of[];                    // [k] the slots' packed rows, then [k] weights
    float* wt = reinterpret_cast<float*>(row_of + k);
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x) {
        for (int j = threadIdx.x; j < k; j += kThreads) {
            const int e = ids[t * k + j];
            int64_t at = -1;
            if (e >= 0 && e < E) {
                int64_t lo = seg[e], hi = lo + seg[E + 1 + e];
                if (lo >= 0 && hi <= rows) {
                    const int64_t end = hi;
                    while (lo < hi) {
                        const int64_t mid = (lo + hi) >> 1;
                        int64_t m = mid;             // (a token that names an expert twice leaves a hole, -1, behind
                        int32_t v = perm[m];         // its row)
                        while (v < 0 && m > lo) v = perm[--m];
                        if (v < (int32_t)t) lo = mid + 1; else hi = m;
                    }
                    if (lo < end && perm[lo] == (int32_t)t) at = lo;
                }
            }
            if (at < 0) clha_record_error(err, CLHA_ERR_INVALID_ARG, (int)t, j, KID_COMBINE);
            row_of[j] = at;
            wt[j] = w ? w[t * k + j] : 1.f;
        }
        __syncthreads();
        for (int c = threadIdx.x * 8; c < d; c += kThreads * 8) {
            float y[8] = {};
            if (add) load8<TA>(add + t * d + c, y);
            for (int j = 0; j < k; ++j) {
                const int64_t r = row_of[j];
                if (r < 0) continue;
                float z[8];
                load8<TZ>(Z + r * d + c, z);
                const float g = wt[j];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = fmaf(g, z[i], y[i]);
            }
            store8(Y + t * d + c, y);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_combine(cudaStream_t s, const void* Z, int z_f32, int64_t rows, int d, const int32_t* ids,
                           const float* w, int64_t n, int k, int E, const int64_t* seg, const int32_t* perm,
                           const void* add, int add_f32, void* Y, int y_f32, int* err) {
    const unsigned blocks = (unsigned)(n < 65536 * 16 ? n : 65536 * 16);
    const size_t smem = (size_t)k * 12;
    typedef __nv_bfloat16 bf;
    const auto launch = [&](auto tz, auto ty, auto ta) {
        typedef decltype(tz) TZ;
        typedef decltype(ty) TY;
        typedef decltype(ta) TA;
        return clha_launch_overlapped(combine_kernel<TZ, TY, TA>, blocks, kThreads, smem, s, 1, (const TZ*)Z, rows, d, ids, w,
                                      n, k, E, seg, perm, (const TA*)add, (TY*)Y, err);
    };
    const auto by_add = [&](auto tz, auto ty) { return add_f32 ? launch(tz, ty, float()) : launch(tz, ty, bf()); };
    const cudaError_t e = z_f32 ? (y_f32 ? by_add(float(), float()) : by_add(float(), bf()))
                                : (y_f32 ? by_add(bf(), float()) : by_add(bf(), bf()));
    if (e != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}
