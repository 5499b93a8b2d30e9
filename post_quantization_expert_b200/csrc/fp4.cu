// Microscaled 4-bit floating point: quantization, decoding and the matrix scale.
//
// A row is cut into blocks of 32 (power-of-two e8m0 scales) or 16 (e4m3 scales). With g the float32 scale
// of the matrix (1 where there is none), a block's scale s and its codes q are
//   e8m0   s = 2^(floor(log2(max|x| / g)) - 2)          (2 = the exponent of e2m1's largest number, 6)
//   e4m3   s = max|x| / (6 g) rounded to nearest even, 2^-9 <= s <= 448 (0 for a block of zeros)
//   q = x / (s g) rounded to the nearest e2m1 number, ties to the even code, saturating at +-6,
// all of it decided as if in exact arithmetic. Divisions make that more than one float32 operation: the
// quotient t is formed with reciprocals (relative error below 2^-21.9), t (1 - 2^-21) and t (1 + 2^-21)
// are both rounded, and only where the two differ (about one block in 10^5) the lane decides again in
// float64, where a quotient of a 24-bit by a 28-bit number cannot round onto a border that it is not on
// (borders have at most 5 bits, so x and border * s * g differ by 2^-33 of their size or not at all).
// A power-of-two scale without g needs no quotient: x times a power of two is exact.
//
// Both kernels stream: a warp takes 256 columns of the four rows r, r + 32, r + 64, r + 96 of a 128-row
// tile (four loads in flight a lane), because those rows' scales of four blocks are 16 consecutive bytes
// of the tiled scale layout and leave in one store.
#include "clha_internal.h"

#include <cuda_fp16.h>

namespace {

constexpr float kLo = 1.f - 0x1p-21f, kHi = 1.f + 0x1p-21f;
constexpr int kThreads = 256;

// Eight e2m1 codes of v[0..7], v[0] in the low bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// e4m3 codes of two floats, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float from_e4m3(uint32_t byte) {   // byte < 0x7f: sign-free, finite
    const uint32_t e = byte >> 3, m = byte & 7;
    return e ? __uint_as_float(((e + 120) << 23) | (m << 20)) : (float)m * 0x1p-9f;
}
__device__ __forceinline__ float pow2_byte(uint32_t byte) {   // 2^(byte - 127)
    return byte ? __uint_as_float(byte << 23) : 0x1p-127f;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ------------------------------------------------------------------ exact decisions, rarely taken
__device__ __noinline__ uint32_t e4m3_exact(double t) {       // t > 0
    if (t >= 448.0) return 0x7e;
    int e;
    frexp(t, &e);                                             // t in [2^(e-1), 2^e)
    e = e - 1 < -6 ? -6 : e - 1;
    const int m = (int)rint(ldexp(t, 3 - e));                 // 0..16 eighths of 2^e
    return (uint32_t)((e + 6) * 8 + m);                       // a carry runs into the exponent
}
__device__ __noinline__ uint32_t e2m1_exact(float x, double d) {
    const double a = fabs((double)x) / d;
    const uint32_t c = (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0);
    return c | (signbit(x) ? 8u : 0u);
}

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
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The block scale's byte for the largest magnitude `top` (finite) of a block, and *r ~ 1 / (s g).
template <int BLOCK, bool SCALED>
__device__ __forceinline__ uint32_t block_scale(float top, float g, float rg, float r6g, float* r) {
    if (BLOCK == 32) {
        uint32_t byte;
        if (!SCALED) {
            const int e = (int)(__float_as_uint(top) >> 23) - 2;
            byte = e > 0 ? e : 0;
        } else {
            const float t = top * rg;
            const uint32_t lo = __float_as_uint(t * kLo) >> 23, hi = __float_as_uint(t * kHi) >> 23;
            int e = (int)lo - 2;
            if (lo != hi || lo == 0 || hi >= 254) {          // near a power of two, or outside float32's range
                int x;
                frexp((double)top / (double)g, &x);          // floor(log2) = x - 1
                e = x - 1 - 2 + 127;
            }
            byte = top == 0.f || e < 0 ? 0 : (e > 254 ? 254 : e);
        }
        // 2^(127 - byte) is a float32 for every byte <= 254 (for 254 a subnormal)
        const float inv = byte == 254 ? 0x1p-127f : __uint_as_float((254 - byte) << 23);
        *r = top == 0.f ? 0.f : (SCALED ? inv * rg : inv);
        return byte;
    }
    const float t = top * r6g;
    uint32_t two = e4m3x2(t * kLo, t * kHi);
    uint32_t byte = two & 0xff;
    if (byte != two >> 8 || !(t > 0x1p-100f && t < 0x1p100f)) byte = top == 0.f ? 0 : e4m3_exact((double)top / (6.0 * (double)g));
    if (byte == 0 && top != 0.f) byte = 1;
    float rs;
    asm("rcp.approx.f32 %0, %1;" : "=f"(rs) : "f"(from_e4m3(byte)));
    *r = byte == 0 ? 0.f : (SCALED ? rs * rg : rs);
    return byte;
}

// ------------------------------------------------------------------------------ quantization
struct QuantArgs {
    const void* X;
    int64_t n, rows;              // rows of X, and of the output
    int d;
    const int32_t* perm;          // null: row r is X's row r
    const int64_t* seg;           // null: all rows; else rows below seg[E]
    int E;
    const float* g;               // null or one an equal share of the rows
    int64_t rows_per_g;
    uint8_t* codes;
    uint8_t* scales;
    int64_t items;                // 128-row tiles * 32 * column chunks
    int chunks;                   // of 256 columns
    int* err;
};

template <typename T, int BLOCK, bool SCALED>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(QuantArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int64_t live = p.seg ? p.seg[p.E] : p.rows;
    constexpr int LPB = BLOCK / 8;                           // lanes a block
    const int atoms = p.d / BLOCK / 4;                       // 512-byte scale tiles across a row tile
    for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < p.items; w += warps) {
        const int64_t slot = w / p.chunks;                   // 32 per row tile
        const int c = (int)(w - slot * p.chunks) * 256 + lane * 8;
        const int64_t r0 = (slot >> 5) * 128 + (slot & 31);
        if ((slot >> 5) * 128 >= live) break;                // (w ascends)
        const bool in_row = c < p.d;
        float v[4][8];
        bool has[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int64_t row = r0 + 32 * a;
            has[a] = in_row && row < live && row < p.rows;
            int64_t src = row;
            if (has[a] && p.perm) src = p.perm[row];
            const bool real = has[a] && src >= 0 && src < p.n;
            if (has[a] && src >= p.n) clha_record_error(p.err, CLHA_ERR_INVALID_ARG, (int)(row & 0x7fffffff), (int)src, KID_FP4);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[a][i] = 0.f;
            if (real) load8<T>(reinterpret_cast<const T*>(p.X) + src * p.d + c, v[a]);
        }
        uint32_t sb[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int64_t row = r0 + 32 * a;
            float g = 1.f;
            if (SCALED) {
                if (has[a]) g = __ldg(p.g + row / p.rows_per_g);
                if (!(g > 0.f && g < INFINITY)) {
                    clha_record_error(p.err, CLHA_ERR_INVALID_ARG, (int)(row & 0x7fffffff), 0, KID_FP4);
                    g = 1.f;
                }
            }
            // outside this range a reciprocal may be subnormal and short of bits: NaN sends every decision to float64
            const float rg = !SCALED ? 1.f : g > 0x1p-100f && g < 0x1p100f ? 1.f / g : NAN;
            const float r6g = rg * (1.f / 6.f);
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(v[a][i]));
#pragma unroll
            for (int o = 1; o < LPB; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            uint32_t q;
            if (!(top < INFINITY)) {                         // the same decision in all lanes of the block
                clha_record_error(p.err, CLHA_ERR_NONFINITE, (int)(row & 0x7fffffff), c, KID_FP4);
                sb[a] = BLOCK == 32 ? 0xff : 0x7f;           // the formats' NaN
                q = 0;
            } else {
                float r;
                sb[a] = block_scale<BLOCK, SCALED>(top, g, rg, r6g, &r);
                float lo[8];
                if (BLOCK == 32 && !SCALED) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) lo[i] = v[a][i] * r;
                    q = e2m1x8(lo);
                } else {
                    float hi[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float t = v[a][i] * r;
                        lo[i] = t * kLo;
                        hi[i] = t * kHi;
                    }
                    q = e2m1x8(lo);
                    if (q != e2m1x8(hi) || (r != 0.f && !(r > 0x1p-100f && r < 0x1p100f))) {
                        const double dd = (BLOCK == 32 ? ldexp(1.0, (int)sb[a] - 127) : (double)from_e4m3(sb[a])) * (double)g;
                        q = 0;
                        if (dd > 0.0)
#pragma unroll
                            for (int i = 0; i < 8; ++i) q |= e2m1_exact(v[a][i], dd) << (4 * i);
                    }
                }
            }
            if (has[a]) __stcs(reinterpret_cast<uint32_t*>(p.codes + row * (p.d / 2) + c / 2), q);
            if (!has[a]) sb[a] = 0;
            // the four blocks of this lane's scale cell, one byte each
            const int kb = (lane / LPB) & 3;
            uint32_t word = sb[a] << (8 * kb);
            word |= __shfl_xor_sync(0xffffffffu, word, LPB);
            word |= __shfl_xor_sync(0xffffffffu, word, 2 * LPB);
            sb[a] = word;
        }
        if (in_row && lane % (4 * LPB) == 0)
            *reinterpret_cast<uint4*>(p.scales + (((slot >> 5) * atoms + c / (4 * BLOCK)) * 32 + (slot & 31)) * 16) =
                make_uint4(sb[0], sb[1], sb[2], sb[3]);
    }
}

template <typename T, int BLOCK>
cudaError_t launch_q(cudaStream_t s, int num_sms, const QuantArgs& p) {
    int64_t blocks = (p.items + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > (int64_t)num_sms * 32) blocks = (int64_t)num_sms * 32;
    if (p.g)
        fp4_quantize_kernel<T, BLOCK, true><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    else
        fp4_quantize_kernel<T, BLOCK, false><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    clha_note_launches(1);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------ decoding
// q s g rounded once: q s is exact (6 bits) and float32's product with g is one rounding. A bfloat16 result
// rounds the product towards zero first and keeps a sticky bit, so that it too is rounded once.
__device__ __forceinline__ uint32_t bf16_once(float v, float g) {
    float t = __fmul_rz(v, g);
    if (__fmaf_rn(v, g, -t) != 0.f) t = __uint_as_float(__float_as_uint(t) | 1u);
    return __bfloat16_as_ushort(__float2bfloat16_rn(t));
}

template <int BLOCK, bool F32>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, int64_t rows, int d,
                                                                  const float* __restrict__ g, int64_t rows_per_g,
                                                                  int64_t items, int chunks, void* __restrict__ out) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int atoms = d / BLOCK / 4;
    for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < items; w += warps) {
        const int64_t slot = w / chunks;
        const int c = (int)(w - slot * chunks) * 256 + lane * 8;
        const int64_t r0 = (slot >> 5) * 128 + (slot & 31);
        if (c >= d) continue;
        uint32_t q[4] = {};
        const uint4 sv = __ldg(reinterpret_cast<const uint4*>(
            scales + (((slot >> 5) * atoms + c / (4 * BLOCK)) * 32 + (slot & 31)) * 16));
        const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int a = 0; a < 4; ++a)
            if (r0 + 32 * a < rows) q[a] = __ldcs(reinterpret_cast<const uint32_t*>(codes + (r0 + 32 * a) * (d / 2) + c / 2));
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int64_t row = r0 + 32 * a;
            if (row >= rows) break;
            const uint32_t byte = (sw[a] >> (8 * ((c / BLOCK) & 3))) & 0xff;
            float s;
            if (BLOCK == 32)
                s = byte == 0xff ? __uint_as_float(0x7fffffffu) : pow2_byte(byte);
            else
                s = byte == 0x7f ? __uint_as_float(0x7fffffffu) : from_e4m3(byte & 0x7f);
            const float gr = g ? __ldg(g + row / rows_per_g) : 1.f;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // e2m1: eem -> the number with exponent and mantissa bits in place, scaled by 2^126
                const uint32_t code = q[a] >> (4 * i);
                const uint32_t mag = code & 7;
                const float m = mag < 2 ? 0.5f * (float)mag : __uint_as_float(((mag >> 1) + 126) << 23 | (mag & 1) << 22);
                v[i] = __uint_as_float(__float_as_uint(m) | (code & 8) << 28) * s;
            }
            if (F32) {
                float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + row * d + c);
                __stcs(o, make_float4(v[0] * gr, v[1] * gr, v[2] * gr, v[3] * gr));
                __stcs(o + 1, make_float4(v[4] * gr, v[5] * gr, v[6] * gr, v[7] * gr));
            } else {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = bf16_once(v[2 * i], gr) | bf16_once(v[2 * i + 1], gr) << 16;
                __stcs(reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + row * d + c),
                       make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
}

// ------------------------------------------------------------------------------ matrix scale
// max|x| as bits (ordered like the magnitudes; NaN above infinity), one atomic a block: order-free.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp4_amax_kernel(const T* __restrict__ X, int64_t per, uint32_t* __restrict__ top) {
    const T* x = X + (int64_t)blockIdx.y * per;
    uint32_t m = 0;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8; i < per; i += (int64_t)gridDim.x * kThreads * 8) {
        float v[8];
        load8<T>(x + i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0 && m) atomicMax(top + blockIdx.y, m);
}

__global__ void fp4_finish_scale_kernel(uint32_t* top, int batch, float largest, int* err) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= batch) return;
    const uint32_t m = top[b];
    if (m >= 0x7f800000u) clha_record_error(err, CLHA_ERR_NONFINITE, b, 0, KID_FP4);
    const float g = __uint_as_float(m) / largest;
    reinterpret_cast<float*>(top)[b] = m < 0x7f800000u && g > 0.f ? g : 1.f;
}

}  // namespace

cudaError_t launch_fp4_quantize(cudaStream_t s, int num_sms, const void* X, int x_f32, int64_t n, int d,
                                const int32_t* perm, int64_t rows, const int64_t* seg, int E, int block, const float* g,
                                int64_t rows_per_g, uint8_t* codes, uint8_t* scales, int* err) {
    QuantArgs p{X, n, rows, d, perm, seg, E, g, rows_per_g, codes, scales, 0, (d + 255) / 256, err};
    p.items = (rows + 127) / 128 * 32 * p.chunks;
    if (x_f32) return block == 32 ? launch_q<float, 32>(s, num_sms, p) : launch_q<float, 16>(s, num_sms, p);
    return block == 32 ? launch_q<__nv_bfloat16, 32>(s, num_sms, p) : launch_q<__nv_bfloat16, 16>(s, num_sms, p);
}

cudaError_t launch_fp4_dequantize(cudaStream_t s, int num_sms, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                  int d, int block, const float* g, int64_t rows_per_g, void* out, int out_f32) {
    const int chunks = (d + 255) / 256;
    const int64_t items = (rows + 127) / 128 * 32 * chunks;
    int64_t blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > (int64_t)num_sms * 32) blocks = (int64_t)num_sms * 32;
#define CLHA_DQ(B, F) \
    fp4_dequantize_kernel<B, F><<<(unsigned)blocks, kThreads, 0, s>>>(codes, scales, rows, d, g, rows_per_g, items, chunks, out)
    if (block == 32) {
        if (out_f32) CLHA_DQ(32, true); else CLHA_DQ(32, false);
    } else {
        if (out_f32) CLHA_DQ(16, true); else CLHA_DQ(16, false);
    }
#undef CLHA_DQ
    clha_note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_fp4_tensor_scale(cudaStream_t s, int num_sms, const void* X, int x_f32, int batch, int64_t per,
                                    int block, float* scale, int* err) {
    cudaError_t e = cudaMemsetAsync(scale, 0, (size_t)batch * sizeof(float), s);
    if (e != cudaSuccess) return e;
    if (per) {
        int64_t blocks = (per + kThreads * 8 * 4 - 1) / (kThreads * 8 * 4);
        const int64_t most = ((int64_t)num_sms * 8 + batch - 1) / batch;
        if (blocks > most) blocks = most;
        const dim3 grid((unsigned)blocks, (unsigned)batch);
        if (x_f32)
            fp4_amax_kernel<float><<<grid, kThreads, 0, s>>>((const float*)X, per, (uint32_t*)scale);
        else
            fp4_amax_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>((const __nv_bfloat16*)X, per, (uint32_t*)scale);
        clha_note_launches(1);
    }
    // the largest value of the format: 6 times the largest scale that a block of it may take
    fp4_finish_scale_kernel<<<(batch + 127) / 128, 128, 0, s>>>((uint32_t*)scale, batch, block == 16 ? 6.f * 448.f : 6.f, err);
    clha_note_launches(1);
    return cudaGetLastError();
}
