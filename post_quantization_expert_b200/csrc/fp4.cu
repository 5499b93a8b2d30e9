// Microscaled 4-bit floating point: quantization, decoding and the matrix scale.
//
// A row is cut into blocks of 32 (power-of-two e8m0 scales) or 16 (e4m3 scales). With g the float32 scale
// of the matrix (1 where there is none), a block's scale s and its codes q are
//   e8m0   s = 2^(floor(log2(max|x| / g)) - 2)          (2 = the exponent of e2m1's largest number, 6)
//   e4m3   s = max|x| / (6 g) rounded to nearest even, 2^-9 <= s <= 448 (0 for a block of zeros)
//   q = x / (s g) rounded to the nearest e2m1 number, ties to the even code, saturating at +-6,
// all of it decided as if in exact arithmetic. Divisions make that more than one float32 operation: the
// quotient t is formed with reciprocals (relative error below 2^-21.9), t (1 - 2^-21) and t (1 + 2^-21)
// are both rounded, and only where the two differ the lane decides again in float64, where a quotient of a 24-bit by
// a 28-bit number cannot round onto a border that it is not on (borders have at most 5 bits, so x and border * s * g differ
// by 2^-33 of their size or not at all). How often that is, counted over normal numbers: one block in 10^4 to 10^5 of
// float32; of bfloat16, whose 8 bits put many values exactly on a border of e4m3 scales, one block in 6 without a matrix
// scale and one in some 30 with one (none under power-of-two scales).
// A power-of-two scale without g needs no quotient: x times a power of two is exact.
//
// Both kernels stream. Eight lanes take 128 columns, 16 a lane (32 bytes of bf16 in one access, 8 bytes of
// codes), of the four rows r, r + 32, r + 64, r + 96 of a 128-row tile: four loads in flight a lane, and the
// scales of four blocks of those rows are 16 consecutive bytes of the tiled layout (the lanes transpose 4 x 4
// bytes by two exchanges and store 4 bytes each). A block is one lane (16) or two (32). 32768 tokens x 2048 of bf16 into
// the segments of 64 experts, top 6, under power-of-two scales take 130 us against 53 us for the bytes: 97 M warp
// instructions in 64 % of the issue slots, half of the warps that an SM can hold, and each token decided once for each
// of its experts (8 columns a lane and a 64-bit division a step took 285 us, routed rows as they lie 142 us, runs of 512
// columns a unit 140 us). Every other variant does more for a block: float32 203 us; a matrix scale 302 us (a division of
// the row's number and a reciprocal stand in the column loop); e4m3 scales 264 us over float32, and over bf16 1148 us, or
// 433 us with a matrix scale: the float64 decisions above. Decoding to bf16 is bound by memory: 167 us, 93 % of the measured
// copy bandwidth.
#include "clha_internal.h"

#include <cuda_fp16.h>

namespace {

constexpr float kLo = 1.f - 0x1p-21f, kHi = 1.f + 0x1p-21f;
constexpr int kThreads = 256;

// Eight e2m1 codes of v[0..7], v[0] in the low bits.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
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
// The eight numbers of a word of codes, as four pairs of halves (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t q, __half2 (&v)[4]) {
    uint32_t o[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(q));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<__half2*>(&o[i]);
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
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ------------------------------------------------------------------ exact decisions
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

// 32 bytes at a time: one access where the address is a multiple of 32 (`wide`), two where it is one of 16.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Sixteen columns as they lie in memory, and as floats.
template <typename T>
struct Raw {
    static constexpr int N = (int)sizeof(T) / 2;             // accesses of 32 bytes
    uint32_t w[N][8];
    __device__ __forceinline__ void load(const T* p, bool wide) {
#pragma unroll
        for (int i = 0; i < N; ++i) load32(reinterpret_cast<const char*>(p) + 32 * i, wide, w[i]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) w[i][j] = 0;
    }
    __device__ __forceinline__ float at(int i) const {       // i a constant once unrolled
        if (sizeof(T) == 4) return __uint_as_float(w[i >> 3 & (N - 1)][i & 7]);
        return __uint_as_float(i & 1 ? w[0][i >> 1] & 0xffff0000u : w[0][i >> 1] << 16);
    }
    // The largest magnitude; NaN if there is one.
    __device__ __forceinline__ float largest() const {
        if (sizeof(T) == 2) {                                // two columns an instruction, signs combined as they come
            uint32_t m = w[0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[0][i]));
            return max_nan(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xffff0000u)));
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max_nan(m, fabsf(at(i)));
        return m;
    }
    // Columns 8 h .. 8 h + 7 times r. A power of two leaves a bfloat16 exact (or far below the smallest code): two
    // products an instruction, before they are taken apart.
    __device__ __forceinline__ void times(int h, float r, bool pow2, float (&t)[8]) const {
        if (sizeof(T) == 2 && pow2) {
            const __nv_bfloat162 rr = __float2bfloat162_rn(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t v = w[0][4 * h + i];
                const __nv_bfloat162 m = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&v), rr);
                v = *reinterpret_cast<const uint32_t*>(&m);
                t[2 * i] = __uint_as_float(v << 16);
                t[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = at(8 * h + i) * r;
        }
    }
};

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

// The work items: 128 columns of four rows, item = slot * chunks + chunk with 32 slots a 128-row tile. Eight
// lanes take one, and go on in steps of all groups of eight; no division after the first item.
struct Items {
    int64_t slot;
    int chunk;
    int64_t step_slot;
    int step_chunk, chunks;
    __device__ __forceinline__ Items(int chunks_) : chunks(chunks_) {
        const int64_t groups = (int64_t)gridDim.x * (kThreads / 8);
        const int64_t id = (int64_t)blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3);
        slot = id / chunks;
        chunk = (int)(id - slot * chunks);
        step_slot = groups / chunks;
        step_chunk = (int)(groups - step_slot * chunks);
    }
    __device__ __forceinline__ void next() {
        slot += step_slot;
        chunk += step_chunk;
        if (chunk >= chunks) { chunk -= chunks; ++slot; }
    }
};

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
    int wide;                     // X is 32-byte aligned
    int bands;                    // 1: row tiles as they lie
    int run;                      // columns of a work unit
    int* err;
};

// Routed rows of a large X in the order of its tokens: a token's rows lie in k segments, so that row tiles taken as
// they lie read X from DRAM once for each (of 726 MB moved for 32768 tokens x 2048 in six experts each, 134 were X once).
// Segments list their tokens in ascending order: the tiles are taken in bands, first the first 1 / bands of every
// segment, and a band's share of X stays in L2. before[b E + e]: the tiles before band b of expert e.
constexpr int kBandEntries = 2048;
__device__ void band_table(const QuantArgs& p, int* before) {
    __shared__ int sums[kThreads];
    const int entries = p.bands * p.E, per = (entries + kThreads - 1) / kThreads;
    const int lo = threadIdx.x * per, hi = min(entries, lo + per);
    int sum = 0;
    for (int i = lo; i < hi; ++i) {
        const int b = i / p.E, e = i - b * p.E;
        const int64_t tiles = (p.seg[e + 1] - p.seg[e]) >> 7;
        before[i] = sum;
        sum += (int)(tiles * (b + 1) / p.bands - tiles * b / p.bands);
    }
    sums[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
        const int v = threadIdx.x >= o ? sums[threadIdx.x - o] : 0;
        __syncthreads();
        sums[threadIdx.x] += v;
        __syncthreads();
    }
    for (int i = lo; i < hi; ++i) before[i] += sums[threadIdx.x] - sum;
    __syncthreads();
}
// The row tile that is taken w-th.
__device__ __forceinline__ int64_t banded(const QuantArgs& p, const int* before, int64_t w) {
    int lo = 0, hi = p.bands * p.E - 1;
    while (lo < hi) {                                        // the last entry with before <= w (empty ones share theirs)
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= w) lo = mid; else hi = mid - 1;
    }
    const int b = lo / p.E, e = lo - b * p.E;
    const int64_t first = p.seg[e] >> 7, tiles = (p.seg[e + 1] >> 7) - first;
    return first + tiles * b / p.bands + (w - before[lo]);
}

template <typename T, int BLOCK, bool SCALED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) fp4_quantize_kernel(QuantArgs p) {
    clha_allow_next();
    clha_wait_inputs();
    const int sub = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int64_t live = p.seg ? min(p.seg[p.E], p.rows) : p.rows;
    constexpr int LPB = BLOCK / 16;                          // lanes a block
    const int atoms = p.d / BLOCK / 4;                       // 512-byte scale tiles across a row tile
    extern __shared__ int before[];
    const bool in_bands = p.bands > 1 && p.seg[p.E] <= p.rows;   // (segments that `rows` cuts off: tiles as they lie)
    if (in_bands) band_table(p, before);
    // a unit: the 128 rows of a tile, rows r, r + 32, r + 64, r + 96 to eight lanes, by p.run columns
    const int runs = (p.d + p.run - 1) / p.run;
    for (int64_t u = blockIdx.x;; u += gridDim.x) {
        int64_t tile = u / runs;
        const int c0 = (int)(u - tile * runs) * p.run, c1 = min(p.d, c0 + p.run);
        if (tile * 128 >= live) break;
        if (in_bands) tile = banded(p, before, tile);
        const int64_t r0 = tile * 128 + r;
        const T* src[4];                                       // null: a row of zeros
        uint8_t* dst[4];                                       // null: behind the last row
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int64_t row = r0 + 32 * a;
            const bool has = row < live;
            int64_t at = has ? row : -1;
            if (has && p.perm) at = p.perm[row];
            if (at >= p.n) {
                clha_record_error(p.err, CLHA_ERR_INVALID_ARG, (int)(row & 0x7fffffff), (int)at, KID_FP4);
                at = -1;
            }
            src[a] = at >= 0 ? reinterpret_cast<const T*>(p.X) + at * p.d : nullptr;
            dst[a] = has ? p.codes + row * (p.d >> 1) : nullptr;
        }
        for (int c = c0 + sub * 16; c < c1; c += 128) {
            Raw<T> x[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                if (src[a])
                    x[a].load(src[a] + c, p.wide);
                else
                    x[a].zero();
            }
            uint32_t sb = 0;                                     // the four rows' scale bytes of this lane's block
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int64_t row = r0 + 32 * a;
                float g = 1.f;
                if (SCALED) {
                    if (dst[a]) g = __ldg(p.g + row / p.rows_per_g);
                    if (!(g > 0.f && g < INFINITY)) {
                        clha_record_error(p.err, CLHA_ERR_INVALID_ARG, (int)(row & 0x7fffffff), 0, KID_FP4);
                        g = 1.f;
                    }
                }
                // outside this range a reciprocal may be subnormal and short of bits: NaN sends every decision to float64
                const float rg = !SCALED ? 1.f : g > 0x1p-100f && g < 0x1p100f ? 1.f / g : NAN;
                const float r6g = rg * (1.f / 6.f);
                float top = x[a].largest();
                if (LPB == 2) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
                uint32_t q[2] = {0u, 0u}, byte;
                if (!(top < INFINITY)) {                         // the same decision in both lanes of a block
                    clha_record_error(p.err, CLHA_ERR_NONFINITE, (int)(row & 0x7fffffff), c, KID_FP4);
                    byte = BLOCK == 32 ? 0xff : 0x7f;            // the formats' NaN
                } else {
                    float r;
                    byte = block_scale<BLOCK, SCALED>(top, g, rg, r6g, &r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float t[8];
                        x[a].times(h, r, BLOCK == 32 && !SCALED, t);
                        q[h] = e2m1x8(t);
                        if (BLOCK == 32 && !SCALED) continue;
                        float lo[8], hi[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            lo[i] = t[i] * kLo;
                            hi[i] = t[i] * kHi;
                        }
                        if (e2m1x8(lo) != e2m1x8(hi) || (r != 0.f && !(r > 0x1p-100f && r < 0x1p100f))) {
                            const double dd = (BLOCK == 32 ? ldexp(1.0, (int)byte - 127) : (double)from_e4m3(byte)) * (double)g;
                            q[h] = 0;
                            if (dd > 0.0)
#pragma unroll
                                for (int i = 0; i < 8; ++i) q[h] |= e2m1_exact(x[a].at(8 * h + i), dd) << (4 * i);
                        }
                    }
                }
                if (dst[a]) {
                    *reinterpret_cast<uint2*>(dst[a] + (c >> 1)) = make_uint2(q[0], q[1]);
                    sb |= byte << (8 * a);
                }
            }
            // lane b of a tile's four blocks holds the bytes of rows 0..3 (32 apart); exchange: it gets row b's four blocks
            const int b = sub / LPB & 3;
            uint32_t o = __shfl_xor_sync(0xffffffffu, sb, LPB);
            sb = b & 1 ? __byte_perm(sb, o, 0x3715) : __byte_perm(sb, o, 0x6240);
            o = __shfl_xor_sync(0xffffffffu, sb, 2 * LPB);
            sb = b & 2 ? __byte_perm(sb, o, 0x3276) : __byte_perm(sb, o, 0x5410);
            if (LPB == 1 || !(sub & 1))
                *reinterpret_cast<uint32_t*>(p.scales + ((tile * atoms + c / (4 * BLOCK)) * 32 + r) * 16 + 4 * b) = sb;
        }
    }
}

// Blocks for `items` of eight lanes, 128 for each SM at most: short blocks that follow one another keep the memory
// evenly busy to the end (196608 x 2048: 167 us; 8 blocks for each SM 189 us, 32 175 us, 512 167 us).
unsigned item_blocks(int64_t items, int num_sms) {
    const int64_t blocks = (items + kThreads / 8 - 1) / (kThreads / 8), most = (int64_t)num_sms * 128;
    return (unsigned)(blocks < most ? blocks : most);
}

template <typename T, int BLOCK>
cudaError_t launch_q(cudaStream_t s, int num_sms, const QuantArgs& p) {
    const int64_t units = (p.rows + 127) / 128 * ((p.d + p.run - 1) / p.run), most = (int64_t)num_sms * (sizeof(T) == 2 ? 4 : 2);
    const unsigned blocks = (unsigned)(units < most ? units : most);
    cudaError_t e = clha_launch_overlapped(p.g ? fp4_quantize_kernel<T, BLOCK, true> : fp4_quantize_kernel<T, BLOCK, false>,
                                           blocks, kThreads, p.bands > 1 ? p.bands * p.E * 4 : 0, s, 1, p);
    if (e != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------ decoding
// q s g rounded once: q s is exact (6 bits) and float32's product with g is one rounding. Under the two largest
// power-of-two scales q s may pass float32's range where q s g does not: a quarter of s then meets four times g,
// both exact (for |g| >= 1 the value overflows with q s). A bfloat16 result rounds the product towards zero first and
// keeps a sticky bit, so that it too is rounded once (without g it is exact). What the rounding towards zero cut off
// may lie below 2^-149, float32's smallest number, where the product is below 2^-120: it is looked at 2^64 times as
// large there. (A product cut off to zero is zero in bfloat16 too.)
__device__ __forceinline__ float sticky(float v, float g) {
    const float t = __fmul_rz(v, g);
    float u = t;
    if (fabsf(t) < 0x1p-100f && t != 0.f) {
        u *= 0x1p64f;
        if (fabsf(v) > 1.f) g *= 0x1p64f; else v *= 0x1p64f;   // |v| > 1: |g| < 2^-100
    }
    return __fmaf_rn(v, g, -u) != 0.f ? __uint_as_float(__float_as_uint(t) | 1u) : t;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    return r;
}

template <int BLOCK, bool F32, bool SCALED>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, int64_t rows, int d,
                                                                  const float* __restrict__ g, int64_t rows_per_g,
                                                                  int wide, void* __restrict__ out) {
    clha_allow_next();
    clha_wait_inputs();
    const int sub = threadIdx.x & 7;
    const int64_t slots = (rows + 127) / 128 * 32;
    const int atoms = d / BLOCK / 4;
    for (Items it(d >> 7); it.slot < slots; it.next()) {
        const int64_t r0 = (it.slot >> 5) * 128 + (it.slot & 31);
        const int c = it.chunk * 128 + sub * 16;
        uint2 q[4];
        const uint4 sv = __ldg(reinterpret_cast<const uint4*>(
            scales + (((it.slot >> 5) * atoms + c / (4 * BLOCK)) * 32 + (it.slot & 31)) * 16));
        const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            q[a] = make_uint2(0, 0);
            if (r0 + 32 * a < rows)
                q[a] = __ldg(reinterpret_cast<const uint2*>(codes + (r0 + 32 * a) * (d >> 1) + (c >> 1)));
        }
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int64_t row = r0 + 32 * a;
            if (row >= rows) break;
            const uint32_t byte = sw[a] >> (8 * (c / BLOCK & 3)) & 0xff;
            float s;
            if (BLOCK == 32)
                s = byte == 0xff ? NAN : pow2_byte(byte);
            else
                s = byte == 0x7f ? NAN : from_e4m3(byte & 0x7f);
            float gr = SCALED ? __ldg(g + row / rows_per_g) : 1.f;
            if (BLOCK == 32 && SCALED && byte >= 253 && byte != 0xff && fabsf(gr) < 1.f) {
                s *= 0.25f;
                gr *= 4.f;
            }
            float v[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __half2 m[4];
                from_e2m1x8(h ? q[a].y : q[a].x, m);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __half22float2(m[i]);
                    v[8 * h + 2 * i] = f.x * s;
                    v[8 * h + 2 * i + 1] = f.y * s;
                }
            }
            uint32_t o[8];
            if (F32) {
                float* y = reinterpret_cast<float*>(out) + row * d + c;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(SCALED ? v[8 * h + i] * gr : v[8 * h + i]);
                    store32(y + 8 * h, wide, o);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = SCALED ? pack_bf16(sticky(v[2 * i], gr), sticky(v[2 * i + 1], gr))
                                  : pack_bf16(v[2 * i], v[2 * i + 1]);
                store32(reinterpret_cast<__nv_bfloat16*>(out) + row * d + c, wide, o);
            }
        }
    }
}

// ------------------------------------------------------------------------------ matrix scale
// max|x| as bits (ordered like the magnitudes; NaN above infinity), one atomic a block: order-free.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp4_amax_kernel(const T* __restrict__ X, int64_t per, int wide, uint32_t* __restrict__ top) {
    const T* x = X + (int64_t)blockIdx.y * per;
    uint32_t m = 0;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 16; i < per; i += (int64_t)gridDim.x * kThreads * 16) {
        Raw<T> v;
        v.load(x + i, wide);
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v.at(j)) & 0x7fffffffu);
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
    // bands of X of at most 24 MB, where that leaves something to gain
    const int64_t bytes = n * d * (x_f32 ? 4 : 2), want = (bytes + (24 << 20) - 1) / (24 << 20);
    int bands = 1;
    if (perm && seg && rows > n) {                            // (E is in 1..1024 then)
        const int most = kBandEntries / E < 8 ? kBandEntries / E : 8;
        bands = (int)(want < most ? want : most);
        if (bands < 1) bands = 1;
    }
    // long runs save work for each row; a few thousand units keep every SM busy
    int run = 1024;
    while (run > 128 && (rows + 127) / 128 * ((d + run - 1) / run) < (int64_t)num_sms * 16) run /= 2;
    const QuantArgs p{X,     n,      rows, d,  perm, seg, E, g, rows_per_g, codes, scales, ((uintptr_t)X & 31) == 0,
                      bands, run, err};
    if (x_f32) return block == 32 ? launch_q<float, 32>(s, num_sms, p) : launch_q<float, 16>(s, num_sms, p);
    return block == 32 ? launch_q<__nv_bfloat16, 32>(s, num_sms, p) : launch_q<__nv_bfloat16, 16>(s, num_sms, p);
}

cudaError_t launch_fp4_dequantize(cudaStream_t s, int num_sms, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                  int d, int block, const float* g, int64_t rows_per_g, void* out, int out_f32) {
    const unsigned blocks = item_blocks((rows + 127) / 128 * 32 * (d >> 7), num_sms);
    const int wide = ((uintptr_t)out & 31) == 0;
    const auto kernel = [&] {
        if (block == 32) {
            if (out_f32) return g ? fp4_dequantize_kernel<32, true, true> : fp4_dequantize_kernel<32, true, false>;
            return g ? fp4_dequantize_kernel<32, false, true> : fp4_dequantize_kernel<32, false, false>;
        }
        if (out_f32) return g ? fp4_dequantize_kernel<16, true, true> : fp4_dequantize_kernel<16, true, false>;
        return g ? fp4_dequantize_kernel<16, false, true> : fp4_dequantize_kernel<16, false, false>;
    }();
    cudaError_t e = clha_launch_overlapped(kernel, blocks, kThreads, 0, s, 1, codes, scales, rows, d, g, rows_per_g, wide, out);
    if (e != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_fp4_tensor_scale(cudaStream_t s, int num_sms, const void* X, int x_f32, int batch, int64_t per,
                                    int block, float* scale, int* err) {
    cudaError_t e = cudaMemsetAsync(scale, 0, (size_t)batch * sizeof(float), s);
    if (e != cudaSuccess) return e;
    if (per) {
        int64_t blocks = (per + kThreads * 16 * 2 - 1) / (kThreads * 16 * 2);
        const int64_t most = ((int64_t)num_sms * 8 + batch - 1) / batch;
        if (blocks > most) blocks = most;
        const dim3 grid((unsigned)blocks, (unsigned)batch);
        const int wide = ((uintptr_t)X & 31) == 0;             // (every matrix then is: per is a multiple of 128)
        if (x_f32)
            fp4_amax_kernel<float><<<grid, kThreads, 0, s>>>((const float*)X, per, wide, (uint32_t*)scale);
        else
            fp4_amax_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>((const __nv_bfloat16*)X, per, wide, (uint32_t*)scale);
        clha_note_launches(1);
    }
    // the largest value of the format: 6 times the largest scale that a block of it may take
    fp4_finish_scale_kernel<<<(batch + 127) / 128, 128, 0, s>>>((uint32_t*)scale, batch, block == 16 ? 6.f * 448.f : 6.f, err);
    clha_note_launches(1);
    return cudaGetLastError();
}
