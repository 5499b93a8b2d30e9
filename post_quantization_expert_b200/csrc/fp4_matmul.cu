// Products of microscaled 4-bit operands on the tensor cores: Y = X W^T, and the experts' gate/up pair
// h = SiLU(X Wg^T) * (X Wu^T), dense or over routed segments.
//
// tcgen05.mma multiplies e2m1 values and applies both operands' block scales, accumulating in float32;
// the matrix scales multiply the finished sums in the epilogue. Two kernels: pairs of SMs on large tiles (further
// down), bound by the tensor pipe under the power limit (28672 -> 8192 on 16384 tokens: 1.6 to 1.7 ms, 4.5 to 4.8
// PFLOP/s), and one for few rows, bound by reading W (1 token of the same: 25 us, the same weights again or four sets in
// turn, 80 % of the measured copy bandwidth); launch_product chooses. Segments start at multiples of 128, so a tile never
// mixes experts. Rows of a segment behind its tokens are written as zero; rows behind the last segment are not touched.
//
// Few rows. The tensor core's 128-row operand is W (for gate and up a block of each), its other operand the
// tile's rows of X, as many as hold tokens, in steps of 16: a decoding step pays for 16 rows, not for 128,
// and more of shared memory is left for W's copies in flight.
//   warp 0       TMA producer: per 256 columns of K, 128 bytes a row of W and of X (128-byte swizzle) and
//                their scale tiles (512 bytes for 128 rows x 4 blocks, copied as they lie).
//   warp 1       copies the stage's scale tiles to TMEM (its own columns for each stage, so that the stage's
//                barriers also order their reuse) and issues the products of 64 columns of K each.
//   warps 2-9    epilogue: two warps for each TMEM lane quadrant (32 columns of Y), rows in turns.
// Warp 1 runs its loop as a whole and one elected lane issues: its instructions' operands are then uniform
// registers. Issued under `if (lane == 0)`, a stage of the large tiles took 730 cycles to issue, whatever the
// products' size, and a scale copy about 60, so that extra warps for the copies paid (28672 -> 8192 on 16384
// tokens: 2.35 ms, 1.73 ms with two warps for the copies, 1.58 ms issued this way, with or without those warps).
// With few tiles, `split` CTAs of a cluster share one tile's K range and add their parts through distributed
// shared memory, in rank order, so that the result does not depend on timing.
#include "clha_internal.h"
#include "tc_ptx.h"
#include "tmap.h"

#include <cfloat>

namespace {

constexpr int kThreads = 320;
constexpr int BKB = 128;                        // bytes of K a stage (256 columns)
constexpr int TILE_BYTES = 128 * BKB;           // 16 KB: 128 rows of a stage
constexpr int MAX_SMEM = 232448;
constexpr int kMaxE = 1024;

// NB blocks of W (2: gate and up), at most XR rows of X a tile
template <int BLOCK, int NB, int XR>
struct Cfg {
    static constexpr int APS = 256 / BLOCK / 4;              // scale tiles of 512 bytes a stage and 128 rows
    static constexpr int SF_BYTES = APS * 512;
    static constexpr int STAGE_BYTES = NB * TILE_BYTES + XR * BKB + (NB + 1) * SF_BYTES;
    static constexpr int ACCS = NB == 1 || XR < 128 ? 2 : 1; // accumulators of NB * XR columns
    static constexpr int SF_COLS = APS * 4 * (1 + NB);       // TMEM columns of a stage's scales
    static constexpr int SF_BASE = ACCS * NB * XR;
    static constexpr int SEG_BYTES = XR < 128 ? 0 : (2 * kMaxE + 2) * 4;   // (fewer than 128 rows: dense)
    static constexpr int CTAS = NB == 1 && XR < 128 ? 2 : 1; // of an SM
    static constexpr int TCOLS = 512 / CTAS;                 // TMEM columns of a CTA
    static constexpr int FIT = (MAX_SMEM / CTAS - 1024 * CTAS - SEG_BYTES - 512) / STAGE_BYTES;
    static constexpr int TFIT = (TCOLS - SF_BASE) / SF_COLS;
    static constexpr int STAGES = FIT < TFIT ? FIT : TFIT;
    static constexpr int SEG_OFF = STAGES * STAGE_BYTES;
    static constexpr int BAR_OFF = SEG_OFF + SEG_BYTES;
    static constexpr int SMEM = BAR_OFF + 8 * (2 * STAGES + 2 * ACCS + 1) + 16 + 1024;
    static_assert((SMEM + 1024) * CTAS <= MAX_SMEM + 1024 && STAGES >= 4, "shared memory");
    static_assert(STAGE_BYTES % 1024 == 0 && BAR_OFF % 8 == 0, "alignment");
    static_assert(STAGES * STAGE_BYTES >= NB * XR * 128 * 4, "partial sums fit the stages");
};

struct MatmulArgs {
    int64_t rows;
    int K, N;                // columns of X; columns of Y (rows of one W)
    const int64_t* seg;      // null: one expert, all rows
    int E;
    const float* xg;         // matrix scales (null: 1): of X, and of each expert's W, Wu
    const float* wg;
    const float* ug;
    void* Y;
    int n_tiles;             // column tiles
    int split;               // CTAs of a cluster that share a tile's K
    int* err;
};

// SiLU(g) u = g / (1 + e^-g) u. With h = e^(-|g| / 2) it is g / (1 + h h) u, and g h / (1 + h h) (u h) for g < 0: nothing
// overflows or is flushed before |g| = 174, where h h u is below float32's range for any u. (1 + e^-g itself passes 2^126 at
// g = -87.4, and the fast division by more than that gives 0, while u may bring the value back.) Off by at most
// (1.5 |g| + 16) 2^-24 of its size: the exponent is rounded twice, h by two steps, six operations follow.
__device__ __forceinline__ float silu_mul(float g, float u) {
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(fabsf(g) * -0.72134752f));   // log2(e) / 2
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 1.f)));
    const float m = g < 0.f ? h : 1.f;
    return g * m * r * (u * m);
}

template <typename OUT>
__device__ __forceinline__ void store4(OUT* y, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void store4<float>(float* y, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(y) = make_float4(a, b, c, d);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    return r;
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* y, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
}
__device__ __forceinline__ void store1(float* y, float v) { *y = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// What the finished sums are multiplied by, first `pre`, then `by`: the product of X's and W's matrix scales, rounded once.
// pre is 1 unless that product leaves float32's normal range, where the scaled sums may well be inside it: pre takes half
// of its exponent then, so that neither step overflows or is flushed before the result is. Two sums an instruction, so
// that the second step costs no more than one step on single sums does.
struct MatrixScale {
    float pre, by;
    __device__ __forceinline__ MatrixScale(float x, float w) : pre(1.f), by(x * w) {
        if (fabsf(by) >= 0x1p-126f && fabsf(by) < INFINITY) return;
        const double p = (double)x * (double)w;
        if (!(fabs(p) < 0x1p256)) return;                          // (an Inf or NaN scale)
        const int h = max(-126, min(127, ((__double2hiint(p) >> 20 & 0x7ff) - 1023) / 2));
        pre = __int_as_float((h + 127) << 23);
        by = fmaxf(-FLT_MAX, fminf(FLT_MAX, (float)(p * __hiloint2double((1023 - h) << 20, 0))));
    }
    template <int N>
    __device__ __forceinline__ void apply(uint32_t (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
                "mul.rn.f32x2 a, a, b;\n\tmul.rn.f32x2 a, a, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
                : "+r"(v[i]), "+r"(v[i + 1]) : "f"(pre), "f"(by));
    }
};

// ------------------------------------------------------------------------------ few rows
struct Tile {
    int64_t m0;              // first row
    int n0, e;               // first column; expert
    int tokens, height;      // rows with a token; rows that are written
};

template <int BLOCK, int NB, int XR, typename OUT>
__global__ void __launch_bounds__(kThreads, Cfg<BLOCK, NB, XR>::CTAS)
fp4_matmul_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
                  const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWs,
                  const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmUs, MatmulArgs p) {
    using C = Cfg<BLOCK, NB, XR>;
    constexpr bool ACT = NB == 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* seg = reinterpret_cast<int*>(smem + C::SEG_OFF);          // starts [E + 1], then token counts [E]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    const uint32_t full0 = tc::smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * C::STAGES;
    const uint32_t tfull0 = empty0 + 8 * C::STAGES;      // accumulator a holds a finished tile
    const uint32_t tempty0 = tfull0 + 8 * C::ACCS;        // accumulator a has been read
    const uint32_t drain = tempty0 + 8 * C::ACCS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 2 * C::ACCS + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int no_abort = 0;                             // for the waits after an abort
    const int warp = tc::warp_index(), lane = threadIdx.x & 31;
    const int S = p.split;
    const int rank = S > 1 ? (int)tc::cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(full0 + 8 * s, 1);
            tc::mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < C::ACCS; ++a) {
            tc::mbar_init(tfull0 + 8 * a, 1);
            tc::mbar_init(tempty0 + 8 * a, 8);            // one arrival per epilogue warp
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::fence_barrier_init();
        tc::prefetch_tmap(&tmX);
        tc::prefetch_tmap(&tmXs);
        tc::prefetch_tmap(&tmW);
        tc::prefetch_tmap(&tmWs);
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_u32(tmem_slot), C::TCOLS);
    clha_allow_next();
    clha_wait_inputs();
    if (p.seg)
        for (int i = threadIdx.x; i <= 2 * p.E; i += kThreads) seg[i] = (int)p.seg[i];
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    const int64_t used = p.seg ? min((int64_t)seg[p.E], p.rows) : p.rows;
    const int64_t total = (used + XR - 1) / XR * p.n_tiles;        // (segments are tiled by 128 rows: XR = 128 then)
    const int64_t w0 = S > 1 ? blockIdx.x / S : blockIdx.x, stride = S > 1 ? gridDim.x / S : gridDim.x;
    const int nk = (p.K + 255) / 256;
    const int atoms = p.K / BLOCK / 4;                     // scale tiles across a row tile
    const int k_lo = (int)((int64_t)nk * rank / S), k_hi = (int)((int64_t)nk * (rank + 1) / S);
    // split > 1 runs one tile a cluster (the grid covers them all): the stages then hold the partial sums

    const auto tile = [&](int64_t w) {
        Tile t;
        t.m0 = w / p.n_tiles * XR;
        t.n0 = (int)(w % p.n_tiles) * 128;
        t.height = (int)min((int64_t)XR, used - t.m0);
        t.e = 0;
        t.tokens = t.height;
        if (p.seg) {
            int lo = 0, hi = p.E - 1;
            while (lo < hi) {                              // last e with seg[e] <= m0
                const int mid = (lo + hi + 1) >> 1;
                if (seg[mid] <= t.m0) lo = mid; else hi = mid - 1;
            }
            t.e = lo;
            t.tokens = max(0, min(t.height, seg[lo] + seg[p.E + 1 + lo] - (int)t.m0));
        }
        return t;
    };

    int issued = 0;                                        // producer: stages asked for
    if (warp == 0) {
        if (lane == 0) {
            int& it = issued;
            bool ok = true;
            for (int64_t w = w0; ok && w < total; w += stride) {
                const Tile t = tile(w);
                const int boxes = (t.tokens + 15) / 16;
                const int wr = t.e * p.N + t.n0;
                for (int kb = k_lo; kb < k_hi; ++kb, ++it) {
                    const int s = it % C::STAGES;
                    if (!tc::mbar_wait_bounded(empty0 + 8 * s, ((it / C::STAGES) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    const uint32_t fb = full0 + 8 * s;
                    tc::mbar_arrive_expect_tx(fb, NB * TILE_BYTES + boxes * 16 * BKB + (NB + 1) * C::SF_BYTES);
                    const uint32_t a = tc::smem_u32(smem + s * C::STAGE_BYTES);
                    const uint32_t b = a + NB * TILE_BYTES, sf = b + XR * BKB;
                    tc::tma_load_2d(a, &tmW, fb, kb * BKB, wr);
                    tc::tma_load_2d(sf, &tmWs, fb, 0, wr / 128 * atoms + kb * C::APS);
                    if (ACT) {
                        tc::tma_load_2d(a + TILE_BYTES, &tmU, fb, kb * BKB, wr);
                        tc::tma_load_2d(sf + C::SF_BYTES, &tmUs, fb, 0, wr / 128 * atoms + kb * C::APS);
                    }
                    tc::tma_load_2d(sf + NB * C::SF_BYTES, &tmXs, fb, 0, (int)(t.m0 / 128) * atoms + kb * C::APS);
                    for (int x = 0; x < boxes; ++x) tc::tma_load_2d(b + x * 16 * BKB, &tmX, fb, kb * BKB, (int)t.m0 + 16 * x);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool issuer = tc::elect_one();
        const uint64_t desc0 = tc::sw128_desc(tc::smem_u32(smem), 16, 1024);
        const uint64_t sdesc0 = tc::plain_desc(tc::smem_u32(smem) + NB * TILE_BYTES + XR * BKB);
        int s = 0, tcount = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int64_t w = w0; ok && w < total; w += stride, ++tcount) {
            const Tile t = tile(w);
            const uint32_t n16 = max(1, (t.tokens + 15) / 16);
            const uint32_t id0 = tc::idesc_fp4(BLOCK == 32, 128, n16 * 16, 0);
            const uint32_t id2 = tc::idesc_fp4(BLOCK == 32, 128, n16 * 16, 2);
            const int acc = tcount % C::ACCS;
            if (!tc::mbar_wait_warp(tempty0 + 8 * acc, ((tcount / C::ACCS) & 1) ^ 1, abort_flag)) { ok = false; break; }
            tc::fence_after_sync();
            const uint32_t d_tmem = tmem + acc * (NB * XR);
            for (int kb = k_lo; kb < k_hi; ++kb) {
                if (!tc::mbar_wait_warp(full0 + 8 * s, ph, abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
                const uint64_t ad = desc0 + (uint32_t)(s * (C::STAGE_BYTES >> 4)), xd = ad + (NB * TILE_BYTES >> 4);
                const uint32_t tw = tmem + C::SF_BASE + s * C::SF_COLS, tx = tw + NB * C::APS * 4;
                const uint64_t sd = sdesc0 + (uint32_t)(s * (C::STAGE_BYTES >> 4));
                const bool full_k = p.K - kb * 256 >= 256;             // else half: K is a multiple of 128
                if (issuer) {
#pragma unroll
                    for (int j = 0; j < (NB + 1) * C::APS; ++j) tc::tmem_copy_scales(tw + 4 * j, sd + j * 32);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= 2 && !full_k) break;
                        const int j = BLOCK == 16 ? kk : kk >> 1;
#pragma unroll
                        for (int x = 0; x < NB; ++x)
                            tc::mma_fp4<BLOCK>(d_tmem + x * XR, ad + (x * (TILE_BYTES >> 4) + 2 * kk), xd + 2 * kk,
                                               BLOCK == 32 && (kk & 1) ? id2 : id0, tw + 4 * (x * C::APS + j), tx + 4 * j,
                                               kb != k_lo || kk != 0);
                    }
                    tc::mma_commit(empty0 + 8 * s);
                    if (kb == k_hi - 1) tc::mma_commit(tfull0 + 8 * acc);
                }
                __syncwarp();
                if (++s == C::STAGES) { s = 0; ph ^= 1; }
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const float xg = p.xg ? __ldg(p.xg) : 1.f;
        OUT* Y = reinterpret_cast<OUT*>(p.Y);
        float* part = reinterpret_cast<float*>(smem);              // [NB][XR][128], for split > 1
        int tcount = 0;
        for (int64_t w = w0; w < total; w += stride, ++tcount) {
            const Tile t = tile(w);
            const int acc = tcount % C::ACCS;
            const MatrixScale ag(xg, p.wg ? __ldg(p.wg + t.e) : 1.f), au(xg, ACT && p.ug ? __ldg(p.ug + t.e) : 1.f);
            if (!tc::mbar_wait_bounded(tfull0 + 8 * acc, (tcount / C::ACCS) & 1, abort_flag)) break;
            tc::fence_after_sync();
            const uint32_t tb = tmem + acc * (NB * XR) + ((uint32_t)(q * 32) << 16);
            const int col = q * 32 + lane;                         // of the tile's 128
            for (int r0 = half * 32; r0 < t.tokens; r0 += 64) {
                uint32_t v[NB][32];
#pragma unroll
                for (int x = 0; x < NB; ++x) tc::tmem_ld_32x32b_x32(tb + x * XR + r0, v[x]);
                tc::tmem_wait_ld();
                if (S > 1) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (r0 + j < t.tokens)
#pragma unroll
                            for (int x = 0; x < NB; ++x)
                                part[(x * XR + r0 + j) * 128 + col] = __uint_as_float(v[x][j]);
                    continue;
                }
                ag.apply(v[0]);
                if (ACT) au.apply(v[NB - 1]);
                OUT* y = Y + (t.m0 + r0) * p.N + t.n0 + col;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (r0 + j < t.tokens) {
                        const float a = __uint_as_float(v[0][j]);
                        store1(y + (int64_t)j * p.N, ACT ? silu_mul(a, __uint_as_float(v[NB - 1][j])) : a);
                    }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tempty0 + 8 * acc);
            if (S > 1) continue;
            // rows behind the segment's tokens: zeros, 16 bytes a lane
            constexpr int PER = 16 / (int)sizeof(OUT);
            const int in_row = 128 / PER;
            for (int i = (warp - 2) * 32 + lane; i < (t.height - t.tokens) * in_row; i += 256)
                *reinterpret_cast<uint4*>(Y + (t.m0 + t.tokens + i / in_row) * p.N + t.n0 + i % in_row * PER) =
                    make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
    }

    if (S > 1) {
        // every CTA's part of the tile is in its shared memory; each CTA adds a 1/S share of it
        __syncthreads();
        tc::cluster_sync();
        if (w0 < total && !*abort_flag) {
            const Tile t = tile(w0);
            const float xg = p.xg ? __ldg(p.xg) : 1.f;
            const MatrixScale ag(xg, p.wg ? __ldg(p.wg + t.e) : 1.f), au(xg, ACT && p.ug ? __ldg(p.ug + t.e) : 1.f);
            const int groups = 32 / S;                             // 4-column groups of this CTA
            const uint32_t part = tc::smem_u32(smem);
            OUT* Y = reinterpret_cast<OUT*>(p.Y);
            for (int i = threadIdx.x; i < t.height * groups; i += kThreads) {
                const int r = i / groups, c4 = rank * groups + i % groups;
                float a[4] = {}, u[4] = {};
                if (r < t.tokens) {
                    for (int s = 0; s < S; ++s) {
                        const uint32_t base = tc::mapa_shared(part, s) + (r * 128 + c4 * 4) * 4;
                        const float4 x = ld_cluster_f4(base);
                        a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
                        if (ACT) {
                            const float4 z = ld_cluster_f4(base + XR * 512);
                            u[0] += z.x; u[1] += z.y; u[2] += z.z; u[3] += z.w;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        a[x] = a[x] * ag.pre * ag.by;
                        if (ACT) a[x] = silu_mul(a[x], u[x] * au.pre * au.by);
                    }
                }
                store4<OUT>(Y + (t.m0 + r) * p.N + t.n0 + c4 * 4, a[0], a[1], a[2], a[3]);
            }
        }
        tc::cluster_sync();                                        // the others have read this CTA's part
    } else {
        __syncthreads();
    }
    if (*abort_flag && warp == 0 && lane == 0)             // the copies asked for land before the CTA ends
        for (int j = max(0, issued - C::STAGES); j < issued; ++j)
            tc::mbar_wait_bounded(full0 + 8 * (j % C::STAGES), (j / C::STAGES) & 1, &no_abort, 100000000ull);
    __syncwarp();
    if (warp == 1) {
        if (tc::elect_one()) {                     // (the lane that issued the products)
            tc::mma_commit(drain);
            tc::mbar_wait_bounded(drain, 0, abort_flag, 100000000ull);
        }
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::TCOLS);
    }
    if (threadIdx.x == 0 && *abort_flag) clha_record_error(p.err, CLHA_ERR_TIMEOUT, blockIdx.x, 0, KID_FP4_MATMUL);
}

// ------------------------------------------------------------------------------ pairs of SMs
// Many tiles: CTA pairs (a cluster of two, cta_group::2) on tiles of 256 rows of X by 256 rows of W (for gate and
// up 128 of each). Each CTA loads its 128 rows of X, one of the two blocks of W and the scales of its rows
// and of both blocks: 38 KB a stage for the tensor work of a 128 x 256 tile, which takes 54 KB on one SM
// alone. The accumulator takes 256 of the 512 TMEM columns and the stages' scales most of the rest, so there
// is only one: the epilogue's warps read all of it into registers at once (128 columns each) and give it
// back before they scale, round and store, while the next tile's products already run. Finished values leave
// through shared memory by TMA (boxes of 32 rows x 128 bytes), which cuts off rows behind the end of Y.
// Tiles of an expert are taken in bands of 8 row tiles, rows fastest, so that the pairs working at one time
// share about 8 row blocks and as many column blocks of L2. Between two tiles the tensor pipe waits about 900
// cycles for the accumulator's hand-over (of 7600 for gate and up with K = 2048, 4.0 PFLOP/s on 32768 tokens).
// (Writing the scales from registers, with tcgen05.st from four warps, took twice the time of the copies.)
template <int BLOCK>
struct PairCfg {
    static constexpr int APS = 256 / BLOCK / 4;
    static constexpr int SF_BYTES = APS * 512;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES + 3 * SF_BYTES;
    static constexpr int STAGES = 5;
    static constexpr int SF_COLS = APS * 4 * 3;
    static constexpr int STG_OFF = STAGES * ((STAGE_BYTES + 1023) / 1024 * 1024);
    static constexpr int STAGE_STRIDE = (STAGE_BYTES + 1023) / 1024 * 1024;
    static constexpr int BAR_OFF = STG_OFF + 8 * 4096;
    static constexpr int SMEM = BAR_OFF + 8 * (2 * STAGES + 3) + 16 + 1024;
    static_assert(SMEM <= MAX_SMEM, "shared memory");
    static_assert(256 + STAGES * SF_COLS <= 512, "tensor memory");
};
constexpr int kBand = 8;

// The tiles in order: expert after expert, each expert's in bands. A role asks with ascending w.
struct Walk {
    int e = 0, mt = 0;
    int64_t base = 0, row0 = 0, pend = 0;    // tiles before expert e; its first row and the end of its segment
    __device__ __forceinline__ bool at(const MatmulArgs& p, int64_t w) {
        for (; e < p.E; ++e) {
            row0 = p.seg ? p.seg[e] : 0;
            pend = p.seg ? p.seg[e + 1] : p.rows;
            mt = (int)((pend - row0 + 255) >> 8);
            if (w < base + (int64_t)mt * p.n_tiles) return true;
            base += (int64_t)mt * p.n_tiles;
        }
        return false;
    }
    // first row and first column tile of tile w
    __device__ __forceinline__ void tile(const MatmulArgs& p, int64_t w, int64_t& m0, int& nt) const {
        const int64_t i = w - base;
        const int band = (int)(i / ((int64_t)kBand * p.n_tiles));
        const int r = (int)(i - (int64_t)band * kBand * p.n_tiles);
        const int h = min(kBand, mt - band * kBand);
        m0 = row0 + (int64_t)(band * kBand + r % h) * 256;
        nt = r / h;
    }
};

template <int BLOCK, bool ACT, typename OUT>
__global__ void __launch_bounds__(kThreads, 1)
fp4_matmul_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
                       const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWs,
                       const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmUs,
                       const __grid_constant__ CUtensorMap tmY, MatmulArgs p) {
    using C = PairCfg<BLOCK>;
    constexpr int TILE_N = ACT ? 128 : 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    const uint32_t full0 = tc::smem_u32(bars);            // leader: both CTAs' copies of a stage
    const uint32_t empty0 = full0 + 8 * C::STAGES;        // each CTA: its stage may be refilled
    const uint32_t tfull = empty0 + 8 * C::STAGES;        // each CTA: the accumulator holds a finished tile
    const uint32_t tempty = tfull + 8;                    // leader: both CTAs' epilogues have read it
    const uint32_t drain = tempty + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 3);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int no_abort = 0;                             // for the waits after an abort
    const uint32_t rank = tc::cluster_ctarank();
    const bool leader = rank == 0;
    const int warp = tc::warp_index(), lane = threadIdx.x & 31;
    const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(full0 + 8 * s, 1);
            tc::mbar_init(empty0 + 8 * s, 1);
        }
        tc::mbar_init(tfull, 1);
        tc::mbar_init(tempty, 16);                        // one arrival per epilogue warp of either CTA
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) tc::tmem_alloc_pair(tc::smem_u32(tmem_slot), 512);
    clha_allow_next();
    clha_wait_inputs();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();   // both CTAs' barriers exist before any copy or arrival reaches them
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int nk = (p.K + 255) / 256;
    const int atoms = p.K / BLOCK / 4;

    int issued = 0;                                        // producer: stages asked for
    if (warp == 0) {
        if (lane == 0) {
            tc::prefetch_tmap(&tmX);
            tc::prefetch_tmap(&tmXs);
            tc::prefetch_tmap(&tmW);
            tc::prefetch_tmap(&tmWs);
            const uint32_t full_leader = tc::mapa_shared(full0, 0);
            const CUtensorMap* mb = ACT && rank ? &tmU : &tmW;      // this CTA's block of W
            Walk k;
            int& it = issued;
            bool ok = true;
            for (int64_t w = pair; ok && k.at(p, w); w += npairs) {
                int64_t m0;
                int nt;
                k.tile(p, w, m0, nt);
                const int ra = (int)m0 + (int)rank * 128;
                const int w0 = k.e * p.N + nt * TILE_N, w1 = ACT ? w0 : w0 + 128;
                const int rb = rank ? w1 : w0;
                const int sa = ra / 128 * atoms, s0 = w0 / 128 * atoms, s1 = w1 / 128 * atoms;
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % C::STAGES;
                    if (!tc::mbar_wait_bounded(empty0 + 8 * s, ((it / C::STAGES) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    if (leader) tc::mbar_arrive_expect_tx(full0 + 8 * s, 2 * C::STAGE_BYTES);
                    const uint32_t fb = full_leader + 8 * s;
                    const uint32_t a = tc::smem_u32(smem + s * C::STAGE_STRIDE);
                    const uint32_t sf = a + 2 * TILE_BYTES;
                    tc::tma_load_2d_pair(a, &tmX, fb, kb * BKB, ra);
                    tc::tma_load_2d_pair(a + TILE_BYTES, mb, fb, kb * BKB, rb);
                    tc::tma_load_2d_pair(sf, &tmXs, fb, 0, sa + kb * C::APS);
                    tc::tma_load_2d_pair(sf + C::SF_BYTES, &tmWs, fb, 0, s0 + kb * C::APS);
                    tc::tma_load_2d_pair(sf + 2 * C::SF_BYTES, ACT ? &tmUs : &tmWs, fb, 0, s1 + kb * C::APS);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            constexpr uint32_t kE8 = BLOCK == 32;
            constexpr uint32_t ID0 = tc::idesc_fp4(kE8, 256, 256, 0), ID2 = tc::idesc_fp4(kE8, 256, 256, 2);
            const bool issuer = tc::elect_one();
            const uint64_t desc0 = tc::sw128_desc(tc::smem_u32(smem), 16, 1024);
            const uint64_t sdesc0 = tc::plain_desc(tc::smem_u32(smem) + 2 * TILE_BYTES);
            Walk k;
            int s = 0, tcount = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int64_t w = pair; ok && k.at(p, w); w += npairs, ++tcount) {
                if (!tc::mbar_wait_warp(tempty, (tcount & 1) ^ 1, abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
                for (int kb = 0; kb < nk; ++kb) {
                    if (!tc::mbar_wait_warp(full0 + 8 * s, ph, abort_flag)) { ok = false; break; }
                    tc::fence_after_sync();
                    const uint64_t ad = desc0 + (uint32_t)(s * (C::STAGE_STRIDE >> 4)), bd = ad + (TILE_BYTES >> 4);
                    const uint32_t ta = tmem + 256 + s * C::SF_COLS, tb = ta + C::APS * 4;
                    const uint64_t sd = sdesc0 + (uint32_t)(s * (C::STAGE_STRIDE >> 4));
                    const bool full_k = p.K - kb * 256 >= 256;         // else half: K is a multiple of 128
                    if (issuer) {
#pragma unroll
                        for (int j = 0; j < C::APS; ++j) {
                            tc::tmem_copy_scales_pair(ta + 4 * j, sd + j * 32);
                            tc::tmem_copy_scales_pair(tb + 8 * j, sd + (C::SF_BYTES >> 4) + j * 32);
                            tc::tmem_copy_scales_pair(tb + 8 * j + 4, sd + (C::SF_BYTES >> 3) + j * 32);
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kk >= 2 && !full_k) break;
                            const int j = BLOCK == 16 ? kk : kk >> 1;
                            tc::mma_fp4_pair<BLOCK>(tmem, ad + 2 * kk, bd + 2 * kk, BLOCK == 32 && (kk & 1) ? ID2 : ID0,
                                                    ta + 4 * j, tb + 8 * j, kk != 0 || kb != 0);
                        }
                        tc::mma_commit_pair(empty0 + 8 * s, 0x3);
                        if (kb == nk - 1) tc::mma_commit_pair(tfull, 0x3);
                    }
                    __syncwarp();
                    if (++s == C::STAGES) { s = 0; ph ^= 1; }
                }
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t stg = tc::smem_u32(smem + C::STG_OFF) + (warp - 2) * 4096;
        const uint32_t tempty_leader = tc::mapa_shared(tempty, 0);
        const float xg = p.xg ? __ldg(p.xg) : 1.f;
        Walk k;
        int tcount = 0;
        for (int64_t w = pair; k.at(p, w); w += npairs, ++tcount) {
            int64_t m0;
            int nt;
            k.tile(p, w, m0, nt);
            const int64_t r0 = m0 + (int)rank * 128 + q * 32;          // this warp's first row
            const int64_t vend = p.seg ? p.seg[k.e] + p.seg[p.E + 1 + k.e] : p.rows;
            const bool real = r0 + lane < vend;
            const MatrixScale ag(xg, p.wg ? __ldg(p.wg + k.e) : 1.f), au(xg, ACT && p.ug ? __ldg(p.ug + k.e) : 1.f);
            if (!tc::mbar_wait_bounded(tfull, tcount & 1, abort_flag)) break;
            tc::fence_after_sync();
            const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
            uint32_t v[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tc::tmem_ld_32x32b_x32(tb + (ACT ? (i >> 1) * 128 + half * 64 + (i & 1) * 32 : half * 128 + i * 32), v[i]);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster_relaxed(tempty_leader);
            const int col = nt * TILE_N + half * (ACT ? 64 : 128);
            if (r0 >= k.pend || col >= p.N) continue;  // rows of another segment; the missing half of an odd N
            constexpr int PER = 128 / (int)sizeof(OUT);                // columns of a 128-byte box
            constexpr int BOXES = (ACT ? 64 : 128) / PER;
#pragma unroll
            for (int b = 0; b < BOXES; ++b) {
#pragma unroll
                for (int i = 0; i < 4 / BOXES; ++i) (ACT && i >= 2 ? au : ag).apply(v[b * (4 / BOXES) + i]);
                if (lane == 0) tc::bulk_wait_read<0>();                // the buffer's last store has read it
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t o[4];
                    if (sizeof(OUT) == 4) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            o[x] = real ? v[b][4 * j + x] : 0u;
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int c = b * 64 + j * 8 + 2 * x;      // the pair of columns among this warp's
                            float f[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                f[y] = __uint_as_float(v[(c + y) >> 5][(c + y) & 31]);
                                if (ACT) f[y] = silu_mul(f[y], __uint_as_float(v[(((c + y) >> 5) + 2) & 3][(c + y) & 31]));
                            }
                            o[x] = real ? pack_bf16(f[0], f[1]) : 0u;
                        }
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 ::"r"(stg + lane * 128 + ((j ^ (lane & 7)) << 4)), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                 : "memory");
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::tma_store_2d(&tmY, stg, col + b * PER, (int)r0);
                    tc::bulk_commit();
                }
            }
        }
        if (lane == 0) tc::bulk_wait_all();
        __syncwarp();
    }

    __syncthreads();
    if (*abort_flag && leader && warp == 0 && lane == 0)   // both CTAs' copies land before either CTA can end
        for (int j = max(0, issued - C::STAGES); j < issued; ++j)
            tc::mbar_wait_bounded(full0 + 8 * (j % C::STAGES), (j / C::STAGES) & 1, &no_abort, 100000000ull);
    __syncwarp();
    if (warp == 1 && leader) {
        if (tc::elect_one()) {                     // (the lane that issued the products)
            tc::mma_commit_pair(drain, 0x1);
            tc::mbar_wait_bounded(drain, 0, abort_flag, 100000000ull);
        }
        __syncwarp();
    }
    tc::fence_before_sync();
    tc::cluster_sync();   // the leader's last products (which read both CTAs' shared memory) are done
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
    if (threadIdx.x == 0 && *abort_flag) clha_record_error(p.err, CLHA_ERR_TIMEOUT, blockIdx.x, 0, KID_FP4_MATMUL);
}

struct Maps {
    CUtensorMap X, Xs, W, Ws, U, Us, Y;
};

template <int BLOCK, bool ACT>
cudaError_t make_maps(const Fp4Product& a, int y_size, int x_box, Maps& t) {
    constexpr int APS = 256 / BLOCK / 4;
    const int atoms = a.K / BLOCK / 4;
    const uint64_t x_tiles = (uint64_t)((a.rows + 127) / 128), w_rows = (uint64_t)a.E * a.N;
    cudaError_t e;
    if ((e = make_tmap_2d(&t.X, a.xq, (uint64_t)a.rows, (uint64_t)a.K / 2, 1, x_box, BKB)) != cudaSuccess) return e;
    if ((e = make_tmap_2d_u32(&t.Xs, a.xs, x_tiles * atoms, 128, APS, 128)) != cudaSuccess) return e;
    if ((e = make_tmap_2d(&t.W, a.wq, w_rows, (uint64_t)a.K / 2, 1, 128, BKB)) != cudaSuccess) return e;
    if ((e = make_tmap_2d_u32(&t.Ws, a.ws, w_rows / 128 * atoms, 128, APS, 128)) != cudaSuccess) return e;
    t.U = t.W;
    t.Us = t.Ws;
    if (ACT) {
        if ((e = make_tmap_2d(&t.U, a.uq, w_rows, (uint64_t)a.K / 2, 1, 128, BKB)) != cudaSuccess) return e;
        if ((e = make_tmap_2d_u32(&t.Us, a.us, w_rows / 128 * atoms, 128, APS, 128)) != cudaSuccess) return e;
    }
    return make_tmap_2d(&t.Y, a.Y, (uint64_t)a.rows, (uint64_t)a.N, y_size, 32, 128 / y_size);
}

// Token slots in segments of `rows` packed rows, at most (clha_packed_rows).
int64_t slots_of(const Fp4Product& a) {
    return a.rows - 128 * (int64_t)a.E > 0 ? a.rows - 128 * (int64_t)a.E : a.rows;
}
// Row tiles of `height` rows to expect.
int64_t expected_row_tiles(const Fp4Product& a, int height) {
    if (!a.seg) return (a.rows + height - 1) / height;
    const int64_t slots = slots_of(a);
    return slots / height + (slots < a.E ? slots : a.E);
}

template <int BLOCK, bool ACT, typename OUT>
cudaError_t launch_pair(cudaStream_t s, int num_sms, const Fp4Product& a, int* err) {
    using C = PairCfg<BLOCK>;
    Maps t;
    cudaError_t e = make_maps<BLOCK, ACT>(a, (int)sizeof(OUT), 128, t);
    if (e != cudaSuccess) return e;
    auto kernel = fp4_matmul_pair_kernel<BLOCK, ACT, OUT>;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    const int tile_n = ACT ? 128 : 256;
    MatmulArgs p{a.rows, a.K, a.N, a.seg, a.E, a.xg, a.wg, a.ug, a.Y, (a.N + tile_n - 1) / tile_n, 1, err};
    e = clha_launch_overlapped(kernel, (unsigned)(num_sms / 2 * 2), kThreads, C::SMEM, s, 2, t.X, t.Xs, t.W, t.Ws, t.U,
                               t.Us, t.Y, p);
    if (e != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}

// CTAs of a cluster that share a tile's K in the kernel for few rows, `places` being the CTAs that run at one time:
// as many as find a place. Clusters of 8 leave an eighth of the places or more unused (a cluster stays within a
// GPC): 16 of them, of one CTA an SM, took 25 us where clusters of 4 take 17 (256 x 16384 -> 1024).
int few_split(int64_t tiles, int64_t places, int nk) {
    int split = 1;
    while (split < 8 && tiles * split * 2 <= (split == 4 ? places * 3 / 4 : places) && nk >= 4 * split) split *= 2;
    return split;
}

template <int BLOCK, int NB, int XR, typename OUT>
cudaError_t launch_few(cudaStream_t s, int num_sms, const Fp4Product& a, int* err) {
    using C = Cfg<BLOCK, NB, XR>;
    Maps t;
    cudaError_t e = make_maps<BLOCK, NB == 2>(a, (int)sizeof(OUT), 16, t);
    if (e != cudaSuccess) return e;
    auto kernel = fp4_matmul_kernel<BLOCK, NB, XR, OUT>;
    // per call: the attribute belongs to the current device's context (a process may drive several)
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    MatmulArgs p{a.rows, a.K, a.N, a.seg, a.E, a.xg, a.wg, a.ug, a.Y, a.N / 128, 1, err};
    const int64_t bound = (a.rows + XR - 1) / XR * p.n_tiles;            // tiles, at most
    const int64_t expect = expected_row_tiles(a, XR) * p.n_tiles;
    const int places = num_sms * C::CTAS;
    p.split = few_split(expect, places, (a.K + 255) / 256);
    const int64_t grid = p.split > 1 ? bound * p.split : (bound < places ? bound : places);
    e = clha_launch_overlapped(kernel, (unsigned)grid, kThreads, C::SMEM, s, (unsigned)p.split, t.X, t.Xs, t.W, t.Ws, t.U,
                               t.Us, p);
    if (e != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}

template <int BLOCK, int NB, typename OUT>
cudaError_t launch_product(cudaStream_t s, int num_sms, const Fp4Product& a, int* err) {
    constexpr bool ACT = NB == 2;
    // Which kernel: the one with the fewer rounds of stages, in units of a pair's stage (0.37 us). A round costs five
    // more for its start and end. A stage of the kernel for few rows costs 1.2 with a few rows a tile, and more with
    // more of them: 2.05 with 128, or 3.5 with 64 or more for gate and up. Measured on both sides, few against pairs:
    // 28672 -> 8192 with 1 row 25 : 58 us, 64 rows 33 : 42, 128 rows 43 : 43, 200 rows 74 : 45; 16384 -> 1024 with 512
    // rows 18 : 25, 1024 rows 28 : 26; gate/up 2048 -> 1408 of 64 experts, top 6, with 64 tokens 28 : 37, 256 tokens
    // 40 : 47, 512 tokens 52 : 50, 4096 tokens 161 : 105.
    const bool short_x = !a.seg && a.rows <= 32;
    const int nk = (a.K + 255) / 256, tile_n = ACT ? 128 : 256, pairs = num_sms / 2;
    const int64_t places = short_x && !ACT ? 2 * num_sms : num_sms, few_rows = expected_row_tiles(a, short_x ? 32 : 128);
    const int64_t few_tiles = few_rows * (a.N / 128), pair_tiles = expected_row_tiles(a, 256) * ((a.N + tile_n - 1) / tile_n);
    const int split = few_split(few_tiles, places, nk);
    const double rows = (double)(a.seg ? slots_of(a) : a.rows) / (few_rows > 0 ? few_rows : 1);
    const double stage = ACT ? 1.2 + 2.3 * (rows < 64 ? rows / 64 : 1) : 1.2 + 0.85 * (rows / 128);
    const double few = (few_tiles * split + places - 1) / places * ((nk + split - 1) / split * stage + 5);
    const double pair = (pair_tiles + pairs - 1) / pairs * (nk + 5.0);
    if (pair <= few) return launch_pair<BLOCK, ACT, OUT>(s, num_sms, a, err);
    // up to 32 dense rows: room for W's copies instead of 128 rows of X
    if (short_x) return launch_few<BLOCK, NB, 32, OUT>(s, num_sms, a, err);
    return launch_few<BLOCK, NB, 128, OUT>(s, num_sms, a, err);
}

}  // namespace

cudaError_t launch_fp4_matmul(cudaStream_t s, int num_sms, const Fp4Product& a, int block, int y_f32, int* err) {
    typedef __nv_bfloat16 bf;
    if (a.uq)
        return block == 32 ? launch_product<32, 2, bf>(s, num_sms, a, err) : launch_product<16, 2, bf>(s, num_sms, a, err);
    if (y_f32)
        return block == 32 ? launch_product<32, 1, float>(s, num_sms, a, err)
                           : launch_product<16, 1, float>(s, num_sms, a, err);
    return block == 32 ? launch_product<32, 1, bf>(s, num_sms, a, err) : launch_product<16, 1, bf>(s, num_sms, a, err);
}
