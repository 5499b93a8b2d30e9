// Products of microscaled 4-bit operands on the tensor cores: Y = X W^T, and the experts' gate/up pair
// h = SiLU(X Wg^T) * (X Wu^T), dense or over routed segments.
//
// tcgen05.mma multiplies e2m1 values and applies both operands' block scales, accumulating in float32;
// the matrix scales multiply the finished sums in the epilogue. One CTA computes 128 rows of X by NB
// blocks of 128 rows of W (for the gate/up pair one block of each, so that SiLU(g) * u needs nothing from
// outside the tile):
//   warp 0     TMA producer: per 256 columns of K, 128 bytes a row of X and of W (128-byte swizzle) and
//              their scale tiles (512 bytes for 128 rows x 4 blocks, copied as they lie).
//   warp 1     copies the stage's scale tiles to TMEM (its own columns for each stage, so that the stage's
//              barrier also orders their reuse) and issues the products of 64 columns of K each.
//   warps 2-9  epilogue: two warps for each TMEM lane quadrant.
// Segments start at multiples of 128, so a tile never mixes experts. Rows of a segment behind its tokens
// are written as zero; rows behind the last segment are not touched.
//
// Few tiles (decoding) are bound by reading W: then `split` CTAs of a cluster share one tile's K range,
// and add their parts through distributed shared memory, in rank order, so that the result does not
// depend on timing.
#include "clha_internal.h"
#include "tc_ptx.h"
#include "tmap.h"

namespace {

constexpr int kThreads = 320;
constexpr int BM = 128, BKB = 128;              // rows of X; bytes of K a stage (256 columns)
constexpr int TILE_BYTES = 128 * BKB;           // 16 KB: one operand block of a stage
constexpr int MAX_SMEM = 232448;

template <int BLOCK, int NB>
struct Cfg {
    static constexpr int APS = 256 / BLOCK / 4;              // scale tiles of 512 bytes a stage and operand block
    static constexpr int SF_BYTES = APS * 512;
    static constexpr int STAGE_BYTES = (1 + NB) * (TILE_BYTES + SF_BYTES);
    static constexpr int STAGES = NB == 1 ? 6 : 4;
    static constexpr int ACCS = NB == 1 ? 2 : 1;             // accumulators of NB * 128 columns: 256 in all
    static constexpr int SF_COLS = APS * 4 * (1 + NB);       // TMEM columns of a stage's scales
    static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
    static constexpr int SMEM = BAR_OFF + 8 * (2 * STAGES + 2 * ACCS + 1) + 16 + 1024;
    static_assert(SMEM <= MAX_SMEM, "shared memory");
    static_assert(256 + STAGES * SF_COLS <= 512, "tensor memory");
    static_assert(STAGES * STAGE_BYTES >= 128 * NB * 128 * 4, "partial sums fit the stages");
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

__device__ __forceinline__ int find_segment(const int64_t* seg, int E, int64_t row) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {  // last e with seg[e] <= row
        int mid = (lo + hi + 1) >> 1;
        if (seg[mid] <= row) lo = mid; else hi = mid - 1;
    }
    return lo;
}

struct Tile {
    int64_t m0, vend;        // first row; end of the rows with a token
    int n0, e;
};

__device__ __forceinline__ Tile decode(const MatmulArgs& p, int64_t w, int tile_n) {
    Tile t;
    t.m0 = w / p.n_tiles * BM;
    t.n0 = (int)(w % p.n_tiles) * tile_n;
    t.e = 0;
    t.vend = p.rows;
    if (p.seg) {
        t.e = find_segment(p.seg, p.E, t.m0);
        t.vend = p.seg[t.e] + p.seg[p.E + 1 + t.e];
    }
    return t;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

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
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// byte of element (row, 4-column group c4) in the partial sums' [128][NB * 128] float32 array; groups of a
// row are permuted by the row so that eight rows' same group fall into different banks
template <int NB>
__device__ __forceinline__ uint32_t part_off(int row, int c4) {
    return (uint32_t)(row * (NB * 512) + ((c4 ^ (row & 7)) << 4));
}

template <int BLOCK, int NB, bool ACT, typename OUT>
__global__ void __launch_bounds__(kThreads, 1)
fp4_matmul_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
                  const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWs,
                  const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmUs, MatmulArgs p) {
    static_assert(!ACT || NB == 2, "gate and up blocks");
    using C = Cfg<BLOCK, NB>;
    constexpr int TILE_N = ACT ? 128 : NB * 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    const uint32_t full0 = tc::smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * C::STAGES;
    const uint32_t tfull0 = empty0 + 8 * C::STAGES;       // accumulator a holds a finished tile
    const uint32_t tempty0 = tfull0 + 8 * C::ACCS;        // accumulator a has been read
    const uint32_t drain = tempty0 + 8 * C::ACCS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 2 * C::ACCS + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    const int64_t used = p.seg ? p.seg[p.E] : p.rows;
    const int64_t total = (used + BM - 1) / BM * p.n_tiles;
    const int64_t w0 = S > 1 ? blockIdx.x / S : blockIdx.x, stride = S > 1 ? gridDim.x / S : gridDim.x;
    const int nk = (p.K + 255) / 256;
    const int atoms = p.K / BLOCK / 4;                     // scale tiles across a row tile
    const int k_lo = (int)((int64_t)nk * rank / S), k_hi = (int)((int64_t)nk * (rank + 1) / S);
    // split > 1 runs one tile a cluster (the grid covers them all): the stages then hold the partial sums

    if (warp == 0) {
        if (lane == 0) {
            tc::prefetch_tmap(&tmX);
            tc::prefetch_tmap(&tmXs);
            tc::prefetch_tmap(&tmW);
            tc::prefetch_tmap(&tmWs);
            int it = 0;
            bool ok = true;
            for (int64_t w = w0; ok && w < total; w += stride) {
                const Tile t = decode(p, w, TILE_N);
                const int wr = t.e * p.N + t.n0;
                for (int kb = k_lo; kb < k_hi; ++kb, ++it) {
                    const int s = it % C::STAGES;
                    if (!tc::mbar_wait_bounded(empty0 + 8 * s, ((it / C::STAGES) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    const uint32_t fb = full0 + 8 * s;
                    tc::mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
                    const uint32_t a = tc::smem_u32(smem + s * C::STAGE_BYTES);
                    const uint32_t b = a + TILE_BYTES;
                    const uint32_t sf = b + NB * TILE_BYTES;
                    tc::tma_load_2d(a, &tmX, fb, kb * BKB, (int)t.m0);
                    tc::tma_load_2d(sf, &tmXs, fb, 0, (int)(t.m0 / 128) * atoms + kb * C::APS);
                    tc::tma_load_2d(b, &tmW, fb, kb * BKB, wr);
                    tc::tma_load_2d(sf + C::SF_BYTES, &tmWs, fb, 0, wr / 128 * atoms + kb * C::APS);
                    if (NB == 2) {   // the up projection's block, or the next 128 columns
                        const int ur = ACT ? wr : wr + 128;
                        tc::tma_load_2d(b + TILE_BYTES, ACT ? &tmU : &tmW, fb, kb * BKB, ur);
                        tc::tma_load_2d(sf + 2 * C::SF_BYTES, ACT ? &tmUs : &tmWs, fb, 0, ur / 128 * atoms + kb * C::APS);
                    }
                }
            }
            if (!ok) {  // the copies already issued land before the CTA exits
                for (int j = it - 1; j >= 0 && j >= it - C::STAGES; --j)
                    tc::mbar_wait_bounded(full0 + 8 * (j % C::STAGES), (j / C::STAGES) & 1, abort_flag, 100000000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t kE8 = BLOCK == 32;
            constexpr uint32_t ID0 = tc::idesc_fp4(kE8, BM, NB * 128, 0), ID2 = tc::idesc_fp4(kE8, BM, NB * 128, 2);
            int it = 0, tcount = 0;
            bool ok = true;
            for (int64_t w = w0; ok && w < total; w += stride, ++tcount) {
                const int acc = tcount % C::ACCS;
                if (!tc::mbar_wait_bounded(tempty0 + 8 * acc, ((tcount / C::ACCS) & 1) ^ 1, abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
                const uint32_t d_tmem = tmem + acc * (NB * 128);
                for (int kb = k_lo; kb < k_hi; ++kb, ++it) {
                    const int s = it % C::STAGES;
                    if (!tc::mbar_wait_bounded(full0 + 8 * s, (it / C::STAGES) & 1, abort_flag)) { ok = false; break; }
                    tc::fence_after_sync();
                    const uint32_t a = tc::smem_u32(smem + s * C::STAGE_BYTES);
                    const uint32_t b = a + TILE_BYTES;
                    const uint32_t sf = b + NB * TILE_BYTES;
                    const uint32_t ta = tmem + 256 + s * C::SF_COLS, tb = ta + C::APS * 4;
#pragma unroll
                    for (int j = 0; j < C::APS; ++j) {
                        tc::tmem_copy_scales(ta + 4 * j, tc::plain_desc(sf + j * 512));
#pragma unroll
                        for (int x = 0; x < NB; ++x)
                            tc::tmem_copy_scales(tb + 4 * (j * NB + x), tc::plain_desc(sf + (1 + x) * C::SF_BYTES + j * 512));
                    }
                    const int steps = p.K - kb * 256 >= 256 ? 4 : 2;   // K is a multiple of 128
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        const int j = BLOCK == 16 ? kk : kk >> 1;
                        tc::mma_fp4<BLOCK>(d_tmem, tc::sw128_desc(a + kk * 32, 16, 1024), tc::sw128_desc(b + kk * 32, 16, 1024),
                                           BLOCK == 32 && (kk & 1) ? ID2 : ID0, ta + 4 * j, tb + 4 * NB * j,
                                           kb != k_lo || kk != 0);
                    }
                    tc::mma_commit(empty0 + 8 * s);
                }
                if (ok) tc::mma_commit(tfull0 + 8 * acc);
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const float xg = p.xg ? __ldg(p.xg) : 1.f;
        OUT* Y = reinterpret_cast<OUT*>(p.Y);
        int tcount = 0;
        for (int64_t w = w0; w < total; w += stride, ++tcount) {
            const Tile t = decode(p, w, TILE_N);
            const int acc = tcount % C::ACCS;
            if (!tc::mbar_wait_bounded(tfull0 + 8 * acc, (tcount / C::ACCS) & 1, abort_flag)) break;
            tc::fence_after_sync();
            // this warp's columns: a half of the tile's (of both blocks' for gate and up)
            const uint32_t tb = tmem + acc * (NB * 128) + ((uint32_t)(q * 32) << 16);
            uint32_t v[2 * NB][32];
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                const int col = ACT ? (i >> 1) * 128 + half * 64 + (i & 1) * 32 : half * (NB * 64) + i * 32;
                tc::tmem_ld_32x32b_x32(tb + col, v[i]);
            }
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tempty0 + 8 * acc);
            const int lr = q * 32 + lane;
            const int64_t row = t.m0 + lr;
            if (S > 1) {
                const uint32_t part = tc::smem_u32(smem);
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
                    const int col = ACT ? (i >> 1) * 128 + half * 64 + (i & 1) * 32 : half * (NB * 64) + i * 32;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                     ::"r"(part + part_off<NB>(lr, col / 4 + j)), "r"(v[i][4 * j]), "r"(v[i][4 * j + 1]),
                                     "r"(v[i][4 * j + 2]), "r"(v[i][4 * j + 3]) : "memory");
                }
                continue;
            }
            if (row >= p.rows) continue;
            const bool real = row < t.vend;
            const float ag = real ? xg * (p.wg ? __ldg(p.wg + t.e) : 1.f) : 0.f;
            const float au = ACT ? (real ? xg * (p.ug ? __ldg(p.ug + t.e) : 1.f) : 0.f) : 0.f;
            const int col = t.n0 + half * (ACT ? 64 : NB * 64);
            if (!ACT && NB == 2 && col >= p.N) continue;       // N is an odd number of 128-column blocks
            OUT* y = Y + row * p.N + col;
#pragma unroll
            for (int i = 0; i < (ACT ? 2 : 2 * NB); ++i)
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float o[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float a = __uint_as_float(v[i][j + x]) * ag;
                        o[x] = ACT ? silu_mul(a, __uint_as_float(v[ACT ? i + 2 : i][j + x]) * au) : a;
                        if (!real) o[x] = 0.f;
                    }
                    store4<OUT>(y + i * 32 + j, o[0], o[1], o[2], o[3]);
                }
        }
        __syncwarp();
    }

    if (S > 1) {
        // every CTA's part of the tile is in its shared memory; each CTA adds a 1/S share of the columns
        __syncthreads();
        tc::cluster_sync();
        if (w0 < total && !*abort_flag) {
            const Tile t = decode(p, w0, TILE_N);
            const float xg = p.xg ? __ldg(p.xg) : 1.f;
            const float ag = xg * (p.wg ? __ldg(p.wg + t.e) : 1.f);
            const float au = ACT ? xg * (p.ug ? __ldg(p.ug + t.e) : 1.f) : 0.f;
            const int groups = TILE_N / 4 / S;                 // 4-column groups of this CTA
            const int64_t last = used < p.rows ? used : p.rows;
            const int n_rows = (int)(last - t.m0 < BM ? last - t.m0 : BM);
            const uint32_t part = tc::smem_u32(smem);
            OUT* Y = reinterpret_cast<OUT*>(p.Y);
            for (int i = threadIdx.x; i < n_rows * groups; i += kThreads) {
                const int lr = i / groups, c4 = rank * groups + i % groups;
                float a[4] = {}, u[4] = {};
                const bool real = t.m0 + lr < t.vend;
                if (real)
                    for (int s = 0; s < S; ++s) {
                        const uint32_t base = tc::mapa_shared(part, s);
                        const float4 x = ld_cluster_f4(base + part_off<NB>(lr, c4));
                        a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
                        if (ACT) {
                            const float4 z = ld_cluster_f4(base + part_off<NB>(lr, c4 + 32));
                            u[0] += z.x; u[1] += z.y; u[2] += z.z; u[3] += z.w;
                        }
                    }
                if (!ACT && NB == 2 && t.n0 + c4 * 4 >= p.N) continue;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    a[x] = !real ? 0.f : ACT ? silu_mul(a[x] * ag, u[x] * au) : a[x] * ag;
                store4<OUT>(Y + (t.m0 + lr) * p.N + t.n0 + c4 * 4, a[0], a[1], a[2], a[3]);
            }
        }
        tc::cluster_sync();                                    // the others have read this CTA's part
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        if (lane == 0) {
            tc::mma_commit(drain);
            tc::mbar_wait_bounded(drain, 0, abort_flag, 100000000ull);
        }
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
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
// share about 8 row blocks and as many column blocks of L2.
//
// Two warps of their own copy the scales to TMEM, every other scale column each. Such a copy takes about 60
// cycles in its issuer's order, and a stage of e4m3 scales has twelve: issued by the products' thread they ran
// in line with its products (measured on 4096 x 16384 -> 9472: 441 us; from one other warp 343, from two 274;
// without any copy 253). Writing the scales with tcgen05.st from registers took 547.
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
    static constexpr int SMEM = BAR_OFF + 8 * (3 * STAGES + 3) + 16 + 1024;
    static_assert(SMEM <= MAX_SMEM, "shared memory");
    static_assert(256 + STAGES * SF_COLS <= 512, "tensor memory");
};
constexpr int kBand = 8;
constexpr int kPairThreads = 384;   // as above, and warps 10 and 11 for the scales

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
__global__ void __launch_bounds__(kPairThreads, 1)
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
    const uint32_t sready0 = drain + 8;                   // leader: a stage's scales are on their way to TMEM
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * C::STAGES + 3);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t rank = tc::cluster_ctarank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            tc::mbar_init(full0 + 8 * s, 1);
            tc::mbar_init(empty0 + 8 * s, 1);
            tc::mbar_init(sready0 + 8 * s, 2);            // one arrival per scale warp
        }
        tc::mbar_init(tfull, 1);
        tc::mbar_init(tempty, 16);                        // one arrival per epilogue warp of either CTA
        tc::mbar_init(drain, 3);                          // the products' thread and the scale warps
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) tc::tmem_alloc_pair(tc::smem_u32(tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();   // both CTAs' barriers exist before any copy or arrival reaches them
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int nk = (p.K + 255) / 256;
    const int atoms = p.K / BLOCK / 4;

    if (warp == 0) {
        if (lane == 0) {
            tc::prefetch_tmap(&tmX);
            tc::prefetch_tmap(&tmXs);
            tc::prefetch_tmap(&tmW);
            tc::prefetch_tmap(&tmWs);
            const uint32_t full_leader = tc::mapa_shared(full0, 0);
            const CUtensorMap* mb = ACT && rank ? &tmU : &tmW;      // this CTA's block of W
            Walk k;
            int it = 0;
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
            if (!ok && leader) {  // the copies already issued (both CTAs') land before either CTA can exit
                for (int j = it - 1; j >= 0 && j >= it - C::STAGES; --j)
                    tc::mbar_wait_bounded(full0 + 8 * (j % C::STAGES), (j / C::STAGES) & 1, abort_flag, 100000000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            constexpr uint32_t kE8 = BLOCK == 32;
            constexpr uint32_t ID0 = tc::idesc_fp4(kE8, 256, 256, 0), ID2 = tc::idesc_fp4(kE8, 256, 256, 2);
            Walk k;
            int it = 0, tcount = 0;
            bool ok = true;
            for (int64_t w = pair; ok && k.at(p, w); w += npairs, ++tcount) {
                if (!tc::mbar_wait_bounded(tempty, (tcount & 1) ^ 1, abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % C::STAGES;
                    const uint32_t ph = (it / C::STAGES) & 1;
                    if (!tc::mbar_wait_bounded(full0 + 8 * s, ph, abort_flag) ||
                        !tc::mbar_wait_bounded(sready0 + 8 * s, ph, abort_flag)) { ok = false; break; }
                    tc::fence_after_sync();
                    const uint32_t a = tc::smem_u32(smem + s * C::STAGE_STRIDE);
                    const uint32_t b = a + TILE_BYTES;
                    const uint32_t ta = tmem + 256 + s * C::SF_COLS, tb = ta + C::APS * 4;
                    const int steps = p.K - kb * 256 >= 256 ? 4 : 2;   // K is a multiple of 128
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        const int j = BLOCK == 16 ? kk : kk >> 1;
                        tc::mma_fp4_pair<BLOCK>(tmem, tc::sw128_desc(a + kk * 32, 16, 1024),
                                                tc::sw128_desc(b + kk * 32, 16, 1024),
                                                BLOCK == 32 && (kk & 1) ? ID2 : ID0, ta + 4 * j, tb + 8 * j, (kb | kk) != 0);
                    }
                    tc::mma_commit_pair(empty0 + 8 * s, 0x3);
                }
                if (ok) tc::mma_commit_pair(tfull, 0x3);
            }
        }
        __syncwarp();
    } else if (warp >= 10) {
        if (lane == 0 && leader) {
            Walk k;
            int it = 0;
            bool ok = true;
            for (int64_t w = pair; ok && k.at(p, w); w += npairs)
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % C::STAGES;
                    if (!tc::mbar_wait_bounded(full0 + 8 * s, (it / C::STAGES) & 1, abort_flag)) { ok = false; break; }
                    tc::fence_after_sync();
                    const uint32_t sf = tc::smem_u32(smem + s * C::STAGE_STRIDE) + 2 * TILE_BYTES;
                    const uint32_t ta = tmem + 256 + s * C::SF_COLS, tb = ta + C::APS * 4;
#pragma unroll
                    for (int j = 0; j < C::APS; ++j) {
                        if ((j & 1) != warp - 10) continue;
                        tc::tmem_copy_scales_pair(ta + 4 * j, tc::plain_desc(sf + j * 512));
                        tc::tmem_copy_scales_pair(tb + 8 * j, tc::plain_desc(sf + C::SF_BYTES + j * 512));
                        tc::tmem_copy_scales_pair(tb + 8 * j + 4, tc::plain_desc(sf + 2 * C::SF_BYTES + j * 512));
                    }
                    tc::mma_commit_pair(sready0 + 8 * s, 0x1);
                }
            // the copies that this thread issued are done before the CTA gives its TMEM back
            tc::mma_commit_pair(drain, 0x1);
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
            const float ag = xg * (p.wg ? __ldg(p.wg + k.e) : 1.f);
            const float au = ACT ? xg * (p.ug ? __ldg(p.ug + k.e) : 1.f) : 0.f;
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
            if (lane == 0) tc::mbar_arrive_cluster(tempty_leader);
            const int col = nt * TILE_N + half * (ACT ? 64 : 128);
            if (r0 >= k.pend || col >= p.N) continue;  // rows of another segment; the missing half of an odd N
            constexpr int PER = 128 / (int)sizeof(OUT);                // columns of a 128-byte box
            constexpr int BOXES = (ACT ? 64 : 128) / PER;
#pragma unroll
            for (int b = 0; b < BOXES; ++b) {
                if (lane == 0) tc::bulk_wait_read<0>();                // the buffer's last store has read it
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t o[4];
                    if (sizeof(OUT) == 4) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            o[x] = real ? __float_as_uint(__uint_as_float(v[b][4 * j + x]) * ag) : 0u;
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int c = b * 64 + j * 8 + 2 * x;      // the pair of columns among this warp's
                            float f[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                f[y] = __uint_as_float(v[(c + y) >> 5][(c + y) & 31]) * ag;
                                if (ACT) f[y] = silu_mul(f[y], __uint_as_float(v[(((c + y) >> 5) + 2) & 3][(c + y) & 31]) * au);
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
    if (warp == 1 && leader) {
        if (lane == 0) {
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
cudaError_t make_maps(const Fp4Product& a, int y_size, Maps& t) {
    constexpr int APS = 256 / BLOCK / 4;
    const int atoms = a.K / BLOCK / 4;
    const uint64_t x_tiles = (uint64_t)((a.rows + 127) / 128), w_rows = (uint64_t)a.E * a.N;
    cudaError_t e;
    if ((e = make_tmap_2d(&t.X, a.xq, (uint64_t)a.rows, (uint64_t)a.K / 2, 1, 128, BKB)) != cudaSuccess) return e;
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

// Row tiles of `height` rows to expect: segments hold rows - 128 E token slots at most (clha_packed_rows).
int64_t expected_row_tiles(const Fp4Product& a, int height) {
    if (!a.seg) return (a.rows + height - 1) / height;
    const int64_t slots = a.rows - 128 * (int64_t)a.E > 0 ? a.rows - 128 * (int64_t)a.E : a.rows;
    return slots / height + (slots < a.E ? slots : a.E);
}

template <int BLOCK, bool ACT, typename OUT>
cudaError_t launch_pair(cudaStream_t s, int num_sms, const Fp4Product& a, int* err) {
    using C = PairCfg<BLOCK>;
    Maps t;
    cudaError_t e = make_maps<BLOCK, ACT>(a, (int)sizeof(OUT), t);
    if (e != cudaSuccess) return e;
    auto kernel = fp4_matmul_pair_kernel<BLOCK, ACT, OUT>;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    const int tile_n = ACT ? 128 : 256;
    MatmulArgs p{a.rows, a.K, a.N, a.seg, a.E, a.xg, a.wg, a.ug, a.Y, (a.N + tile_n - 1) / tile_n, 1, err};
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.gridDim = dim3((unsigned)(num_sms / 2 * 2));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, t.X, t.Xs, t.W, t.Ws, t.U, t.Us, t.Y, p)) != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}

template <int BLOCK, int NB, bool ACT, typename OUT>
cudaError_t launch_one(cudaStream_t s, int num_sms, const Fp4Product& a, int* err) {
    using C = Cfg<BLOCK, NB>;
    Maps t;
    cudaError_t e = make_maps<BLOCK, ACT>(a, (int)sizeof(OUT), t);
    if (e != cudaSuccess) return e;
    auto kernel = fp4_matmul_kernel<BLOCK, NB, ACT, OUT>;
    // per call: the attribute belongs to the current device's context (a process may drive several)
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    const int tile_n = ACT ? 128 : NB * 128;
    MatmulArgs p{a.rows, a.K, a.N, a.seg, a.E, a.xg, a.wg, a.ug, a.Y, (a.N + tile_n - 1) / tile_n, 1, err};
    const int64_t bound = (a.rows + 127) / 128 * p.n_tiles;              // tiles, at most
    const int64_t expect = expected_row_tiles(a, 128) * p.n_tiles;
    const int nk = (a.K + 255) / 256;
    while (p.split < 8 && expect * p.split * 2 <= num_sms && nk >= 4 * p.split) p.split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? bound * p.split : (bound < num_sms ? bound : num_sms)));
    e = cudaLaunchKernelEx(&cfg, kernel, t.X, t.Xs, t.W, t.Ws, t.U, t.Us, p);
    if (e != cudaSuccess) return e;
    clha_note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_matmul(cudaStream_t s, int num_sms, const Fp4Product& a, int block, int y_f32, int* err) {
    typedef __nv_bfloat16 bf;
    const int tile_n = a.uq ? 128 : 256;
    const bool pair = expected_row_tiles(a, 256) * ((a.N + tile_n - 1) / tile_n) >= num_sms / 2;
#define CLHA_PRODUCT(B)                                                                                              \
    (a.uq ? (pair ? launch_pair<B, true, bf>(s, num_sms, a, err) : launch_one<B, 2, true, bf>(s, num_sms, a, err))    \
     : y_f32 ? (pair ? launch_pair<B, false, float>(s, num_sms, a, err)                                               \
                     : launch_one<B, 1, false, float>(s, num_sms, a, err))                                            \
             : (pair ? launch_pair<B, false, bf>(s, num_sms, a, err) : launch_one<B, 1, false, bf>(s, num_sms, a, err)))
    return block == 32 ? CLHA_PRODUCT(32) : CLHA_PRODUCT(16);
#undef CLHA_PRODUCT
}
