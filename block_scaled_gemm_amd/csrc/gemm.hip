// gemm.hip -- block-scaled FP8 GEMM for gfx950.
//
// D[m][n] = sum_g sa[g][m] * SB(n,g) * P_g[m][n], P_g the 128-element group
// partial.  Each group's partial is formed on the matrix cores from zero and
// promoted into an FP32 register accumulator with one FMA per output element
// (the per-group dequantisation rides on that FMA), as the pages' promotion
// every 128 elements does.
//
// Three ways of forming P_g (the `accum` argument):
//
//  ACC_F32 (0, default).  The gfx950 FP8 matrix cores do not add their
//  products at FP32 accuracy: on crafted inputs every FP8 MFMA form loses
//  about 2^-12 of the largest product inside one instruction -- the limited
//  accumulation the pages measure on their own tensor cores.  This path
//  widens each E4M3 fragment exactly to f16 right after reading it from LDS
//  (v_cvt_scalef32_pk_f16_fp8 with scale 1 is exact for every finite code)
//  and forms P_g with v_mfma_f32_32x32x16_f16, whose products are exact and
//  whose sums are FP32-accurate.  Workgroup tile 256 (m) x 128 (n); 8 waves
//  of 64x64, each 2x2 sub-tiles of 32x32, 8 MFMAs per sub-tile per group.
//
//  ACC_MFMA8 (1).  P_g straight from v_mfma_f32_16x16x128_f8f6f4 (one MFMA
//  is one K group of a 16x16 sub-tile) at twice the matrix-core rate, with
//  the matrix core's own limited accumulation inside the group.  Dense
//  launches: workgroup tile 256 (m) x 256 (n), 8 waves of 64x128 (4x8
//  sub-tiles of 16x16), the last partial round of tiles as 256 x 128 tiles
//  (waves of 64x64); split-K launches: 256 x 128; grouped launches: 128
//  columns by 64, 128, 192 or 256 rows, with loader and compute waves apart
//  (grouped_split_kernel).
//
//  ACC_MFMA8_POW2 (2).  As ACC_MFMA8, for power-of-two scales: they enter
//  the scaled MFMA as E8M0 block scales and every group is accumulated by
//  the matrix core itself, so there is no promotion step on the VALU.
//
// All: the MFMA's first operand is the B (weight) tile and its second the
// A (activation) tile, so each result sub-tile is D^T: every lane holds runs
// of four consecutive output columns of one row and needs one activation
// scale per sub-tile.  Each lane's k positions depend only on its lane
// index, identically for both operands, so whatever order the hardware
// pairs elements in, equal k meet.
//
// Staging: 512 threads (two waves per SIMD).  Each K group of both tiles
// goes global -> LDS with global_load_lds_dwordx4 (no register staging:
// lane i of a wave instruction lands at LDS base + 16*i, so each
// instruction fills 8 rows of 128 B), the group's scales with 4-byte
// global_load_lds (see dma16s, Stager).  Tiles sit in LDS as FP8 codes,
// rows of 128 B whose 16-byte chunks are XOR-swizzled by (row & 7) ^ (row>>3 & 1)
// -- lanes fetch the permuted chunk of their row, so coalescing is unchanged
// and the fragment reads of 16 consecutive rows spread over all banks.
// STAGES groups are in flight; one barrier per group both publishes the
// landed group and frees the stage the next issue overwrites.
//
// Epilogue: the tile goes through a row-major fp32 image in the freed stage
// memory and leaves in whole row segments (bf16, fp32, or -- fused -- the
// bf16 result quantised 1x128 along n, one group per tile row).
#include "gemm_tile.h"

namespace fp8bs {

// ==== kernels ==========================================================================

template <int ACC, int SH, int KIND, int OUT, bool SPLIT>
__global__ __launch_bounds__(THREADS) void gemm_kernel(GemmArgs p, int64_t tiles_m, int64_t tiles_n) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Lds<SH>::BYTES];
    const int64_t ntiles = tiles_m * tiles_n;
    const int64_t wid = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t split = SPLIT ? wid / ntiles : 0;
    int64_t tm, tn;
    tile_coords(wid % ntiles, tiles_m, tiles_n, tm, tn);

    Tile T;
    T.m0 = tm * Shape<SH>::BM;
    T.m_end = p.M;
    T.n0 = tn * Shape<SH>::BN;
    T.n_end = p.N;
    T.a = p.a;
    T.lda = p.lda;
    T.sa = p.sa;
    T.ldsa = p.ldsa;
    T.b = p.b;
    T.ldb = p.ldb;
    T.sb = p.sb;
    T.sb_s0 = p.sb_s0;
    T.sb_s1 = p.sb_s1;
    T.qs = p.qs;
    T.qlds = p.qlds;

    const int64_t groups = p.K / 128;
    if (SPLIT) {
        const int64_t per = (groups + p.splits - 1) / p.splits;
        const int64_t g0 = split * per;
        const int64_t g1 = g0 + per < groups ? g0 + per : groups;
        run_tile<ACC, SH, KIND, 1, true>(T, g0, g1, p.ws + split * p.M * p.ws_ld, p.ws_ld, smem);
    } else {
        run_tile<ACC, SH, KIND, OUT, true>(T, 0, groups, p.d, p.ldd, smem);
    }
}

// FP8 dense paths: one launch, two tile shapes.  Output columns [0, n1)
// (n1 a multiple of 256, possibly past N) run on 256 x 256 tiles
// (workgroups 0 .. wide-1), the rest on 256 x 128
// tiles (the following workgroups): a last, partial round of wide tiles
// becomes a full round of narrow ones.  Each region is XCD-remapped on its
// own, so both spread over all XCDs in dispatch order.
template <int ACC, int KIND, int OUT>
__global__ __launch_bounds__(THREADS) void gemm_wide_kernel(GemmArgs p, int64_t n1) {
    constexpr int LDS_BYTES = Lds<0>::BYTES > Lds<1>::BYTES ? Lds<0>::BYTES : Lds<1>::BYTES;
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];
    static_assert(Shape<0>::BM == Shape<1>::BM, "both regions share the m tiling");
    const int64_t tiles_m = (p.M + Shape<1>::BM - 1) / Shape<1>::BM;
    const int64_t wide = tiles_m * (n1 / Shape<1>::BN);
    Tile T;
    T.m_end = p.M;
    T.a = p.a;
    T.lda = p.lda;
    T.sa = p.sa;
    T.ldsa = p.ldsa;
    T.b = p.b;
    T.ldb = p.ldb;
    T.sb = p.sb;
    T.sb_s0 = p.sb_s0;
    T.sb_s1 = p.sb_s1;
    T.qs = p.qs;
    T.qlds = p.qlds;
    const int64_t groups = p.K / 128;
    int64_t tm, tn;
    if ((int64_t)blockIdx.x < wide) {
        tile_coords(xcd_remap(blockIdx.x, wide), tiles_m, n1 / Shape<1>::BN, tm, tn);
        T.m0 = tm * Shape<1>::BM;
        T.n0 = tn * Shape<1>::BN;
        T.n_end = n1 < p.N ? n1 : p.N;
        run_tile<ACC, 1, KIND, OUT, true>(T, 0, groups, p.d, p.ldd, smem);
    } else {
        // only launched when n1 < N
        const int64_t tiles_n = (p.N - n1 + Shape<0>::BN - 1) / Shape<0>::BN;
        tile_coords(xcd_remap(blockIdx.x - wide, gridDim.x - wide), tiles_m, tiles_n, tm, tn);
        T.m0 = tm * Shape<0>::BM;
        T.n0 = n1 + tn * Shape<0>::BN;
        T.n_end = p.N;
        run_tile<ACC, 0, KIND, OUT, true>(T, 0, groups, p.d, p.ldd, smem);
    }
}

// Grouped, exact mode: workgroup (expert e, n-tile) walks the expert's
// m-tiles.  (The FP8 modes run grouped_split_kernel below.)
template <int ACC, int KIND, int OUT>
__global__ __launch_bounds__(THREADS) void grouped_kernel(GemmArgs p, int64_t tiles_n) {
    static_assert(ACC == 0, "the exact mode");
    __shared__ __attribute__((aligned(16))) uint8_t smem[Lds<0>::BYTES];
    const int64_t wid = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t e = wid / tiles_n;
    const int64_t tn = wid % tiles_n;
    const int64_t r0 = p.offsets[e], r1 = p.offsets[e + 1];

    Tile T;
    T.m_end = r1;
    T.n0 = tn * Shape<0>::BN;
    T.n_end = p.N;
    T.a = p.a;
    T.lda = p.lda;
    T.sa = p.sa;
    T.ldsa = p.ldsa;
    T.b = p.b + e * p.b_estride;
    T.ldb = p.ldb;
    T.sb = p.sb + e * p.sb_estride;
    T.sb_s0 = p.sb_s0;
    T.sb_s1 = p.sb_s1;
    for (int64_t m0 = r0; m0 < r1; m0 += Shape<0>::BM) {
        T.m0 = m0;
        run_tile<ACC, 0, KIND, OUT>(T, 0, p.K / 128, p.d, p.ldd, smem);
    }
}

// ==== grouped GEMMs with the roles apart ===================================================
//
// The FP8 paths of the grouped GEMMs stream every weight tile once and are
// bound by that staging, not by the matrix cores.  Waves 0..3 only issue
// the direct loads (the weight codes with the non-temporal hint) and waves
// 4..7 only compute, so a loader's issue of the next groups never waits
// behind its own MFMA and promotion work.  Compute wave c (on SIMD c) owns
// columns 32c..32c+31: its two B fragments stay in registers while the A
// fragments of the tile's 16-row blocks stream past them.  A row tile is
// the smallest of 64, 128, 192 or 256 rows that holds the expert's
// remaining rows, so an expert with few rows stages and multiplies few.

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const u32x4_t lds_u4;
typedef __attribute__((address_space(3))) const float lds_f32;

// The fragment of rows 16i + lane % 16 from per-lane LDS byte addresses of
// the two chunks in row lane % 16 (rows 16 apart share the swizzle, so row
// block i is at +2048 i, an immediate offset).
__device__ __forceinline__ v8i f8_frag_at(uint32_t lo, uint32_t hi, int i) {
    const u32x4_t x = *(lds_u4*)(uintptr_t)(lo + 2048 * i);
    const u32x4_t y = *(lds_u4*)(uintptr_t)(hi + 2048 * i);
    v8i r;
    r[0] = (int)x.x; r[1] = (int)x.y; r[2] = (int)x.z; r[3] = (int)x.w;
    r[4] = (int)y.x; r[5] = (int)y.y; r[6] = (int)y.z; r[7] = (int)y.w;
    return r;
}

// `stage`: LDS byte address of the stage, opaque to the compiler.  The
// stage offsets of the later stages do not fit a DS instruction's 16-bit
// offset; folded into every read they made the compiler keep an address
// register per row block and spill them.  From one per-lane base per
// operand, every read of a step takes an immediate offset.
template <int ACC, int SH, int KIND>
__device__ __forceinline__ void compute_cols(uint32_t stage, int c, int lane, v4f (&acc)[Shape<SH>::BM / 16][2]) {
    constexpr int MI = Shape<SH>::BM / 16;
    static_assert(Shape<SH>::BN == 128, "one block column per tile");
    const int nbase = 32 * c, c0 = 2 * (lane >> 4), l16 = lane & 15;
    const uint32_t alo = stage + Lds<SH>::A + f8_off(l16, c0), ahi = stage + Lds<SH>::A + f8_off(l16, c0 + 1);
    const uint32_t bb = stage + Lds<SH>::B + 128 * nbase;
    const v8i b0 = f8_frag_at(bb + f8_off(l16, c0), bb + f8_off(l16, c0 + 1), 0);
    const v8i b1 = f8_frag_at(bb + f8_off(l16, c0), bb + f8_off(l16, c0 + 1), 1);
    lds_f32* sal = (lds_f32*)(uintptr_t)(stage + Lds<SH>::SA + 4 * l16);  // row scales, +16 per row block
    lds_f32* sb = (lds_f32*)(uintptr_t)(stage + Lds<SH>::SB);  // block scalar, or per-column scales
    // Every row block of the tile (rows past m_valid come from the stage's
    // clamped rows and are never stored; a data-dependent exit made the
    // compiler copy the accumulators at every exit and spill), in pairs,
    // software-pipelined: the next pair's A fragments and scales are read
    // from LDS before this pair's MFMAs, and the previous pair's partials
    // are promoted while this pair's MFMAs run.
    v8i a[2];
    float sv[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        a[h] = f8_frag_at(alo, ahi, h);
        sv[h] = sal[16 * h];
    }
    if constexpr (ACC == 2) {
        const int s0 = e8m0(KIND == 0 ? sb[0] : sb[nbase + (lane & 15)]);
        const int s1 = e8m0(KIND == 0 ? sb[0] : sb[nbase + 16 + (lane & 15)]);
#pragma unroll
        for (int i = 0; i < MI; i += 2) {
            v8i na[2];
            float ns[2];
            if (i + 2 < MI) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    na[h] = f8_frag_at(alo, ahi, i + 2 + h);
                    ns[h] = sal[16 * (i + 2 + h)];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int sab = e8m0(sv[h]);
                acc[i + h][0] =
                    __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b0, a[h], acc[i + h][0], 0, 0, 0, s0, 0, sab);
                acc[i + h][1] =
                    __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b1, a[h], acc[i + h][1], 0, 0, 0, s1, 0, sab);
            }
            if (i + 2 < MI) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    a[h] = na[h];
                    sv[h] = ns[h];
                }
            }
        }
    } else {
        const float sbk = KIND == 0 ? sb[0] : 1.f;
        v4f sbn0 = {1.f, 1.f, 1.f, 1.f}, sbn1 = sbn0;
        if (KIND == 1) {
            sbn0 = *(__attribute__((address_space(3))) const v4f*)(sb + nbase + 4 * (lane >> 4));
            sbn1 = *(__attribute__((address_space(3))) const v4f*)(sb + nbase + 16 + 4 * (lane >> 4));
        }
        v4f pp[2][2];
        float pc[2];
        auto promote = [&](int i) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (KIND == 0) {
                    acc[i + h][0] += pp[h][0] * pc[h];
                    acc[i + h][1] += pp[h][1] * pc[h];
                } else {
                    acc[i + h][0] += (pp[h][0] * pc[h]) * sbn0;
                    acc[i + h][1] += (pp[h][1] * pc[h]) * sbn1;
                }
            }
        };
#pragma unroll
        for (int i = 0; i < MI; i += 2) {
            v8i na[2];
            float ns[2];
            if (i + 2 < MI) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    na[h] = f8_frag_at(alo, ahi, i + 2 + h);
                    ns[h] = sal[16 * (i + 2 + h)];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            v4f p[2][2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                p[h][0] = mfma8_group(b0, a[h]);
                p[h][1] = mfma8_group(b1, a[h]);
            }
            if (i > 0) promote(i - 2);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                pp[h][0] = p[h][0];
                pp[h][1] = p[h][1];
                pc[h] = KIND == 0 ? sv[h] * sbk : sv[h];
            }
            if (i + 2 < MI) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    a[h] = na[h];
                    sv[h] = ns[h];
                }
            }
        }
        promote(MI - 2);
    }
}

template <int ACC, int SH, int KIND, int OUT>
__device__ __forceinline__ void run_tile_split(const Tile& T, int64_t g1, void* d, int64_t ldd, uint8_t* smem) {
    static_assert(ACC != 0 && OUT <= 1, "FP8 paths, bf16 or fp32 output");
    constexpr int S = Shape<SH>::STAGES, MI = Shape<SH>::BM / 16;
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    float* ep = (float*)smem;

    // The two roles run separate loops that meet at the same barriers (one
    // per group and one after the last): s_barrier waits for every wave of
    // the workgroup whichever barrier instruction each one is at.  Kept
    // apart, the compute loop's accumulators never merge with a path that
    // leaves them untouched (such merges cost a copy of every accumulator).
    if (wave < LOADERS) {
        Stager<SH, KIND, true> stg;
        stg.init(T, wave, lane);
#pragma unroll
        for (int s = 0; s < S - 1; s++)
            if (s < g1) stg.issue(T, s, smem, s * Lds<SH>::STAGE, wave);
        // as in run_tile: wait until group g has landed (the S - 2 following
        // groups may still be in flight), meet the compute waves at the
        // barrier, refill the stage of group g - 1.  This loader's tile
        // loads per group: its valid A instructions and its B ones; its
        // scale loads come on top, so waiting for k * per outstanding is
        // conservative.
        constexpr int PER = (Shape<SH>::BM + Shape<SH>::BN) / 8 / LOADERS;
        static_assert((S == 4 || S == 3) && (S - 2) * PER <= 63, "wait counts cover this pipeline");
        const int per = stg.na_valid + Stager<SH, KIND, true>::NB;
        auto step = [&](auto ss, int64_t g) {
            constexpr int SS = decltype(ss)::value;
            if (S == 4 && g + 2 < g1)
                wait_n_and_barrier<2 * PER>(2 * per);
            else if (S >= 3 && g + 1 < g1)
                wait_n_and_barrier<PER>(per);
            else
                asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
            if (g + S - 1 < g1) stg.issue(T, g + S - 1, smem, ((SS + S - 1) % S) * Lds<SH>::STAGE, wave);
        };
        for (int64_t g = 0; g < g1; g += S) {
            step(std::integral_constant<int, 0>(), g);
            if (g + 1 < g1) step(std::integral_constant<int, 1>(), g + 1);
            if (g + 2 < g1) step(std::integral_constant<int, 2>(), g + 2);
            if constexpr (S == 4)
                if (g + 3 < g1) step(std::integral_constant<int, 3>(), g + 3);
        }
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");  // every group used
    } else {
        const int c = wave - LOADERS;
        v4f acc[MI][2];
#pragma unroll
        for (int i = 0; i < MI; i++) acc[i][0] = acc[i][1] = v4f{0.f, 0.f, 0.f, 0.f};
        auto step = [&](auto ss) {
            constexpr int SS = decltype(ss)::value;
            asm volatile("s_barrier" ::: "memory");
            uint32_t stage = lds_addr(smem) + SS * Lds<SH>::STAGE;
            asm volatile("" : "+s"(stage));
            compute_cols<ACC, SH, KIND>(stage, c, lane, acc);
        };
        for (int64_t g = 0; g < g1; g += S) {
            step(std::integral_constant<int, 0>());
            if (g + 1 < g1) step(std::integral_constant<int, 1>());
            if (g + 2 < g1) step(std::integral_constant<int, 2>());
            if constexpr (S == 4)
                if (g + 3 < g1) step(std::integral_constant<int, 3>());
        }
        asm volatile("s_barrier" ::: "memory");  // the stages hold the output image next
#pragma unroll
        for (int i = 0; i < MI; i++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                put4<SH>(ep, 16 * i + (lane & 15), 32 * c + 16 * j + 4 * (lane >> 4), acc[i][j][0], acc[i][j][1],
                         acc[i][j][2], acc[i][j][3]);
    }
    __syncthreads();
    write_tile_image<SH, OUT, true>(ep, T, T.n0, d, ldd);
    __syncthreads();  // a following row tile refills the stages
}

// Grouped, FP8 paths: workgroup (expert e, n-tile) walks the expert's rows
// in 256-row tiles, a last tile of fewer rows on the smallest shape that
// holds them.
template <int ACC, int KIND, int OUT>
__global__ __launch_bounds__(THREADS) void grouped_split_kernel(GemmArgs p, int64_t tiles_n) {
    constexpr int LDS_BYTES = Lds<11>::BYTES;
    static_assert(Lds<10>::BYTES <= LDS_BYTES && Lds<12>::BYTES <= LDS_BYTES && Lds<13>::BYTES <= LDS_BYTES,
                  "every row-tile shape fits");
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];
    const int64_t wid = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t e = wid / tiles_n;
    const int64_t tn = wid % tiles_n;
    const int64_t r0 = p.offsets[e], r1 = p.offsets[e + 1];

    Tile T;
    T.m_end = r1;
    T.n0 = tn * 128;
    T.n_end = p.N;
    T.a = p.a;
    T.lda = p.lda;
    T.sa = p.sa;
    T.ldsa = p.ldsa;
    T.b = p.b + e * p.b_estride;
    T.ldb = p.ldb;
    T.sb = p.sb + e * p.sb_estride;
    T.sb_s0 = p.sb_s0;
    T.sb_s1 = p.sb_s1;
    for (int64_t m0 = r0; m0 < r1; m0 += Shape<11>::BM) {
        T.m0 = m0;
        const int64_t rows = r1 - m0;
        if (rows <= Shape<13>::BM)
            run_tile_split<ACC, 13, KIND, OUT>(T, p.K / 128, p.d, p.ldd, smem);
        else if (rows <= Shape<10>::BM)
            run_tile_split<ACC, 10, KIND, OUT>(T, p.K / 128, p.d, p.ldd, smem);
        else if (rows <= Shape<12>::BM)
            run_tile_split<ACC, 12, KIND, OUT>(T, p.K / 128, p.d, p.ldd, smem);
        else
            run_tile_split<ACC, 11, KIND, OUT>(T, p.K / 128, p.d, p.ldd, smem);
    }
}

// K-grouped (MoE Wgrad over each expert's tokens): workgroup (expert e,
// output tile) sums the expert's K groups, which sit consecutively on the
// padded token axis starting at group sum_{e'<e} ceil(n_e'/128).  An expert
// without tokens writes zeros.
__device__ __forceinline__ int64_t expert_first_group(const int32_t* __restrict__ offsets, int64_t e) {
    __shared__ int64_t wsum[WAVES];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int64_t acc = 0;
    for (int64_t i = t; i < e; i += THREADS) acc += ((int64_t)offsets[i + 1] - offsets[i] + 127) / 128;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) acc += __shfl_xor(acc, d);
    if (lane == 0) wsum[wave] = acc;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) total += wsum[w];
    __syncthreads();
    return total;
}

// Each workgroup takes a strip of KSTRIP n-tiles of one (expert, m-tile):
// experts hold few tokens, so a tile's K loop is short and the expert's
// group range (two dependent reads of the offsets) is looked up once per
// strip rather than once per tile.
constexpr int KSTRIP = 8;

template <int ACC, int OUT>
__global__ __launch_bounds__(THREADS) void kgrouped_kernel(GemmArgs p, int64_t tiles_m, int64_t tiles_n) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Lds<0>::BYTES];
    const int64_t strips = (tiles_n + KSTRIP - 1) / KSTRIP;
    const int64_t per = tiles_m * strips;
    const int64_t wid = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t e = wid / per;
    const int64_t tm = (wid % per) % tiles_m, strip = (wid % per) / tiles_m;
    const int64_t g0 = expert_first_group(p.offsets, e);
    const int64_t g1 = g0 + ((int64_t)p.offsets[e + 1] - p.offsets[e] + 127) / 128;

    Tile T;
    T.m0 = tm * Shape<0>::BM;
    T.m_end = p.M;
    T.n_end = p.N;
    T.a = p.a;
    T.lda = p.lda;
    T.sa = p.sa;
    T.ldsa = p.ldsa;
    T.b = p.b;
    T.ldb = p.ldb;
    T.sb = p.sb;
    T.sb_s0 = p.sb_s0;
    T.sb_s1 = 0;
    void* d = (uint8_t*)p.d + e * p.d_estride * (OUT ? 4 : 2);
    const int64_t tn_end = (strip + 1) * KSTRIP < tiles_n ? (strip + 1) * KSTRIP : tiles_n;
    for (int64_t tn = strip * KSTRIP; tn < tn_end; tn++) {
        T.n0 = tn * Shape<0>::BN;
        run_tile<ACC, 0, 1, OUT>(T, g0, g1, d, p.ldd, smem);
    }
}

// K-grouped Wgrad, experts of at most two K groups: the workgroup's B tile
// (its column tile of every group of the expert) is staged once and stays
// in LDS while the strip's row tiles stage only their A groups; a tile's
// fp32 output goes out through the A ring in two 64-column images.  Other
// experts run each tile through the two-stage pipeline of shape 5.  LDS:
// B groups [2][codes 16 KB + 128
// column scales], then the A ring [2][codes 16 KB + 128 row scales, padded
// so that the ring holds a 128 x 64 fp32 image].
constexpr int KG3_BGROUP = 128 * 128 + 128 * 4;
constexpr int KG3_ASTAGE = 128 * 128 + 128 * 4 + 512;
constexpr int KG3_A = 2 * KG3_BGROUP;
constexpr int KG3_BYTES = KG3_A + 2 * KG3_ASTAGE;
static_assert(128 * Epi<8>::LD * 4 <= 2 * KG3_ASTAGE && Lds<5>::BYTES <= KG3_BYTES, "the K-grouped LDS map");

__device__ __forceinline__ void kg3_issue_a(const Stager<5, 1>& stg, const Tile& T, int64_t g, uint8_t* dst,
                                            int wave) {
    const uint8_t* a = T.a + T.m0 * T.lda + g * 128;
    const uint32_t base = lds_addr(dst);
#pragma unroll
    for (int ins = 0; ins < Stager<5, 1>::NA; ins++) dma16s(stg.va[ins], a, base + (ins * LOADERS + wave) * 8 * 128);
    if (wave < Stager<5, 1>::SA_INS) dma4s(stg.vsa, T.sa + g * T.ldsa + T.m0, base + 128 * 128 + wave * 256);
}

__device__ __forceinline__ void kg3_issue_b(const Stager<5, 1>& stg, const Tile& T, int64_t g, uint8_t* dst,
                                            int wave) {
    const uint8_t* b = T.b + T.n0 * T.ldb + g * 128;
    const uint32_t base = lds_addr(dst);
#pragma unroll
    for (int ins = 0; ins < Stager<5, 1>::NB; ins++) dma16s(stg.vb[ins], b, base + (ins * LOADERS + wave) * 8 * 128);
    if (wave < Stager<5, 1>::SB_INS) dma4s(stg.vsb, T.sb + g * T.sb_s0 + T.n0, base + 128 * 128 + wave * 256);
}

template <int ACC, int OUT>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(4, 4))) void kgrouped3_kernel(
    GemmArgs p, int64_t tiles_m, int64_t tiles_n) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[KG3_BYTES];
    const int64_t strips = (tiles_m + KSTRIP - 1) / KSTRIP;
    const int64_t per = tiles_n * strips;
    const int64_t wid = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t e = wid / per;
    const int64_t tn = (wid % per) % tiles_n, strip = (wid % per) / tiles_n;
    const int64_t g0 = expert_first_group(p.offsets, e);
    const int64_t ng = ((int64_t)p.offsets[e + 1] - p.offsets[e] + 127) / 128;

    Tile T;
    T.n0 = tn * 128;
    T.m_end = p.M;
    T.n_end = p.N;
    T.a = p.a;
    T.lda = p.lda;
    T.sa = p.sa;
    T.ldsa = p.ldsa;
    T.b = p.b;
    T.ldb = p.ldb;
    T.sb = p.sb;
    T.sb_s0 = p.sb_s0;
    T.sb_s1 = 0;
    void* d = (uint8_t*)p.d + e * p.d_estride * (OUT ? 4 : 2);
    const int64_t tm0 = strip * KSTRIP, tm1 = tm0 + KSTRIP < tiles_m ? tm0 + KSTRIP : tiles_m;
    if (ng == 0 || ng > 2) {
        for (int64_t tm = tm0; tm < tm1; tm++) {
            T.m0 = tm * 128;
            run_tile<ACC, 5, 1, OUT>(T, g0, g0 + ng, d, p.ldd, smem);
        }
        return;
    }
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    int wm, wn;
    Shape<8>::wave_grid(wave, wm, wn);
    Stager<5, 1> stg;
    T.m0 = tm0 * 128;
    stg.init(T, wave, lane);
    if (wave < LOADERS)
        for (int k = 0; k < ng; k++) kg3_issue_b(stg, T, g0 + k, smem + k * KG3_BGROUP, wave);
    for (int64_t tm = tm0; tm < tm1; tm++) {
        T.m0 = tm * 128;
        if (tm != tm0) stg.init(T, wave, lane);
        if (wave < LOADERS)
            for (int k = 0; k < ng; k++) kg3_issue_a(stg, T, g0 + k, smem + KG3_A + k * KG3_ASTAGE, wave);
        wait_and_barrier<0>(wave);  // this tile's A groups (and, the first time, B) have landed
        const int m_valid = (int)(T.m_end - T.m0 < 128 ? T.m_end - T.m0 : 128);
        v4f acc[Sub<8>::MI][Sub<8>::NJ];
#pragma unroll
        for (int i = 0; i < Sub<8>::MI; i++)
#pragma unroll
            for (int j = 0; j < Sub<8>::NJ; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < ng; k++) {
            const uint8_t* as = smem + KG3_A + k * KG3_ASTAGE;
            const uint8_t* bg = smem + k * KG3_BGROUP;
            const StagePtrs sp{as, bg, (const float*)(as + 128 * 128), (const float*)(bg + 128 * 128)};
            if constexpr (ACC == 1)
                compute_mfma8<8, 1>(sp, wm, wn, lane, m_valid, acc);
            else
                compute_mfma8_pow2<8, 1>(sp, wm, wn, lane, m_valid, acc);
        }
        __syncthreads();  // every wave is done with the A ring, which the images reuse
        store_mfma8<8, OUT>(acc, T, wm, wn, lane, d, p.ldd, smem + KG3_A);
    }
}

// Sum split-K partials in split order and convert.
template <int OUT>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ ws, int splits,
                                                            int64_t M, int64_t N, int64_t ws_ld,
                                                            void* __restrict__ d, int64_t ldd) {
    const int64_t cols4 = (N + 3) / 4;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (idx >= M * cols4) return;
    const int64_t m = idx / cols4, n = (idx % cols4) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < splits; k++) {
        const float4 v = *(const float4*)(ws + (int64_t)k * M * ws_ld + m * ws_ld + n);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    if (n + 4 <= N)
        store4_full<OUT>(d, ldd, m, n, s.x, s.y, s.z, s.w);
    else
        store4<OUT>(d, ldd, m, n, N, s.x, s.y, s.z, s.w);
}

// ==== host side ==========================================================================

int gemm_splits(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = ((M + Shape<0>::BM - 1) / Shape<0>::BM) * ((N + Shape<0>::BN - 1) / Shape<0>::BN);
    const int64_t groups = K / 128;
    if (tiles == 0 || groups < 16 || tiles >= 128) return 1;
    int64_t s = 256 / tiles;         // about one workgroup per CU
    const int64_t cap = groups / 8;  // at least 8 groups per split
    if (s > cap) s = cap;
    if (s > 256) s = 256;
    return s < 2 ? 1 : (int)s;
}

size_t gemm_workspace(int64_t M, int64_t N, int64_t K) {
    const int s = gemm_splits(M, N, K);
    if (s <= 1) return 0;
    return (size_t)s * (size_t)M * (size_t)((N + 3) / 4 * 4) * sizeof(float);
}

template <int ACC, int SH, int KIND, int OUT, bool SPLIT>
static void launch_shape(const GemmArgs& g, hipStream_t st) {
    const int64_t tiles_m = (g.M + Shape<SH>::BM - 1) / Shape<SH>::BM;
    const int64_t tiles_n = (g.N + Shape<SH>::BN - 1) / Shape<SH>::BN;
    const int64_t wgs = tiles_m * tiles_n * (SPLIT ? g.splits : 1);
    hipLaunchKernelGGL((gemm_kernel<ACC, SH, KIND, OUT, SPLIT>), dim3((unsigned)wgs), dim3(THREADS), 0, st, g,
                       tiles_m, tiles_n);
}

// Compute units of the current device (one workgroup of either shape fills
// a CU's LDS, so this is also the number of tiles in flight).
int device_cus() {
    static int cache[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cache[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
        cache[dev] = n;
    }
    return cache[dev];
}

// The FP8 paths run the first n1 output columns on 256 x 256 tiles and the
// rest on 256 x 128 tiles.  n1 (a multiple of 256; n1 >= N puts every
// column on wide tiles) minimises the rounds of
// workgroups, counting a round of the narrow tiles as 0.65 of a round of
// the wide ones (their measured time per tile): 4096 x 18432, 4.5 rounds
// of wide tiles, becomes 4 rounds of wide tiles and one of narrow ones.
int64_t wide_columns(int64_t M, int64_t N, int cus, double* cost_out) {
    const int64_t tm = (M + 255) / 256, tn = (N + 255) / 256;
    int64_t best_n1 = 256 * tn;  // every column on wide tiles
    double best = (double)((tm * tn + cus - 1) / cus);
    for (int64_t n1t = 0; n1t < tn; n1t++) {
        const int64_t t1 = tm * n1t, t0 = tm * ((N - 256 * n1t + 127) / 128);
        const double cost = (double)((t1 + cus - 1) / cus) + 0.65 * (double)((t0 + cus - 1) / cus);
        if (cost < best - 1e-9) {
            best = cost;
            best_n1 = 256 * n1t;
        }
    }
    if (cost_out) *cost_out = best;
    return best_n1;
}

// Rounds of 256 x 224 tiles, in the wide tile's rounds (a 256 x 224 tile is
// 7/8 of a wide tile's work).
static double cols224_cost(int64_t M, int64_t N, int cus) {
    const int64_t tiles = ((M + 255) / 256) * ((N + 223) / 224);
    return 0.875 * (double)((tiles + cus - 1) / cus);
}

// Split-K and the f16 path use shape 0; the FP8 paths gemm_wide_kernel,
// shape 1 on the first wide_columns() columns and shape 0 on the rest.
template <int ACC, int KIND, int OUT, bool SPLIT>
static void launch_dense(const GemmArgs& g, hipStream_t st) {
    if constexpr (ACC == 0 || SPLIT) {
        launch_shape<ACC, 0, KIND, OUT, SPLIT>(g, st);
    } else {
        const int cus = device_cus();
        double wide_cost = 0.0;
        const int64_t n1 = wide_columns(g.M, g.N, cus, &wide_cost);
        if constexpr (ACC == 1 && KIND == 1 && OUT <= 1) {
            // per-column scales, FP32-scale mode: 256 x 224 tiles where
            // their rounds come out fuller (2048 x 7168: one full round)
            if (cols224_cost(g.M, g.N, cus) < wide_cost - 0.05) {
                launch_shape<1, 7, 1, OUT, false>(g, st);
                return;
            }
        }
        const int64_t tiles_m = (g.M + Shape<1>::BM - 1) / Shape<1>::BM;
        const int64_t narrow_n = n1 < g.N ? (g.N - n1 + Shape<0>::BN - 1) / Shape<0>::BN : 0;
        const int64_t wgs = tiles_m * (n1 / Shape<1>::BN) + tiles_m * narrow_n;
        hipLaunchKernelGGL((gemm_wide_kernel<ACC, KIND, OUT>), dim3((unsigned)wgs), dim3(THREADS), 0, st, g, n1);
    }
}

template <int ACC>
static hipError_t launch_gemm_acc(const GemmArgs& g, hipStream_t st) {
    if (g.splits > 1 && !g.out_quant) {
        if (g.bscale_kind == 0)
            launch_dense<ACC, 0, 1, true>(g, st);
        else
            launch_dense<ACC, 1, 1, true>(g, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t n = g.M * ((g.N + 3) / 4);
        const dim3 grid((unsigned)((n + 255) / 256));
        if (g.out_f32)
            hipLaunchKernelGGL(splitk_reduce_kernel<1>, grid, dim3(256), 0, st, g.ws, g.splits, g.M, g.N, g.ws_ld,
                               g.d, g.ldd);
        else
            hipLaunchKernelGGL(splitk_reduce_kernel<0>, grid, dim3(256), 0, st, g.ws, g.splits, g.M, g.N, g.ws_ld,
                               g.d, g.ldd);
        return hipGetLastError();
    }
    if (g.out_quant) {
        if (g.bscale_kind == 0) {
            if (g.out_quant == 1)
                launch_dense<ACC, 0, 2, false>(g, st);
            else
                launch_dense<ACC, 0, 3, false>(g, st);
        } else {
            if (g.out_quant == 1)
                launch_dense<ACC, 1, 2, false>(g, st);
            else
                launch_dense<ACC, 1, 3, false>(g, st);
        }
        return hipGetLastError();
    }
    if (g.bscale_kind == 0) {
        if (g.out_f32)
            launch_dense<ACC, 0, 1, false>(g, st);
        else
            launch_dense<ACC, 0, 0, false>(g, st);
    } else {
        if (g.out_f32)
            launch_dense<ACC, 1, 1, false>(g, st);
        else
            launch_dense<ACC, 1, 0, false>(g, st);
    }
    return hipGetLastError();
}

hipError_t launch_gemm(const GemmArgs& g, hipStream_t st) {
    if (g.M == 0 || g.N == 0) return hipSuccess;
    if (g.accum == 0) return launch_gemm_acc<0>(g, st);
    return g.accum == 1 ? launch_gemm_acc<1>(g, st) : launch_gemm_acc<2>(g, st);
}

template <int ACC>
static hipError_t launch_grouped_acc(const GemmArgs& g, hipStream_t st) {
    const int64_t tiles_n = (g.N + Shape<0>::BN - 1) / Shape<0>::BN;
    const dim3 grid((unsigned)(tiles_n * g.G));
    if constexpr (ACC != 0) {
        if (g.bscale_kind == 0) {
            if (g.out_f32)
                hipLaunchKernelGGL((grouped_split_kernel<ACC, 0, 1>), grid, dim3(THREADS), 0, st, g, tiles_n);
            else
                hipLaunchKernelGGL((grouped_split_kernel<ACC, 0, 0>), grid, dim3(THREADS), 0, st, g, tiles_n);
        } else {
            if (g.out_f32)
                hipLaunchKernelGGL((grouped_split_kernel<ACC, 1, 1>), grid, dim3(THREADS), 0, st, g, tiles_n);
            else
                hipLaunchKernelGGL((grouped_split_kernel<ACC, 1, 0>), grid, dim3(THREADS), 0, st, g, tiles_n);
        }
        return hipGetLastError();
    }
    else {
        if (g.bscale_kind == 0) {
            if (g.out_f32)
                hipLaunchKernelGGL((grouped_kernel<ACC, 0, 1>), grid, dim3(THREADS), 0, st, g, tiles_n);
            else
                hipLaunchKernelGGL((grouped_kernel<ACC, 0, 0>), grid, dim3(THREADS), 0, st, g, tiles_n);
        } else {
            if (g.out_f32)
                hipLaunchKernelGGL((grouped_kernel<ACC, 1, 1>), grid, dim3(THREADS), 0, st, g, tiles_n);
            else
                hipLaunchKernelGGL((grouped_kernel<ACC, 1, 0>), grid, dim3(THREADS), 0, st, g, tiles_n);
        }
        return hipGetLastError();
    }
}

template <int ACC>
static hipError_t launch_kgrouped_acc(const GemmArgs& g, hipStream_t st) {
    if constexpr (ACC != 0) {
        const int64_t tiles_m = (g.M + 127) / 128, tiles_n = (g.N + 127) / 128;
        const dim3 grid((unsigned)(tiles_n * ((tiles_m + KSTRIP - 1) / KSTRIP) * g.G));
        if (g.out_f32)
            hipLaunchKernelGGL((kgrouped3_kernel<ACC, 1>), grid, dim3(THREADS), 0, st, g, tiles_m, tiles_n);
        else
            hipLaunchKernelGGL((kgrouped3_kernel<ACC, 0>), grid, dim3(THREADS), 0, st, g, tiles_m, tiles_n);
        return hipGetLastError();
    }
    const int64_t tiles_m = (g.M + Shape<0>::BM - 1) / Shape<0>::BM;
    const int64_t tiles_n = (g.N + Shape<0>::BN - 1) / Shape<0>::BN;
    const dim3 grid((unsigned)(tiles_m * ((tiles_n + KSTRIP - 1) / KSTRIP) * g.G));
    if (g.out_f32)
        hipLaunchKernelGGL((kgrouped_kernel<ACC, 1>), grid, dim3(THREADS), 0, st, g, tiles_m, tiles_n);
    else
        hipLaunchKernelGGL((kgrouped_kernel<ACC, 0>), grid, dim3(THREADS), 0, st, g, tiles_m, tiles_n);
    return hipGetLastError();
}

hipError_t launch_kgrouped_gemm(const GemmArgs& g, hipStream_t st) {
    if (g.G == 0 || g.M == 0 || g.N == 0) return hipSuccess;
    if (g.accum == 0) return launch_kgrouped_acc<0>(g, st);
    return g.accum == 1 ? launch_kgrouped_acc<1>(g, st) : launch_kgrouped_acc<2>(g, st);
}

hipError_t launch_grouped_gemm(const GemmArgs& g, hipStream_t st) {
    if (g.G == 0 || g.N == 0) return hipSuccess;
    if (g.accum == 0) return launch_grouped_acc<0>(g, st);
    return g.accum == 1 ? launch_grouped_acc<1>(g, st) : launch_grouped_acc<2>(g, st);
}

}  // namespace fp8bs
