// block_kernels.h -- internal launch interface of the feed-forward block's
// kernels (gated.hip, norm.hip, clip.hip).  Launchers assume their arguments
// were validated (block_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8bs {

// ---- gated feed-forward, forward ------------------------------------------------------

// Output H: 0 bf16, 1 fp32, 2 / 3 codes with FP32 / power-of-two scales.
enum { GATED_BF16 = 0, GATED_F32 = 1, GATED_QUANT = 2, GATED_QUANT_POW2 = 3 };

struct GatedArgs {
    int64_t M, N, K;
    const uint8_t* a;  // codes [M][lda]
    int64_t lda;
    const float* sa;  // [K/128][ldsa]
    int64_t ldsa;
    const uint8_t* b;  // codes [2N][ldb]: N gate rows, then N up rows
    int64_t ldb;
    const float* sb;  // [2N/128][ldsb]
    int64_t ldsb;
    int act;
    int out;
    void* d;
    int64_t ldd;
    float* qs;  // quantised H: scales qs[(n/128)*qlds + m]
    int64_t qlds;
    uint16_t* gu;  // optional: the pre-activations, bf16 [M][ldgu], gate | up
    int64_t ldgu;
    int accum;
    float* ws;  // split-K partials [splits][M][2N], or H of few rows [M][N]
    int splits;
    const int32_t* offsets;  // grouped: device [G+1]
    int G;
    int64_t b_estride, sb_estride;
};

int gated_splits(int64_t M, int64_t N, int64_t K);
size_t gated_workspace(int64_t M, int64_t N, int64_t K, bool quant);
hipError_t launch_gated(const GatedArgs& g, hipStream_t st);
hipError_t launch_grouped_gated(const GatedArgs& g, hipStream_t st);

// ---- gated feed-forward, backward -------------------------------------------------------

struct GatedBwdArgs {
    int64_t M, N;
    const uint16_t* dh;
    int64_t lddh;
    const uint16_t* gu;
    int64_t ldgu;
    int act;
    int pow2;
    uint8_t* qr;  // 1x128 groups of dG | dU: [M][ldqr]; scales sr[g*ldsr + m]
    int64_t ldqr;
    float* sr;
    int64_t ldsr;
    uint8_t* qc;  // 128x1 groups of dG | dU, transposed: [2N][ldqc]; sc[p*ldsc + c]
    int64_t ldqc;
    float* sc;
    int64_t ldsc;
    uint8_t* qh;  // 128x1 groups of H, transposed: [N][ldqh]; sh[p*ldsh + c]
    int64_t ldqh;
    float* sh;
    int64_t ldsh;
    const int32_t* offsets;  // grouped: device [G+1]; null: one range of M rows
    int G;
};

hipError_t launch_gated_backward(const GatedBwdArgs& g, hipStream_t st);

// ---- norms, gate and residual between two blocks ------------------------------------------

constexpr int64_t NORM_MAX_COLS = 32768;

struct NormArgs {
    int64_t M, D;
    const uint16_t* x;  // residual stream, bf16 [M][ldx]
    int64_t ldx;
    const uint16_t* y;  // optional: the block's output, bf16 [M][ldy]
    int64_t ldy;
    const float* w_post;  // optional: norm of y, [D]
    const float* gate;    // optional: [ceil(M/gate_rows)][D]
    int64_t gate_rows;
    float alpha, eps;
    uint16_t* xo;  // the new residual stream (with y), bf16 [M][ldxo]
    int64_t ldxo;
    const float* w_pre;  // optional: the next norm, [D]
    uint16_t* h;         // its result: bf16 [M][ldh] and / or codes
    int64_t ldh;
    uint8_t* q;
    int64_t ldq;
    float* s;  // s[g*lds + m]
    int64_t lds;
    int pow2;
    float* rstd_y;  // optional: [M]
    float* rstd_x;
};

hipError_t launch_norm(const NormArgs& g, hipStream_t st);

struct NormBwdArgs {
    int64_t M, D;
    const uint16_t* dxo;  // optional: gradient of x' from the residual stream
    int64_t lddxo;
    const uint16_t* dh;  // optional, with w_pre: gradient of h
    int64_t lddh;
    const uint16_t* xo;  // x' (x, without y)
    int64_t ldxo;
    const float* rstd_x;
    const float* w_pre;
    const uint16_t* y;
    int64_t ldy;
    const float* rstd_y;
    const float* w_post;
    const float* gate;
    int64_t gate_rows;
    float alpha;
    uint16_t* dx;
    int64_t lddx;
    uint16_t* dy;
    int64_t lddy;
    float* dw_pre;   // [D]
    float* dw_post;  // [D]
    float* dgate;    // [ceil(M/gate_rows)][D]
    float* ws;       // [parts] x ([D] pre, [D] post, [2][D] gate)
    int parts;
};

int norm_bwd_parts(int64_t M, int64_t D);
size_t norm_bwd_workspace(int64_t M, int64_t D);
hipError_t launch_norm_bwd(const NormBwdArgs& g, hipStream_t st);

// ---- global gradient norm and clipping -----------------------------------------------------

constexpr int CLIP_TABLE = 96;  // tensors of one launch

// Passed by value (a kernel's arguments may hold 4 KiB).
struct ClipTable {
    const void* g[CLIP_TABLE];
    void* out[CLIP_TABLE];
    int64_t count[CLIP_TABLE];
    int32_t first[CLIP_TABLE + 1];  // first chunk of each tensor in the launch
    uint8_t f32[CLIP_TABLE];
    int n;
};

constexpr int64_t CLIP_CHUNK = 1 << 15;  // elements a workgroup takes at a time

// Workgroups of one launch over `chunks` chunks, one of `tables` launches.
int clip_grid(int64_t chunks, int64_t tables);
hipError_t launch_grad_sumsq(const ClipTable& t, int grid, double* part, hipStream_t st);
// norm and coef may be null
hipError_t launch_grad_finish(const double* part, int parts, float max_norm, float* norm, float* coef,
                              hipStream_t st);
hipError_t launch_grad_scale(const ClipTable& t, int grid, const double* part, int parts, float max_norm, float* norm,
                             float* coef, hipStream_t st);

}  // namespace fp8bs
