// norm.hip -- the seam between two blocks for gfx950: the norm after a block,
// its gate and the residual scale, and the norm before the next block with
// its result quantised in 1x128 groups; and the backward pass.
//
//   r_y = 1/sqrt(mean(y^2) + eps)   n = y r_y w_post      (n = y without w_post)
//   x'  = alpha x + gate n                                (x' = x without y)
//   r_x = 1/sqrt(mean(x'^2) + eps)  h = x' r_x w_pre
//
// HBM-bound: 4 B read and 2 + 1 B written per element forward, 8 B read and
// 4 B written backward.  A workgroup holds whole rows in registers (8 columns
// per thread and vector), so every row is read once; it walks consecutive
// rows, so the fp32 vectors w_pre, w_post and gate are read once per
// workgroup and stay in registers.
#include "block_kernels.h"
#include "device.h"

namespace fp8bs {

__device__ __forceinline__ uint32_t pk_bf16(float lo, float hi) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){lo, hi}, bf2));
}

// Eight bf16 (zeros where !on) widened to fp32.
__device__ __forceinline__ void load8(const uint16_t* p, bool on, float (&v)[8]) {
    const uint4 w = on ? *(const uint4*)p : make_uint4(0, 0, 0, 0);
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

__device__ __forceinline__ void loadf8(const float* p, bool on, float (&v)[8]) {
    const float4 a = on ? *(const float4*)p : make_float4(0, 0, 0, 0);
    const float4 b = on ? *(const float4*)(p + 4) : make_float4(0, 0, 0, 0);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    *(uint4*)p = make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Sums of N values over the workgroup, in a fixed order; every thread gets
// them.  `slot` alternates between calls, so one barrier per call keeps a
// call's values apart from the next one's.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*lds)[16][N], int& slot) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = (blockDim.x + 63) >> 6;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = wave_sum(v[i]);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; i++) lds[slot][wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = 0.f;
    for (int w = 0; w < waves; w++)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += lds[slot][w][i];
    slot ^= 1;
}

// Thread t owns columns 8(t + j*threads) ..+7, j < NV.
template <int NV>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs p, int64_t rows_per) {
    __shared__ float red[2][16][1];
    int slot = 0;
    const int t = threadIdx.x, nt = blockDim.x;
    const int64_t r0 = blockIdx.x * rows_per, r1 = r0 + rows_per < p.M ? r0 + rows_per : p.M;
    const float inv_d = 1.0f / (float)p.D;
    int64_t col[NV];
    bool on[NV];
    float wpre[NV][8], wpost[NV][8], gate[NV][8];
#pragma unroll
    for (int j = 0; j < NV; j++) {
        col[j] = 8 * (int64_t)(t + j * nt);
        on[j] = col[j] < p.D;
        if (p.w_pre) loadf8(p.w_pre + col[j], on[j], wpre[j]);
        if (p.w_post) loadf8(p.w_post + col[j], on[j], wpost[j]);
    }
    int64_t have = -1;  // the row of `gate` in registers
    for (int64_t r = r0; r < r1; r++) {
        float x[NV][8], y[NV][8];
#pragma unroll
        for (int j = 0; j < NV; j++) {
            load8(p.x + r * p.ldx + col[j], on[j], x[j]);
            if (p.y) load8(p.y + r * p.ldy + col[j], on[j], y[j]);
        }
        if (p.y) {
            if (p.gate && r / p.gate_rows != have) {
                have = r / p.gate_rows;
#pragma unroll
                for (int j = 0; j < NV; j++) loadf8(p.gate + have * p.D + col[j], on[j], gate[j]);
            }
            float ry = 1.0f;
            if (p.w_post) {
                float s[1] = {0.f};
#pragma unroll
                for (int j = 0; j < NV; j++)
#pragma unroll
                    for (int k = 0; k < 8; k++) s[0] += y[j][k] * y[j][k];
                block_sum<1>(s, red, slot);
                ry = 1.0f / sqrtf(s[0] * inv_d + p.eps);
                if (t == 0 && p.rstd_y) p.rstd_y[r] = ry;
            }
#pragma unroll
            for (int j = 0; j < NV; j++) {
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    float n = y[j][k];
                    if (p.w_post) n = n * ry * wpost[j][k];
                    if (p.gate) n *= gate[j][k];
                    x[j][k] = p.alpha * x[j][k] + n;
                }
                if (on[j]) store8(p.xo + r * p.ldxo + col[j], x[j]);
            }
        }
        if (!p.w_pre) continue;
        // the norm takes x' in fp32, before its rounding for the residual stream
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; j++)
#pragma unroll
            for (int k = 0; k < 8; k++) s[0] += x[j][k] * x[j][k];
        block_sum<1>(s, red, slot);
        const float rx = 1.0f / sqrtf(s[0] * inv_d + p.eps);
        if (t == 0 && p.rstd_x) p.rstd_x[r] = rx;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            float h[8];
            uint32_t am = 0;
#pragma unroll
            for (int k = 0; k < 8; k++) {
                h[k] = x[j][k] * rx * wpre[j][k];
                am = max(am, __float_as_uint(h[k]) & 0x7FFFFFFFu);
            }
            if (p.q) {
                // 16 lanes hold a group; lanes past D are whole groups
                const GroupScale gs = group_scale(row16_max(am), p.pow2);
                if (on[j]) {
                    *(uint2*)(p.q + r * p.ldq + col[j]) =
                        make_uint2(pack4(h[0] * gs.inv, h[1] * gs.inv, h[2] * gs.inv, h[3] * gs.inv),
                                   pack4(h[4] * gs.inv, h[5] * gs.inv, h[6] * gs.inv, h[7] * gs.inv));
                    if ((t & 15) == 0) p.s[(col[j] >> 7) * p.lds + r] = gs.s;
                }
            }
            if (p.h && on[j]) store8(p.h + r * p.ldh + col[j], h);
        }
    }
}

// Threads (a multiple of 64) that hold D columns in nv vectors of 8.
static int norm_threads(int64_t D, int nv) { return (int)((D / 8 + nv - 1) / nv + 63) / 64 * 64; }

hipError_t launch_norm(const NormArgs& g, hipStream_t st) {
    if (g.M == 0 || g.D == 0) return hipSuccess;
    const int64_t rows_per = g.M >= 4096 ? 8 : g.M >= 1024 ? 2 : 1;
    const dim3 grid((unsigned)((g.M + rows_per - 1) / rows_per));
    if (g.D <= 8192)
        hipLaunchKernelGGL(norm_kernel<1>, grid, dim3(norm_threads(g.D, 1)), 0, st, g, rows_per);
    else if (g.D <= 16384)
        hipLaunchKernelGGL(norm_kernel<2>, grid, dim3(norm_threads(g.D, 2)), 0, st, g, rows_per);
    else
        hipLaunchKernelGGL(norm_kernel<4>, grid, dim3(norm_threads(g.D, 4)), 0, st, g, rows_per);
    return hipGetLastError();
}

// ==== backward =============================================================================
//
// With v = dh w_pre, xhat = x' r_x, yhat = y r_y, mean over a row's columns:
//   t  = dx' + r_x (v - xhat mean(v xhat))       the whole gradient of x'
//   dx = alpha t,  dn = gate t,  dgate = sum over rows of t n
//   z  = dn w_post,  dy = r_y (z - yhat mean(z yhat))
//   dw_pre = sum of dh xhat,  dw_post = sum of dn yhat
// mean(z yhat) is linear in t, so with c = mean(v xhat)
//   sum z yhat = sum k (dx' + r_x v) - c r_x sum k xhat,  k = gate w_post yhat:
// the three row sums come from one reduction.
//
// The column sums are held in fp32 registers over a workgroup's consecutive
// rows, written as partials, and added in a fixed order by a second kernel.
// A gate row whose rows all lie in one workgroup is written at once; one
// that crosses workgroups leaves a partial in each of them: in its first slot
// where the gate row is the workgroup's first, else in its second.

__device__ __forceinline__ float* part_pre(const NormBwdArgs& p, int64_t b) { return p.ws + b * 4 * p.D; }
__device__ __forceinline__ float* part_gate(const NormBwdArgs& p, int64_t b, int slot) {
    return p.ws + (b * 4 + 2 + slot) * p.D;
}

template <int NV>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdArgs p, int64_t rows_per) {
    __shared__ float red[2][16][3];
    int slot = 0;
    const int t = threadIdx.x, nt = blockDim.x;
    const int64_t r0 = blockIdx.x * rows_per, r1 = r0 + rows_per < p.M ? r0 + rows_per : p.M;
    const float inv_d = 1.0f / (float)p.D;
    int64_t col[NV];
    bool on[NV];
    float wpre[NV][8], wpost[NV][8], gate[NV][8];
    float apre[NV][8], apost[NV][8], agate[NV][8];
#pragma unroll
    for (int j = 0; j < NV; j++) {
        col[j] = 8 * (int64_t)(t + j * nt);
        on[j] = col[j] < p.D;
        if (p.dh) loadf8(p.w_pre + col[j], on[j], wpre[j]);
        if (p.w_post) loadf8(p.w_post + col[j], on[j], wpost[j]);
#pragma unroll
        for (int k = 0; k < 8; k++) apre[j][k] = apost[j][k] = agate[j][k] = 0.f;
    }
    int64_t have = -1;
    auto flush = [&](int64_t last_row) {  // the gate row `have`, whose rows here end at last_row
        const int64_t first = have * p.gate_rows;
        const int64_t end = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
        const bool whole = first >= r0 && end == last_row;
        float* to = whole ? p.dgate + have * p.D : part_gate(p, blockIdx.x, first <= r0 ? 0 : 1);
#pragma unroll
        for (int j = 0; j < NV; j++) {
            if (on[j]) {
                *(float4*)(to + col[j]) = make_float4(agate[j][0], agate[j][1], agate[j][2], agate[j][3]);
                *(float4*)(to + col[j] + 4) = make_float4(agate[j][4], agate[j][5], agate[j][6], agate[j][7]);
            }
#pragma unroll
            for (int k = 0; k < 8; k++) agate[j][k] = 0.f;
        }
    };
    for (int64_t r = r0; r < r1; r++) {
        float dxo[NV][8], dh[NV][8], xo[NV][8], y[NV][8];
#pragma unroll
        for (int j = 0; j < NV; j++) {
            load8(p.dxo + r * p.lddxo + col[j], on[j] && p.dxo, dxo[j]);
            if (p.dh) {
                load8(p.dh + r * p.lddh + col[j], on[j], dh[j]);
                load8(p.xo + r * p.ldxo + col[j], on[j], xo[j]);
            }
            if (p.y) load8(p.y + r * p.ldy + col[j], on[j], y[j]);
        }
        if (p.gate && r / p.gate_rows != have) {
            if (have >= 0) flush(r);
            have = r / p.gate_rows;
#pragma unroll
            for (int j = 0; j < NV; j++) loadf8(p.gate + have * p.D + col[j], on[j], gate[j]);
        }
        const float rx = p.dh ? p.rstd_x[r] : 0.f;
        const float ry = p.w_post ? p.rstd_y[r] : 1.f;
        // sums of v xhat, k (dx' + r_x v), k xhat
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; j++)
#pragma unroll
            for (int k = 0; k < 8; k++) {
                float xhat = 0.f;
                if (p.dh) {
                    xhat = xo[j][k] * rx;
                    const float v = dh[j][k] * wpre[j][k];
                    apre[j][k] += dh[j][k] * xhat;
                    s[0] += v * xhat;
                    dxo[j][k] += rx * v;
                    xo[j][k] = xhat;
                }
                if (p.w_post) {
                    float q = wpost[j][k] * (y[j][k] * ry);
                    if (p.gate) q *= gate[j][k];
                    s[1] += q * dxo[j][k];
                    s[2] += q * xhat;
                }
            }
        block_sum<3>(s, red, slot);
        const float c = rx * s[0] * inv_d;
        const float m = (s[1] - c * s[2]) * inv_d;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; k++) {
                if (p.dh) dxo[j][k] -= c * xo[j][k];
                o[k] = p.y ? p.alpha * dxo[j][k] : dxo[j][k];
            }
            if (on[j]) store8(p.dx + r * p.lddx + col[j], o);
            if (!p.y) continue;
#pragma unroll
            for (int k = 0; k < 8; k++) {
                float n = y[j][k], dn = dxo[j][k];
                const float yhat = n * ry;
                if (p.w_post) n = yhat * wpost[j][k];
                if (p.gate) {
                    agate[j][k] += dn * n;
                    dn *= gate[j][k];
                }
                if (p.w_post) {
                    apost[j][k] += dn * yhat;
                    dn = ry * (dn * wpost[j][k] - yhat * m);
                }
                o[k] = dn;
            }
            if (on[j]) store8(p.dy + r * p.lddy + col[j], o);
        }
    }
    if (p.gate && have >= 0) flush(r1);
#pragma unroll
    for (int j = 0; j < NV; j++) {
        if (!on[j]) continue;
        float* w = part_pre(p, blockIdx.x) + col[j];
        if (p.dh) {
            *(float4*)w = make_float4(apre[j][0], apre[j][1], apre[j][2], apre[j][3]);
            *(float4*)(w + 4) = make_float4(apre[j][4], apre[j][5], apre[j][6], apre[j][7]);
        }
        if (p.w_post) {
            *(float4*)(w + p.D) = make_float4(apost[j][0], apost[j][1], apost[j][2], apost[j][3]);
            *(float4*)(w + p.D + 4) = make_float4(apost[j][4], apost[j][5], apost[j][6], apost[j][7]);
        }
    }
}

// Adds the workgroups' partials: 64 columns, 16 interleaved runs of
// workgroups, then the runs in order.  blockIdx.y: 0 dw_pre, 1 dw_post, then
// the gate rows that cross workgroups -- by gate row, or (where there are more
// gate rows than workgroups) by the workgroup in which one starts.
__global__ __launch_bounds__(1024) void norm_bwd_reduce_kernel(NormBwdArgs p, int64_t rows_per, int by_part) {
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    int64_t b0 = 0, b1 = p.parts, row = 0;
    const int kind = blockIdx.y < 2 ? (int)blockIdx.y : 2;
    float* to;
    if (kind == 0) {
        to = p.dw_pre;
    } else if (kind == 1) {
        to = p.dw_post;
    } else {
        const int64_t i = (int64_t)blockIdx.y - 2;
        if (by_part) {
            // the gate row of workgroup i's last row, if it starts there
            const int64_t end = (i + 1) * rows_per < p.M ? (i + 1) * rows_per : p.M;
            row = (end - 1) / p.gate_rows;
            if (row * p.gate_rows < i * rows_per) return;
        } else {
            row = i;
        }
        const int64_t first = row * p.gate_rows;
        const int64_t end = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
        b0 = first / rows_per;
        b1 = (end - 1) / rows_per + 1;
        if (b1 - b0 == 1) return;  // written whole by its workgroup
        to = p.dgate + row * p.D;
    }
    if (!to) return;
    float v = 0.f;
    if (c < p.D)
        for (int64_t b = b0 + run; b < b1; b += 16)
            v += kind == 2 ? part_gate(p, b, row * p.gate_rows <= b * rows_per ? 0 : 1)[c]
                           : (part_pre(p, b) + kind * p.D)[c];
    lds[run][lane] = v;
    __syncthreads();
    if (run == 0 && c < p.D) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i++) v += lds[i][lane];
        to[c] = v;
    }
}

int norm_bwd_parts(int64_t M) {
    const int64_t per = (M + 511) / 512;
    return M == 0 ? 0 : (int)((M + per - 1) / per);
}

size_t norm_bwd_workspace(int64_t M, int64_t D) {
    return (size_t)norm_bwd_parts(M) * 4 * (size_t)D * sizeof(float);
}

hipError_t launch_norm_bwd(const NormBwdArgs& g, hipStream_t st) {
    if (g.D == 0) return hipSuccess;
    const int64_t rows_per = (g.M + g.parts - 1) / (g.parts > 0 ? g.parts : 1);
    if (g.M > 0) {
        const dim3 grid((unsigned)g.parts);
        if (g.D <= 8192)
            hipLaunchKernelGGL(norm_bwd_kernel<1>, grid, dim3(norm_threads(g.D, 1)), 0, st, g, rows_per);
        else if (g.D <= 16384)
            hipLaunchKernelGGL(norm_bwd_kernel<2>, grid, dim3(norm_threads(g.D, 2)), 0, st, g, rows_per);
        else
            hipLaunchKernelGGL(norm_bwd_kernel<4>, grid, dim3(norm_threads(g.D, 4)), 0, st, g, rows_per);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    int64_t ys = 2, by_part = 0;
    if (g.gate && g.M > 0) {
        const int64_t B = (g.M + g.gate_rows - 1) / g.gate_rows;
        by_part = B > g.parts;
        ys += by_part ? g.parts : B;
    }
    hipLaunchKernelGGL(norm_bwd_reduce_kernel, dim3((unsigned)((g.D + 63) / 64), (unsigned)ys), dim3(1024), 0, st, g,
                       rows_per, (int)by_part);
    return hipGetLastError();
}

}  // namespace fp8bs
