// actgrad.hip -- the elementwise half of a linear layer's backward pass, for
// gfx950 (MI355X): dZ = dC act'(Z) with the bias gradient's column sums, the
// reduction that finishes column sums, and the fp32 transpose.
//
// dZ is written in the products' input format: the matrix instructions take
// 16-bit operands, so for 16-bit layers this is the one rounding between dC and
// the gradients (half a step, 2^-8 relative for bf16, as the rounding of the
// gradients it feeds).  dbias sums the unrounded fp32 values.
//
// Bound by memory: 4096 x 4096 bf16, dC and Z read and dZ written once, 22-26 us
// (100 MB at 3.9 to 4.6 TB/s), beside 223 us of products.

#include "kern_common.h"

namespace dgemm {
namespace {

// act'(z) times d, with the forward's own forms for Z's format CF (kern_common.h):
//   z sigmoid(p), p = a z + b z^3:  s + z s (1 - s)(a + 3 b z^2), s = sigmoid(p)
//   z Phi(z):                       Phi(z) + z phi(z)
//   relu:                           z > 0
// With e = exp(-|p|) and r = 1 / (1 + e), s is r or, for p < 0, e r, and s (1 - s) = e r^2:
// 1 - s itself would carry s's rounding, near s = 1 many times the term (off by, in half
// steps of 1, gelu_tanh at 4 to 8: 33, so 2.0; silu at 8 to 20: 16, so 2.4; so nowhere more
// than 3.7).  Far out the term is 0 while
// z^3 stays finite; where z^2 itself overflows or z is infinite, the factor is taken as 0
// or 1 by z's sign.
template <int CF, int NE>
__device__ __forceinline__ void apply_act_grad(float (&d)[NE], const float (&z)[NE], int act) {
    if (act >= ACT_GELU_TANH) {
        const float a = act == ACT_SILU ? 1.0f : GELU_A, b = act == ACT_SILU ? 0.0f : GELU_B;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float p = z[i] * (a + b * z[i] * z[i]);
            const float e = __builtin_amdgcn_exp2f(-LOG2E * __builtin_fabsf(p));
            const float r = __builtin_amdgcn_rcpf(1.0f + e);
            const float er = e * r;
            const float f = (p < 0.0f ? er : r) + z[i] * (er * r) * (a + 3.0f * b * z[i] * z[i]);
            const float far = z[i] > 0.0f ? 1.0f : 0.0f;
            d[i] *= __builtin_fabsf(z[i]) > 1e4f ? far : f;
        }
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float x = z[i];
            float e;
            const float far = x > 0.0f ? 1.0f : 0.0f;
            const float cdf = normal_cdf<CF>(x, e);
            const float f = cdf + x * (0.3989422804014327f * e);
            d[i] *= __builtin_fabsf(x) > 1e4f ? far : f;
        }
    } else if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < NE; ++i) d[i] = z[i] > 0.0f ? d[i] : (z[i] != z[i] ? z[i] : 0.0f);
    }
}

constexpr int AG_COLS = 512;     // columns per workgroup: 64 lanes x 8

// One workgroup of W waves: columns blockIdx.x * 512 .., rows blockIdx.y *
// rows_per ...  T lanes share a row, so narrow layers put 64 / T rows into a wave
// (64 columns, 300000 rows: 497 us with a wave per row, 38.5 with 16 lanes,
// the column sums' second step included); the
// W 64 / T rows of a pass interleave.  The column sums of a workgroup's lanes are
// added in LDS in order and go to the workspace, one row of partial sums per
// blockIdx.y.  Sixteen waves where one workgroup takes all the rows.
template <int CF, int DF, int W, int T>
__global__ __launch_bounds__(64 * W) void act_grad_kernel(ActGradArgs a) {
    constexpr int RP = 64 / T;  // rows per wave and pass
    __shared__ float sums[W * AG_COLS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int lr = lane / T;
    const int c = (int)blockIdx.x * AG_COLS + (lane % T) * 8;
    const int nvalid = a.N - c;
    const int64_t r0 = (int64_t)blockIdx.y * a.rows_per;
    const int64_t r1 = r0 + a.rows_per < a.M ? r0 + a.rows_per : a.M;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 2
    for (int64_t row = r0 + wave * RP; row < r1; row += W * RP) {
        const int n = r1 - row < RP ? (int)(r1 - row) : RP;  // this wave's rows
        auto rows = [&](const char* p, int ld, int es) {
            return make_rsrc(p + row * ld * es, ((int64_t)(n - 1) * ld + a.N) * es);
        };
        // Rows and columns outside load as 0 and are not stored.
        auto at = [&](int ld, int es) {
            return lr < n && nvalid > 0 ? (uint32_t)((lr * ld + c) * es) : OOB_LANE;
        };
        Row8<CF> x, zz;
        x.load(rows(a.dC, a.lddc, fmt_es<CF>), at(a.lddc, fmt_es<CF>), nvalid);
        float d[8];
        if (a.Z) {
            zz.load(rows(a.Z, a.ldz, fmt_es<CF>), at(a.ldz, fmt_es<CF>), nvalid);
            float z[8];
            x.get(d);
            zz.get(z);
            apply_act_grad<CF>(d, z, a.act);
        } else {
            x.get(d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += d[j];
        if (a.dZ) {
            Row8<DF> o;
            o.set(d);
            o.store(rows(a.dZ, a.lddz, fmt_es<DF>), at(a.lddz, fmt_es<DF>), nvalid);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[wave * AG_COLS + lane * 8 + j] = sum[j];
    __syncthreads();
    for (int j = threadIdx.x; j < T * 8; j += 64 * W) {
        const int col = (int)blockIdx.x * AG_COLS + j;
        if (col >= a.N) break;
        float v = sums[j];
#pragma unroll
        for (int q = 1; q < W * RP; ++q) v += sums[q * T * 8 + j];
        a.part[(int64_t)blockIdx.y * a.ldp + col] = v;
    }
}

// The same for a gated layer: dG = dC U act'(G) and dU = dC act(G), with both column sums.  Bound by
// memory too, five arrays instead of three.
//
// In 16 bits dG and dU are rounded to the operands' format, since the products that read them run at
// the 16-bit matrix rate (a second term for what the rounding drops would double their work): the
// gradients are off by 2.3e-3 of their 2-norm in bf16 and 2.9e-4 in fp16, where products of the
// unrounded values give, with the results' own rounding, 1.7e-3 and 2.1e-4.  The column sums take the
// unrounded values.
template <int CF, int DF, int W, int T>
__global__ __launch_bounds__(64 * W) void gated_grad_kernel(GatedGradArgs a) {
    constexpr int RP = 64 / T;  // rows per wave and pass
    __shared__ float sums[2][W * AG_COLS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int lr = lane / T;
    const int c = (int)blockIdx.x * AG_COLS + (lane % T) * 8;
    const int nvalid = a.N - c;
    const int64_t r0 = (int64_t)blockIdx.y * a.rows_per;
    const int64_t r1 = r0 + a.rows_per < a.M ? r0 + a.rows_per : a.M;
    float sg[8] = {0, 0, 0, 0, 0, 0, 0, 0}, su[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 2
    for (int64_t row = r0 + wave * RP; row < r1; row += W * RP) {
        const int n = r1 - row < RP ? (int)(r1 - row) : RP;  // this wave's rows
        auto rows = [&](const char* p, int ld, int es) {
            return make_rsrc(p + row * ld * es, ((int64_t)(n - 1) * ld + a.N) * es);
        };
        auto at = [&](int ld, int es) {
            return lr < n && nvalid > 0 ? (uint32_t)((lr * ld + c) * es) : OOB_LANE;
        };
        Row8<CF> x, y, z;
        x.load(rows(a.dC, a.lddc, fmt_es<CF>), at(a.lddc, fmt_es<CF>), nvalid);
        y.load(rows(a.G, a.ldg, fmt_es<CF>), at(a.ldg, fmt_es<CF>), nvalid);
        z.load(rows(a.U, a.ldu, fmt_es<CF>), at(a.ldu, fmt_es<CF>), nvalid);
        float d[8], g[8], u[8], dg[8], du[8];
        x.get(d);
        y.get(g);
        z.get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dg[j] = d[j] * u[j];
            du[j] = g[j];
        }
        apply_act_grad<CF>(dg, g, a.act);
        apply_act<CF>(du, a.act);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            du[j] *= d[j];
            sg[j] += dg[j];
            su[j] += du[j];
        }
        if (a.dG) {
            Row8<DF> o;
            o.set(dg);
            o.store(rows(a.dG, a.lddz, fmt_es<DF>), at(a.lddz, fmt_es<DF>), nvalid);
            o.set(du);
            o.store(rows(a.dU, a.lddz, fmt_es<DF>), at(a.lddz, fmt_es<DF>), nvalid);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sums[0][wave * AG_COLS + lane * 8 + j] = sg[j];
        sums[1][wave * AG_COLS + lane * 8 + j] = su[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * T * 8; i += 64 * W) {
        const int which = i / (T * 8), j = i % (T * 8);
        const int col = (int)blockIdx.x * AG_COLS + j;
        if (col >= a.N) continue;
        float v = sums[which][j];
#pragma unroll
        for (int q = 1; q < W * RP; ++q) v += sums[which][q * T * 8 + j];
        a.part[((int64_t)blockIdx.y * 2 + which) * a.ldp + col] = v;
    }
}

template <int CF, int DF, int T>
hipError_t go_gg(const GatedGradArgs& a, hipStream_t stream) {
    GatedGradArgs b = a;
    void* args[] = {&b};
    const bool one = a.M > 16 && a.M <= a.rows_per;
    const void* fn = one ? (const void*)gated_grad_kernel<CF, DF, 16, T> : (const void*)gated_grad_kernel<CF, DF, 4, T>;
    return hipLaunchKernel(fn,
                           dim3((unsigned)((a.N + AG_COLS - 1) / AG_COLS),
                                (unsigned)((a.M + a.rows_per - 1) / a.rows_per)),
                           dim3(one ? 1024 : 256), args, 0, stream);
}

template <int CF, int DF>
hipError_t gg_by_size(const GatedGradArgs& a, hipStream_t stream) {
    if (a.N <= 128) return go_gg<CF, DF, 16>(a, stream);
    if (a.N <= 256) return go_gg<CF, DF, 32>(a, stream);
    return go_gg<CF, DF, 64>(a, stream);
}

template <int CF, int DF, int T>
hipError_t go_ag(const ActGradArgs& a, hipStream_t stream) {
    ActGradArgs b = a;
    void* args[] = {&b};
    const bool one = a.M > 16 && a.M <= a.rows_per;
    const void* fn = one ? (const void*)act_grad_kernel<CF, DF, 16, T> : (const void*)act_grad_kernel<CF, DF, 4, T>;
    return hipLaunchKernel(fn,
                           dim3((unsigned)((a.N + AG_COLS - 1) / AG_COLS),
                                (unsigned)((a.M + a.rows_per - 1) / a.rows_per)),
                           dim3(one ? 1024 : 256), args, 0, stream);
}

template <int CF, int DF>
hipError_t ag_by_size(const ActGradArgs& a, hipStream_t stream) {
    if (a.N <= 128) return go_ag<CF, DF, 16>(a, stream);
    if (a.N <= 256) return go_ag<CF, DF, 32>(a, stream);
    return go_ag<CF, DF, 64>(a, stream);
}

__global__ __launch_bounds__(256) void col_reduce_kernel(ColReduceArgs a) {
    __shared__ float lds[COL_REDUCE_LDS];
    col_reduce((int)blockIdx.x, a, lds);
}

__global__ __launch_bounds__(256) void col_reduce2_kernel(ColReduceArgs a, ColReduceArgs b, int blocks_a) {
    __shared__ float lds[COL_REDUCE_LDS];
    if ((int)blockIdx.x < blocks_a) col_reduce((int)blockIdx.x, a, lds);
    else col_reduce((int)blockIdx.x - blocks_a, b, lds);
}

// Y[n][m] = X[m][n], fp32, in 32 x 32 tiles through LDS (rows padded to 33 words):
// small enough that the backward pass of a small layer still fills the CUs.
__global__ __launch_bounds__(256) void transpose32_kernel(const float* X, int ldx, int M, int N,
                                                          float* Y, int ldy, int tiles_n) {
    __shared__ float tile[32][33];
    const int m0 = (int)(blockIdx.x / tiles_n) * 32, n0 = (int)(blockIdx.x % tiles_n) * 32;
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (m0 + r + i < M && n0 + c < N) tile[r + i][c] = X[(int64_t)(m0 + r + i) * ldx + n0 + c];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (n0 + r + i < N && m0 + c < M) Y[(int64_t)(n0 + r + i) * ldy + m0 + c] = tile[c][r + i];
}

}  // namespace

// Rows per workgroup of act_grad_kernel, one row of partial sums each.  Up to 64 rows: one
// workgroup's, whose sums are dbias without a second launch (4 rows for each of 16 waves;
// 16 rows each measured 16-35 us where two launches take 10).  More: as many rows as
// leave at most 512 workgroups per column block, or 2048 in all where there are fewer than
// four blocks, but at least 16, or an M / 256th if that is fewer, and never below 8 (4096 x
// 4096, column sums alone: 20.5 us with 8 rows, 19.1 with 16), in whole passes of four waves.
int act_grad_rows(int M, int N) {
    if (M <= 64) return 64;
    const int blocks = (N + AG_COLS - 1) / AG_COLS;
    const int most = blocks >= 4 ? 512 : 2048 / (blocks > 0 ? blocks : 1);
    const int unit = N <= 128 ? 16 : N <= 256 ? 8 : 4;  // rows of a pass of four waves
    const int64_t share = ((int64_t)M + 255) / 256;
    int64_t r = ((int64_t)M + most - 1) / most;
    if (r < (share < 16 ? share : 16)) r = share < 16 ? share : 16;
    if (r < 8) r = 8;
    return (int)((r + unit - 1) / unit * unit);
}

hipError_t launch_act_grad(const ActGradArgs& a, int cf, int df, hipStream_t stream) {
    if (cf == OUT_F32 && df == OUT_F32) return ag_by_size<OUT_F32, OUT_F32>(a, stream);
    if (cf == OUT_F32 && df == OUT_BF16) return ag_by_size<OUT_F32, OUT_BF16>(a, stream);
    if (cf == OUT_F32 && df == OUT_F16) return ag_by_size<OUT_F32, OUT_F16>(a, stream);
    if (cf == OUT_BF16 && df == OUT_BF16) return ag_by_size<OUT_BF16, OUT_BF16>(a, stream);
    if (cf == OUT_F16 && df == OUT_F16) return ag_by_size<OUT_F16, OUT_F16>(a, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int cf, int df, hipStream_t stream) {
    if (cf == OUT_F32 && df == OUT_F32) return gg_by_size<OUT_F32, OUT_F32>(a, stream);
    if (cf == OUT_F32 && df == OUT_BF16) return gg_by_size<OUT_F32, OUT_BF16>(a, stream);
    if (cf == OUT_F32 && df == OUT_F16) return gg_by_size<OUT_F32, OUT_F16>(a, stream);
    if (cf == OUT_BF16 && df == OUT_BF16) return gg_by_size<OUT_BF16, OUT_BF16>(a, stream);
    if (cf == OUT_F16 && df == OUT_F16) return gg_by_size<OUT_F16, OUT_F16>(a, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_col_reduce(const ColReduceArgs& a, hipStream_t stream) {
    ColReduceArgs b = a;
    void* args[] = {&b};
    return hipLaunchKernel((const void*)col_reduce_kernel, dim3((unsigned)col_reduce_blocks(a.N)),
                           dim3(256), args, 0, stream);
}

hipError_t launch_col_reduce2(const ColReduceArgs& a, const ColReduceArgs& b, hipStream_t stream) {
    ColReduceArgs x = a, y = b;
    int na = a.N > 0 ? col_reduce_blocks(a.N) : 0;
    const int nb = b.N > 0 ? col_reduce_blocks(b.N) : 0;
    if (na + nb == 0) return hipSuccess;
    void* args[] = {&x, &y, &na};
    return hipLaunchKernel((const void*)col_reduce2_kernel, dim3((unsigned)(na + nb)), dim3(256), args, 0,
                           stream);
}

hipError_t launch_transpose32(const float* X, int ldx, int M, int N, float* Y, int ldy,
                              hipStream_t stream) {
    const int64_t tm = ((int64_t)M + 31) / 32, tn = ((int64_t)N + 31) / 32;
    if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
    int tiles_n = (int)tn;
    void* args[] = {&X, &ldx, &M, &N, &Y, &ldy, &tiles_n};
    return hipLaunchKernel((const void*)transpose32_kernel, dim3((unsigned)(tm * tn)), dim3(256), args,
                           0, stream);
}

}  // namespace dgemm
