// norm.hip -- root-mean-square norms with the residual's addition, forward and
// backward, and the quantizers that make 8-bit operands, for gfx950 (MI355X).
//
// Forward, per row: s = x + r, S := s, rstd = (mean s^2 + eps)^-1/2,
// y = s rstd w, then Y := y or, in 8 bits, scale = max(max|y| / 448, 2^-100),
// Y := e4m3(y / scale).  The quantizer alone is the same row pass without the
// norm.  Bound by HBM (16384 x 4096 bf16 with the residual: forward 94 us = 5.7
// TB/s, backward 100 and 4 for dweight): every row is read once, held in registers (eight columns
// per lane and piece) between the sum of squares, the row maximum and the
// stores, and written once.
//
// A row of up to 1024 columns belongs to one wave (no barrier), several rows of up
// to 256 columns (the norms of attention heads) to one wave, 16 or 32 lanes each:
// with a wave per row, 64 columns leave 56 lanes idle (16-bit 64 Mi values: 361 us,
// 118 with 16 lanes).  Longer rows belong to a workgroup of 256 or 1024 threads,
// so that a lane holds at most 32 columns (64 columns in registers spill at 1024
// threads, so longer rows are refused).

#include "rows.h"

namespace dgemm {
namespace {

template <int FMT>
hipError_t row_by_mode(const RowArgs& a, bool norm, int rows, hipStream_t s) {
    if (!norm) return row_by_size<FMT, QUANT>(a, s);
    if (rows == ROWS_F8_BLOCK) return row_by_size<FMT, NORM_F8B>(a, s);
    return rows == ROWS_F8 ? row_by_size<FMT, NORM_F8>(a, s) : row_by_size<FMT, NORM>(a, s);
}

// ------------------------------------------------------- columns to 8 bits
//
// Q[n][m] := e4m3(X[m][n] / scale[n]), scale[n] from column n's largest
// magnitude: a weight matrix stored per input becomes gemm_f8's operand, stored
// per output.  One workgroup of 512 threads per 64 columns, two passes over
// them: the columns' maxima, then 64 x 64 tiles quantized and transposed in LDS
// (byte rows padded to 68 so that the eight columns a lane writes fall in
// different banks).  Done once per weight: 4096 x 4096 bf16 90 us (its bytes 10), 4096 x
// 14336 (K x N) 115 (34), 14336 x 4096 372 (34), bound by the latency of a workgroup's loads,
// one per thread in flight, and by CUs without one of the few workgroups.

constexpr int QT_THREADS = 512;

template <int FMT>
__global__ __launch_bounds__(QT_THREADS) void quant_cols_kernel(RowArgs a) {
    __shared__ uint32_t cmax[64][64];  // [row lane][column]
    __shared__ float cscale[64];
    __shared__ __attribute__((aligned(16))) unsigned char tile[64][68];
    const int n0 = (int)blockIdx.x * 64;
    const int t = threadIdx.x;
    const int c8 = (t & 7) * 8, rl = t >> 3;  // this thread's columns and row lane
    const int nvalid = a.N - (n0 + c8);
    uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int row = rl; row < a.M; row += 64) {
        Row8<FMT> x;
        x.load_from(a.X + ((int64_t)row * a.ldx + n0 + c8) * fmt_es<FMT>, nvalid);
        float v[8];
        x.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = mag_bits(v[j]);
            m[j] = b > m[j] ? b : m[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[rl][c8 + j] = m[j];
    __syncthreads();
    if (t < 64) {
        uint32_t s = 0;
        for (int i = 0; i < 64; ++i) s = cmax[i][t] > s ? cmax[i][t] : s;
        const float scale = f8_scale(s);
        cscale[t] = scale;
        if (n0 + t < a.N) a.scale[n0 + t] = scale;
    }
    __syncthreads();
    float sc[8], inv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sc[j] = cscale[c8 + j];
        inv[j] = 1.0f / sc[j];
    }
    for (int k0 = 0; k0 < a.M; k0 += 64) {
        const int row = k0 + rl;
        if (row < a.M) {
            Row8<FMT> x;
            x.load_from(a.X + ((int64_t)row * a.ldx + n0 + c8) * fmt_es<FMT>, nvalid);
            float v[8];
            x.get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t w = f8_pack4(f8_clamp(quotient(v[j], sc[j], inv[j])), 0.0f, 0.0f, 0.0f);
                tile[c8 + j][rl] = (unsigned char)(w & 0xffu);
            }
        }
        __syncthreads();
        // thread t: bytes 8 (t & 7) .. + 7 of output row t >> 3
        const int n = n0 + (t >> 3), k = k0 + (t & 7) * 8;
        if (n < a.N && k < a.M) {
            unsigned char* q = (unsigned char*)a.Y + (int64_t)n * a.ldy + k;
            const unsigned char* p = &tile[t >> 3][(t & 7) * 8];
            if (k + 8 <= a.M) {
                const uint32_t lo = *(const uint32_t*)p, hi = *(const uint32_t*)(p + 4);
                *(u32x2*)q = u32x2{lo, hi};
            } else {
                for (int j = 0; j < a.M - k; ++j) q[j] = p[j];
            }
        }
        __syncthreads();
    }
}

template <int FMT>
hipError_t go_quant_cols(const RowArgs& a, hipStream_t stream) {
    RowArgs b = a;
    void* args[] = {&b};
    return hipLaunchKernel((const void*)quant_cols_kernel<FMT>, dim3((unsigned)((a.N + 63) / 64)),
                           dim3(QT_THREADS), args, 0, stream);
}

// --------------------------------------------------------------- backward
//
// With xh = s rstd, g = dy w:  dx = rstd (g - xh mean(g xh)) + ds, and
// dw = sum over rows of dy xh.  Each workgroup walks rows blockIdx, blockIdx +
// grid, ...; a row's dy and s are loaded once, held in registers over the row's
// reduction, and the next row's loads are issued before it.  The thread's
// columns are the same in every row, so dw is a running fp32 sum in registers,
// written once per workgroup to the workspace and added over workgroups by
// col_reduce_kernel in a fixed order: no atomics, the same bits every time.

template <int FMT, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_bwd_kernel(NormBwdArgs a) {
    using P = Place<T>;
    constexpr int ES = fmt_es<FMT>;
    __shared__ float red[2][P::WG / 64];
    __shared__ float dwl[P::RPW > 1 ? P::WG * NV * 8 : 1];
    const P pl;
    const int t = pl.t;
    const int64_t step = (int64_t)gridDim.x * P::RPW;
    auto col = [&](int i) { return (i * T + t) * 8; };
    // 1024 threads have 128 registers each: no room for the next row's loads, nor
    // to keep the weights over the rows.
    constexpr bool PRE = T < 1024;
    float w[PRE ? NV : 1][8], dw[NV][8];
    const auto rw = make_rsrc((const char*)a.weight, (int64_t)a.N * 4);
    auto load_w = [&](int i, float (&to)[8]) {
        Row8<OUT_F32> w8;
        w8.load(rw, (uint32_t)col(i) * 4, a.N - col(i));
        w8.get(to);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if constexpr (PRE) load_w(i, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    Row8<FMT> y[NV], s[NV], d[NV];
    float next_rstd = 0.0f;
    // The rows of this wave from row0 on; rows past M and columns past N load as 0.
    auto load = [&](int64_t row0) {
        next_rstd = row0 + pl.lr < a.M ? a.rstd[row0 + pl.lr] : 0.0f;
        const auto ry = P::rows(a.dY, row0, a.M, a.N, a.lddy, ES);
        const auto rs = P::rows(a.S, row0, a.M, a.N, a.lds, ES);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            y[i].load(ry, pl.at(row0, a.M, a.N, col(i), a.lddy, ES), a.N - col(i));
            s[i].load(rs, pl.at(row0, a.M, a.N, col(i), a.lds, ES), a.N - col(i));
        }
        if (a.dS) {
            const auto rd = P::rows(a.dS, row0, a.M, a.N, a.ldds, ES);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                d[i].load(rd, pl.at(row0, a.M, a.N, col(i), a.ldds, ES), a.N - col(i));
        }
    };
    int64_t row0 = (int64_t)blockIdx.x * P::RPW + P::first();
    if (PRE && row0 < a.M) load(row0);
    int par = 0;
    for (; row0 < a.M; row0 += step, par ^= 1) {
        if (!PRE) load(row0);
        const float rstd = next_rstd;
        // The row stays in its storage format (half the registers of fp32 for
        // 16-bit rows); the few products are formed again after the reduction.
        Row8<FMT> cy[NV], cs[NV], cd[NV];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cy[i] = y[i];
            cs[i] = s[i];
            cd[i] = d[i];
            float dy[8], x[8];
            cy[i].get(dy);
            cs[i].get(x);
            float wt[8];
            if constexpr (!PRE) load_w(i, wt);
            const float(&wi)[8] = PRE ? w[PRE ? i : 0] : wt;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = x[j] * rstd;
                dot += dy[j] * wi[j] * xh;
                dw[i][j] += dy[j] * xh;
            }
        }
        if (PRE && row0 + step < a.M) load(row0 + step);
        // The reduction's words alternate between rows, so one barrier per row
        // is enough: a wave reaches the next but one row's write only after
        // every wave has passed the next row's barrier.
        const float mean = row_sum<T>(dot, red[par]) / (float)a.N;
        const auto ro = P::rows(a.dX, row0, a.M, a.N, a.lddx, ES);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float dy[8], x[8], o[8], e[8];
            cy[i].get(dy);
            cs[i].get(x);
            if (a.dS) cd[i].get(e);
            float wt[8];
            if constexpr (!PRE) load_w(i, wt);
            const float(&wi)[8] = PRE ? w[PRE ? i : 0] : wt;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = rstd * (dy[j] * wi[j] - x[j] * rstd * mean);
                if (a.dS) o[j] += e[j];
            }
            Row8<FMT> out;
            out.set(o);
            out.store(ro, pl.at(row0, a.M, a.N, col(i), a.lddx, ES), a.N - col(i));
        }
    }
    if (!a.part) return;
    if constexpr (P::RPW > 1) {
        // The workgroup's groups of T lanes hold the same columns: add them in order.
        const int sub = (int)threadIdx.x / T;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) dwl[(sub * NV * 8 + i * 8 + j) * T + t] = dw[i][j];
        __syncthreads();
        if (sub != 0) return;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                for (int q = 1; q < P::RPW; ++q) dw[i][j] += dwl[(q * NV * 8 + i * 8 + j) * T + t];
    }
    const auto rp = make_rsrc((const char*)(a.part + (int64_t)blockIdx.x * a.ldp), (int64_t)a.N * 4);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        Row8<OUT_F32> out;
        out.set(dw[i]);
        out.store(rp, (uint32_t)col(i) * 4, a.N - col(i));
    }
}

template <int FMT, int T, int NV>
hipError_t go_bwd(const NormBwdArgs& a, int grid, hipStream_t stream) {
    NormBwdArgs b = a;
    void* args[] = {&b};
    return hipLaunchKernel((const void*)norm_bwd_kernel<FMT, T, NV>, dim3((unsigned)grid),
                           dim3(T < 256 ? 256 : T), args, 0, stream);
}

template <int FMT>
hipError_t bwd_by_size(const NormBwdArgs& a, int grid, hipStream_t s) {
    if (a.N <= 128) return go_bwd<FMT, 16, 1>(a, grid, s);
    if (a.N <= 256) return go_bwd<FMT, 32, 1>(a, grid, s);
    if (a.N <= 512) return go_bwd<FMT, 64, 1>(a, grid, s);
    if (a.N <= 1024) return go_bwd<FMT, 64, 2>(a, grid, s);
    if (a.N <= 2048) return go_bwd<FMT, 256, 1>(a, grid, s);
    if (a.N <= 4096) return go_bwd<FMT, 256, 2>(a, grid, s);
    if (a.N <= 8192) return go_bwd<FMT, 512, 2>(a, grid, s);
    if (a.N <= NORM_BWD_MAX) return go_bwd<FMT, 1024, 2>(a, grid, s);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rows(const RowArgs& a, int fmt, bool norm, int rows, hipStream_t stream) {
    if (fmt == OUT_F32) return row_by_mode<OUT_F32>(a, norm, rows, stream);
    if (fmt == OUT_BF16) return row_by_mode<OUT_BF16>(a, norm, rows, stream);
    if (fmt == OUT_F16) return row_by_mode<OUT_F16>(a, norm, rows, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_quant_cols(const RowArgs& a, int fmt, hipStream_t stream) {
    if (fmt == OUT_F32) return go_quant_cols<OUT_F32>(a, stream);
    if (fmt == OUT_BF16) return go_quant_cols<OUT_BF16>(a, stream);
    if (fmt == OUT_F16) return go_quant_cols<OUT_F16>(a, stream);
    return hipErrorInvalidValue;
}

// Workgroups of the backward pass: enough to keep the rows' loads in flight (four
// per CU where a thread holds 8 columns, two where it holds 16, one of 1024
// threads); more only adds partial sums of dweight.
int norm_bwd_grid(int M, int N) {
    const int per = N <= 128 ? 16 : N <= 256 ? 8 : N <= 1024 ? 4 : 1;  // rows per workgroup
    const int64_t rows = ((int64_t)M + per - 1) / per;
    const bool light = N <= 512 || (N > 1024 && N <= 2048);
    const int64_t most = (N > 8192 ? 1 : light ? 4 : 2) * NUM_CU;
    // Two passes per workgroup before there are more workgroups than CUs: a row of
    // partial sums is written and read back per workgroup (512 x 8192 bf16 19.1 us
    // with a row each, 14.6 with two; 2000 x 1024 9.5 and 7.5).
    const int64_t two = (rows + 1) / 2 > NUM_CU ? (rows + 1) / 2 : rows < NUM_CU ? rows : NUM_CU;
    return (int)(two < most ? two : most);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int fmt, hipStream_t stream) {
    const int grid = norm_bwd_grid(a.M, a.N);
    if (fmt == OUT_F32) return bwd_by_size<OUT_F32>(a, grid, stream);
    if (fmt == OUT_BF16) return bwd_by_size<OUT_BF16>(a, grid, stream);
    if (fmt == OUT_F16) return bwd_by_size<OUT_F16>(a, grid, stream);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
