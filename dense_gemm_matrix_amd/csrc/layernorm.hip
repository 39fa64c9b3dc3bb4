// layernorm.hip -- layer norm with the residual's addition, forward and backward, for
// gfx950 (MI355X).
//
// The forward pass is the row pass of rows.h.  Bound by HBM, as the root-mean-square
// norm's: each row is read once, held in registers over its two reductions (mean, then
// the deviations and their squares) and written once.
//
// Backward: with xh = (s - mean) rstd and g = dy w,
//   dx = rstd (g - mean(g) - xh mean(g xh)) + ds,  dw = sum over rows of dy xh,
//   db = sum over rows of dy.
// As the root-mean-square norm's (norm.hip): each workgroup walks rows blockIdx, blockIdx +
// grid, ..., the next row's loads in flight over this one's reduction, whose two sums share one
// barrier; a thread's columns are the same in every row, so dw and db are running fp32 sums in
// registers (from 8193 columns on in LDS), written once per workgroup and added over workgroups
// in a fixed order by one more launch for both.

#include "rows.h"

namespace dgemm {
namespace {

// Two sums over the T threads that share a row, with one barrier; red: T / 64 words each.
template <int T>
__device__ __forceinline__ void row_sum2(float& x, float& y, float (*red)[Place<T>::WG / 64]) {
#pragma unroll
    for (int m = (T < 64 ? T : 64) / 2; m > 0; m >>= 1) {
        x += __shfl_xor(x, m);
        y += __shfl_xor(y, m);
    }
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) {
            red[0][threadIdx.x >> 6] = x;
            red[1][threadIdx.x >> 6] = y;
        }
        __syncthreads();
        x = red[0][0];
        y = red[1][0];
#pragma unroll
        for (int i = 1; i < T / 64; ++i) {
            x += red[0][i];
            y += red[1][i];
        }
    }
}

template <int FMT>
hipError_t ln_by_rows(const RowArgs& a, int rows, hipStream_t s) {
    if (rows == ROWS_F8_BLOCK) return row_by_size<FMT, LN_F8B>(a, s);
    return rows == ROWS_F8 ? row_by_size<FMT, LN_F8>(a, s) : row_by_size<FMT, LN>(a, s);
}

template <int FMT, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void ln_bwd_kernel(NormBwdArgs a) {
    using P = Place<T>;
    constexpr int ES = fmt_es<FMT>;
    __shared__ float red[2][2][P::WG / 64];
    __shared__ float dwl[P::RPW > 1 ? P::WG * NV * 8 : 1];
    const P pl;
    const int t = pl.t;
    const int64_t step = (int64_t)gridDim.x * P::RPW;
    auto col = [&](int i) { return (i * T + t) * 8; };
    // 1024 threads have 128 registers each: no room for the next row's loads, nor to keep the
    // weights over the rows, and the running sums are in LDS, a thread's own in its own words (4000 x
    // 16384 bf16 130 us, fp32 218; with the sums in registers, 30 of them in scratch, 197 and 275).
    constexpr bool PRE = T < 1024, IN_LDS = T == 1024;
    __shared__ f32x4 lsum[IN_LDS ? 4 * NV : 1][IN_LDS ? T : 1];  // dw's halves of eight columns, then db's
    float w[PRE ? NV : 1][8], dw[NV][8], db[NV][8];
    auto to_lds = [&](int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            lsum[2 * i + h][t] = f32x4{dw[i][4 * h], dw[i][4 * h + 1], dw[i][4 * h + 2], dw[i][4 * h + 3]};
            lsum[2 * (NV + i) + h][t] = f32x4{db[i][4 * h], db[i][4 * h + 1], db[i][4 * h + 2], db[i][4 * h + 3]};
        }
    };
    auto from_lds = [&](int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 x = lsum[2 * i + h][t], y = lsum[2 * (NV + i) + h][t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dw[i][4 * h + j] = x[j];
                db[i][4 * h + j] = y[j];
            }
        }
    };
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
        for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
        if (IN_LDS) to_lds(i);
    }
    // Rows in flight beside the one at work: its time is far below memory's latency, so two where eight
    // 16-bit columns per thread leave them room (8192 x 2048 bf16 27.9 us, 31.2 with one; with 16 columns
    // 16384 x 4096 112 us, 106 with one).
    constexpr int D = PRE && FMT != OUT_F32 && NV == 1 ? 2 : 1;
    const bool ragged = (a.N & 7) != 0;
    Row8<FMT> y[D][NV], s[D][NV], d[D][NV];
    float next_rstd[D], next_mean[D];
    // The rows of this wave from row0 on; rows past M load as 0.  Columns past N are zeroed where the
    // values are used: here that would wait for them (1000 x 2999 f16 17.0 us, 15.1 this way).
    auto load = [&](int64_t row0, auto slot) {
        constexpr int q = decltype(slot)::value;
        next_rstd[q] = row0 + pl.lr < a.M ? a.rstd[row0 + pl.lr] : 0.0f;
        next_mean[q] = row0 + pl.lr < a.M ? a.mean[row0 + pl.lr] : 0.0f;
        const auto ry = P::rows(a.dY, row0, a.M, a.N, a.lddy, ES);
        const auto rs = P::rows(a.S, row0, a.M, a.N, a.lds, ES);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            y[q][i].load_whole(ry, pl.at(row0, a.M, a.N, col(i), a.lddy, ES));
            s[q][i].load_whole(rs, pl.at(row0, a.M, a.N, col(i), a.lds, ES));
        }
        if (a.dS) {
            const auto rd = P::rows(a.dS, row0, a.M, a.N, a.ldds, ES);
#pragma unroll
            for (int i = 0; i < NV; ++i) d[q][i].load_whole(rd, pl.at(row0, a.M, a.N, col(i), a.ldds, ES));
        }
    };
    using Slot0 = std::integral_constant<int, 0>;
    using Slot1 = std::integral_constant<int, D - 1>;
    int par = 0;
    auto pass = [&](int64_t row0, auto slot) {
        constexpr int q = decltype(slot)::value;
        if (!PRE) load(row0, slot);
        const float rstd = next_rstd[q], mean = next_mean[q];
        // The row stays in its storage format (half the registers of fp32 for
        // 16-bit rows); the few products are formed again after the reduction.
        Row8<FMT> cy[NV], cs[NV], cd[NV];
        float dot = 0.0f, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cy[i] = y[q][i];
            cs[i] = s[q][i];
            cd[i] = d[q][i];
            if (ragged && a.N - col(i) < 8) {
                cy[i].mask(a.N - col(i));
                cs[i].mask(a.N - col(i));
            }
            float dy[8], x[8];
            cy[i].get(dy);
            cs[i].get(x);
            float wt[8];
            if constexpr (!PRE) load_w(i, wt);
            const float(&wi)[8] = PRE ? w[PRE ? i : 0] : wt;
            if (IN_LDS) from_lds(i);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = (x[j] - mean) * rstd, gj = dy[j] * wi[j];
                sum += gj;
                dot += gj * xh;
                dw[i][j] += dy[j] * xh;
                db[i][j] += dy[j];
            }
            if (IN_LDS) to_lds(i);
        }
        if (PRE && row0 + D * step < a.M) load(row0 + D * step, slot);
        // The reduction's words alternate between rows, so one barrier per row
        // is enough: a wave reaches the next but one row's write only after
        // every wave has passed the next row's barrier.
        row_sum2<T>(sum, dot, red[par]);
        const float mg = sum / (float)a.N, mgx = dot / (float)a.N;
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
                o[j] = rstd * (dy[j] * wi[j] - mg - (x[j] - mean) * rstd * mgx);
                if (a.dS) o[j] += e[j];
            }
            Row8<FMT> out;
            out.set(o);
            out.store(ro, pl.at(row0, a.M, a.N, col(i), a.lddx, ES), a.N - col(i));
        }
        par ^= 1;
    };
    int64_t row0 = (int64_t)blockIdx.x * P::RPW + P::first();
    if (PRE && row0 < a.M) load(row0, Slot0{});
    if (D > 1 && row0 + step < a.M) load(row0 + step, Slot1{});
    for (; row0 < a.M; row0 += D * step) {
        pass(row0, Slot0{});
        if (D > 1 && row0 + step < a.M) pass(row0 + step, Slot1{});
    }
    if (!a.part) return;
    if (IN_LDS)
#pragma unroll
        for (int i = 0; i < NV; ++i) from_lds(i);
    // dw's partial sums, then db's, a row of ldp each per workgroup.
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        auto& v = which ? db : dw;
        if constexpr (P::RPW > 1) {
            // The workgroup's groups of T lanes hold the same columns: add them in order.
            const int sub = (int)threadIdx.x / T;
            if (which) __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) dwl[(sub * NV * 8 + i * 8 + j) * T + t] = v[i][j];
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        for (int q = 1; q < P::RPW; ++q) v[i][j] += dwl[(q * NV * 8 + i * 8 + j) * T + t];
            }
        }
        if (P::RPW > 1 && (int)threadIdx.x >= T) continue;
        const auto rp = make_rsrc((const char*)(a.part + ((int64_t)blockIdx.x * 2 + which) * a.ldp),
                                  (int64_t)a.N * 4);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Row8<OUT_F32> out;
            out.set(v[i]);
            out.store(rp, (uint32_t)col(i) * 4, a.N - col(i));
        }
    }
}

template <int FMT, int T, int NV>
hipError_t go_bwd(const NormBwdArgs& a, int grid, hipStream_t stream) {
    NormBwdArgs b = a;
    void* args[] = {&b};
    return hipLaunchKernel((const void*)ln_bwd_kernel<FMT, T, NV>, dim3((unsigned)grid),
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

hipError_t launch_layernorm(const RowArgs& a, int fmt, int rows, hipStream_t stream) {
    if (fmt == OUT_F32) return ln_by_rows<OUT_F32>(a, rows, stream);
    if (fmt == OUT_BF16) return ln_by_rows<OUT_BF16>(a, rows, stream);
    if (fmt == OUT_F16) return ln_by_rows<OUT_F16>(a, rows, stream);
    return hipErrorInvalidValue;
}

// Workgroups of the backward pass.  Each writes two rows of partial sums, which are read once
// more, so every CU has one workgroup before any has two, and a second only from four passes
// each on (1000 x 8192 bf16 24.0 us with 256, 32.8 with 500; 1000 x 3000 f16 17.1 and 18.7;
// 8192 x 512 bf16 11.5 with 512, 13.5 with 256, 13.2 with 1024).  In fp32 a row takes twice as long
// and one per CU is enough (16384 x 4096 194 us with 256, 206 with 512; 4096 x 1024 15.6 and 17.2;
// 8192 x 512 15.1 and 15.7), as it is from 8192 columns on, with 16 waves each.
int layernorm_bwd_grid(int M, int N, int fmt) {
    const int per = N <= 128 ? 16 : N <= 256 ? 8 : N <= 1024 ? 4 : 1;  // rows per pass of a workgroup
    const int64_t rows = ((int64_t)M + per - 1) / per;
    if (rows <= NUM_CU) return (int)rows;
    const int most = fmt == OUT_F32 || N > 8192 ? NUM_CU : 2 * NUM_CU;
    const int64_t four = rows / 4;
    return four < NUM_CU ? NUM_CU : four < most ? (int)four : most;
}

hipError_t launch_layernorm_bwd(const NormBwdArgs& a, int fmt, hipStream_t stream) {
    const int grid = layernorm_bwd_grid(a.M, a.N, fmt);
    if (fmt == OUT_F32) return bwd_by_size<OUT_F32>(a, grid, stream);
    if (fmt == OUT_BF16) return bwd_by_size<OUT_BF16>(a, grid, stream);
    if (fmt == OUT_F16) return bwd_by_size<OUT_F16>(a, grid, stream);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
