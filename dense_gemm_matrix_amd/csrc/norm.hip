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

#include <type_traits>

#include "kern_common.h"

namespace dgemm {
namespace {

constexpr float F8_MAX = 448.0f;                       // largest e4m3 value
constexpr float SCALE_MIN = 7.888609052210118e-31f;    // 2^-100: a row of zeros divides by it

// Reductions over the T threads that share a row (T <= 64: lanes of one wave;
// else the whole workgroup, in wave order), every thread getting the same bits.
// `red` holds T / 64 words and is not shared with another reduction of the row.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int m = (T < 64 ? T : 64) / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (T <= 64) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) s += red[i];
    return s;
}
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
#pragma unroll
    for (int m = (T < 64 ? T : 64) / 2; m > 0; m >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, m);
        v = o > v ? o : v;
    }
    if constexpr (T <= 64) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t s = red[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) s = red[i] > s ? red[i] : s;
    return s;
}

// |v| as an integer that orders like the magnitudes, infinities and NaN on top.
__device__ __forceinline__ uint32_t mag_bits(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

// The scale of a row (or column) whose largest magnitude is `bits`.  A row that
// holds an infinity or a NaN has no scale: NaN, so every value it stands for is one.
__device__ __forceinline__ float f8_scale(uint32_t bits) {
    if (bits >= 0x7f800000u) return __builtin_nanf("");
    const float s = as_float(bits) / F8_MAX;
    return s > SCALE_MIN ? s : SCALE_MIN;
}

// v / scale, correctly rounded: the product with the rounded reciprocal and one
// correction by the exact remainder (Markstein's division), three operations where
// the compiler's general division takes a dozen and made the quantizer wait for
// arithmetic.  The quotient has to be fp32's own: e4m3 rounding has ties (the 16-bit
// inputs meet them often), and a product with the reciprocal falls on their wrong
// side.  Equal to the fp32 quotient on every pair of 16-bit significands and on 5e7
// fp32 pairs, half of them next to a tie.  scale is in [2^-100, 2^120] and the quotient
// below 449 in magnitude, so only the remainder of the smallest scales leaves the normal
// range, by less than the correction's own rounding (equal down to rows of 2^-126).
__device__ __forceinline__ float quotient(float v, float scale, float inv) {
    const float q = v * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, scale, v), inv, q);
}
__device__ __forceinline__ float f8_clamp(float q) {
    return q > F8_MAX ? F8_MAX : q < -F8_MAX ? -F8_MAX : q;
}
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Eight values quantized and stored at byte offset `off` of a row of bytes.
__device__ __forceinline__ void store_f8(__amdgpu_buffer_rsrc_t r, uint32_t off, int nvalid,
                                         const float (&v)[8], float scale, float inv) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = f8_clamp(quotient(v[j], scale, inv));
    const u32x2 w = {f8_pack4(q[0], q[1], q[2], q[3]), f8_pack4(q[4], q[5], q[6], q[7])};
    if (nvalid >= 8) {
        __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)off, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < nvalid)
                __builtin_amdgcn_raw_buffer_store_b8((unsigned char)(w[j >> 2] >> (8 * (j & 3))), r,
                                                     (int)(off + j), 0, 0);
    }
}

// Where a lane works: the rows of its wave start at `row0` (wave-uniform, so that
// the rows' resources live in scalar registers), its own is row0 + lr.  Fewer than
// 64 threads per row put 64 / T rows into a wave.
template <int T>
struct Place {
    static constexpr int WG = T < 256 ? 256 : T;
    static constexpr int RPWAVE = T < 64 ? 64 / T : 1;
    static constexpr int RPW = WG / T;  // rows per workgroup
    int t, lr;

    __device__ __forceinline__ Place() : t(threadIdx.x % T), lr(T < 64 ? (threadIdx.x & 63) / T : 0) {}
    // The first row of this wave among the workgroup's.
    __device__ __forceinline__ static int first() {
        return RPW > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) * RPWAVE : 0;
    }
    // A resource over the wave's rows of a matrix of es-byte elements.
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rows(const void* p, int64_t row0, int M,
                                                                  int N, int ld, int es) {
        const int64_t n = M - row0 < RPWAVE ? M - row0 : RPWAVE;
        return make_rsrc((const char*)p + row0 * ld * es, ((n - 1) * ld + N) * es);
    }
    // Byte offset of column c of this lane's row in it.
    __device__ __forceinline__ uint32_t at(int64_t row0, int M, int N, int c, int ld, int es) const {
        if constexpr (RPWAVE == 1) return (uint32_t)(c * es);  // past N: outside the resource
        return row0 + lr < M && c < N ? (uint32_t)((lr * ld + c) * es) : OOB_LANE;
    }
};

// FMT: format of X, R, S and (MODE NORM) Y.
enum RowMode { NORM = 0, NORM_F8 = 1, QUANT = 2 };

template <int FMT, int MODE, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void row_kernel(RowArgs a) {
    constexpr int ES = fmt_es<FMT>;
    using P = Place<T>;
    __shared__ float red_s[P::WG / 64];
    __shared__ uint32_t red_m[P::WG / 64];
    const P pl;
    const int64_t row0 = (int64_t)blockIdx.x * P::RPW + P::first();
    if (row0 >= a.M) return;  // T <= 64 only: no barrier follows
    const int64_t row = row0 + pl.lr;
    auto col = [&](int i) { return (i * T + pl.t) * 8; };
    auto at = [&](int i, int ld, int es) { return pl.at(row0, a.M, a.N, col(i), ld, es); };
    float v[NV][8];
    Row8<FMT> x[NV], r[NV];
    const auto rx = P::rows(a.X, row0, a.M, a.N, a.ldx, ES);
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i].load(rx, at(i, a.ldx, ES), a.N - col(i));
    const bool res = MODE != QUANT && a.R;
    if (res) {
        const auto rr = P::rows(a.R, row0, a.M, a.N, a.ldr, ES);
#pragma unroll
        for (int i = 0; i < NV; ++i) r[i].load(rr, at(i, a.ldr, ES), a.N - col(i));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        x[i].get(v[i]);
        if (res) {
            float w[8];
            r[i].get(w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += w[j];
        }
    }
    if constexpr (MODE != QUANT) {
        if (a.S) {
            const auto rs = P::rows(a.S, row0, a.M, a.N, a.lds, ES);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                Row8<FMT> o;
                o.set(v[i]);
                o.store(rs, at(i, a.lds, ES), a.N - col(i));
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
        ss = row_sum<T>(ss, red_s);
        const float rstd = rsqrtf(ss / (float)a.N + a.eps);
        if (a.rstd && pl.t == 0 && row < a.M) a.rstd[row] = rstd;
        const auto rw = make_rsrc((const char*)a.weight, (int64_t)a.N * 4);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Row8<OUT_F32> w8;
            w8.load(rw, (uint32_t)col(i) * 4, a.N - col(i));
            float w[8];
            w8.get(w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
        }
    }
    if constexpr (MODE == NORM) {
        const auto ry = P::rows(a.Y, row0, a.M, a.N, a.ldy, ES);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Row8<FMT> o;
            o.set(v[i]);
            o.store(ry, at(i, a.ldy, ES), a.N - col(i));
        }
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = col(i) + j < a.N ? mag_bits(v[i][j]) : 0u;
                m = b > m ? b : m;
            }
        m = row_max<T>(m, red_m);
        const float scale = f8_scale(m), inv = 1.0f / scale;
        if (pl.t == 0 && row < a.M) a.scale[row] = scale;
        const auto ry = P::rows(a.Y, row0, a.M, a.N, a.ldy, 1);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (col(i) < a.N) store_f8(ry, at(i, a.ldy, 1), a.N - col(i), v[i], scale, inv);
    }
}

template <int FMT, int MODE, int T, int NV>
hipError_t go_row(const RowArgs& a, hipStream_t stream) {
    using P = Place<T>;
    constexpr int ES = fmt_es<FMT>, EY = MODE == NORM ? ES : 1;
    // A launch has fewer than 2^32 threads: 2^21 workgroups at a time.
    constexpr int64_t ROWS = (int64_t)P::RPW << 21;
    for (int64_t r0 = 0; r0 < a.M; r0 += ROWS) {
        RowArgs b = a;
        b.M = (int)(a.M - r0 < ROWS ? a.M - r0 : ROWS);
        b.X += r0 * a.ldx * ES;
        b.Y += r0 * a.ldy * EY;
        if (a.R) b.R += r0 * a.ldr * ES;
        if (a.S) b.S += r0 * a.lds * ES;
        if (a.scale) b.scale += r0;
        if (a.rstd) b.rstd += r0;
        void* args[] = {&b};
        const hipError_t e = hipLaunchKernel((const void*)row_kernel<FMT, MODE, T, NV>,
                                             dim3((unsigned)((b.M + P::RPW - 1) / P::RPW)), dim3(P::WG), args,
                                             0, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int FMT, int MODE>
hipError_t row_by_size(const RowArgs& a, hipStream_t s) {
    if (a.N <= 128) return go_row<FMT, MODE, 16, 1>(a, s);
    if (a.N <= 256) return go_row<FMT, MODE, 32, 1>(a, s);
    if (a.N <= 512) return go_row<FMT, MODE, 64, 1>(a, s);
    if (a.N <= 1024) return go_row<FMT, MODE, 64, 2>(a, s);
    if (a.N <= 2048) return go_row<FMT, MODE, 256, 1>(a, s);
    if (a.N <= 4096) return go_row<FMT, MODE, 256, 2>(a, s);
    if (a.N <= 8192) return go_row<FMT, MODE, 256, 4>(a, s);
    if (a.N <= 16384) return go_row<FMT, MODE, 1024, 2>(a, s);
    if (a.N <= ROW_MAX) return go_row<FMT, MODE, 1024, 4>(a, s);
    return hipErrorInvalidValue;
}

template <int FMT>
hipError_t row_by_mode(const RowArgs& a, bool norm, bool f8, hipStream_t s) {
    if (!norm) return row_by_size<FMT, QUANT>(a, s);
    return f8 ? row_by_size<FMT, NORM_F8>(a, s) : row_by_size<FMT, NORM>(a, s);
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

hipError_t launch_rows(const RowArgs& a, int fmt, bool norm, bool f8, hipStream_t stream) {
    if (fmt == OUT_F32) return row_by_mode<OUT_F32>(a, norm, f8, stream);
    if (fmt == OUT_BF16) return row_by_mode<OUT_BF16>(a, norm, f8, stream);
    if (fmt == OUT_F16) return row_by_mode<OUT_F16>(a, norm, f8, stream);
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
