// rows.h -- the pass over rows that norms and row quantizers share (norm.hip,
// layernorm.hip), its reductions, and the rounding to 8 bits.
//
// Per row: s = x + r, S := s, then
//   root-mean-square norm: y = s rstd w, rstd = (mean s^2 + eps)^-1/2
//   layer norm: y = (s - mean) rstd w + b, rstd = (mean (s - mean)^2 + eps)^-1/2.  An fp32
//     sum gives the mean to a few half steps of |s|, many of the deviations' where the mean
//     is large.  So the deviations from it, d = s - m in registers, are summed beside their
//     squares (one barrier for both): c = mean d is what m lacks, d - c are the deviations
//     and mean d^2 - c^2 their variance, where nothing cancels as it does in mean s^2 - mean^2
// and Y := y or, in 8 bits, Y := e4m3(y / scale) with scale = max(max|y| / 448, 2^-100)
// over the row or over each block of 128 of its columns.  The quantizer alone is the
// same pass without the norm.
//
// A lane holds eight consecutive columns per piece, so a block of 128 columns is 16
// neighbouring lanes' piece and its maximum four shuffles, with no barrier.
#pragma once

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
// The sum over T lanes of a wave (64 for T above), the same bits in each.  The lanes trade values by
// DPP and lane swaps, not through LDS as __shfl_xor does: a layer norm's sums are what a short row
// waits for (1 x 4096 bf16 with its residual 2.8 us, through LDS 3.2).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int T>
__device__ __forceinline__ float lane_sum(float v) {
    v += dpp<0xb1>(v);   // neighbours within pairs
    v += dpp<0x4e>(v);   // pairs within four lanes, which then hold the same
    v += dpp<0x141>(v);  // mirrored within eight
    v += dpp<0x140>(v);  // mirrored within 16
    typedef uint32_t pair __attribute__((ext_vector_type(2)));
    if constexpr (T >= 32) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        const pair p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        v = as_float(p[0]) + as_float(p[1]);
    }
    if constexpr (T >= 64) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        const pair p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        v = as_float(p[0]) + as_float(p[1]);
    }
    return v;
}
// K sums over the T threads that share a row, with one barrier; red: T / 64 words each.
template <int T, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*red)[(T < 256 ? 256 : T) / 64]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane_sum<T>(v[k]);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) red[k][threadIdx.x >> 6] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = red[k][0];
#pragma unroll
            for (int i = 1; i < T / 64; ++i) v[k] += red[k][i];
        }
    }
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
// The same, as what rounds to e4m3 once: where fp32's quotient is inexact and its last bit
// is even, moved by that bit towards the remainder's side, so that a quotient which fp32
// rounds to a border between two codes still falls on its own side of it (one 16-bit value
// in a thousand does, the ratio to the block's largest being one of small integers; fp32 sums
// over such rows would show the other code).  The remainder is exact while the scale is
// above 2^-84.
__device__ __forceinline__ float quotient_odd(float v, float scale, float inv) {
    const float q = quotient(v, scale, inv);
    const float r = __builtin_fmaf(-q, scale, v);
    const int t = __builtin_bit_cast(int, q);
    const int side = ((__builtin_bit_cast(int, r) ^ t) >> 31) | 1;
    return __builtin_bit_cast(float, r != 0.0f && !(t & 1) ? t + side : t);
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

// Eight values quantized and stored at byte offset `off` of a row of bytes (ODD: by
// quotient_odd).
template <bool ODD>
__device__ __forceinline__ void store_f8(__amdgpu_buffer_rsrc_t r, uint32_t off, int nvalid,
                                         const float (&v)[8], float scale, float inv) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        q[j] = f8_clamp(ODD ? quotient_odd(v[j], scale, inv) : quotient(v[j], scale, inv));
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

// FMT: format of X, R, S and, without 8 bits, Y.
//   NORM, NORM_F8, NORM_F8B: root-mean-square norm, Y in FMT, in 8 bits with a scale per
//     row, in 8 bits with a scale per block;  LN, LN_F8, LN_F8B: layer norm;  QUANT: none
enum RowMode { NORM = 0, NORM_F8 = 1, QUANT = 2, NORM_F8B = 3, LN = 4, LN_F8 = 5, LN_F8B = 6 };

template <int FMT, int MODE, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void row_kernel(RowArgs a) {
    constexpr int ES = fmt_es<FMT>;
    using P = Place<T>;
    constexpr bool CENTER = MODE >= LN, PLAIN = MODE == NORM || MODE == LN;
    constexpr bool BLOCKS = MODE == NORM_F8B || MODE == LN_F8B;
    __shared__ float red_s[CENTER ? 2 : 1][P::WG / 64];
    __shared__ float red_c[1][CENTER ? P::WG / 64 : 1];
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
        float ss = 0.0f, rstd, off = 0.0f;  // y = (v rstd - off) w + b
        if constexpr (CENTER) {
            float sum[1] = {0.0f}, d[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[0] += v[i][j];
            row_sums<T>(sum, red_c);
            const float m = sum[0] / (float)a.N;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] = col(i) + j < a.N ? v[i][j] - m : 0.0f;
                    d[0] += v[i][j];
                    d[1] += v[i][j] * v[i][j];
                }
            row_sums<T>(d, red_s);
            const float c = d[0] / (float)a.N, var = d[1] / (float)a.N - c * c;
            rstd = rsqrtf((var < 0.0f ? 0.0f : var) + a.eps);
            off = c * rstd;
            if (a.mean && pl.t == 0 && row < a.M) a.mean[row] = c == c ? m + c : m;  // infinite: m
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
            ss = row_sum<T>(ss, red_s[0]);
            rstd = rsqrtf(ss / (float)a.N + a.eps);
        }
        if (a.rstd && pl.t == 0 && row < a.M) a.rstd[row] = rstd;
        const auto rw = make_rsrc((const char*)a.weight, (int64_t)a.N * 4);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Row8<OUT_F32> w8;
            w8.load(rw, (uint32_t)col(i) * 4, a.N - col(i));
            float w[8];
            w8.get(w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = (CENTER ? __builtin_fmaf(v[i][j], rstd, -off) : v[i][j] * rstd) * w[j];
        }
        if constexpr (CENTER) {
            if (a.bias) {
                const auto rb = make_rsrc((const char*)a.bias, (int64_t)a.N * 4);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    Row8<OUT_F32> b8;
                    b8.load(rb, (uint32_t)col(i) * 4, a.N - col(i));
                    float b[8];
                    b8.get(b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += b[j];
                }
            }
        }
    }
    if constexpr (PLAIN) {
        const auto ry = P::rows(a.Y, row0, a.M, a.N, a.ldy, ES);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Row8<FMT> o;
            o.set(v[i]);
            o.store(ry, at(i, a.ldy, ES), a.N - col(i));
        }
    } else if constexpr (BLOCKS) {
        const auto ry = P::rows(a.Y, row0, a.M, a.N, a.ldy, 1);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = col(i) + j < a.N ? mag_bits(v[i][j]) : 0u;
                m = b > m ? b : m;
            }
            m = row_max<16>(m, red_m);  // 16 lanes hold a block
            const float scale = f8_scale(m);
            if (col(i) < a.N) {
                if ((pl.t & 15) == 0 && row < a.M)
                    a.scale[row * a.s_row + (int64_t)(col(i) / F8_BLOCK) * a.s_blk] = scale;
                store_f8<true>(ry, at(i, a.ldy, 1), a.N - col(i), v[i], scale, 1.0f / scale);
            }
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
            if (col(i) < a.N) store_f8<false>(ry, at(i, a.ldy, 1), a.N - col(i), v[i], scale, inv);
    }
}

template <int FMT, int MODE, int T, int NV>
hipError_t go_row(const RowArgs& a, hipStream_t stream) {
    using P = Place<T>;
    constexpr int ES = fmt_es<FMT>, EY = MODE == NORM || MODE == LN ? ES : 1;
    // A launch has fewer than 2^32 threads: 2^21 workgroups at a time.
    constexpr int64_t ROWS = (int64_t)P::RPW << 21;
    for (int64_t r0 = 0; r0 < a.M; r0 += ROWS) {
        RowArgs b = a;
        b.M = (int)(a.M - r0 < ROWS ? a.M - r0 : ROWS);
        b.X += r0 * a.ldx * ES;
        b.Y += r0 * a.ldy * EY;
        if (a.R) b.R += r0 * a.ldr * ES;
        if (a.S) b.S += r0 * a.lds * ES;
        if (a.scale) b.scale += MODE == NORM_F8B || MODE == LN_F8B ? r0 * a.s_row : r0;
        if (a.rstd) b.rstd += r0;
        if (a.mean) b.mean += r0;
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
    // Rows that have a CU each: eight columns per thread, for the time of one row (bf16, us, 8 and 16
    // columns per thread or more: 8-bit blocks 1 x 4096 3.3 and 3.8, 1 x 8192 4.3 and 5.7, 256 x 8192 5.4
    // and 6.7, root-mean-square 1 x 8192 3.6 and 5.2; a scale per row 1 x 8192 4.3 and 4.5; plain output
    // 256 x 3000 3.1 and 3.4, 1 x 4096 2.6 both, 256 x 8192 4.2 and 4.1).  The order of a row's sums
    // differs, and so its last bits between the two sides of this rule; the root-mean-square norm's other
    // outputs, which were there before it, keep one width.
    if constexpr (MODE >= NORM_F8B) {
        if (a.M <= NUM_CU && a.N > 2048 && a.N <= 4096) return go_row<FMT, MODE, 512, 1>(a, s);
        if (a.M <= NUM_CU && a.N > 4096 && a.N <= 8192) return go_row<FMT, MODE, 1024, 1>(a, s);
    }
    if (a.N <= 4096) return go_row<FMT, MODE, 256, 2>(a, s);
    if (a.N <= 8192) return go_row<FMT, MODE, 256, 4>(a, s);
    if (a.N <= 16384) return go_row<FMT, MODE, 1024, 2>(a, s);
    if (a.N <= ROW_MAX) return go_row<FMT, MODE, 1024, 4>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace
}  // namespace dgemm
