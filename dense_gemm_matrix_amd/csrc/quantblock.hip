// quantblock.hip -- matrices to 8 bits with a scale per block, for gfx950 (MI355X): the
// operands of gemm_f8_block.
//
// Q = e4m3(X / scale) or its transpose, scale = max(max|x| / 448, 2^-100) over a block of
// `rows` x 128 of Q (rows = 1: activations and gradients; 128: weights).  Every value is
// read once and written once, and the quotient is rounded to e4m3 once.
//
// Rows as they lie (quant_rows): a block is 16 lanes of eight columns, its maximum four
// shuffles; no LDS, no barrier.  Four blocks per lane, their loads in flight together,
// where there are enough of them to fill the chip.
//
// The other three (quant_tile) need a 128 x 128 tile of X at once: for its maximum, to
// take the maxima of columns, to write rows of the transpose in whole lines.  A workgroup
// of 256 threads holds it in registers, eight consecutive rows of eight columns per
// thread, so that a thread's values of one column are eight neighbouring bytes of the
// transpose: it goes through LDS as 8-byte pieces, in rows of 128 bytes whose pieces trade
// places by the column's eighth, so that the 16 columns that are written at once, eight apart,
// and the 16 pieces of a row that are read at once each meet all banks.

#include "rows.h"

namespace dgemm {
namespace {

// A block's scale and what its quotients need.
//
// fp32 values: quotient_odd.  16-bit ones have significands of at most 11 bits, the border t
// between two codes one of 5, and scale = amax / 448 (1 + d) with |d| <= 2^-24: v / scale lies
// within 2^-24 of t, relatively, only if v 448 / amax is t itself (two products of at most 16 bits
// differ by 2^-16 or not at all).  Then d's sign says on which side of t it lies, for the whole
// block, and the fp32 quotient (t, or its neighbour on that side) times 1 + 2^-22 or 1 - 2^-22
// falls there; d = 0 leaves a tie, which goes to the even code.  No other quotient is near
// enough a border to cross it.  Four operations a value instead of eleven.
template <int FMT>
struct Divisor {
    float scale, inv, bias;
    __device__ __forceinline__ explicit Divisor(uint32_t amax_bits) {
        scale = f8_scale(amax_bits);
        inv = 1.0f / scale;
        const float d = __builtin_fmaf(-scale, F8_MAX, as_float(amax_bits));  // exact
        bias = d == 0.0f || scale == SCALE_MIN ? 1.0f : d > 0.0f ? 1.0f + 0x1p-22f : 1.0f - 0x1p-22f;
    }
    Divisor() = default;
    __device__ __forceinline__ Divisor(float s, float i, float b) : scale(s), inv(i), bias(b) {}
    // The quotient, as rounding to e4m3 takes it; at most 448 and a few steps, which rounds to 448.
    __device__ __forceinline__ float operator()(float v) const {
        return FMT == OUT_F32 ? quotient_odd(v, scale, inv) : quotient(v, scale, inv) * bias;
    }
};

template <int FMT>
__device__ __forceinline__ u32x2 quantize8(const float (&v)[8], const Divisor<FMT>& d) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = d(v[j]);
    return u32x2{f8_pack4(q[0], q[1], q[2], q[3]), f8_pack4(q[4], q[5], q[6], q[7])};
}

// n <= 8 bytes of w to p, which is 8-byte aligned.
__device__ __forceinline__ void put8(char* p, u32x2 w, int n) {
    if (n >= 8) {
        *(u32x2*)p = w;
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) p[j] = (char)(w[j >> 2] >> (8 * (j & 3)));
    }
}

template <int FMT, int U>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantBlockArgs a, uint32_t blocks, uint32_t total) {
    const int l = threadIdx.x & 15;
    const uint32_t g0 = blockIdx.x * 16 * U + (threadIdx.x >> 4);
    Row8<FMT> x[U];
    uint32_t row[U], blk[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t g = g0 + u * 16 < total ? g0 + u * 16 : total - 1;
        row[u] = g / blocks;
        blk[u] = g - row[u] * blocks;
        const int c = (int)blk[u] * F8_BLOCK + l * 8;
        x[u].load_from(a.X + ((int64_t)row[u] * a.ldx + c) * fmt_es<FMT>, a.N - c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[8];
        x[u].get(v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = mag_bits(v[j]);
            m = b > m ? b : m;
        }
        m = row_max<16>(m, nullptr);
        if (g0 + u * 16 >= total) continue;
        const int c = (int)blk[u] * F8_BLOCK + l * 8;
        const Divisor<FMT> d(m);
        if (l == 0) a.scale[row[u] * a.s_row + blk[u] * a.s_blk] = d.scale;
        if (c < a.N) put8(a.Q + (int64_t)row[u] * a.ldq + c, quantize8<FMT>(v, d), a.N - c);
    }
}

// TR: Q is X transposed.  ROWS: a block's rows of Q, 1 (with TR) or 128.
template <int FMT, bool TR, int ROWS>
__global__ __launch_bounds__(256) void quant_tile_kernel(QuantBlockArgs a, int tiles_n) {
    static_assert(TR || ROWS == F8_BLOCK, "rows as they lie are quant_rows_kernel's");
    constexpr int P = F8_BLOCK;
    __shared__ uint32_t wmax[4][ROWS == 1 ? F8_BLOCK : 1];
    __shared__ __attribute__((aligned(16))) float cdiv[3][ROWS == 1 ? F8_BLOCK : 4];
    __shared__ __attribute__((aligned(16))) char tile[TR ? F8_BLOCK * P : 8];
    const int tm = (int)(blockIdx.x / tiles_n), tn = (int)(blockIdx.x % tiles_n);
    const int m0 = tm * F8_BLOCK, n0 = tn * F8_BLOCK;
    const int t = threadIdx.x, wave = t >> 6;
    const int c8 = (t & 15) * 8, r8 = (t >> 4) * 8;  // this thread's columns and rows
    const int nvalid = a.N - (n0 + c8);
    Row8<FMT> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = m0 + r8 + i;
        const int n = row < a.M ? nvalid : 0;
        x[i].load_from(a.X + ((int64_t)(n > 0 ? row : 0) * a.ldx + (n > 0 ? n0 + c8 : 0)) * fmt_es<FMT>, n);
    }
    uint32_t m[ROWS == 1 ? 8 : 1] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        x[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = mag_bits(v[j]);
            uint32_t& to = m[ROWS == 1 ? j : 0];
            to = b > to ? b : to;
        }
    }
    Divisor<FMT> div[ROWS == 1 ? 8 : 1];
    if constexpr (ROWS == 1) {
        // A column's 128 rows are 16 threads': four lanes of each wave.
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int s = 16; s <= 32; s *= 2) {
                const uint32_t o = (uint32_t)__shfl_xor((int)m[j], s);
                m[j] = o > m[j] ? o : m[j];
            }
            if ((t & 63) < 16) wmax[wave][c8 + j] = m[j];
        }
        __syncthreads();
        if (t < F8_BLOCK) {
            uint32_t s = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) s = wmax[w][t] > s ? wmax[w][t] : s;
            const Divisor<FMT> d(s);
            cdiv[0][t] = d.scale;
            cdiv[1][t] = d.inv;
            cdiv[2][t] = d.bias;
            if (n0 + t < a.N) a.scale[(int64_t)(n0 + t) * a.s_row + (int64_t)tm * a.s_blk] = d.scale;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) div[j] = Divisor<FMT>(cdiv[0][c8 + j], cdiv[1][c8 + j], cdiv[2][c8 + j]);
    } else {
        div[0] = Divisor<FMT>(row_max<256>(m[0], &wmax[0][0]));
        if (t == 0) a.scale[(int64_t)(TR ? tn : tm) * a.s_row + (int64_t)(TR ? tm : tn) * a.s_blk] = div[0].scale;
    }
    if constexpr (!TR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
            x[i].get(v);
            const int row = m0 + r8 + i;
            if (row < a.M && nvalid > 0)
                put8(a.Q + (int64_t)row * a.ldq + n0 + c8, quantize8<FMT>(v, div[0]), nvalid);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float w[8];
                x[i].get(w);
                v[i] = w[j];
            }
            *(u32x2*)(tile + (c8 + j) * P + (r8 ^ c8)) = quantize8<FMT>(v, div[ROWS == 1 ? j : 0]);
        }
        __syncthreads();
        // Row n0 + r of Q: bytes m0 + 8 (t % 16) .., 16 rows at a time.
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 16 + (t >> 4), c = (t & 15) * 8;
            if (n0 + r < a.N && m0 + c < a.M)
                put8(a.Q + (int64_t)(n0 + r) * a.ldq + m0 + c, *(const u32x2*)(tile + r * P + (c ^ (r & ~7))), a.M - (m0 + c));
        }
    }
}

template <int FMT>
hipError_t go_quant_block(const QuantBlockArgs& a, int rows, bool transpose, hipStream_t stream) {
    QuantBlockArgs b = a;
    if (rows == 1 && !transpose) {
        uint32_t blocks = ((uint32_t)a.N + F8_BLOCK - 1) / F8_BLOCK;
        const int64_t all = (int64_t)a.M * blocks;
        // Four blocks per 16 lanes from 4 workgroups of them per CU on; at most 2^26 blocks in a
        // launch (fewer than 2^32 threads), or a row's.
        const bool four = all >= (int64_t)16 * 4 * 4 * NUM_CU;
        const int64_t most = ((int64_t)1 << 26) / blocks > 0 ? ((int64_t)1 << 26) / blocks : 1;  // rows
        for (int64_t r0 = 0; r0 < a.M; r0 += most) {
            const int64_t n = a.M - r0 < most ? a.M - r0 : most;
            b.M = (int)n;
            b.X = a.X + r0 * a.ldx * fmt_es<FMT>;
            b.Q = a.Q + r0 * a.ldq;
            b.scale = a.scale + r0 * a.s_row;
            uint32_t total = (uint32_t)(n * blocks);
            const int64_t per = four ? 64 : 16;
            void* args[] = {&b, &blocks, &total};
            const hipError_t e =
                hipLaunchKernel(four ? (const void*)quant_rows_kernel<FMT, 4> : (const void*)quant_rows_kernel<FMT, 1>,
                                dim3((unsigned)((total + per - 1) / per)), dim3(256), args, 0, stream);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    int tiles_n = (a.N + F8_BLOCK - 1) / F8_BLOCK;
    const int64_t tiles = (int64_t)tiles_n * ((a.M + F8_BLOCK - 1) / F8_BLOCK);
    if (tiles >= (int64_t)1 << 23) return hipErrorInvalidValue;
    const void* fn = !transpose ? (const void*)quant_tile_kernel<FMT, false, F8_BLOCK>
                     : rows == 1 ? (const void*)quant_tile_kernel<FMT, true, 1>
                                 : (const void*)quant_tile_kernel<FMT, true, F8_BLOCK>;
    void* args[] = {&b, &tiles_n};
    return hipLaunchKernel(fn, dim3((unsigned)tiles), dim3(256), args, 0, stream);
}

}  // namespace

hipError_t launch_quant_block(const QuantBlockArgs& a, int fmt, int rows, bool transpose, hipStream_t stream) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    if (fmt == OUT_F32) return go_quant_block<OUT_F32>(a, rows, transpose, stream);
    if (fmt == OUT_BF16) return go_quant_block<OUT_BF16>(a, rows, transpose, stream);
    if (fmt == OUT_F16) return go_quant_block<OUT_F16>(a, rows, transpose, stream);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
