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
// of 16 waves holds it in registers, eight consecutive rows per wave and two columns per lane,
// so that a thread's values of one column are eight neighbouring bytes of the transpose: it
// goes through LDS in rows of 128 bytes whose 8-byte pieces trade places by the column, so that
// the columns that are written at once meet different banks.  (Eight rows and columns per thread
// in 4 waves: a small call 5.8 us bf16 and 7.2 fp32, four times the arithmetic one after another,
// where this takes 3.8 and 4.3; 8192 x 2048 bf16 transposed 10.8 and 10.7, 8192 x 4096 fp32 28.3 and
// 26.6, with a scale per 128 x 128 10.1 and 11.7, 27.6 and 27.5.)

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

template <int FMT>
__device__ __forceinline__ float half_value(uint32_t h) {
    if constexpr (FMT == OUT_BF16) return as_float(h << 16);
    else return (float)__builtin_bit_cast(_Float16, (unsigned short)h);
}

// The first n bytes of w (at most 8, none if negative) to p, which is 8-byte aligned.
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
__global__ __launch_bounds__(1024) void quant_tile_kernel(QuantBlockArgs a, int tiles_n, int first) {
    static_assert(TR || ROWS == F8_BLOCK, "rows as they lie are quant_rows_kernel's");
    constexpr bool F32 = FMT == OUT_F32;
    __shared__ uint32_t wmax[16][ROWS == 1 ? F8_BLOCK : 1];
    __shared__ Divisor<FMT> cdiv[ROWS == 1 ? F8_BLOCK : 1];
    __shared__ __attribute__((aligned(16))) char tile[F8_BLOCK * F8_BLOCK];
    const int b = first + (int)blockIdx.x, tm = b / tiles_n, tn = b - tm * tiles_n;
    const int m0 = tm * F8_BLOCK, n0 = tn * F8_BLOCK;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int c2 = lane * 2, r8 = wave * 8;  // this thread's columns and rows
    const int nvalid = a.N - (n0 + c2);
    float v[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = m0 + r8 + i;
        const bool in = row < a.M && nvalid > 0;
        const char* p = a.X + ((int64_t)(in ? row : 0) * a.ldx + (in ? n0 + c2 : 0)) * fmt_es<FMT>;
        if constexpr (F32) {
            const u32x2 w = in ? *(const u32x2*)p : u32x2{0u, 0u};
            v[i][0] = as_float(w[0]);
            v[i][1] = as_float(w[1]);
        } else {
            const uint32_t w = in ? *(const uint32_t*)p : 0u;
            v[i][0] = half_value<FMT>(w & 0xffffu);
            v[i][1] = half_value<FMT>(w >> 16);
        }
        if (nvalid < 2) v[i][1] = 0.0f;
    }
    uint32_t m[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t b = mag_bits(v[i][j]);
            m[j] = b > m[j] ? b : m[j];
        }
    Divisor<FMT> div[ROWS == 1 ? 2 : 1];
    if constexpr (ROWS == 1) {
        wmax[wave][c2] = m[0];
        wmax[wave][c2 + 1] = m[1];
        __syncthreads();
        if (t < F8_BLOCK) {
            uint32_t s = wmax[0][t];
#pragma unroll
            for (int w = 1; w < 16; ++w) s = wmax[w][t] > s ? wmax[w][t] : s;
            const Divisor<FMT> d(s);
            cdiv[t] = d;
            if (n0 + t < a.N) a.scale[(int64_t)(n0 + t) * a.s_row + (int64_t)tm * a.s_blk] = d.scale;
        }
        __syncthreads();
        div[0] = cdiv[c2];
        div[1] = cdiv[c2 + 1];
    } else {
        div[0] = Divisor<FMT>(row_max<1024>(m[0] > m[1] ? m[0] : m[1], &wmax[0][0]));
        if (t == 0) a.scale[(int64_t)(TR ? tn : tm) * a.s_row + (int64_t)(TR ? tm : tn) * a.s_blk] = div[0].scale;
    }
    if constexpr (TR) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float x[8] = {v[0][j], v[1][j], v[2][j], v[3][j], v[4][j], v[5][j], v[6][j], v[7][j]};
            *(u32x2*)(tile + (c2 + j) * F8_BLOCK + ((wave ^ (lane & 15)) << 3)) =
                quantize8<FMT>(x, div[ROWS == 1 ? j : 0]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float x[8] = {v[4 * h][0], v[4 * h][1], v[4 * h + 1][0], v[4 * h + 1][1],
                                v[4 * h + 2][0], v[4 * h + 2][1], v[4 * h + 3][0], v[4 * h + 3][1]};
            const u32x2 q = quantize8<FMT>(x, div[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(uint16_t*)(tile + (r8 + 4 * h + i) * F8_BLOCK + c2) = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
        }
    }
    __syncthreads();
    // Row r of Q's tile, its bytes c .. c + 15.
    const int r = t >> 3, c = (t & 7) * 16;
    u32x4 w;
    if constexpr (TR) {
        const int s = (r >> 1) & 15;  // the pieces' exchange: 16-byte units, and the halves of one
        w = *(const u32x4*)(tile + r * F8_BLOCK + ((c >> 4 ^ s >> 1) << 4));
        if (s & 1) w = u32x4{w[2], w[3], w[0], w[1]};
    } else {
        w = *(const u32x4*)(tile + r * F8_BLOCK + c);
    }
    const int64_t row = (TR ? n0 : m0) + r;
    const int col = (TR ? m0 : n0) + c;
    const int rows = TR ? a.N : a.M, cols = TR ? a.M : a.N;
    if (row >= rows || col >= cols) return;
    char* const q = a.Q + row * a.ldq + col;
    if (cols - col >= 16) {
        *(u32x4*)q = w;
    } else {
        put8(q, u32x2{w[0], w[1]}, cols - col);
        put8(q + 8, u32x2{w[2], w[3]}, cols - col - 8);
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
    // A launch has fewer than 2^32 threads: 2^21 tiles at a time.
    for (int first = 0; first < (int)tiles; first += 1 << 21) {
        void* args[] = {&b, &tiles_n, &first};
        const int n = (int)tiles - first < 1 << 21 ? (int)tiles - first : 1 << 21;
        const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)n), dim3(1024), args, 0, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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
