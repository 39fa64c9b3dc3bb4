// splitk.hip -- the reduction that finishes a split-K GEMM on gfx950.
//
// A split-K launch leaves `splits` fp32 partial products W[z] (each M x ldw,
// ldw a multiple of 4) in the caller's workspace; this kernel sums them in
// ascending z (so the result does not depend on timing), applies the fused
// epilogue and rounds once to C's format.  It is elementwise and bound by HBM:
// per output it reads 4 * splits bytes and writes one element (plus C_old
// when beta != 0), so each thread takes four consecutive columns of one row
// and moves 16-byte pieces.

#include "kern_common.h"

namespace dgemm {
namespace {

constexpr int RED_THREADS = 256;

typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));

// Four consecutive elements, an aligned 16- or 8-byte piece.
template <int OUT>
__device__ __forceinline__ void store4(char* p, int64_t idx, const float (&v)[4]) {
    if constexpr (OUT == OUT_F32) {
        *(f32x4*)(p + idx * 4) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
        u16x4 h;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (OUT == OUT_BF16)
                h[j] = __builtin_bit_cast(unsigned short, (__bf16)v[j]);
            else
                h[j] = __builtin_bit_cast(unsigned short, (_Float16)v[j]);
        }
        *(u16x4*)(p + idx * 2) = h;
    }
}

template <int OUT>
__device__ __forceinline__ void load4(const char* p, int64_t idx, float (&v)[4]) {
    if constexpr (OUT == OUT_F32) {
        const f32x4 x = *(const f32x4*)(p + idx * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = x[j];
    } else {
        const u16x4 x = *(const u16x4*)(p + idx * 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned short h = x[j];
            if constexpr (OUT == OUT_BF16) v[j] = as_float((uint32_t)h << 16);
            else v[j] = (float)__builtin_bit_cast(_Float16, h);
        }
    }
}

template <int OUT, int EPI>
__global__ __launch_bounds__(RED_THREADS) void splitk_reduce_kernel(
    const float* __restrict__ W, int splits, int64_t zstride, int ldw, char* __restrict__ C,
    int ldc, int M, int N, EpiArgs e) {
    const int nq = ldw >> 2;
    const int64_t t = (int64_t)blockIdx.x * RED_THREADS + threadIdx.x;
    if (t >= (int64_t)M * nq) return;
    const int row = (int)(t / nq);
    const int col0 = (int)(t - (int64_t)row * nq) * 4;
    if (col0 >= N) return;

    const float* p = W + (int64_t)row * ldw + col0;
    f32x4 s = *(const f32x4*)p;
    // In ascending z, four partials' loads in flight.
#pragma unroll 4
    for (int z = 1; z < splits; ++z) s += *(const f32x4*)(p + z * zstride);

    if constexpr (EPI == EPI_FULL) {
        float f[4] = {s[0], s[1], s[2], s[3]};
        if (col0 + 4 <= N) {
            // Four columns of one row, 8- or 16-byte aligned in R, Z and C.
            float res[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (e.res) load4<OUT>(e.res, (int64_t)row * e.ldr + col0, res);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (e.scale_a) f[j] = f[j] * e.scale_a[row] * e.scale_b[col0 + j];
                if (e.bias) f[j] += e.bias[col0 + j];
            }
            if (e.pre) store4<OUT>(e.pre, (int64_t)row * e.ldz + col0, f);
            apply_act<OUT>(f, e.act);
            if (e.res) {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] += res[j];
            }
            store4<OUT>(C, (int64_t)row * ldc + col0, f);
        } else {
            const int rows[4] = {row, row, row, row};
            const int cols[4] = {col0, col0 + 1, col0 + 2, col0 + 3};
            finish_full<OUT, 4>(f, rows, cols, C, M, N, ldc, e);
        }
        return;
    }
    const int64_t base = (int64_t)row * ldc + col0;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = s[j];
        if constexpr (EPI == EPI_BASIC) {
            if (col0 + j < N) {
                const float bias = e.bias ? e.bias[col0 + j] : 0.0f;
                v[j] = epilogue<OUT>(v[j], C, base + j, bias, e);
            }
        }
    }
    if (col0 + 4 <= N) {
        // C's base and row pitch are 16-byte aligned and col0 is a multiple
        // of 4, so the four outputs form one aligned 16- or 8-byte piece.
        store4<OUT>(C, base, v);
    } else {
        for (int j = 0; j < 4; ++j)
            if (col0 + j < N) store_c<OUT>(C, base + j, v[j]);
    }
}

// The plain sums of up to three products in one launch.
struct Reduce3 {
    SplitSum s[3];
    int64_t end[3];  // the blocks up to each product's last
};

template <int OUT>
__global__ __launch_bounds__(RED_THREADS) void splitk_reduce3_kernel(Reduce3 r) {
    const int64_t b = blockIdx.x;
    const int i = b < r.end[0] ? 0 : b < r.end[1] ? 1 : 2;
    const SplitSum a = i == 0 ? r.s[0] : i == 1 ? r.s[1] : r.s[2];
    const int64_t t = (b - (i == 0 ? 0 : i == 1 ? r.end[0] : r.end[1])) * RED_THREADS + threadIdx.x;
    const int nq = a.ldw >> 2;
    if (t >= (int64_t)a.M * nq) return;
    const int row = (int)(t / nq);
    const int col0 = (int)(t - (int64_t)row * nq) * 4;
    if (col0 >= a.N) return;
    const float* p = a.W + (int64_t)row * a.ldw + col0;
    f32x4 s = *(const f32x4*)p;
#pragma unroll 4
    for (int z = 1; z < a.splits; ++z) s += *(const f32x4*)(p + z * a.zstride);
    const int64_t base = (int64_t)row * a.ldc + col0;
    const float v[4] = {s[0], s[1], s[2], s[3]};
    if (col0 + 4 <= a.N) {
        store4<OUT>(a.C, base, v);
    } else {
        for (int j = 0; j < 4; ++j)
            if (col0 + j < a.N) store_c<OUT>(a.C, base + j, v[j]);
    }
}

template <int OUT, int EPI>
hipError_t go(const float* W, int splits, int64_t zstride, int ldw, char* C, int ldc, int M, int N,
              const EpiArgs& e, hipStream_t stream) {
    const int64_t threads = (int64_t)M * (ldw / 4);
    const int64_t blocks = (threads + RED_THREADS - 1) / RED_THREADS;
    if (blocks <= 0) return hipSuccess;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    EpiArgs ea = e;
    void* args[] = {&W, &splits, &zstride, &ldw, &C, &ldc, &M, &N, &ea};
    return hipLaunchKernel((const void*)splitk_reduce_kernel<OUT, EPI>, dim3((unsigned)blocks),
                           dim3(RED_THREADS), args, 0, stream);
}

template <int OUT>
hipError_t by_epi(int epi, const float* W, int splits, int64_t zstride, int ldw, char* C, int ldc,
                  int M, int N, const EpiArgs& e, hipStream_t stream) {
    if (epi == EPI_FULL) return go<OUT, EPI_FULL>(W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    if (epi == EPI_BASIC) return go<OUT, EPI_BASIC>(W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    return go<OUT, EPI_NONE>(W, splits, zstride, ldw, C, ldc, M, N, e, stream);
}

}  // namespace

hipError_t launch_splitk_reduce(const float* W, int splits, int64_t zstride, int ldw, char* C,
                                int ldc, int M, int N, int out, int epi, const EpiArgs& e,
                                hipStream_t stream) {
    if (ldw % 4 != 0 || splits < 1) return hipErrorInvalidValue;
    if (out == OUT_F32) return by_epi<OUT_F32>(epi, W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    if (out == OUT_BF16) return by_epi<OUT_BF16>(epi, W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    if (out == OUT_F16) return by_epi<OUT_F16>(epi, W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_splitk_reduce3(const SplitSum* sums, int count, int out, hipStream_t stream) {
    if (count < 1 || count > 3 || (out != OUT_BF16 && out != OUT_F16)) return hipErrorInvalidValue;
    Reduce3 r{};
    int64_t blocks = 0;
    for (int i = 0; i < 3; ++i) {
        if (i < count) {
            if (sums[i].ldw % 4 != 0 || sums[i].splits < 1) return hipErrorInvalidValue;
            r.s[i] = sums[i];
            blocks += ((int64_t)sums[i].M * (sums[i].ldw / 4) + RED_THREADS - 1) / RED_THREADS;
        }
        r.end[i] = blocks;
    }
    if (blocks <= 0) return hipSuccess;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    void* args[] = {&r};
    return hipLaunchKernel(out == OUT_BF16 ? (const void*)splitk_reduce3_kernel<OUT_BF16>
                                           : (const void*)splitk_reduce3_kernel<OUT_F16>,
                           dim3((unsigned)blocks), dim3(RED_THREADS), args, 0, stream);
}

}  // namespace dgemm
