// skinny.hip -- products of at most 16 rows (tokens being generated) on gfx950
// (MI355X): bf16 / fp16 A[M x K] B[K x N], and e4m3 A[M x K] B[N x K]^T.
//
// Such a product reads B once and computes little: the floor is B's bytes over
// the HBM rate.  So no LDS staging: B goes straight from memory into the
// registers that the matrix instruction reads, with many loads in flight.  A
// workgroup owns a strip of columns, its W waves take its k steps in turn, and
// their partial sums are added in LDS in wave order (deterministic).  K may be
// split over workgroups too, with fp32 partials in the caller's workspace.
//
// 16-bit: lane (g, c) of 64 (g = lane / 16, c = lane % 16) loads the CPL
// consecutive columns CPL c .. of the eight k-rows 8 g .. 8 g + 7 of a 32-k
// step.  v_mfma_f32_16x16x32 wants eight k of one column per lane; the lane
// holds eight rows of CPL columns, and one v_perm_b32 per output word picks a
// column's halves from two rows' words: half an operation per element, instead
// of a transpose through LDS.  Matrix instruction j covers columns n0 + CPL c +
// j, c = 0 .. 15.  Rows past M come as zeros from A's resource.
//
// e4m3: B's rows are K-contiguous, so a lane loads its operand as it is: 32 k
// of row n0 + c per 128-k step, in two 16-byte pieces 64 bytes apart, so that
// the four lane groups read 64 consecutive bytes of a row at a time (A's pieces
// the same: the order of k inside the instruction cancels).  The values are
// widened to bf16 in registers, exactly, for the bf16 instruction: the kernel
// waits for memory, and the sums are fp32 (the 8-bit instruction's are not quite:
// gemmt.hip).

#include <type_traits>

#include "kern_common.h"

namespace dgemm {
namespace {

// Zero the bytes of a 16-byte piece at and past `valid` (<= 0: all of them).
__device__ __forceinline__ u32x4 mask_bytes(u32x4 v, int valid) {
    u32x4 out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int n = valid - 4 * w;  // bytes of this word to keep
        out[w] = n >= 4 ? v[w] : n <= 0 ? 0u : v[w] & (0xffffffffu >> (32 - 8 * n));
    }
    return out;
}

// The elements of a strip that a lane finishes, and what the epilogue reads for
// them, loaded before the K loop (at its end they would wait for memory once
// more).  CPL accumulators of 16 x 16 per wave: value idx = 4 j + r of lane (g, c)
// is row 4 g + r, column n0 + CPL c + j; wave w finishes idx in [w PER, ..).
template <int OUT, int EPI, int CPL, int W>
struct Strip {
    static constexpr int NV = CPL * 4;            // values per lane
    static constexpr int PER = (NV + W - 1) / W;  // of them, finished by one wave
    int row[PER], col[PER];
    float res[PER], bias[PER], scale[PER];

    __device__ __forceinline__ void prefetch(int M, int N, int n0, int wave, int lane,
                                             const EpiArgs& e) {
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int idx = wave * PER + q;
            row[q] = 4 * (lane >> 4) + idx % 4;
            col[q] = n0 + CPL * (lane & 15) + idx / 4;
            if (idx >= NV) row[q] = M;  // W larger than the values: none
            if constexpr (EPI == EPI_FULL) {
                const bool in = row[q] < M && col[q] < N;
                res[q] = in && e.res ? load_c<OUT>(e.res, (int64_t)row[q] * e.ldr + col[q]) : 0.0f;
                bias[q] = in && e.bias ? e.bias[col[q]] : 0.0f;
                scale[q] = in && e.scale_a ? e.scale_a[row[q]] * e.scale_b[col[q]] : 1.0f;
            }
        }
    }
    // Adds the W waves' sums in wave order and stores: the full epilogue, or an
    // fp32 partial.
    __device__ __forceinline__ void finish(const f32x4 (&acc)[CPL], float* red, char* C, int M, int N,
                                           int ldc, int wave, int lane, const EpiArgs& e) {
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[(wave * NV + j * 4 + r) * 64 + lane] = acc[j][r];
        __syncthreads();
        if (wave * PER >= NV) return;
        float v[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int idx = wave * PER + q;
            v[q] = red[idx * 64 + lane];
#pragma unroll
            for (int w = 1; w < W; ++w) v[q] += red[(w * NV + idx) * 64 + lane];
            if constexpr (EPI == EPI_FULL) {
                v[q] = v[q] * scale[q] + bias[q];
                if (e.pre && row[q] < M && col[q] < N)
                    store_c<OUT>(e.pre, (int64_t)row[q] * e.ldz + col[q], v[q]);
            }
        }
        if constexpr (EPI == EPI_FULL) apply_act(v, e.act);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if constexpr (EPI == EPI_FULL) v[q] = e.res ? v[q] + res[q] : v[q];
            if (row[q] < M && col[q] < N) store_c<OUT>(C, (int64_t)row[q] * ldc + col[q], v[q]);
        }
    }
};

// A wave's n steps in chunks of D: the next chunk's loads are issued before the
// current one is used, so D to 2 D steps are in flight, and the last chunk loads
// only the steps there are (a load past the end costs as much issue as a real
// one).  load(i, slot) and use(i, slot): step i in register slot `slot`, which is
// a constant once unrolled.
template <int D, class Load, class Use>
__device__ __forceinline__ void run_steps(int n, Load load, Use use) {
    const int full = n > 0 ? n / D : 0, rem = n > 0 ? n - full * D : 0;
    auto rest = [&](int base) {  // the last chunk's loads, into slots base ..
#pragma unroll
        for (int s = 0; s < D - 1; ++s)
            if (s < rem) load(full * D + s, base + s);
    };
    auto use_rest = [&](int base) {
#pragma unroll
        for (int s = 0; s < D - 1; ++s)
            if (s < rem) use(full * D + s, base + s);
    };
    if (full == 0) {
        rest(0);
        use_rest(0);
        return;
    }
#pragma unroll
    for (int s = 0; s < D; ++s) load(s, s);
    int c = 0;
    for (; c + 2 < full; c += 2) {
#pragma unroll
        for (int s = 0; s < D; ++s) load((c + 1) * D + s, D + s);
#pragma unroll
        for (int s = 0; s < D; ++s) use(c * D + s, s);
#pragma unroll
        for (int s = 0; s < D; ++s) load((c + 2) * D + s, s);
#pragma unroll
        for (int s = 0; s < D; ++s) use((c + 1) * D + s, D + s);
    }
    if (c + 1 < full) {
#pragma unroll
        for (int s = 0; s < D; ++s) load((c + 1) * D + s, D + s);
#pragma unroll
        for (int s = 0; s < D; ++s) use(c * D + s, s);
        rest(0);
#pragma unroll
        for (int s = 0; s < D; ++s) use((c + 1) * D + s, D + s);
        use_rest(0);
    } else {
        rest(D);
#pragma unroll
        for (int s = 0; s < D; ++s) use(c * D + s, s);
        use_rest(D);
    }
}

// Workgroup strip map: consecutive strips to one XCD (workgroups are dealt to
// the 8 XCDs in turn), so that strips narrower than a 128-byte line share it in
// one L2.
__device__ __forceinline__ int strip_of(int wg, int strips) {
    int tm, tn;
    map_tile(wg, 1, strips, tm, tn);
    return tn;
}

template <int IN, int OUT, int EPI, int CPL, int W>
__global__ __launch_bounds__(64 * W) void skinny16_kernel(
    const char* __restrict__ A, const char* __restrict__ B, char* C, int M, int N, int K, int lda,
    int ldb, int ldc, int strips, int kchunk, int64_t c_zstride, EpiArgs epi) {
    constexpr int WD = CPL / 2;   // words per lane and k-row
    constexpr int D = CPL == 8 ? 2 : 4;  // steps per chunk; two chunks in registers
    __shared__ float red[W * CPL * 4 * 64];
    {
        const int kbeg = (int)blockIdx.y * kchunk;
        A += (int64_t)kbeg * 2;
        B += (int64_t)kbeg * ldb * 2;
        C += (int)blockIdx.y * c_zstride;
        K = (K - kbeg) < kchunk ? (K - kbeg) : kchunk;
    }
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int n0 = strip_of((int)blockIdx.x, strips) * 16 * CPL;
    const int cols = (N - n0) < 16 * CPL ? (N - n0) : 16 * CPL;
    const int nstep = (K + 31) / 32;
    Strip<OUT, EPI, CPL, W> strip;
    strip.prefetch(M, N, n0, wave, lane, epi);

    uint32_t b[2 * D][8][WD];
    u32x4 a[2 * D];
    auto load = [&](int t, int S) {  // S: a constant once unrolled
        const int k0 = t * 32;
        const int rows = (K - k0) < 32 ? (K - k0) : 32;
        const auto rb = make_rsrc(B + ((int64_t)k0 * ldb + n0) * 2,
                                  rows > 0 ? ((int64_t)(rows - 1) * ldb + cols) * 2 : 0);
        const auto ra = make_rsrc(A + (int64_t)k0 * 2,
                                  rows > 0 ? ((int64_t)(M - 1) * lda + rows) * 2 : 0);
        a[S] = load16(ra, (c * lda + 8 * g) * 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int off = ((8 * g + j) * ldb + CPL * c) * 2;
            if constexpr (WD == 4) {
                const u32x4 v = load16(rb, off);
#pragma unroll
                for (int w = 0; w < 4; ++w) b[S][j][w] = v[w];
            } else if constexpr (WD == 2) {
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rb, off, 0, 0);
                b[S][j][0] = v[0];
                b[S][j][1] = v[1];
            } else {
                b[S][j][0] = __builtin_amdgcn_raw_buffer_load_b32(rb, off, 0, 0);
            }
        }
    };
    f32x4 acc[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto use = [&](int t, int S) {
        const int k0 = t * 32;
        u32x4 av = a[S];
        if (k0 + 32 > K) av = mask_bytes(av, (K - k0 - 8 * g) * 2);  // A's row padding
#pragma unroll
        for (int w = 0; w < WD; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 bv;
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    bv[p] = __builtin_amdgcn_perm(b[S][2 * p + 1][w], b[S][2 * p][w],
                                                  h ? 0x07060302u : 0x05040100u);
                const int j = 2 * w + h;
                if constexpr (IN == IN_BF16)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, av), __builtin_bit_cast(bf16x8, bv), acc[j], 0, 0, 0);
                else
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_bit_cast(f16x8, av), __builtin_bit_cast(f16x8, bv), acc[j], 0, 0, 0);
            }
    };
    // Wave w takes steps w, w + W, ...: the workgroup reads B's rows in order.
    run_steps<D>((nstep - wave + W - 1) / W, [&](int i, int slot) { load(wave + i * W, slot); },
                 [&](int i, int slot) { use(wave + i * W, slot); });
    strip.finish(acc, red, C, M, N, ldc, wave, lane, epi);
}

template <int OUT, int W>
__global__ __launch_bounds__(64 * W) void skinny8_kernel(
    const char* __restrict__ A, const char* __restrict__ B, char* C, int M, int N, int K, int lda,
    int ldb, int ldc, int strips, EpiArgs epi) {
    __shared__ float red[W * 4 * 64];
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int n0 = strip_of((int)blockIdx.x, strips) * 16;
    const int rows_b = (N - n0) < 16 ? (N - n0) : 16;
    const int nstep = (K + 127) / 128;
    Strip<OUT, EPI_FULL, 1, W> strip;
    strip.prefetch(M, N, n0, wave, lane, epi);
    constexpr int D = 2;  // steps per chunk; two chunks in registers
    u32x4 a[2 * D][2], b[2 * D][2];
    auto load = [&](int t, int S) {  // S: a constant once unrolled
        const int k0 = t * 128;
        const int krem = (K - k0) < 128 ? (K - k0) : 128;
        const auto ra = make_rsrc(A + k0, krem > 0 ? (int64_t)(M - 1) * lda + krem : 0);
        const auto rb = make_rsrc(B + (int64_t)n0 * ldb + k0,
                                  krem > 0 ? (int64_t)(rows_b - 1) * ldb + krem : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            a[S][h] = load16(ra, c * lda + 64 * h + 16 * g);
            b[S][h] = load16(rb, c * ldb + 64 * h + 16 * g);
        }
    };
    f32x4 acc[1] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
    auto use = [&](int t, int S) {
        const int k0 = t * 128;
        u32x4 x[2], y[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x[h] = a[S][h];
            y[h] = b[S][h];
            if (k0 + 128 > K) {  // the rows' padding: 0 * NaN would be a NaN, so both
                const int valid = K - (k0 + 64 * h + 16 * g);
                x[h] = mask_bytes(x[h], valid);
                y[h] = mask_bytes(y[h], valid);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; q += 2)
                acc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_f8(x[h][q], x[h][q + 1]),
                                                                 widen_f8(y[h][q], y[h][q + 1]), acc[0],
                                                                 0, 0, 0);
    };
    run_steps<D>((nstep - wave + W - 1) / W, [&](int i, int slot) { load(wave + i * W, slot); },
                 [&](int i, int slot) { use(wave + i * W, slot); });
    strip.finish(acc, red, C, M, N, ldc, wave, lane, epi);
}

template <int IN, int OUT, int EPI, int CPL, int W>
hipError_t go16(const GemmLaunch& L) {
    const char* a = L.A;
    const char* b = L.B;
    char* c = L.C;
    int M = L.M, N = L.N, K = L.K, lda = L.lda, ldb = L.ldb, ldc = L.ldc, strips = L.tiles_n;
    int kchunk = L.kchunk;
    int64_t zs = L.c_zstride;
    EpiArgs e = L.e;
    void* args[] = {&a, &b, &c, &M, &N, &K, &lda, &ldb, &ldc, &strips, &kchunk, &zs, &e};
    return hipLaunchKernel((const void*)skinny16_kernel<IN, OUT, EPI, CPL, W>,
                           dim3((unsigned)strips, (unsigned)L.splits), dim3(64 * W), args, 0, L.stream);
}

template <int IN, int OUT, int EPI>
hipError_t by_strip(const GemmLaunch& L) {
    if (L.tbn == 128 && L.slice_waves == 8) return go16<IN, OUT, EPI, 8, 8>(L);
    if (L.tbn == 64 && L.slice_waves == 8) return go16<IN, OUT, EPI, 4, 8>(L);
    if (L.tbn == 32 && L.slice_waves == 16) return go16<IN, OUT, EPI, 2, 16>(L);
    return hipErrorInvalidValue;
}

template <int IN>
hipError_t by_out16(const GemmLaunch& L) {
    constexpr int SAME = IN == IN_BF16 ? OUT_BF16 : OUT_F16;
    if (L.epi == EPI_NONE && L.out == OUT_F32) return by_strip<IN, OUT_F32, EPI_NONE>(L);
    if (L.epi != EPI_FULL) return hipErrorInvalidValue;
    if (L.out == OUT_F32) return by_strip<IN, OUT_F32, EPI_FULL>(L);
    if (L.out == SAME) return by_strip<IN, SAME, EPI_FULL>(L);
    return hipErrorInvalidValue;
}

template <int OUT, int W>
hipError_t go8(const GemmLaunch& L) {
    const char* a = L.A;
    const char* b = L.B;
    char* c = L.C;
    int M = L.M, N = L.N, K = L.K, lda = L.lda, ldb = L.ldb, ldc = L.ldc, strips = L.tiles_n;
    EpiArgs e = L.e;
    void* args[] = {&a, &b, &c, &M, &N, &K, &lda, &ldb, &ldc, &strips, &e};
    return hipLaunchKernel((const void*)skinny8_kernel<OUT, W>, dim3((unsigned)strips), dim3(64 * W),
                           args, 0, L.stream);
}

template <int OUT>
hipError_t by_waves8(const GemmLaunch& L) {
    if (L.tbn != 16) return hipErrorInvalidValue;
    if (L.slice_waves == 8) return go8<OUT, 8>(L);
    if (L.slice_waves == 16) return go8<OUT, 16>(L);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_skinny(const GemmLaunch& L) {
    if (L.M < 1 || L.M > SKINNY_M || L.splits < 1) return hipErrorInvalidValue;
    if (L.in == IN_BF16 && L.layout == LAY_NN) return by_out16<IN_BF16>(L);
    if (L.in == IN_F16 && L.layout == LAY_NN) return by_out16<IN_F16>(L);
    if (L.in != IN_F8W || L.layout != LAY_NT || L.splits != 1 || L.epi != EPI_FULL)
        return hipErrorInvalidValue;
    if (L.out == OUT_F32) return by_waves8<OUT_F32>(L);
    if (L.out == OUT_BF16) return by_waves8<OUT_BF16>(L);
    if (L.out == OUT_F16) return by_waves8<OUT_F16>(L);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
