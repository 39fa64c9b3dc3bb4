// skinny.hip -- products of at most 16 rows (tokens being generated) on gfx950
// (MI355X): A[M x K] B[K x N] (NN) and A[M x K] B[N x K]^T (NT), and the rank-M
// update A[M x K]^T D[M x N] of their backward pass.
//
// Such a product reads B once and computes little: the floor is B's bytes over
// the HBM rate.  So no LDS staging: B goes straight from memory into the
// registers that the matrix instruction reads, with many loads in flight.  A
// workgroup owns a strip of columns, its W waves take its k steps in turn, and
// their partial sums are added in LDS in wave order (deterministic).  K may be
// split over workgroups too, with fp32 partials in the caller's workspace.
//
// NN (bf16, fp16, fp32): lane (g, c) of 64 (g = lane / 16, c = lane % 16) loads
// the CPL consecutive columns CPL c .. of the eight k-rows 8 g .. 8 g + 7 of a
// 32-k step, and matrix instruction j covers columns n0 + CPL c + j, c = 0 .. 15.
// 16-bit: v_mfma_f32_16x16x32 wants eight k of one column per lane; the lane
// holds eight rows of CPL columns, and one v_perm_b32 per output word picks a
// column's halves from two rows' words: half an operation per element, instead
// of a transpose through LDS.  fp32: v_mfma_f32_16x16x4_f32 wants one k per lane,
// which each loaded word is.
//
// NT (bf16, fp16, fp32, e4m3): B's rows are K-contiguous, so a lane loads its
// operand as it is: row n0 + c, two 16-byte pieces 64 bytes apart per 128-byte
// step, so that the four lane groups read 64 consecutive bytes of a row at a time
// (A's pieces the same: the order of k inside the instructions cancels).  e4m3
// values are widened to bf16 in registers, exactly, for the bf16 instruction: the
// kernel waits for memory, and the sums are fp32 (the 8-bit instruction's are not
// quite: gemmt.hip).
//
// Measured, weights from HBM: 1 x 4096 x 4096 bf16 12.3 us (2.7 TB/s, its second
// launch included), 1 x 4096 x 14336 28.0 (4.2), 16 x 4096 x 4096 e4m3 7.2 (2.3),
// 1 x 8192 x 8192 e4m3 15.3 (4.4).  Small ones are bound by latency.
//
// Rows past M come as zeros from A's resource.

#include <type_traits>

#include "kern_common.h"

namespace dgemm {
namespace {


template <int IN>
__device__ __forceinline__ f32x4 mfma_16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (IN == IN_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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
    // As loaded (a conversion or a product would wait for the loads here).
    uint32_t res[PER], bias[PER], sa[PER], sb[PER];

    __device__ __forceinline__ void prefetch(int M, int N, int n0, int wave, int lane,
                                             const EpiArgs& e) {
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int idx = wave * PER + q;
            row[q] = 4 * (lane >> 4) + idx % 4;
            col[q] = n0 + CPL * (lane & 15) + idx / 4;
            if (idx >= NV) row[q] = M;  // W larger than the values: none
        }
        if constexpr (EPI == EPI_FULL) {
            constexpr int ES = fmt_es<OUT>;
#pragma unroll
            for (int q = 0; q < PER; ++q) res[q] = bias[q] = sa[q] = sb[q] = 0u;
            if (wave * PER >= NV) return;
            // Elements outside C: an offset outside the resource, which loads 0.
            if (e.res) {
                const auto r = c_rsrc((char*)e.res, M, N, e.ldr, 0, 0, ES);
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    const int at = inside(q, M, N) ? (row[q] * e.ldr + col[q]) * ES : (int)OOB_LANE;
                    if constexpr (OUT == OUT_F32) res[q] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
                    else res[q] = __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
                }
            }
            auto words = [&](const float* p, int n, auto index, uint32_t (&to)[PER]) {
                const auto r = make_rsrc((const char*)p, (int64_t)n * 4);
#pragma unroll
                for (int q = 0; q < PER; ++q)
                    to[q] = __builtin_amdgcn_raw_buffer_load_b32(
                        r, inside(q, M, N) ? index(q) * 4 : (int)OOB_LANE, 0, 0);
            };
            if (e.bias) words(e.bias, N, [&](int q) { return col[q]; }, bias);
            if (e.scale_a) {
                words(e.scale_a, M, [&](int q) { return row[q]; }, sa);
                words(e.scale_b, N, [&](int q) { return col[q]; }, sb);
            }
        }
    }
    __device__ __forceinline__ bool inside(int q, int M, int N) const {
        return row[q] < M && col[q] < N;
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
                if (e.scale_a) v[q] = v[q] * as_float(sa[q]) * as_float(sb[q]);
                v[q] += as_float(bias[q]);
                if (e.pre && row[q] < M && col[q] < N)
                    store_c<OUT>(e.pre, (int64_t)row[q] * e.ldz + col[q], v[q]);
            }
        }
        if constexpr (EPI == EPI_FULL) apply_act<OUT>(v, e.act);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if constexpr (EPI == EPI_FULL) {
                if (e.res) v[q] += OUT == OUT_F32    ? as_float(res[q])
                                   : OUT == OUT_BF16 ? as_float(res[q] << 16)
                                   : (float)__builtin_bit_cast(_Float16, (unsigned short)res[q]);
            }
            if (row[q] < M && col[q] < N) store_c<OUT>(C, (int64_t)row[q] * ldc + col[q], v[q]);
        }
    }
};

// Workgroup strip map: consecutive strips to one XCD (workgroups are dealt to
// the 8 XCDs in turn), so that strips narrower than a 128-byte line share it in
// one L2.
__device__ __forceinline__ int strip_of(int wg, int strips) {
    int tm, tn;
    map_tile(wg, 1, strips, tm, tn);
    return tn;
}

template <int IN, int OUT, int EPI, int CPL, int W>
__global__ __launch_bounds__(64 * W) void skinny_nn_kernel(
    const char* __restrict__ A, const char* __restrict__ B, char* C, int M, int N, int K, int lda,
    int ldb, int ldc, int strips, int kchunk, int64_t c_zstride, EpiArgs epi) {
    constexpr bool F32 = IN == IN_F32;
    constexpr int ES = F32 ? 4 : 2;
    constexpr int WD = CPL * ES / 4;    // words per lane and k-row
    constexpr int AW = ES / 2;          // 16-byte pieces of A per lane and step
    // Steps per chunk; two chunks in registers, within 128 of them for 16 waves.
    constexpr int D = WD == 4 || F32 ? 2 : 3;
    __shared__ float red[W * CPL * 4 * 64];
    {
        const int kbeg = (int)blockIdx.y * kchunk;
        A += (int64_t)kbeg * ES;
        B += (int64_t)kbeg * ldb * ES;
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
    u32x4 a[2 * D][AW];
    auto load = [&](int t, int S) {  // S: a constant once unrolled
        const int k0 = t * 32;
        const int rows = (K - k0) < 32 ? (K - k0) : 32;
        const auto rb = make_rsrc(B + ((int64_t)k0 * ldb + n0) * ES,
                                  rows > 0 ? ((int64_t)(rows - 1) * ldb + cols) * ES : 0);
        const auto ra = make_rsrc(A + (int64_t)k0 * ES,
                                  rows > 0 ? ((int64_t)(M - 1) * lda + rows) * ES : 0);
#pragma unroll
        for (int h = 0; h < AW; ++h) a[S][h] = load16(ra, (c * lda + 8 * g) * ES + 16 * h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int off = ((8 * g + j) * ldb + CPL * c) * ES;
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
        u32x4 av[AW];
#pragma unroll
        for (int h = 0; h < AW; ++h) {
            av[h] = a[S][h];
            if (k0 + 32 > K) av[h] = mask_bytes(av[h], (K - k0 - 8 * g) * ES - 16 * h);  // row padding
        }
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int w = 0; w < WD; ++w)
                    acc[w] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_float(av[j >> 2][j & 3]),
                                                                  as_float(b[S][j][w]), acc[w], 0, 0, 0);
        } else {
#pragma unroll
            for (int w = 0; w < WD; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u32x4 bv;
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        bv[p] = __builtin_amdgcn_perm(b[S][2 * p + 1][w], b[S][2 * p][w],
                                                      h ? 0x07060302u : 0x05040100u);
                    acc[2 * w + h] = mfma_16<IN>(av[0], bv, acc[2 * w + h]);
                }
        }
    };
    // Wave w takes steps w, w + W, ...: the workgroup reads B's rows in order.
    run_steps<D>((nstep - wave + W - 1) / W, [&](int i, int slot) { load(wave + i * W, slot); },
                 [&](int i, int slot, auto) { use(wave + i * W, slot); });
    strip.finish(acc, red, C, M, N, ldc, wave, lane, epi);
}

template <int IN, int OUT, int W>
__global__ __launch_bounds__(64 * W) void skinny_nt_kernel(
    const char* __restrict__ A, const char* __restrict__ B, char* C, int M, int N, int K, int lda,
    int ldb, int ldc, int strips, EpiArgs epi) {
    constexpr int ES = IN == IN_F32 ? 4 : IN == IN_F8W ? 1 : 2;
    __shared__ float red[W * 4 * 64];
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int n0 = strip_of((int)blockIdx.x, strips) * 16;
    const int rows_b = (N - n0) < 16 ? (N - n0) : 16;
    constexpr int SK = 128 / ES;  // k per step
    const int nstep = (K + SK - 1) / SK;
    Strip<OUT, EPI_FULL, 1, W> strip;
    strip.prefetch(M, N, n0, wave, lane, epi);
    constexpr int D = 2;  // steps per chunk; two chunks in registers
    u32x4 a[2 * D][2], b[2 * D][2];
    auto load = [&](int t, int S) {  // S: a constant once unrolled
        const int k0 = t * SK;
        const int krem = (K - k0) < SK ? (K - k0) : SK;
        const auto ra = make_rsrc(A + (int64_t)k0 * ES,
                                  krem > 0 ? ((int64_t)(M - 1) * lda + krem) * ES : 0);
        const auto rb = make_rsrc(B + ((int64_t)n0 * ldb + k0) * ES,
                                  krem > 0 ? ((int64_t)(rows_b - 1) * ldb + krem) * ES : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            a[S][h] = load16(ra, c * lda * ES + 64 * h + 16 * g);
            b[S][h] = load16(rb, c * ldb * ES + 64 * h + 16 * g);
        }
    };
    f32x4 acc[1] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
    auto use = [&](int t, int S) {
        const int k0 = t * SK;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 x = a[S][h], y = b[S][h];
            if (k0 + SK > K) {  // the rows' padding: 0 * NaN would be a NaN, so both
                const int valid = (K - k0) * ES - (64 * h + 16 * g);
                x = mask_bytes(x, valid);
                y = mask_bytes(y, valid);
            }
            if constexpr (IN == IN_F32) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_float(x[q]), as_float(y[q]), acc[0],
                                                                  0, 0, 0);
            } else if constexpr (IN == IN_F8W) {
#pragma unroll
                for (int q = 0; q < 4; q += 2)
                    acc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        widen_f8(x[q], x[q + 1]), widen_f8(y[q], y[q + 1]), acc[0], 0, 0, 0);
            } else {
                acc[0] = mfma_16<IN>(x, y, acc[0]);
            }
        }
    };
    run_steps<D>((nstep - wave + W - 1) / W, [&](int i, int slot) { load(wave + i * W, slot); },
                 [&](int i, int slot, auto) { use(wave + i * W, slot); });
    strip.finish(acc, red, C, M, N, ldc, wave, lane, epi);
}

// The rank-M update: C[k][n] = sum over m < M <= 16 of A[m][k] D[m][n], a weight's
// gradient from a few tokens.  Its floor is writing C; at 16 rows the fp32 multiply-adds,
// 1024 per lane, bound it (4096 x 4096 bf16 16 us, floor 6.5).  A wave owns 8 rows of 512
// columns (8 per lane), reads D's pieces once, takes its rows' eight values of
// A[m] as wave-uniform scalars, and stores 16-byte pieces.
template <int FMT>
__global__ __launch_bounds__(256) void outer_kernel(const char* __restrict__ A,
                                                    const char* __restrict__ D, char* C, int M, int N,
                                                    int K, int lda, int ldd, int ldc, int col_blocks) {
    constexpr int ES = fmt_es<FMT>;
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = ((int)blockIdx.x % col_blocks) * 512 + lane * 8;
    const int k0 = ((int)blockIdx.x / col_blocks) * 32 + wave * 8;
    if (k0 >= K) return;
    const int nvalid = N - c;
    float acc[8][8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
    // Every row's loads in flight at once.  Pieces past a row's end hold other
    // data or zeros and feed outputs that are not stored.
    Row8<FMT> d[SKINNY_M], a[SKINNY_M];
#pragma unroll
    for (int m = 0; m < SKINNY_M; ++m)
        if (m < M) {
            d[m].load_whole(make_rsrc(D + (int64_t)m * ldd * ES, (int64_t)N * ES),
                            nvalid > 0 ? (uint32_t)c * ES : OOB_LANE);
            a[m].load_whole(make_rsrc(A + (int64_t)m * lda * ES, (int64_t)K * ES), (uint32_t)k0 * ES);
        }
#pragma unroll
    for (int m = 0; m < SKINNY_M; ++m)
        if (m < M) {
            float x[8], y[8];
            d[m].get(x);
            a[m].get(y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[j][i] += y[j] * x[i];
        }
    const __amdgpu_buffer_rsrc_t rc =
        make_rsrc(C + (int64_t)k0 * ldc * ES,
                  ((int64_t)((K - k0 < 8 ? K - k0 : 8) - 1) * ldc + N) * ES);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Row8<FMT> o;
        o.set(acc[j]);
        if (k0 + j < K && nvalid > 0) o.store(rc, (uint32_t)(j * ldc + c) * ES, nvalid);
    }
}

template <int IN, int OUT, int EPI, int CPL, int W>
hipError_t go_nn(const GemmLaunch& L) {
    const char* a = L.A;
    const char* b = L.B;
    char* c = L.C;
    int M = L.M, N = L.N, K = L.K, lda = L.lda, ldb = L.ldb, ldc = L.ldc, strips = L.tiles_n;
    int kchunk = L.kchunk;
    int64_t zs = L.c_zstride;
    EpiArgs e = L.e;
    void* args[] = {&a, &b, &c, &M, &N, &K, &lda, &ldb, &ldc, &strips, &kchunk, &zs, &e};
    return hipLaunchKernel((const void*)skinny_nn_kernel<IN, OUT, EPI, CPL, W>,
                           dim3((unsigned)strips, (unsigned)L.splits), dim3(64 * W), args, 0, L.stream);
}

template <int IN, int OUT, int EPI>
hipError_t by_strip(const GemmLaunch& L) {
    if constexpr (IN != IN_F32)
        if (L.tbn == 128 && L.slice_waves == 8) return go_nn<IN, OUT, EPI, 8, 8>(L);
    if (L.tbn == 64 && L.slice_waves == 8) return go_nn<IN, OUT, EPI, 4, 8>(L);
    if (L.tbn == 32 && L.slice_waves == 16) return go_nn<IN, OUT, EPI, 2, 16>(L);
    return hipErrorInvalidValue;
}

template <int IN>
hipError_t nn_by_out(const GemmLaunch& L) {
    if (L.epi == EPI_NONE && L.out == OUT_F32) return by_strip<IN, OUT_F32, EPI_NONE>(L);
    if (L.epi != EPI_FULL) return hipErrorInvalidValue;
    if (L.out == OUT_F32) return by_strip<IN, OUT_F32, EPI_FULL>(L);
    if constexpr (IN == IN_BF16)
        if (L.out == OUT_BF16) return by_strip<IN, OUT_BF16, EPI_FULL>(L);
    if constexpr (IN == IN_F16)
        if (L.out == OUT_F16) return by_strip<IN, OUT_F16, EPI_FULL>(L);
    return hipErrorInvalidValue;
}

template <int IN, int OUT, int W>
hipError_t go_nt_w(const GemmLaunch& L) {
    const char* a = L.A;
    const char* b = L.B;
    char* c = L.C;
    int M = L.M, N = L.N, K = L.K, lda = L.lda, ldb = L.ldb, ldc = L.ldc, strips = L.tiles_n;
    EpiArgs e = L.e;
    void* args[] = {&a, &b, &c, &M, &N, &K, &lda, &ldb, &ldc, &strips, &e};
    return hipLaunchKernel((const void*)skinny_nt_kernel<IN, OUT, W>, dim3((unsigned)strips), dim3(64 * W),
                           args, 0, L.stream);
}

template <int IN, int OUT>
hipError_t go_nt(const GemmLaunch& L) {
    if (L.tbn != 16 || L.splits != 1 || L.epi != EPI_FULL) return hipErrorInvalidValue;
    if (L.slice_waves == 16) return go_nt_w<IN, OUT, 16>(L);
    if (L.slice_waves == 8) return go_nt_w<IN, OUT, 8>(L);
    if (L.slice_waves == 4) return go_nt_w<IN, OUT, 4>(L);
    return hipErrorInvalidValue;
}

template <int FMT>
hipError_t go_outer(const GemmLaunch& L) {
    const char* a = L.A;
    const char* d = L.B;
    char* c = L.C;
    int M = L.K, N = L.N, K = L.M, lda = L.lda, ldd = L.ldb, ldc = L.ldc;
    int col_blocks = (N + 511) / 512;
    const int64_t blocks = (int64_t)col_blocks * (((int64_t)K + 31) / 32);
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    void* args[] = {&a, &d, &c, &M, &N, &K, &lda, &ldd, &ldc, &col_blocks};
    return hipLaunchKernel((const void*)outer_kernel<FMT>, dim3((unsigned)blocks), dim3(256), args, 0,
                           L.stream);
}

}  // namespace

hipError_t launch_skinny(const GemmLaunch& L) {
    if (L.layout == LAY_TN) {
        if (L.K < 0 || L.K > SKINNY_M || L.splits != 1) return hipErrorInvalidValue;
        if (L.in == IN_F32 && L.out == OUT_F32) return go_outer<OUT_F32>(L);
        if (L.in == IN_BF16 && L.out == OUT_BF16) return go_outer<OUT_BF16>(L);
        if (L.in == IN_F16 && L.out == OUT_F16) return go_outer<OUT_F16>(L);
        return hipErrorInvalidValue;
    }
    if (L.M < 1 || L.M > SKINNY_M || L.splits < 1) return hipErrorInvalidValue;
    if (L.layout == LAY_NN) {
        if (L.in == IN_BF16) return nn_by_out<IN_BF16>(L);
        if (L.in == IN_F16) return nn_by_out<IN_F16>(L);
        if (L.in == IN_F32) return nn_by_out<IN_F32>(L);
        return hipErrorInvalidValue;
    }
    if (L.in == IN_F8W) {
        if (L.out == OUT_F32) return go_nt<IN_F8W, OUT_F32>(L);
        if (L.out == OUT_BF16) return go_nt<IN_F8W, OUT_BF16>(L);
        if (L.out == OUT_F16) return go_nt<IN_F8W, OUT_F16>(L);
    }
    if (L.in == IN_F32 && L.out == OUT_F32) return go_nt<IN_F32, OUT_F32>(L);
    if (L.in == IN_BF16 && L.out == OUT_BF16) return go_nt<IN_BF16, OUT_BF16>(L);
    if (L.in == IN_F16 && L.out == OUT_F16) return go_nt<IN_F16, OUT_F16>(L);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
