// slicet.hip -- small outputs of the transposed layouts and of 8-bit operands
// (gemmt.hip's products), for gfx950 (MI355X).
//
// As slicek16.hip does for A[M x K] B[K x N]: a workgroup of W waves owns a small
// TS x TS tile (TS = 32 MI), each wave takes an equal run of 128-byte K blocks
// (64 k of 16-bit operands, 128 of e4m3) and holds the whole tile's accumulators
// for its own k; the W partial tiles are added in LDS in wave order, and each wave
// finishes its share of the tile with the full epilogue.  No workspace, no second
// kernel: such a product is a few us, a split's second launch another three.
//
// No operand is shared between the waves, so each wave moves its own:
//   NT: both operands K-contiguous: TS rows x 128 bytes of each go into the wave's
//     own LDS region by direct-to-LDS loads, eight lanes to a row's line (loading
//     the matrix instruction's operands straight from memory touches 32 lines per
//     instruction: 299 x 2164 with 2517 terms took 24.9 us that way, 17.0 this), in
//     gemm16's swizzled layout, and are read with ds_read_b128.  Per 16-k half h of a 16-bit
//     block lane (g, li) takes chunk 2 h + g of row li; of an e4m3 block, per 64 k,
//     chunks 4 q + 2 g and 4 q + 2 g + 1 (the order of k inside the instruction
//     cancels).
//   TN: both along the output: 64 k-rows x TS columns of each as they lie in
//     memory, read back through the transpose read (slicek16.hip's B).
// fp32 operands (the backward pass of small fp32 layers, which would otherwise
// transpose A and B in launches of their own): blocks of 32 k, instructions of 2 k;
// NT takes k = 4 (2 h + g) + w of both operands together, TN reads k-row
// 2 (4 h + w) + g as it lies.
// D to 2 D blocks are in flight per wave.

#include <type_traits>

#include "kern_common.h"
#include "stage16.h"

namespace dgemm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int cmax(int a, int b) { return a > b ? a : b; }

// One product's arguments.
struct SliceArgs {
    const char* X;
    const char* Y;
    char* C;
    int M, N, K, ldx, ldy, ldc, tiles_m, tiles_n;
};

template <int MI, int W>
struct SliceTile {
    // Blocks per chunk, two chunks in LDS.
    static constexpr int D = MI == 1 && W == 4 ? 2 : 1;
    static constexpr int BLKB = 128 * 32 * MI;  // bytes of one operand's block
    static constexpr int STAGES = W * 2 * D * 2 * BLKB;
    static constexpr int RED = W * MI * MI * 16 * 64 * 4;
    static constexpr int LDS = cmax(STAGES, RED);
};

// Tile `wg` of a product.
template <int IN, int LAY, int OUT, int MI, int W>
__device__ __forceinline__ void slice_tile(const SliceArgs& a, int wg, const EpiArgs& epi, char* smem) {
    const char* __restrict__ X = a.X;
    const char* __restrict__ Y = a.Y;
    char* const C = a.C;
    const int M = a.M, N = a.N, K = a.K, ldx = a.ldx, ldy = a.ldy, ldc = a.ldc;
    constexpr bool KC = LAY == LAY_NT;  // K-contiguous operands
    constexpr bool F8 = IN == IN_F8 || IN == IN_F8W;
    static_assert(KC || !F8, "8-bit operands are K-contiguous");
    constexpr int ES = F8 ? 1 : IN == IN_F32 ? 4 : 2;
    constexpr int BK = 128 / ES;
    constexpr int TS = 32 * MI;
    constexpr int NB = MI * MI;
    using T = SliceTile<MI, W>;
    constexpr int D = T::D, BLKB = T::BLKB;
    constexpr int NDB = BLKB / 1024;          // an operand block's direct-to-LDS loads
    int tm, tn;
    map_tile(wg, a.tiles_m, a.tiles_n, tm, tn);
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 5, li = lane & 31;
    const int m0 = tm * TS, n0 = tn * TS;
    const int rows_x = (M - m0) < TS ? (M - m0) : TS;
    const int rows_y = (N - n0) < TS ? (N - n0) : TS;
    const int nblk = (K + BK - 1) / BK;
    const int kb0 = (int)((int64_t)wave * nblk / W);
    const int nb = (int)((int64_t)(wave + 1) * nblk / W) - kb0;

    f32x16 acc[MI][MI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int nj = 0; nj < MI; ++nj)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[mi][nj][r] = 0.0f;

    // One block's operand fragments: [32-row block][16-byte chunk].
    struct Block {
        u32x4 x[MI][4], y[MI][4];
    };
    auto mul = [&](const Block& f) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int nj = 0; nj < MI; ++nj) {
                f32x16 c = acc[mi][nj];
                if constexpr (IN == IN_F8) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const i32x8 a = __builtin_shufflevector(
                            __builtin_bit_cast(i32x4, f.x[mi][2 * q]),
                            __builtin_bit_cast(i32x4, f.x[mi][2 * q + 1]), 0, 1, 2, 3, 4, 5, 6, 7);
                        const i32x8 b = __builtin_shufflevector(
                            __builtin_bit_cast(i32x4, f.y[nj][2 * q]),
                            __builtin_bit_cast(i32x4, f.y[nj][2 * q + 1]), 0, 1, 2, 3, 4, 5, 6, 7);
                        c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
                    }
                } else if constexpr (IN == IN_F8W) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int w = 0; w < 4; w += 2)
                            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                widen_f8(f.x[mi][q][w], f.x[mi][q][w + 1]),
                                widen_f8(f.y[nj][q][w], f.y[nj][q][w + 1]), c, 0, 0, 0);
                } else if constexpr (IN == IN_F32) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            c = __builtin_amdgcn_mfma_f32_32x32x2f32(as_float(f.x[mi][h][w]),
                                                                     as_float(f.y[nj][h][w]), c, 0, 0, 0);
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if constexpr (IN == IN_BF16)
                            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                __builtin_bit_cast(bf16x8, f.x[mi][h]),
                                __builtin_bit_cast(bf16x8, f.y[nj][h]), c, 0, 0, 0);
                        else
                            c = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                                __builtin_bit_cast(f16x8, f.x[mi][h]),
                                __builtin_bit_cast(f16x8, f.y[nj][h]), c, 0, 0, 0);
                    }
                }
                acc[mi][nj] = c;
            }
    };

    char* const mine = smem + wave * 2 * D * 2 * BLKB;
    // Load j's 16 bytes of this lane belong at bytes 1024 j + 16 lane of the stage.
    int vx[NDB], vy[NDB];
#pragma unroll
    for (int j = 0; j < NDB; ++j) {
        const int row = A16_RPB * j + lane / A16_CH;
        const int c = (lane % A16_CH) ^ a16_phi(row);
        const int q = 1024 * j + 16 * lane;  // k-row q / RB, byte q % RB of the row
        constexpr int RB = ES * TS;
        vx[j] = KC ? row * ldx * ES + 16 * c : (q / RB) * ldx * ES + q % RB;
        vy[j] = KC ? row * ldy * ES + 16 * c : (q / RB) * ldy * ES + q % RB;
    }
    // The transpose read's slot: lane 16 G + 4 a + q reads k-row 8 (G / 2) + a,
    // columns 16 (G & 1) + 4 q ...
    const int grp = lane >> 4;
    const int slot = ((8 * (grp >> 1) + ((lane >> 2) & 3)) * TS + 16 * (grp & 1) + 4 * (lane & 3)) * 2;
    auto chunk = [&](int h) { return F8 ? 4 * (h >> 1) + 2 * g + (h & 1) : 2 * h + g; };
    auto operand = [&](const char* p, int ld, int o0, int rows, int k0) {
        const int krem = (K - k0) < BK ? (K - k0) : BK;
        if constexpr (KC)
            return make_rsrc(p + ((int64_t)o0 * ld + k0) * ES, ((int64_t)(rows - 1) * ld + krem) * ES);
        else
            return make_rsrc(p + ((int64_t)k0 * ld + o0) * ES, ((int64_t)(krem - 1) * ld + rows) * ES);
    };
    auto load = [&](int i, int s) {
        const int k0 = (kb0 + i) * BK;
        const auto rx = operand(X, ldx, m0, rows_x, k0);
        const auto ry = operand(Y, ldy, n0, rows_y, k0);
        char* st = mine + s * 2 * BLKB;
#pragma unroll
        for (int j = 0; j < NDB; ++j) dma16(rx, lds_addr(st + 1024 * j), vx[j]);
#pragma unroll
        for (int j = 0; j < NDB; ++j) dma16(ry, lds_addr(st + BLKB + 1024 * j), vy[j]);
    };
    run_steps<D>(nb, load, [&](int i, int s, auto newer) {
        // This step's loads have landed; at most the newer steps' are in flight.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(decltype(newer)::value * 2 * NDB, 15));
        __builtin_amdgcn_sched_barrier(0);
        const char* st = mine + s * 2 * BLKB;
        Block f;
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int mi = 0; mi < MI; ++mi) {
                if constexpr (KC) {
                    const int at = a16_off(mi * 32 + li, chunk(h));
                    f.x[mi][h] = *(const u32x4*)(st + at);
                    f.y[mi][h] = *(const u32x4*)(st + BLKB + at);
                } else if constexpr (IN == IN_F32) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const char* at = st + ((2 * (4 * h + w) + g) * TS + 32 * mi + li) * 4;
                        f.x[mi][h][w] = *(const uint32_t*)at;
                        f.y[mi][h][w] = *(const uint32_t*)(at + BLKB);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const char* at = st + slot + ((16 * h + 4 * t) * TS + 32 * mi) * 2;
                        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                        const u32x2 p = __builtin_bit_cast(
                            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)at));
                        const u32x2 q = __builtin_bit_cast(
                            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(at + BLKB)));
                        f.x[mi][h][2 * t] = p[0];
                        f.x[mi][h][2 * t + 1] = p[1];
                        f.y[mi][h][2 * t] = q[0];
                        f.y[mi][h][2 * t + 1] = q[1];
                    }
                }
            }
        // The reads are done before the slot's next loads are issued.
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        __builtin_amdgcn_sched_barrier(0);
        const int k0 = (kb0 + i) * BK;
        if (KC && k0 + BK > K) {  // the rows' padding: 0 * NaN would be a NaN, so both operands
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const int valid = (K - k0) * ES - 16 * chunk(h);
                    f.x[mi][h] = mask_bytes(f.x[mi][h], valid);
                    f.y[mi][h] = mask_bytes(f.y[mi][h], valid);
                }
        }
        mul(f);
    });
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();  // every wave is done with its stages: the sums reuse them

    // As in slicek16.hip: value idx = 16 b + r of every lane, wave w finishing
    // idx in [w PER, w PER + PER).
    float* const red = (float*)smem;
    constexpr int PER = NB * 16 / W;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            red[(wave * NB * 16 + b * 16 + r) * 64 + lane] = acc[b / MI][b % MI][r];
    __syncthreads();
    float v[PER];
    int row[PER], col[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int idx = wave * PER + q;
        const int b = idx / 16, r = idx % 16;
        v[q] = red[idx * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v[q] += red[(w * NB * 16 + idx) * 64 + lane];
        row[q] = m0 + (b / MI) * 32 + 8 * (r >> 2) + 4 * g + (r & 3);
        col[q] = n0 + (b % MI) * 32 + li;
    }
    finish_full<OUT, PER>(v, row, col, C, M, N, ldc, epi);
}

template <int IN, int LAY, int OUT, int MI, int W>
__global__ __launch_bounds__(64 * W) void slicet_kernel(SliceArgs a, EpiArgs epi) {
    __shared__ __attribute__((aligned(1024))) char smem[SliceTile<MI, W>::LDS];
    slice_tile<IN, LAY, OUT, MI, W>(a, (int)blockIdx.x, epi, smem);
}

// The products of a small backward pass (either may have no tiles) and its bias
// gradient's column sums: independent, and each a few us, so one launch instead of three (2.4 us of host
// time each).  The tiles of both products come first, NT's before TN's counted
// from workgroup `first` on, cyclically (0, or TN's first); then the column sums.
template <int IN, int MI_NT, int MI_TN>
__global__ __launch_bounds__(256) void slicet_pair_kernel(SliceArgs nt, SliceArgs tn, int first,
                                                          ColReduceArgs r) {
    constexpr int OUT = IN == IN_BF16 ? OUT_BF16 : IN == IN_F16 ? OUT_F16 : OUT_F32;
    __shared__ __attribute__((
        aligned(1024))) char smem[cmax(SliceTile<MI_NT, 4>::LDS, SliceTile<MI_TN, 4>::LDS)];
    const int n_nt = nt.tiles_m * nt.tiles_n, n_tn = tn.tiles_m * tn.tiles_n;
    int wg = (int)blockIdx.x;
    if (wg < n_nt + n_tn) {
        wg += first;
        if (wg >= n_nt + n_tn) wg -= n_nt + n_tn;
    }
    EpiArgs e{};
    if (wg < n_nt) slice_tile<IN, LAY_NT, OUT, MI_NT, 4>(nt, wg, e, smem);
    else if (wg < n_nt + n_tn) slice_tile<IN, LAY_TN, OUT, MI_TN, 4>(tn, wg - n_nt, e, smem);
    else col_reduce(wg - n_nt - n_tn, r, (float*)smem);
}

SliceArgs args_of(const GemmLaunch& L) {
    return SliceArgs{L.A, L.B, L.C, L.M, L.N, L.K, L.lda, L.ldb, L.ldc, L.tiles_m, L.tiles_n};
}

template <int IN, int LAY, int OUT, int MI, int W>
hipError_t go(const GemmLaunch& L) {
    SliceArgs a = args_of(L);
    EpiArgs e = L.e;
    void* args[] = {&a, &e};
    return hipLaunchKernel((const void*)slicet_kernel<IN, LAY, OUT, MI, W>,
                           dim3((unsigned)(L.tiles_m * L.tiles_n)), dim3(64 * W), args, 0, L.stream);
}

template <int IN>
hipError_t go_pair(const GemmLaunch& nt, const GemmLaunch& tn, bool tn_first, const ColReduceArgs& r) {
    const bool m2 = nt.tbm == 64, n2 = tn.tbm == 64;
    const void* fn = m2 ? (n2 ? (const void*)slicet_pair_kernel<IN, 2, 2> : (const void*)slicet_pair_kernel<IN, 2, 1>)
                        : (n2 ? (const void*)slicet_pair_kernel<IN, 1, 2> : (const void*)slicet_pair_kernel<IN, 1, 1>);
    SliceArgs a = args_of(nt), b = args_of(tn);
    ColReduceArgs c = r;
    int first = tn_first ? nt.tiles_m * nt.tiles_n : 0;
    void* args[] = {&a, &b, &first, &c};
    const int blocks = nt.tiles_m * nt.tiles_n + tn.tiles_m * tn.tiles_n + (r.N > 0 ? col_reduce_blocks(r.N) : 0);
    if (blocks == 0) return hipSuccess;
    return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(256), args, 0, nt.stream);
}

template <int IN, int LAY, int OUT>
hipError_t by_variant(const GemmLaunch& L) {
    if (L.tbm == 32 && L.slice_waves == 4) return go<IN, LAY, OUT, 1, 4>(L);
    if (L.tbm == 32 && L.slice_waves == 8) return go<IN, LAY, OUT, 1, 8>(L);
    if (L.tbm == 64 && L.slice_waves == 4) return go<IN, LAY, OUT, 2, 4>(L);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_slicet(const GemmLaunch& L) {
    if (L.splits != 1 || L.tbm != L.tbn || L.epi != EPI_FULL) return hipErrorInvalidValue;
    if (L.layout == LAY_NT) {
        if (L.in == IN_F8W && L.out == OUT_F32) return by_variant<IN_F8W, LAY_NT, OUT_F32>(L);
        if (L.in == IN_F8 && L.out == OUT_BF16) return by_variant<IN_F8, LAY_NT, OUT_BF16>(L);
        if (L.in == IN_F8 && L.out == OUT_F16) return by_variant<IN_F8, LAY_NT, OUT_F16>(L);
        if (L.in == IN_BF16 && L.out == OUT_BF16) return by_variant<IN_BF16, LAY_NT, OUT_BF16>(L);
        if (L.in == IN_F16 && L.out == OUT_F16) return by_variant<IN_F16, LAY_NT, OUT_F16>(L);
    } else if (L.layout == LAY_TN) {
        if (L.in == IN_BF16 && L.out == OUT_BF16) return by_variant<IN_BF16, LAY_TN, OUT_BF16>(L);
        if (L.in == IN_F16 && L.out == OUT_F16) return by_variant<IN_F16, LAY_TN, OUT_F16>(L);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_slicet_pair(const GemmLaunch& nt, const GemmLaunch& tn, bool tn_first,
                              const ColReduceArgs& r) {
    for (const GemmLaunch* L : {&nt, &tn})
        if (L->splits != 1 || L->tbm != L->tbn || (L->tbm != 32 && L->tbm != 64) || L->in != nt.in)
            return hipErrorInvalidValue;
    if (nt.in == IN_BF16) return go_pair<IN_BF16>(nt, tn, tn_first, r);
    if (nt.in == IN_F16) return go_pair<IN_F16>(nt, tn, tn_first, r);
    if (nt.in == IN_F32) return go_pair<IN_F32>(nt, tn, tn_first, r);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
