// blockf8.hip -- products of e4m3 operands with a scale per block of 128 along K, for
// gfx950 (MI355X):
//
//   C = act(sum over blocks b of sa[i][b] sb[j'][b] sum_{k in b} A[i][k] B[j][k] + bias) + R,
//   j' = j / 128 (weights) or j (gradients: a scale per row and block on both sides)
//
// A: M x K, B: N x K, both K-contiguous.  A K step of the matrix kernels is 128 bytes of every
// row, which is one block: a step's matrix instructions start from zero, and their sums are
// added to the running ones scaled, in fp32: one multiply-add per output and block. Matrix and
// fp32 vector instructions hardly overlap on a SIMD (4096^3 on the large tile: 53 % of its
// cycles the one, 35 % the other; with two vector instructions per output, on the small tile,
// 42 % and 46 %), so what is left to save is vector instructions: the loop has next to none but
// these, with the stages' addresses in the reads' offsets (two steps written out) and no copies
// of scales.  To have few factors per lane, the operands trade places: the instruction's rows
// are B's, its columns (a lane each) A's, and sb is the same for all of a lane's sums where a
// weight has a scale per 128 x 128.  With a scale per row of B they differ, a second
// multiplication each.
//
// The vector unit adds to ordinary registers only, not to the accumulation half of the register
// file, so a wave cannot hold 256 running sums as gemmt.hip's do: a wave owns 128 x 64 outputs
// (256 x 256 tile, 8 waves, two to a SIMD) or 64 x 64 (128 x 128 tile, 4 waves, two workgroups
// to a CU), and one wave's instructions fill the other's waits.  4096^3, bf16 C: 62-67 us with
// a scale per 128 x 128 (2.1 PFLOP/s; gemm_f8 with a scale per row 58-61), 70.5 with one per
// row and block.
//
// The scales of a step come with its operands, by 4-byte direct-to-LDS loads (one per
// wave and step), and are read back one per lane.  Operands, LDS layout, tile map and
// edges as in gemmt.hip's NT kernel; the smallest outputs take slicet.hip's split of K over
// a workgroup's waves.
//
// 16-bit outputs use the 8-bit matrix instructions, whose sums over a block drop bits below
// 2^-13 of the largest of neighbouring products; fp32 outputs (IN_F8W) widen the values to
// bf16, exactly, for fp32 sums.  Both as in gemmt.hip.

#include <type_traits>

#include "kern_common.h"
#include "stage16.h"

namespace dgemm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int cmax(int a, int b) { return a > b ? a : b; }

// A product's arguments.
struct BlockArgs {
    const char* A;
    const char* B;
    char* C;
    int M, N, K, lda, ldb, ldc, tiles_m, tiles_n;
    BlockScales s;
};

// Four 16-byte chunks of one row: all 128 of its bytes in a step that a lane's half (g) takes,
// k group q = 64 k in chunks 4 q + 2 g and 4 q + 2 g + 1.
struct RowFrag {
    u32x4 w[4];
};

__device__ __forceinline__ i32x8 both(u32x4 lo, u32x4 hi) {
    return __builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1, 2,
                                   3, 4, 5, 6, 7);
}

// Half q (0, 1) of a step's product of 32 rows of B and 32 rows of A: c + B A^T over 64 k.
template <int IN>
__device__ __forceinline__ f32x16 half_product(const RowFrag& b, const RowFrag& a, int q, f32x16 c) {
    if constexpr (IN == IN_F8) {
        // both operands e4m3 (format code 0), block scales 1 (none applied)
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(both(b.w[2 * q], b.w[2 * q + 1]),
                                                               both(a.w[2 * q], a.w[2 * q + 1]), c, 0, 0, 0,
                                                               0, 0, 0);
    } else {
#pragma unroll
        for (int h = 2 * q; h < 2 * q + 2; ++h)
#pragma unroll
            for (int w = 0; w < 4; w += 2)
                c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_f8(b.w[h][w], b.w[h][w + 1]),
                                                            widen_f8(a.w[h][w], a.w[h][w + 1]), c, 0, 0, 0);
        return c;
    }
}

__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.0f;
    return z;
}

// Byte offset of this lane's row in a column of scales, or outside any range.
__device__ __forceinline__ int scale_off(int row, int rows, int stride) {
    return row < rows ? row * stride * 4 : (int)OOB_LANE;
}

// A resource over the scales of `rows` rows of block kb; empty past the end (kb >= nk).  Lanes
// without a row have offsets outside any range, so the rounded-up end is never read.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rsrc(const float* p, int64_t row, int rows, int s_row,
                                                             int kb, int s_blk, int nk) {
    const float* at = p + row * s_row + (int64_t)kb * s_blk;
    return make_rsrc((const char*)at, kb < nk ? ((int64_t)(rows - 1) * s_row + 1) * 4 : 0);
}

// ------------------------------------------------------------------ small outputs

// As slicet.hip: a TS x TS tile (TS = 32 MI) per workgroup of W waves, each with a run of
// the blocks and its own LDS stages; the waves' sums are added in LDS in wave order.  32 x 32 with
// eight waves, 64 x 64 with four (32 x 32 with four, more blocks in flight in each: 12 to 37 % slower).
template <int MI>
struct SliceTile {
    static constexpr int W = MI == 1 ? 8 : 4;
    static constexpr int D = 1;                           // blocks per chunk, two chunks in LDS
    static constexpr int BLKB = 128 * 32 * MI;            // bytes of one operand's block
    static constexpr int STAGE = 2 * BLKB + 512;          // and 64 scales of either
    static constexpr int RED = W * MI * MI * 16 * 64 * 4;
    static constexpr int LDS = cmax(W * 2 * D * STAGE, RED);
};

// NB: B's scales are per row.
template <int IN, int OUT, int MI, bool NB>
__global__ __launch_bounds__(64 * SliceTile<MI>::W) void block_slice_kernel(BlockArgs a, EpiArgs epi) {
    using T = SliceTile<MI>;
    constexpr int W = T::W;
    constexpr int TS = 32 * MI, NBLK = MI * MI, D = T::D, BLKB = T::BLKB;
    constexpr int NDB = BLKB / 1024;  // an operand block's direct-to-LDS loads
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
    int tm, tn;
    map_tile((int)blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 5, li = lane & 31;
    const int m0 = tm * TS, n0 = tn * TS;
    const int rows_a = (a.M - m0) < TS ? (a.M - m0) : TS;
    const int rows_b = (a.N - n0) < TS ? (a.N - n0) : TS;
    const int nblk = (a.K + F8_BLOCK - 1) / F8_BLOCK;
    const int kb0 = (int)((int64_t)wave * nblk / W);
    const int nb = (int)((int64_t)(wave + 1) * nblk / W) - kb0;

    f32x16 acc[MI][MI];  // [A's 32 rows][B's]
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int nj = 0; nj < MI; ++nj) acc[mi][nj] = zero16();

    char* const mine = smem + wave * 2 * D * T::STAGE;
    int va[NDB], vb[NDB];
#pragma unroll
    for (int j = 0; j < NDB; ++j) {
        const int row = A16_RPB * j + lane / A16_CH;
        const int c = (lane % A16_CH) ^ a16_phi(row);
        va[j] = row * a.lda + 16 * c;
        vb[j] = row * a.ldb + 16 * c;
    }
    // A tile lies in one block of 128 rows of B.
    const int64_t sb_row0 = NB ? n0 : n0 / F8_BLOCK;
    const int sb_rows = NB ? rows_b : 1;
    const int vsa = scale_off(lane, rows_a, a.s.sa_row);
    const int vsb = scale_off(NB ? lane : lane < TS ? 0 : 1, sb_rows, a.s.sb_row);
    auto load = [&](int i, int s) {
        const int kb = kb0 + i, k0 = kb * F8_BLOCK;
        const int krem = (a.K - k0) < F8_BLOCK ? (a.K - k0) : F8_BLOCK;
        const auto ra = make_rsrc(a.A + (int64_t)m0 * a.lda + k0, (int64_t)(rows_a - 1) * a.lda + krem);
        const auto rb = make_rsrc(a.B + (int64_t)n0 * a.ldb + k0, (int64_t)(rows_b - 1) * a.ldb + krem);
        char* st = mine + s * T::STAGE;
#pragma unroll
        for (int j = 0; j < NDB; ++j) dma16(ra, lds_addr(st + 1024 * j), va[j]);
#pragma unroll
        for (int j = 0; j < NDB; ++j) dma16(rb, lds_addr(st + BLKB + 1024 * j), vb[j]);
        dma4(scale_rsrc(a.s.sa, m0, rows_a, a.s.sa_row, kb, a.s.sa_blk, nblk), lds_addr(st + 2 * BLKB), vsa);
        dma4(scale_rsrc(a.s.sb, sb_row0, sb_rows, a.s.sb_row, kb, a.s.sb_blk, nblk),
             lds_addr(st + 2 * BLKB + 256), vsb);
    };
    run_steps<D>(nb, load, [&](int i, int s, auto newer) {
        // This step's loads have landed; at most the newer steps' are in flight.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(decltype(newer)::value * (2 * NDB + 2), 15));
        __builtin_amdgcn_sched_barrier(0);
        const char* st = mine + s * T::STAGE;
        RowFrag fa[MI], fb[MI];
        float sa[MI], sb[MI][NB ? 16 : 1];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int at = a16_off(mi * 32 + li, 4 * (h >> 1) + 2 * g + (h & 1));
                fa[mi].w[h] = *(const u32x4*)(st + at);
                fb[mi].w[h] = *(const u32x4*)(st + BLKB + at);
            }
            const float* ps = (const float*)(st + 2 * BLKB);
            sa[mi] = ps[mi * 32 + li];
            if constexpr (NB) {
#pragma unroll
                for (int r = 0; r < 16; ++r) sb[mi][r] = ps[64 + mi * 32 + 8 * (r >> 2) + 4 * g + (r & 3)];
            } else {
                sb[mi][0] = ps[64];
            }
        }
        // The reads are done before the slot's next loads are issued.
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        __builtin_amdgcn_sched_barrier(0);
        const int k0 = (kb0 + i) * F8_BLOCK;
        if (k0 + F8_BLOCK > a.K) {  // the rows' padding: 0 * NaN would be a NaN, so both operands
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const int valid = a.K - k0 - 16 * (4 * (h >> 1) + 2 * g + (h & 1));
                    fa[mi].w[h] = mask_bytes(fa[mi].w[h], valid);
                    fb[mi].w[h] = mask_bytes(fb[mi].w[h], valid);
                }
        }
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int nj = 0; nj < MI; ++nj) {
                f32x16 p = half_product<IN>(fb[nj], fa[mi], 0, zero16());
                p = half_product<IN>(fb[nj], fa[mi], 1, p);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[mi][nj][r] = __builtin_fmaf(p[r], sa[mi] * sb[nj][NB ? r : 0], acc[mi][nj][r]);
            }
    });
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();  // every wave is done with its stages: the sums reuse them

    // Value idx = 16 b + r of every lane, wave w finishing idx in [w PER, w PER + PER).
    float* const red = (float*)smem;
    constexpr int PER = NBLK * 16 / W;
#pragma unroll
    for (int b = 0; b < NBLK; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            red[(wave * NBLK * 16 + b * 16 + r) * 64 + lane] = acc[b / MI][b % MI][r];
    __syncthreads();
    float v[PER];
    int row[PER], col[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int idx = wave * PER + q;
        const int b = idx / 16, r = idx % 16;
        v[q] = red[idx * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v[q] += red[(w * NBLK * 16 + idx) * 64 + lane];
        row[q] = m0 + (b / MI) * 32 + li;
        col[q] = n0 + (b % MI) * 32 + 8 * (r >> 2) + 4 * g + (r & 3);
    }
    finish_full<OUT, PER>(v, row, col, a.C, a.M, a.N, a.ldc, epi);
}

// ------------------------------------------------------------------ grid tiles

// TBM x TBN tile, WM x WN waves, S = 2 stages of 128 bytes per row.
template <int TBM, int TBN, int WM, int WN>
struct GridTile {
    static constexpr int NW = WM * WN, S = 2;
    static constexpr int MI = TBM / WM / 32, NJ = TBN / WN / 32;  // a wave's blocks of 32 x 32
    static constexpr int A_STAGE = TBM * 128, B_STAGE = TBN * 128, S_STAGE = (TBM + TBN) * 4;
    static constexpr int A_DMA = A_STAGE / 1024 / NW, B_DMA = B_STAGE / 1024 / NW;
    static constexpr int LOADS = A_DMA + B_DMA + 1;  // and the scales of 64 rows
    static constexpr int LDS = S * (A_STAGE + B_STAGE + S_STAGE);
    static_assert((TBM + TBN) / 64 == NW && TBM % 64 == 0 && TBN % 64 == 0, "a load of scales per wave");
    static_assert(NW * full_lds<NJ> <= LDS && LDS <= 160 * 1024, "LDS budget");
};

// IN_F8 (16-bit outputs, and the fp32 partial sums of their K splits): the 16 x 16 x 128 instruction
// takes a whole block of K: its sums, rows 4 (lane / 16) .. of B and column lane % 16 of A, are four registers
// that the next instruction's cycles scale and add, so that two sets of four do for the
// products in flight; with a scale per row of B (NB) a lane needs four of them per 16 rows.  Two
// waves to a SIMD, at 247 of their 256 registers on the large tile.
//
// Against 32 x 32 x 64 instructions, two to a block (4096^3: 69 us with a scale per 128 x 128; with
// a scale per row, whose 32 factors per 64 rows leave no registers for the large tile, 95 on the
// small one), it takes 65 and 70.5 us, and the small tile 78 and 82 where it took 85 and 95.
//
// IN_F8W (fp32 outputs): four 16 x 16 x 32 bf16 instructions a block, on fragments widened once per
// step (B's) and per 16 rows (A's).  4096^3 122 us, with a scale per row of B 135 (32 x 32
// instructions whose fragments were widened per use 128 and 255).
template <int IN, int OUT, int TBM, int TBN, int WM, int WN, bool NB>
__global__ __launch_bounds__(64 * WM * WN, 2) void block_grid_kernel(BlockArgs a, int kchunk, int64_t c_zstride,
                                                                     EpiArgs epi) {
    using T = GridTile<TBM, TBN, WM, WN>;
    constexpr int S = T::S, NW = T::NW, MI = TBM / WM / 16, NJ = TBN / WN / 16;
    constexpr bool WIDE = IN == IN_F8W;
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
    char* const smA = smem;
    char* const smB = smem + S * T::A_STAGE;
    char* const smS = smB + S * T::B_STAGE;
    {
        const int z = (int)blockIdx.y;
        const int kbeg = z * kchunk;
        a.A += kbeg;
        a.B += kbeg;
        a.s.sa += (int64_t)(kbeg / F8_BLOCK) * a.s.sa_blk;
        a.s.sb += (int64_t)(kbeg / F8_BLOCK) * a.s.sb_blk;
        a.C += z * c_zstride;
        a.K = (a.K - kbeg) < kchunk ? (a.K - kbeg) : kchunk;
    }
    int tm, tn;
    map_tile((int)blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * TBM, n0 = tn * TBN;
    const int rows_a = (a.M - m0) < TBM ? (a.M - m0) : TBM;
    const int rows_b = (a.N - n0) < TBN ? (a.N - n0) : TBN;
    const int tid = (int)threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int g = lane >> 4, c = lane & 15;
    const int K = a.K, nk = (K + F8_BLOCK - 1) / F8_BLOCK;
    const int row0 = wave * A16_RPB + lane / A16_CH;
    const int ch = ((lane % A16_CH) ^ a16_phi(row0)) << 4;
    const int va = row0 * a.lda + ch, vb = row0 * a.ldb + ch;
    const int ja = NW * A16_RPB * a.lda, jb = NW * A16_RPB * a.ldb;
    const int64_t sb_row0 = NB ? n0 : n0 / F8_BLOCK;
    const int sb_rows = NB ? rows_b : (n0 + rows_b - 1) / F8_BLOCK - n0 / F8_BLOCK + 1;
    const bool for_a = wave < TBM / 64;
    const int srow = (for_a ? wave : wave - TBM / 64) * 64 + lane;
    const int vs = for_a ? scale_off(srow, rows_a, a.s.sa_row)
                         : scale_off(NB ? srow : srow / F8_BLOCK, sb_rows, a.s.sb_row);
    struct Desc { __amdgpu_buffer_rsrc_t a, b, s; int st; };
    auto desc = [&](int kt) {
        const int k0 = kt * F8_BLOCK;
        const int krem = (K - k0) < F8_BLOCK ? (K - k0) : F8_BLOCK;
        Desc d;
        d.a = make_rsrc(a.A + (int64_t)m0 * a.lda + k0, krem > 0 ? (int64_t)(rows_a - 1) * a.lda + krem : 0);
        d.b = make_rsrc(a.B + (int64_t)n0 * a.ldb + k0, krem > 0 ? (int64_t)(rows_b - 1) * a.ldb + krem : 0);
        d.s = for_a ? scale_rsrc(a.s.sa, m0, rows_a, a.s.sa_row, kt, a.s.sa_blk, nk)
                    : scale_rsrc(a.s.sb, sb_row0, sb_rows, a.s.sb_row, kt, a.s.sb_blk, nk);
        d.st = kt % S;
        return d;
    };
    auto dma_one = [&](const Desc& d, int j) {
        if (j < T::A_DMA)
            dma16(d.a, lds_addr(smA + d.st * T::A_STAGE + (j * NW + wave) * 1024), va + j * ja);
        else if (j < T::A_DMA + T::B_DMA)
            dma16(d.b, lds_addr(smB + d.st * T::B_STAGE + ((j - T::A_DMA) * NW + wave) * 1024),
                  vb + (j - T::A_DMA) * jb);
        else
            dma4(d.s, lds_addr(smS + d.st * T::S_STAGE + wave * 256), vs);
    };
    const bool ragged = K % F8_BLOCK != 0;
    auto fix_tail = [&]() {
        const int valid = K - (nk - 1) * F8_BLOCK, s = (nk - 1) % S;
        for (int r = tid; r < TBM + TBN; r += 64 * NW) {
            char* st = r < TBM ? smA + s * T::A_STAGE : smB + s * T::B_STAGE;
            const int row = r < TBM ? r : r - TBM;
            for (int q = valid >> 4; q < A16_CH; ++q) {
                u32x4* p = (u32x4*)(st + a16_off(row, q));
                *p = mask_bytes(*p, valid - 16 * q);
            }
        }
    };
    // Chunks g and g + 4 of row c of 16 (both operands' k in the same order, which is any); the
    // swizzle has a period of 32 rows.  An LDS read of 16 bytes serves lanes 0-3, 12-15, 20-23, 24-27
    // at once, then the others likewise, from a 256-byte window: with chunks 2 g and 2 g + 1 the
    // two lane groups of such a set met in the same banks.
    int off[2][2];
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int h = 0; h < 2; ++h) off[o][h] = a16_off(16 * o + c, g + 4 * h);
    struct Half { u32x4 w[2]; };
    auto read = [&](const char* st, int strip, int h, Half& f) {  // of the wave's 16-row strips
        f.w[h] = *(const u32x4*)(st + (strip >> 1) * 4096 + off[strip & 1][h]);
    };
    // st: the stage, a constant where it counts, so that it is part of the LDS reads' offsets.
    auto read_a = [&](int st, int mi, int h, Half& f) {
        read(smA + st * T::A_STAGE + wm * (TBM / WM) * 128, mi, h, f);
    };
    auto read_b = [&](int st, int nj, int h, Half& f) {
        read(smB + st * T::B_STAGE + wn * (TBN / WN) * 128, nj, h, f);
    };
    auto sync = [&](auto vm_tag) {
        constexpr int VM = decltype(vm_tag)::value;
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(VM, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    using FirstIn = std::integral_constant<int, T::LOADS>;
    using AllIn = std::integral_constant<int, 0>;

    f32x4 acc[MI][NJ];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int nj = 0; nj < NJ; ++nj) acc[mi][nj] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (nk > 0) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const Desc d = desc(s);
#pragma unroll
            for (int j = 0; j < T::LOADS; ++j) dma_one(d, j);
        }
        sync(FirstIn{});
        if (ragged && nk == 1) { fix_tail(); sync(FirstIn{}); }
        Half fa[2], fb[NJ];
        bf16x8 wa[WIDE ? 4 : 1], wb[WIDE ? NJ : 1][4];
        auto widen = [&](const Half& f, bf16x8* to) {
#pragma unroll
            for (int q = 0; q < 4; ++q) to[q] = widen_f8(f.w[q >> 1][2 * (q & 1)], f.w[q >> 1][2 * (q & 1) + 1]);
        };
        constexpr int NS = NB ? NJ : 1;
        float sa[MI];
        f32x4 sb[NS];
        auto read_sb = [&](int st, int nj) {
            const float* p = (const float*)(smS + st * T::S_STAGE) + TBM + wn * (TBN / WN);
            if constexpr (NB) sb[nj] = *(const f32x4*)(p + nj * 16 + 4 * g);
            else if (nj == 0) sb[0][0] = p[0];
        };
        auto read_sa = [&](int st, int mi) {
            sa[mi] = ((const float*)(smS + st * T::S_STAGE))[TBM / WM * wm + mi * 16 + c];
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) read_a(0, 0, h, fa[0]);
#pragma unroll
        for (int nj = 0; nj < NJ; ++nj) {
#pragma unroll
            for (int h = 0; h < 2; ++h) read_b(0, nj, h, fb[nj]);
            read_sb(0, nj);
        }
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) read_sa(0, mi);
        f32x4 part[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
        float a_prev = 0.0f;
        constexpr int NBLK = MI * NJ;
        // Block i's sums times its scales, added to the running ones.
        auto add = [&](int i) {
            const int mi = i / NJ, nj = i % NJ;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float f = NB ? a_prev * sb[NB ? nj : 0][r] : a_prev;
                acc[mi][nj][r] = __builtin_fmaf(part[i & 1][r], f, acc[mi][nj][r]);
            }
            // Here, in program order: the scheduling barriers order only what has side effects,
            // and the compiler would otherwise leave a step's additions to its end.
            asm volatile("" : "+v"(acc[mi][nj]));
        };
        auto step = [&](int kt, auto stage) {
            constexpr int P = decltype(stage)::value, Q = (P + 1) % S;
            Desc d;
#pragma unroll
            for (int i = 0; i < NBLK; ++i) {
                const int mi = i / NJ, nj = i % NJ;
                if (mi == MI - 1 && nj == 0) {
                    d = desc(kt + S);
                    sync(AllIn{});
                    if (ragged && kt + 2 == nk) { fix_tail(); sync(AllIn{}); }
                }
                if (!NB && nj == 0) sa[mi] *= sb[0][0];
                const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (WIDE) {
                    if (mi == 0) widen(fb[nj], wb[nj]);
                    if (nj == 0) widen(fa[mi & 1], wa);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        part[i & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[nj][q], wa[q], q ? part[i & 1] : zero,
                                                                              0, 0, 0);
                } else {
                    part[i & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        both(fb[nj].w[0], fb[nj].w[1]), both(fa[mi & 1].w[0], fa[mi & 1].w[1]), zero, 0, 0, 0, 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                add(i == 0 ? NBLK - 1 : i - 1);
                a_prev = sa[mi];
                if (nj < 2) {
                    if (mi + 1 < MI) read_a(P, mi + 1, nj, fa[(mi + 1) & 1]);
                    else read_a(Q, 0, nj, fa[MI & 1]);
                }
                if (mi == MI - 1) {
#pragma unroll
                    for (int j = (nj * T::LOADS) / NJ; j < ((nj + 1) * T::LOADS) / NJ; ++j) dma_one(d, j);
#pragma unroll
                    for (int h = 0; h < 2; ++h) read_b(Q, nj, h, fb[nj]);
                    // A's scales of the strips that are done, so that the next step's first factor, a
                    // product with B's, does not wait for them (2 % of 16384 x 4096 x 4096; with a scale
                    // per row of B the factors are formed later, and the step ends with these reads).
                    if (!NB && nj == 1)
#pragma unroll
                        for (int m = 0; m + 1 < MI; ++m) read_sa(Q, m);
                    // B's scales, each after its last use here.
                    if (!NB && nj == 0) read_sb(Q, 0);
                    if (NB && nj > 0) read_sb(Q, nj - 1);
                }
                if (NB && i == 0) read_sb(P, NJ - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int m = NB ? 0 : MI - 1; m < MI; ++m) read_sa(Q, m);
        };
        static_assert(S == 2, "the loop's two steps are the stages");
        for (int kt = 0; kt < nk; kt += 2) {
            step(kt, std::integral_constant<int, 0>{});
            if (kt + 1 < nk) step(kt + 1, std::integral_constant<int, 1>{});
        }
        add(NBLK - 1);
    }
    // No direct-to-LDS write may still be in flight when the LDS is reused.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();  // every wave is done with the operand ring
    store_tile_full<OUT, MI / 2, NJ / 2, true>(acc, a.C, a.M, a.N, a.ldc, m0 + wm * (TBM / WM), n0 + wn * (TBN / WN),
                                            lane, epi, smem + wave * full_lds<NJ / 2>);
}

// ------------------------------------------------------------------ launches

BlockArgs block_args(const GemmLaunch& L, const BlockScales& s) {
    return BlockArgs{L.A, L.B, L.C, L.M, L.N, L.K, L.lda, L.ldb, L.ldc, L.tiles_m, L.tiles_n, s};
}

template <int IN, int OUT, bool NB>
hipError_t go(const GemmLaunch& L, const BlockScales& s) {
    BlockArgs a = block_args(L, s);
    EpiArgs e = L.e;
    int kchunk = L.kchunk;
    int64_t zs = L.c_zstride;
    if (L.slice_waves > 0) {
        const void* fn = nullptr;
        if constexpr (!(IN == IN_F8 && OUT == OUT_F32)) {  // that is a K split's, and slices have none
            if (L.tbm == 32 && L.slice_waves == 8) fn = (const void*)block_slice_kernel<IN, OUT, 1, NB>;
            if (L.tbm == 64 && L.slice_waves == 4) fn = (const void*)block_slice_kernel<IN, OUT, 2, NB>;
        }
        if (!fn || L.tbm != L.tbn || L.splits != 1) return hipErrorInvalidValue;
        void* args[] = {&a, &e};
        return hipLaunchKernel(fn, dim3((unsigned)(L.tiles_m * L.tiles_n)), dim3(64 * L.slice_waves), args, 0,
                               L.stream);
    }
    const void* fn = nullptr;
    int threads = 256;
    if constexpr (IN == IN_F8) {
        if (L.tbm == 256 && L.tbn == 256) {
            fn = (const void*)block_grid_kernel<IN, OUT, 256, 256, 2, 4, NB>;
            threads = 512;
        }
    }
    if (L.tbm == 128 && L.tbn == 128) fn = (const void*)block_grid_kernel<IN, OUT, 128, 128, 2, 2, NB>;
    if (!fn) return hipErrorInvalidValue;
    void* args[] = {&a, &kchunk, &zs, &e};
    return hipLaunchKernel(fn, dim3((unsigned)(L.tiles_m * L.tiles_n), (unsigned)L.splits), dim3(threads), args,
                           0, L.stream);
}

template <int IN, int OUT>
hipError_t by_rows(const GemmLaunch& L, const BlockScales& s) {
    return s.rows_b == 1 ? go<IN, OUT, true>(L, s) : go<IN, OUT, false>(L, s);
}

}  // namespace

hipError_t launch_blockf8(const GemmLaunch& L, const BlockScales& s) {
    if (L.in == IN_F8W && L.out == OUT_F32) return by_rows<IN_F8W, OUT_F32>(L, s);
    if (L.in == IN_F8 && L.out == OUT_F32 && L.splits > 1) return by_rows<IN_F8, OUT_F32>(L, s);
    if (L.in == IN_F8 && L.out == OUT_BF16) return by_rows<IN_F8, OUT_BF16>(L, s);
    if (L.in == IN_F8 && L.out == OUT_F16) return by_rows<IN_F8, OUT_F16>(L, s);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
