// gemmt.hip -- matrix products whose operands are not both stored as A[M x K]
// B[K x N], for gfx950 (MI355X): the two products of a linear layer's backward
// pass, and the product of 8-bit operands.
//
//   NT  C = X Y^T   X: M x K, Y: N x K, both K-contiguous
//                   (dA = dZ B^T over N; 8-bit weights stored per output)
//   TN  C = X^T Y   X: K x M, Y: K x N, both along the output
//                   (dB = A^T dZ over the rows of the batch)
//
// so no transposed copy of an operand is ever written: a copy of each costs two
// passes over it, 13-15 us per 4096^2 operand next to a ~110 us product.  The
// kernel is gemm16.hip's SLAB2 schedule (one barrier per step of 128 bytes of
// K per row, an LDS ring of S stages filled by direct-to-LDS loads, every load
// and LDS read placed between two matrix instructions), with each operand's
// staging chosen by how it lies in memory:
//   K-contiguous: 128-byte row pieces, read with ds_read_b128 (gemm16's A);
//   along the output: 64 k-rows, read with ds_read_b64_tr_b16 (gemm16's B).
//
// 8-bit operands (e4m3) are K-contiguous; a step is 128 k and each
// v_mfma_f32_32x32x64_f8f6f4 takes 32 k per lane, two 16-byte chunks of its
// row: bytes, loads and LDS reads per step are those of the 16-bit NT kernel,
// at half the matrix instructions of twice the length, so one step costs the
// same time and covers twice the k.  (The 8-bit matrix instructions without the
// f8f6f4 form run at the 16-bit rate.)  Matrix instructions' internal k order is
// not observable: both operands' lanes hold the same k.
//
// That instruction aligns neighbouring products before it adds them and drops
// bits below 2^-13 of the largest (measured: 2^16 + 2^2 - 2^16 gives 0 in one
// lane's k).  Against 64 bits that leaves 1.5e-5 of the result's 2-norm for
// normal operands and 5e-5 with outliers, whatever K: far below the rounding of
// a 16-bit output (1.7e-3 bf16, 2e-4 fp16) and far above fp32's.  So 16-bit
// outputs use it, and fp32 outputs (IN_F8W) widen the e4m3 values to bf16 in
// registers, exactly, and take the bf16 instruction, whose sums are fp32.
//
// At 4096^3, one launch of 256 workgroups: 16-bit NT 111 us, TN 113 (1.2 PFLOP/s,
// at the power cap); e4m3 with bias, gelu_tanh and a bf16 C 59-61 us (2.3 PFLOP/s).  Its
// K loop takes 1.37 us a step, the matrix pipe busy 91 % of it at 1.64 GHz (counters of
// 4096 less those of 2048 terms): the pipe and the power cap bound it.  Over the whole
// kernel the pipe is busy 58 %: a single round of workgroups hides neither its launch and
// first loads nor its epilogue, together 42 of 114 thousand cycles.
//
// Edges: rows past the output read zeros or feed unstored outputs; k-rows past K
// fall outside the descriptors and read zeros; K-contiguous rows' bytes past K
// (row padding) are zeroed in LDS for both operands, since 0 * NaN is a NaN.

#include <type_traits>

#include "kern_common.h"
#include "stage16.h"

namespace dgemm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

template <int IN, int LAY, int TBM, int TBN, int S_>
struct TileT {
    static constexpr bool F8 = IN == IN_F8 || IN == IN_F8W;
    static constexpr bool KC = LAY == LAY_NT;            // operands K-contiguous
    static constexpr int ES = F8 ? 1 : 2;
    static constexpr int S = S_;                         // ring stages
    static constexpr int STEPK = 128 / ES;               // k per step
    static constexpr int KP = F8 ? 2 : 4;                // matrix-instruction k groups per step
    static constexpr int NW = 4;
    static constexpr int MI = TBM / 64, NJ = TBN / 64;
    static constexpr int A_STAGE = TBM * 128, B_STAGE = TBN * 128;
    static constexpr int A_DMA = A_STAGE / 1024 / NW, B_DMA = B_STAGE / 1024 / NW;
    static constexpr int LOADS = A_DMA + B_DMA;
    static constexpr int RPF = (F8 || !KC) ? 2 : 1;      // LDS reads per 32-row fragment
    static constexpr int NREAD = RPF * (MI + NJ);        // LDS reads per k group
    // Matrix instructions per k group: IN_F8W takes a 64-k group in four 16-k slices.
    static constexpr int SL = IN == IN_F8W ? 4 : 1;
    static constexpr int NMFMA = MI * NJ * SL;
    static constexpr int LDS = S * (A_STAGE + B_STAGE);
    // The step's schedule (mainloop_t), in slots of one matrix instruction.
    // Half a step each for the reads and the refill: issuing the refill earlier or
    // in a shorter burst was never faster (8-bit 4096^3: 61 us with the loads spread
    // over slots 16-31, 61.1-61.6 over 12-27 and 8-23, 63-65 in bursts of 8).
    static constexpr int BAR = KP * NMFMA / 2;
    static constexpr int LEND = KP * NMFMA;
    static_assert(!F8 || KC, "8-bit operands are K-contiguous");
    static_assert(LDS <= 160 * 1024 && (S - 1) * LOADS <= 63, "LDS budget, vmcnt range");
};

// One operand fragment: 32 rows' (or columns') values of one k group.  16-bit:
// 16 bytes per lane, as one chunk or as two transpose reads; 8-bit: two chunks.
template <bool F8>
struct Frag {
    u32x4 w[F8 ? 2 : 1];
};

// A second pair of operands of the same sizes, whose product is added (the gradient of a gated
// layer's input: dG Bg^T + dU Bu^T); X2 has X's row pitch.  Of the steps of both, one pair's
// after the other's, the loop takes `count` from `first` on.
struct Second {
    const char* X2;
    const char* Y2;
    int ldy2;
    int first, count;
};

// SEG: the K loop runs on over the second pair's k.
template <int IN, int LAY, int TBM, int TBN, int S, bool SEG = false>
__device__ __forceinline__ void mainloop_t(const char* __restrict__ X, const char* __restrict__ Y,
                                           int K, int ldx, int ldy, int m0, int n0, int rows_x,
                                           int rows_y, char* smem,
                                           f32x16 (&acc)[TBM / 64][TBN / 64], const Second& two = Second{}) {
    using T = TileT<IN, LAY, TBM, TBN, S>;
    static_assert(!SEG || LAY == LAY_NT, "a second pair");
    constexpr int MI = T::MI, NJ = T::NJ, ES = T::ES;
    constexpr bool KC = T::KC, F8 = T::F8;
    char* const smA = smem;
    char* const smB = smem + S * T::A_STAGE;
    const int tid = (int)threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nk1 = (K + T::STEPK - 1) / T::STEPK;  // steps of one pair
    const int nk = SEG ? two.count : nk1;
    const int g0 = SEG ? two.first : 0;
    // Whether step kt is the last of a pair (or of the only one).
    auto last = [&](int kt) { return kt + g0 == nk1 - 1 || (SEG && kt + g0 == 2 * nk1 - 1); };

    // Global byte offset of the 16 bytes that belong in this lane's slot of load
    // block `blk` (1 KiB, filled lane-linearly) of an operand with `TB` rows: the
    // swizzle is applied by choosing the source chunk.
    auto voff = [&](int blk, int ld, int tb) {
        if constexpr (KC) {
            const int row = blk * A16_RPB + lane / A16_CH;
            return row * ld * ES + (((lane % A16_CH) ^ a16_phi(row)) << 4);
        } else {
            const int ch = tb / 8, rpb = 512 / tb;  // chunks per k-row, k-rows per block
            const int k = blk * rpb + lane / ch;
            return k * ld * 2 + (((lane % ch) ^ b16_swz(k)) << 4);
        }
    };
    int vx[T::A_DMA], vy[T::B_DMA], vy2[SEG ? T::B_DMA : 1];
#pragma unroll
    for (int j = 0; j < T::A_DMA; ++j) vx[j] = voff(wave * T::A_DMA + j, ldx, TBM);
#pragma unroll
    for (int j = 0; j < T::B_DMA; ++j) {
        vy[j] = voff(wave * T::B_DMA + j, ldy, TBN);
        if constexpr (SEG) vy2[j] = voff(wave * T::B_DMA + j, two.ldy2, TBN);
    }

    // Step kt's two resources; steps past the end get empty ones, whose loads
    // fill zeros and keep the count per step uniform.
    struct Desc { __amdgpu_buffer_rsrc_t a, b; int s; bool second; };
    auto operand = [&](const char* p, int ld, int o0, int rows, int kt) {
        const int k0 = kt * T::STEPK;
        const int krem = (K - k0) < T::STEPK ? (K - k0) : T::STEPK;
        if constexpr (KC)
            return make_rsrc(p + ((int64_t)o0 * ld + k0) * ES,
                             krem > 0 ? ((int64_t)(rows - 1) * ld + krem) * ES : 0);
        else
            return make_rsrc(p + ((int64_t)k0 * ld + o0) * ES,
                             krem > 0 ? ((int64_t)(krem - 1) * ld + rows) * ES : 0);
    };
    auto desc = [&](int kt) {
        if constexpr (SEG) {
            const bool q = kt + g0 >= nk1;
            const int k = kt >= nk ? 2 * nk1 : q ? kt + g0 - nk1 : kt + g0;  // past the run: past K
            return Desc{operand(q ? two.X2 : X, ldx, m0, rows_x, k),
                        operand(q ? two.Y2 : Y, q ? two.ldy2 : ldy, n0, rows_y, k), kt % S, q};
        }
        return Desc{operand(X, ldx, m0, rows_x, kt), operand(Y, ldy, n0, rows_y, kt), kt % S, false};
    };
    auto dma_one = [&](const Desc& d, int j) {
        if (j < T::A_DMA)
            dma16(d.a, lds_addr(smA + d.s * T::A_STAGE + (wave * T::A_DMA + j) * 1024), vx[j]);
        else
            dma16(d.b, lds_addr(smB + d.s * T::B_STAGE + (wave * T::B_DMA + j - T::A_DMA) * 1024),
                  SEG && d.second ? vy2[SEG ? j - T::A_DMA : 0] : vy[j - T::A_DMA]);
    };

    // K-contiguous operands: zero the last step's bytes at and past K in LDS.
    const bool ragged = KC && K % T::STEPK != 0;
    auto fix_row = [&](char* stage, int row, int valid) {  // valid: bytes inside K, 1 .. 127
        const int chunk0 = valid >> 4;
        if (valid & 15) {
            char* p = stage + a16_off(row, chunk0);
            for (int e = valid & 15; e < 16; e += ES) {
                if constexpr (F8) p[e] = 0;
                else *(short*)(p + e) = 0;
            }
        }
        for (int c = chunk0 + ((valid & 15) ? 1 : 0); c < A16_CH; ++c)
            *(u32x4*)(stage + a16_off(row, c)) = u32x4{0u, 0u, 0u, 0u};
    };
    auto fix_tail = [&](int kt) {  // of step kt, the last of a pair
        const int valid = (K - (nk1 - 1) * T::STEPK) * ES, s = kt % S;
        if (tid < TBM) fix_row(smA + s * T::A_STAGE, tid, valid);
        if (tid < TBN) fix_row(smB + s * T::B_STAGE, tid, valid);
    };

    const int wm = wave >> 1, wn = wave & 1;
    const int g = lane >> 5, li = lane & 31;
    const int ta = (lane >> 2) & 3, tq = lane & 3, tg = (lane >> 4) & 1;  // transpose reads

#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int nj = 0; nj < NJ; ++nj)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[mi][nj][r] = 0.0f;

    // Fragment read h (0 .. RPF - 1) of k group kp for the 32 rows from `o` of an
    // operand stage with `tb` rows.
    auto read_frag = [&](const char* st, int tb, int o, int kp, int h, Frag<F8>& f) {
        if constexpr (KC) {
            const int chunk = F8 ? 4 * kp + 2 * g + h : 2 * kp + g;
            f.w[h] = *(const u32x4*)(st + a16_off(o + li, chunk));
        } else {
            const int k = kp * 16 + 8 * g + 4 * h + ta;
            const int c = (o >> 3) + 2 * tg + (tq >> 1);
            const s16x4 p = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4_t*)(st + b16_off(k, c, tb * 2) + (tq & 1) * 8));
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 q = __builtin_bit_cast(u32x2, p);
            f.w[0][2 * h] = q[0];
            f.w[0][2 * h + 1] = q[1];
        }
    };
    // Read o (0 .. NREAD - 1) of k group kp of step kt in the order of first use:
    // A block 0, the B blocks, A blocks 1 ...
    Frag<F8> fa[T::KP][MI], fb[T::KP][NJ];
    auto read_piece = [&](int kt, int kp, int o) {
        const int f = o / T::RPF, h = o % T::RPF;
        if (f == 0 || f > NJ) {
            const int mi = f == 0 ? 0 : f - NJ;
            read_frag(smA + (kt % S) * T::A_STAGE, TBM, wm * (TBM / 2) + mi * 32, kp, h, fa[kp][mi]);
        } else {
            const int nj = f - 1;
            read_frag(smB + (kt % S) * T::B_STAGE, TBN, wn * (TBN / 2) + nj * 32, kp, h, fb[kp][nj]);
        }
    };
    // IN_F8W: the fragments of a 16-k slice as bf16.  While a slice's matrix
    // instructions run, the next slice's fragments are widened, a piece after each,
    // into the other half of the buffer (all at once before the group, the
    // conversions took half as long again as the matrix instructions).
    constexpr bool WIDE = IN == IN_F8W;
    constexpr int NP = MI + NJ;  // fragments per slice
    bf16x8 wide[WIDE ? 2 : 1][WIDE ? NP : 1];
    auto widen = [&](int kp, int q, int f) {
        const u32x4& w = f < MI ? fa[kp][f].w[q >> 1] : fb[kp][f - MI].w[q >> 1];
        wide[q & 1][f] = widen_f8(w[2 * (q & 1)], w[2 * (q & 1) + 1]);
    };
    auto snake = [](int i) { return ((i / NJ) & 1) ? NJ - 1 - i % NJ : i % NJ; };
    auto mfma_one = [&](int kp, int n) {
        constexpr int PER = MI * NJ;
        const int q = n / PER, i = n % PER;  // slice (0 but for IN_F8W), block
        const int mi = i / NJ, nj = snake(i);
        const Frag<F8>&a = fa[kp][mi], &b = fb[kp][nj];
        if constexpr (WIDE) {
            if (n == 0) {
#pragma unroll
                for (int f = 0; f < NP; ++f) widen(kp, 0, f);
            }
            acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide[q & 1][mi], wide[q & 1][MI + nj],
                                                                  acc[mi][nj], 0, 0, 0);
            if (q < 3) {
#pragma unroll
                for (int f = (i * NP) / PER; f < ((i + 1) * NP) / PER; ++f) widen(kp, q + 1, f);
            }
        } else if constexpr (F8) {
            const i32x8 av = __builtin_shufflevector(__builtin_bit_cast(i32x4, a.w[0]),
                                                     __builtin_bit_cast(i32x4, a.w[1]), 0, 1, 2, 3, 4,
                                                     5, 6, 7);
            const i32x8 bv = __builtin_shufflevector(__builtin_bit_cast(i32x4, b.w[0]),
                                                     __builtin_bit_cast(i32x4, b.w[1]), 0, 1, 2, 3, 4,
                                                     5, 6, 7);
            // both operands e4m3 (format code 0), block scales 1 (none applied)
            acc[mi][nj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[mi][nj], 0, 0,
                                                                          0, 0, 0, 0);
        } else if constexpr (IN == IN_BF16) {
            acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, a.w[0]), __builtin_bit_cast(bf16x8, b.w[0]), acc[mi][nj],
                0, 0, 0);
        } else {
            acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                __builtin_bit_cast(f16x8, a.w[0]), __builtin_bit_cast(f16x8, b.w[0]), acc[mi][nj],
                0, 0, 0);
        }
    };
    auto sync = [&](auto vm_tag) {
        constexpr int VM = decltype(vm_tag)::value;
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(VM, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    using FirstIn = std::integral_constant<int, (S - 1) * T::LOADS>;
    using NextIn = std::integral_constant<int, (S - 2) * T::LOADS>;
    constexpr int NR = T::NREAD * (T::KP - 1);       // reads of a step's k groups 1 ..
    constexpr int TOT = T::KP * T::NMFMA;            // matrix instructions per step
    constexpr int BAR = T::BAR, LEND = T::LEND, RBEG = T::NMFMA > BAR ? T::NMFMA : BAR;
    static_assert(BAR <= TOT - T::NMFMA && LEND > BAR && LEND <= TOT, "schedule");

    if (nk > 0) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const Desc d = desc(s);
#pragma unroll
            for (int j = 0; j < T::LOADS; ++j) dma_one(d, j);
        }
        sync(FirstIn{});
        if (ragged && last(0)) { fix_tail(0); sync(FirstIn{}); }
#pragma unroll
        for (int o = 0; o < T::NREAD; ++o) {
            read_piece(0, 0, o);
            __builtin_amdgcn_sched_barrier(0);
        }
        // Step kt, in slots of one matrix instruction: slots 0 .. BAR - 1 carry the
        // reads of its k groups 1 .., each group's before its first use; then the
        // wait for step kt + 1 and the barrier, which retires every wave's reads of
        // the stage; slots BAR .. LEND - 1 carry the stage's refill (step kt + S),
        // and from slot RBEG on, group 0's registers being free, the reads of step
        // kt + 1's group 0.
        for (int kt = 0; kt < nk; ++kt) {
            Desc d;
#pragma unroll
            for (int i = 0; i < TOT; ++i) {
                if (i == BAR) {
                    d = desc(kt + S);
                    sync(NextIn{});
                    if (ragged && kt + 1 < nk && last(kt + 1)) { fix_tail(kt + 1); sync(NextIn{}); }
                }
                mfma_one(i / T::NMFMA, i % T::NMFMA);
                __builtin_amdgcn_sched_barrier(0);
                if (i < BAR) {
#pragma unroll
                    for (int r = (i * NR) / BAR; r < ((i + 1) * NR) / BAR; ++r)
                        read_piece(kt, 1 + r / T::NREAD, r % T::NREAD);
                }
                if (i >= BAR && i < LEND) {
#pragma unroll
                    for (int j = ((i - BAR) * T::LOADS) / (LEND - BAR);
                         j < ((i - BAR + 1) * T::LOADS) / (LEND - BAR); ++j)
                        dma_one(d, j);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (i >= RBEG) {
#pragma unroll
                    for (int r = ((i - RBEG) * T::NREAD) / (TOT - RBEG);
                         r < ((i - RBEG + 1) * T::NREAD) / (TOT - RBEG); ++r)
                        read_piece(kt + 1, 0, r);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // No direct-to-LDS write may still be in flight when the LDS is reused.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
}

// One product's arguments.
struct GridArgs {
    const char* X;
    const char* Y;
    char* C;
    int M, N, K, ldx, ldy, ldc, tiles_m, tiles_n;
};

// Macro-tile `wg` of a product (of one K split of it).
template <int IN, int LAY, int OUT, int TBM, int TBN, int EPI, int S, bool SEG = false>
__device__ __forceinline__ void grid_tile(const GridArgs& a, int wg, const EpiArgs& epi, char* smem,
                                          const Second& two = Second{}) {
    using T = TileT<IN, LAY, TBM, TBN, S>;
    int tm, tn;
    map_tile(wg, a.tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * TBM, n0 = tn * TBN;
    const int rows_x = (a.M - m0) < TBM ? (a.M - m0) : TBM;
    const int rows_y = (a.N - n0) < TBN ? (a.N - n0) : TBN;
    f32x16 acc[T::MI][T::NJ];
    mainloop_t<IN, LAY, TBM, TBN, S, SEG>(a.X, a.Y, a.K, a.ldx, a.ldy, m0, n0, rows_x, rows_y, smem, acc, two);
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int row0 = m0 + (wave >> 1) * (TBM / 2), col0 = n0 + (wave & 1) * (TBN / 2);
    if constexpr (EPI == EPI_FULL) {
        static_assert(4 * full_lds<T::NJ> <= T::LDS, "LDS for the full epilogue");
        __syncthreads();  // every wave is done with the operand ring
        store_tile_full<OUT, T::MI, T::NJ>(acc, a.C, a.M, a.N, a.ldc, row0, col0, lane, epi,
                                           smem + wave * full_lds<T::NJ>);
    } else {
        store_tile<OUT, T::MI, T::NJ, EPI, false>(acc, a.C, a.M, a.N, a.ldc, row0, col0, lane >> 5,
                                                  lane & 31, epi);
    }
}

// One macro-tile per workgroup and K split, as gemm16_kernel.
template <int IN, int LAY, int OUT, int TBM, int TBN, int EPI, int S>
__global__ __launch_bounds__(256) void gemmt_kernel(GridArgs a, int kchunk, int64_t c_zstride,
                                                    EpiArgs epi) {
    using T = TileT<IN, LAY, TBM, TBN, S>;
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
    const int z = (int)blockIdx.y;
    const int kbeg = z * kchunk;
    a.X += (T::KC ? (int64_t)kbeg : (int64_t)kbeg * a.ldx) * T::ES;
    a.Y += (T::KC ? (int64_t)kbeg : (int64_t)kbeg * a.ldy) * T::ES;
    a.C += z * c_zstride;
    a.K = (a.K - kbeg) < kchunk ? (a.K - kbeg) : kchunk;
    grid_tile<IN, LAY, OUT, TBM, TBN, EPI, S>(a, (int)blockIdx.x, epi, smem);
}

// Both products of a backward pass and its column sums in one launch: the CUs that
// one product's last round leaves idle take the other's tiles.  Tiles counted from
// `first` on as in slicet.hip's pair.
template <int IN, int TB>
__global__ __launch_bounds__(256) void gemmt_pair_kernel(GridArgs nt, GridArgs tn, int first,
                                                         ColReduceArgs r) {
    constexpr int OUT = IN == IN_BF16 ? OUT_BF16 : OUT_F16;
    constexpr int L1 = TileT<IN, LAY_NT, TB, TB, 2>::LDS, L2 = TileT<IN, LAY_TN, TB, TB, 2>::LDS;
    __shared__ __attribute__((aligned(1024))) char smem[L1 > L2 ? L1 : L2];
    const int n_nt = nt.tiles_m * nt.tiles_n, n_tn = tn.tiles_m * tn.tiles_n;
    int wg = (int)blockIdx.x;
    if (wg < n_nt + n_tn) {
        wg += first;
        if (wg >= n_nt + n_tn) wg -= n_nt + n_tn;
    }
    EpiArgs e{};
    if (wg < n_nt) grid_tile<IN, LAY_NT, OUT, TB, TB, EPI_FULL, 2>(nt, wg, e, smem);
    else if (wg < n_nt + n_tn) grid_tile<IN, LAY_TN, OUT, TB, TB, EPI_FULL, 2>(tn, wg - n_nt, e, smem);
    else col_reduce(wg - n_nt - n_tn, r, (float*)smem);
}

// Sums in `splits` runs of `per` steps at most (nt) or rows (tn), run z's in fp32 at C + z zstride.
struct Runs {
    int splits, per;
    int64_t zstride;
};

// A gated layer's: dA = X Y^T + X2 Y2^T (nt, in ra's runs), both weights' gradients (tn, tn2, in
// rb's), both biases' column sums.  Any of the products may have no tiles.
template <int IN, int TB>
__global__ __launch_bounds__(256) void gemmt_gated_kernel(GridArgs nt, Second two, Runs ra, GridArgs tn,
                                                          GridArgs tn2, Runs rb, int first,
                                                          ColReduceArgs r, ColReduceArgs r2) {
    constexpr int OUT = IN == IN_BF16 ? OUT_BF16 : OUT_F16;
    constexpr int L1 = TileT<IN, LAY_NT, TB, TB, 2>::LDS, L2 = TileT<IN, LAY_TN, TB, TB, 2>::LDS;
    __shared__ __attribute__((aligned(1024))) char smem[L1 > L2 ? L1 : L2];
    const int tiles = nt.tiles_m * nt.tiles_n;
    const int n_nt = tiles * ra.splits, n_tn = tn.tiles_m * tn.tiles_n * rb.splits;
    const int n_all = n_nt + n_tn + tn2.tiles_m * tn2.tiles_n * rb.splits;
    int wg = (int)blockIdx.x;
    if (wg < n_all) {
        wg += first;
        if (wg >= n_all) wg -= n_all;
    }
    EpiArgs e{};
    if (wg < n_nt) {
        const int z = wg / tiles;
        const int steps = 2 * ((nt.K + TileT<IN, LAY_NT, TB, TB, 2>::STEPK - 1) / TileT<IN, LAY_NT, TB, TB, 2>::STEPK);
        two.first = z * ra.per;
        two.count = steps - two.first < ra.per ? steps - two.first : ra.per;
        if (ra.splits > 1) {
            nt.C += z * ra.zstride;
            grid_tile<IN, LAY_NT, OUT_F32, TB, TB, EPI_NONE, 2, true>(nt, wg - z * tiles, e, smem, two);
        } else {
            grid_tile<IN, LAY_NT, OUT, TB, TB, EPI_FULL, 2, true>(nt, wg, e, smem, two);
        }
    } else if (wg < n_all) {
        const bool b = wg >= n_nt + n_tn;
        GridArgs a = b ? tn2 : tn;
        wg -= n_nt + (b ? n_tn : 0);
        if (rb.splits > 1) {
            const int t = a.tiles_m * a.tiles_n, z = wg / t;
            const int64_t at = (int64_t)z * rb.per;
            a.X += at * a.ldx * TileT<IN, LAY_TN, TB, TB, 2>::ES;
            a.Y += at * a.ldy * TileT<IN, LAY_TN, TB, TB, 2>::ES;
            a.C += z * rb.zstride;
            a.K = a.K - at < rb.per ? (int)(a.K - at) : rb.per;
            grid_tile<IN, LAY_TN, OUT_F32, TB, TB, EPI_NONE, 2>(a, wg - z * t, e, smem);
        } else {
            grid_tile<IN, LAY_TN, OUT, TB, TB, EPI_FULL, 2>(a, wg, e, smem);
        }
    } else {
        const int c = wg - n_all, n1 = r.N > 0 ? (r.N + 15) / 16 : 0;
        col_reduce(c < n1 ? c : c - n1, c < n1 ? r : r2, (float*)smem);
    }
}

GridArgs grid_args(const GemmLaunch& L) {
    return GridArgs{L.A, L.B, L.C, L.M, L.N, L.K, L.lda, L.ldb, L.ldc, L.tiles_m, L.tiles_n};
}

template <int IN>
hipError_t go_pair_t(const GemmLaunch& nt, const GemmLaunch& tn, bool tn_first, const ColReduceArgs& r) {
    const void* fn = nt.tbm == 256 ? (const void*)gemmt_pair_kernel<IN, 256>
                                   : (const void*)gemmt_pair_kernel<IN, 128>;
    GridArgs a = grid_args(nt), b = grid_args(tn);
    int first = tn_first ? nt.tiles_m * nt.tiles_n : 0;
    ColReduceArgs c = r;
    void* args[] = {&a, &b, &first, &c};
    const int blocks =
        nt.tiles_m * nt.tiles_n + tn.tiles_m * tn.tiles_n + (r.N > 0 ? col_reduce_blocks(r.N) : 0);
    return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(256), args, 0, nt.stream);
}

template <int IN>
hipError_t go_gated_t(const GatedBwdLaunch& L) {
    const void* fn = L.nt.tbm == 256 ? (const void*)gemmt_gated_kernel<IN, 256>
                                     : (const void*)gemmt_gated_kernel<IN, 128>;
    GridArgs a = grid_args(L.nt), b = grid_args(L.tn[0]), c = grid_args(L.tn[1]);
    Second two{L.A2, L.B2, L.ldb2, 0, 0};
    Runs ra{L.nt.splits, L.nt.kchunk, L.nt.c_zstride}, rb{L.tn[0].splits, L.tn[0].kchunk, L.tn[0].c_zstride};
    const int tiles = a.tiles_m * a.tiles_n * ra.splits;
    const int tns = (b.tiles_m * b.tiles_n + c.tiles_m * c.tiles_n) * rb.splits;
    int first = L.tn_first ? tiles : 0;
    ColReduceArgs r = L.sums[0], r2 = L.sums[1];
    const int blocks = tiles + tns + (r.N > 0 ? col_reduce_blocks(r.N) : 0) + (r2.N > 0 ? col_reduce_blocks(r2.N) : 0);
    if (blocks == 0) return hipSuccess;
    void* args[] = {&a, &two, &ra, &b, &c, &rb, &first, &r, &r2};
    return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(256), args, 0, L.nt.stream);
}

template <int IN, int LAY, int OUT, int EPI>
hipError_t go_t(const GemmLaunch& L) {
    const void* fn = nullptr;
    if (L.tbm == 256 && L.tbn == 256)
        fn = (const void*)gemmt_kernel<IN, LAY, OUT, 256, 256, EPI, 2>;
    else if (L.tbm == 128 && L.tbn == 128)
        fn = L.stages == 4 ? (const void*)gemmt_kernel<IN, LAY, OUT, 128, 128, EPI, 4>
                           : (const void*)gemmt_kernel<IN, LAY, OUT, 128, 128, EPI, 2>;
    if (!fn) return hipErrorInvalidValue;
    GridArgs a = grid_args(L);
    int kchunk = L.kchunk;
    int64_t zs = L.c_zstride;
    EpiArgs e = L.e;
    void* args[] = {&a, &kchunk, &zs, &e};
    return hipLaunchKernel(fn, dim3((unsigned)(L.tiles_m * L.tiles_n), (unsigned)L.splits), dim3(256),
                           args, 0, L.stream);
}

// A whole product (the full epilogue) or a split's fp32 partials (none).
template <int IN, int LAY>
hipError_t by_out(const GemmLaunch& L) {
    if (L.epi == EPI_NONE && L.out == OUT_F32) return go_t<IN, LAY, OUT_F32, EPI_NONE>(L);
    if (L.epi != EPI_FULL) return hipErrorInvalidValue;
    if constexpr (IN == IN_F8W) {
        if (L.out == OUT_F32) return go_t<IN, LAY, OUT_F32, EPI_FULL>(L);
    } else if constexpr (IN == IN_F8) {
        if (L.out == OUT_BF16) return go_t<IN, LAY, OUT_BF16, EPI_FULL>(L);
        if (L.out == OUT_F16) return go_t<IN, LAY, OUT_F16, EPI_FULL>(L);
    } else {
        constexpr int SAME = IN == IN_BF16 ? OUT_BF16 : OUT_F16;
        if (L.out == SAME) return go_t<IN, LAY, SAME, EPI_FULL>(L);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_gemmt(const GemmLaunch& L) {
    if (L.in == IN_F8 && L.layout == LAY_NT) return by_out<IN_F8, LAY_NT>(L);
    if (L.in == IN_F8W && L.layout == LAY_NT) return by_out<IN_F8W, LAY_NT>(L);
    if (L.in == IN_BF16 && L.layout == LAY_NT) return by_out<IN_BF16, LAY_NT>(L);
    if (L.in == IN_BF16 && L.layout == LAY_TN) return by_out<IN_BF16, LAY_TN>(L);
    if (L.in == IN_F16 && L.layout == LAY_NT) return by_out<IN_F16, LAY_NT>(L);
    if (L.in == IN_F16 && L.layout == LAY_TN) return by_out<IN_F16, LAY_TN>(L);
    return hipErrorInvalidValue;
}

hipError_t launch_gemmt_pair(const GemmLaunch& nt, const GemmLaunch& tn, bool tn_first,
                             const ColReduceArgs& r) {
    for (const GemmLaunch* L : {&nt, &tn})
        if (L->splits != 1 || L->tbm != nt.tbm || L->tbn != nt.tbm || (nt.tbm != 128 && nt.tbm != 256) ||
            L->in != nt.in)
            return hipErrorInvalidValue;
    if (nt.in == IN_BF16) return go_pair_t<IN_BF16>(nt, tn, tn_first, r);
    if (nt.in == IN_F16) return go_pair_t<IN_F16>(nt, tn, tn_first, r);
    return hipErrorInvalidValue;
}

hipError_t launch_gemmt_gated(const GatedBwdLaunch& L) {
    for (const GemmLaunch* p : {&L.nt, &L.tn[0], &L.tn[1]})
        if (p->tbm != L.nt.tbm || p->tbn != L.nt.tbm || (p->tbm != 128 && p->tbm != 256)) return hipErrorInvalidValue;
    if (L.nt.in == IN_BF16) return go_gated_t<IN_BF16>(L);
    if (L.nt.in == IN_F16) return go_gated_t<IN_F16>(L);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
