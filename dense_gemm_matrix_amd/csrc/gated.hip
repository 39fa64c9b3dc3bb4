// gated.hip -- gated projections on gfx950 (MI355X): two products of the same rows and the
// activation of one times the other, in one kernel,
//
//   G = A Bg + bias_g,  U = A Bu + bias_u,  C = act(G) o U      A: M x K, Bg, Bu: K x N
//
// bf16, fp16 and fp32.  As one grid kernel per macro-tile, gemm16.hip's SLAB2 schedule (a ring
// of S stages of 128 bytes of K per row, one barrier per step, every load and LDS read placed
// between two matrix instructions): A is staged and read once for both products, and a
// tile's columns are TBP of G and the same TBP of U, so that a wave holds both values of
// each of its outputs (accumulator blocks 0 .. NJ - 1 are G's, the rest U's) and the
// activation and the product cost no memory traffic.  Compared with two products, A's loads
// and LDS reads are halved, and U is neither written nor read back: bf16 8192 x 8192 x
// 4096, G and U kept for the backward pass, 908 to 950 us (1.16 to 1.21 PFLOP/s, at the power cap).
//
// The two weights are separate matrices (or windows of one; their row pitches may
// differ).  A direct-to-LDS load takes one base for its 64 lanes, so each weight has its
// own half of a stage: k-rows of TBP columns.  With 128 columns of 16 bits a k-row is 256
// bytes, gemm16's layout; with 64 it is 128 and two k-rows share the 256-byte window that a
// transpose read draws its 4 k-rows x 64 bytes from: the second pair of k-rows trades the
// halves of a row.  fp32 (64 columns, 256 bytes): a lane reads its column's value of four k-rows
// one by one, the two lane halves 4 k-rows apart; k-rows with bit 2 set are rotated by
// half a row, so that the halves meet different banks (gemm32.hip's layout).
//
// Edges as in gemm16.hip: rows past M and k-rows past K read zeros, A's bytes past K are
// zeroed in LDS, columns past N feed outputs that are not stored.
//
// With K split over workgroups the tiles write both products' fp32 partial sums to the
// workspace, and gated_reduce_kernel adds them in order and finishes.  Up to 16 rows:
// skinny.hip.

#include <type_traits>

#include "kern_common.h"
#include "stage16.h"

namespace dgemm {
namespace {

// Byte offset of 16-byte chunk `c` of k-row `k` in a weight's half of a stage.
template <int ROW_BYTES, bool F32>
__device__ __forceinline__ int w_off(int k, int c) {
    if constexpr (F32) return k * ROW_BYTES + (((c + ((k >> 2) & 1) * 8) & (ROW_BYTES / 16 - 1)) << 4);
    else if constexpr (ROW_BYTES == 128) return k * 128 + ((c ^ (((k >> 1) & 1) << 2)) << 4);
    else return b16_off(k, c, ROW_BYTES);
}
// Chunk that belongs in slot `s` of k-row `k` (the inverse of w_off).
template <int ROW_BYTES, bool F32>
__device__ __forceinline__ int w_chunk(int k, int s) {
    if constexpr (F32) return (s + ((k >> 2) & 1) * 8) & (ROW_BYTES / 16 - 1);
    else if constexpr (ROW_BYTES == 128) return s ^ (((k >> 1) & 1) << 2);
    else return s ^ b16_swz(k);
}

template <int IN, int TBM, int TBP, int S_>
struct TileG {
    static constexpr bool F32 = IN == IN_F32;
    static constexpr int ES = F32 ? 4 : 2;
    static constexpr int S = S_;                       // ring stages
    static constexpr int STEPK = 128 / ES;             // k per step
    static constexpr int KP = 4;                       // k groups per step: 16 k, or 8 of fp32
    static constexpr int NW = 4;
    static constexpr int MI = TBM / 64, NJ = TBP / 64 * 2;  // a wave's blocks: NJ / 2 of G, NJ / 2 of U
    static constexpr int NJP = NJ / 2;
    static constexpr int ROWB = TBP * ES;              // bytes of a weight's k-row
    static constexpr int A_STAGE = TBM * 128, W_STAGE = STEPK * ROWB;
    static constexpr int A_DMA = A_STAGE / 1024 / NW, W_DMA = 2 * W_STAGE / 1024 / NW;
    static constexpr int LOADS = A_DMA + W_DMA;
    static constexpr int RPB = F32 ? 4 : 2;            // LDS reads per weight fragment
    static constexpr int NREAD = MI + RPB * NJ;        // LDS reads per k group
    static constexpr int SL = F32 ? 4 : 1;             // matrix instructions per block and k group
    static constexpr int NMFMA = MI * NJ * SL;
    static constexpr int LDS = S * (A_STAGE + 2 * W_STAGE);
    static constexpr int BAR = KP * NMFMA / 2, TOT = KP * NMFMA;
    static_assert(LDS <= 160 * 1024 && (S - 1) * LOADS <= 63, "LDS budget, vmcnt range");
    static_assert(NW * full_lds<NJ> <= LDS, "LDS for the epilogue");
    static_assert(W_STAGE % 2048 == 0 && (ROWB == 128 || ROWB == 256) && !(F32 && ROWB != 256), "layout");
};

// One product's arguments; either weight's row pitch is its own.
struct GatedArgs {
    const char* A;
    const char* Bg;
    const char* Bu;
    char* C;
    int M, N, K, lda, ldbg, ldbu, ldc, tiles_m, tiles_n;
};

// acc := the wave's blocks of G and U over k in [0, K).
template <int IN, int TBM, int TBP, int S>
__device__ __forceinline__ void mainloop_g(const GatedArgs& p, int m0, int n0, int rows_a, int cols_b,
                                           char* smem,
                                           f32x16 (&acc)[TBM / 64][TBP / 64 * 2]) {
    using T = TileG<IN, TBM, TBP, S>;
    constexpr int MI = T::MI, NJ = T::NJ, ES = T::ES;
    constexpr bool F32 = T::F32;
    char* const smA = smem;
    char* const smW = smem + S * T::A_STAGE;
    const int K = p.K;
    const int tid = (int)threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nk = (K + T::STEPK - 1) / T::STEPK;

    // Waves 0 and 1 load Bg's k-rows, 2 and 3 Bu's.
    const bool up = wave >= 2;
    const char* const W = up ? p.Bu : p.Bg;
    const int ldw = up ? p.ldbu : p.ldbg;
    int va[T::A_DMA], vw[T::W_DMA];
#pragma unroll
    for (int j = 0; j < T::A_DMA; ++j) {
        const int row = (wave * T::A_DMA + j) * A16_RPB + lane / A16_CH;
        va[j] = row * p.lda * ES + (((lane % A16_CH) ^ a16_phi(row)) << 4);
    }
    constexpr int CH = T::ROWB / 16;  // chunks per k-row
#pragma unroll
    for (int j = 0; j < T::W_DMA; ++j) {
        const int k = ((wave & 1) * T::W_DMA + j) * (64 / CH) + lane / CH;
        vw[j] = k * ldw * ES + (w_chunk<T::ROWB, F32>(k, lane % CH) << 4);
    }
    // Step kt's resources; steps past the end get empty ones, whose loads fill zeros.
    struct Desc { __amdgpu_buffer_rsrc_t a, w; int s; };
    auto desc = [&](int kt) {
        const int k0 = kt * T::STEPK;
        const int krem = (K - k0) < T::STEPK ? (K - k0) : T::STEPK;
        return Desc{make_rsrc(p.A + ((int64_t)m0 * p.lda + k0) * ES,
                              krem > 0 ? ((int64_t)(rows_a - 1) * p.lda + krem) * ES : 0),
                    make_rsrc(W + ((int64_t)k0 * ldw + n0) * ES,
                              krem > 0 ? ((int64_t)(krem - 1) * ldw + cols_b) * ES : 0),
                    kt % S};
    };
    auto dma_one = [&](const Desc& d, int j) {
        if (j < T::A_DMA)
            dma16(d.a, lds_addr(smA + d.s * T::A_STAGE + (wave * T::A_DMA + j) * 1024), va[j]);
        else
            dma16(d.w, lds_addr(smW + (2 * d.s + (up ? 1 : 0)) * T::W_STAGE +
                                ((wave & 1) * T::W_DMA + j - T::A_DMA) * 1024),
                  vw[j - T::A_DMA]);
    };
    // The last step's bytes of A at and past K hold other data: zeroed in LDS.
    const bool ragged = K % T::STEPK != 0;
    auto fix_tail = [&]() {
        const int valid = (K - (nk - 1) * T::STEPK) * ES, s = (nk - 1) % S;
        if (tid < TBM)
            for (int c = valid >> 4; c < A16_CH; ++c) {
                u32x4* q = (u32x4*)(smA + s * T::A_STAGE + a16_off(tid, c));
                *q = mask_bytes(*q, valid - 16 * c);
            }
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

    u32x4 fa[T::KP][MI], fb[T::KP][NJ];
    // Read o (0 .. NREAD - 1) of k group kp of step kt, in the order of first use: A block 0,
    // the weights' blocks, A blocks 1 ..
    auto read_piece = [&](int kt, int kp, int o) {
        if (o == 0 || o > T::RPB * NJ) {
            const int mi = o == 0 ? 0 : o - T::RPB * NJ;
            fa[kp][mi] = *(const u32x4*)(smA + (kt % S) * T::A_STAGE +
                                         a16_off(wm * (TBM / 2) + mi * 32 + li, 2 * kp + g));
            return;
        }
        const int nj = (o - 1) / T::RPB, h = (o - 1) % T::RPB;
        const char* st = smW + (2 * (kt % S) + nj / T::NJP) * T::W_STAGE;
        const int col = wn * (TBP / 2) + (nj % T::NJP) * 32;
        if constexpr (F32) {
            const int k = 8 * kp + 4 * g + h;
            fb[kp][nj][h] = *(const uint32_t*)(st + w_off<T::ROWB, true>(k, (col + li) >> 2) + (li & 3) * 4);
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            const int k = kp * 16 + 8 * g + 4 * h + ta;
            const u32x2 q = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                           (lds_s16x4_t*)(st + w_off<T::ROWB, false>(k, (col >> 3) + 2 * tg + (tq >> 1)) +
                                          (tq & 1) * 8)));
            fb[kp][nj][2 * h] = q[0];
            fb[kp][nj][2 * h + 1] = q[1];
        }
    };
    auto snake = [](int i) { return ((i / NJ) & 1) ? NJ - 1 - i % NJ : i % NJ; };
    auto mfma_one = [&](int kp, int n) {
        constexpr int PER = MI * NJ;
        const int e = n / PER, mi = (n % PER) / NJ, nj = snake(n % PER);
        const u32x4 &a = fa[kp][mi], &b = fb[kp][nj];
        if constexpr (F32)
            acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x2f32(as_float(a[e]), as_float(b[e]), acc[mi][nj], 0, 0, 0);
        else if constexpr (IN == IN_BF16)
            acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc[mi][nj], 0, 0, 0);
        else
            acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                __builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc[mi][nj], 0, 0, 0);
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
    constexpr int NR = T::NREAD * (T::KP - 1);  // reads of a step's k groups 1 ..
    constexpr int BAR = T::BAR, TOT = T::TOT, RBEG = T::NMFMA > BAR ? T::NMFMA : BAR;
    if (nk > 0) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const Desc d = desc(s);
#pragma unroll
            for (int j = 0; j < T::LOADS; ++j) dma_one(d, j);
        }
        sync(FirstIn{});
        if (ragged && nk == 1) { fix_tail(); sync(FirstIn{}); }
#pragma unroll
        for (int o = 0; o < T::NREAD; ++o) {
            read_piece(0, 0, o);
            __builtin_amdgcn_sched_barrier(0);
        }
        // As gemmt.hip's: slots 0 .. BAR - 1 carry the reads of the step's k groups 1 ..; then the
        // wait for step kt + 1 and the barrier that retires the stage; the other slots carry its
        // refill and, group 0's registers being free, the reads of step kt + 1's group 0.
        for (int kt = 0; kt < nk; ++kt) {
            Desc d;
#pragma unroll
            for (int i = 0; i < TOT; ++i) {
                if (i == BAR) {
                    d = desc(kt + S);
                    sync(NextIn{});
                    if (ragged && kt + 2 == nk) { fix_tail(); sync(NextIn{}); }
                }
                mfma_one(i / T::NMFMA, i % T::NMFMA);
                __builtin_amdgcn_sched_barrier(0);
                if (i < BAR) {
#pragma unroll
                    for (int r = (i * NR) / BAR; r < ((i + 1) * NR) / BAR; ++r)
                        read_piece(kt, 1 + r / T::NREAD, r % T::NREAD);
                } else {
#pragma unroll
                    for (int j = ((i - BAR) * T::LOADS) / (TOT - BAR);
                         j < ((i - BAR + 1) * T::LOADS) / (TOT - BAR); ++j)
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

// The epilogue of one wave's MI x 2 NJP blocks (NJP of G, NJP of U), as store_tile_full's: each
// 32-row strip goes through the wave's LDS region and comes back eight consecutive columns
// of G and of U per lane; C, G and U move in 16-byte pieces.  C, G, U: NULL where not wanted.
template <int OUT, int MI, int NJP>
__device__ __forceinline__ void store_gated(const f32x16 (&acc)[MI][2 * NJP], char* C, int M, int N, int ldc,
                                            int row0, int col0, int lane, const GatedEpi& e, char* lds) {
    if (row0 >= M || col0 >= N) return;  // this wave's part of the tile lies outside C
    constexpr int ES = fmt_es<OUT>;
    constexpr int NJ = 2 * NJP, P = full_pitch<NJ>;
    constexpr int LPR = NJP * 4;       // lanes per row
    constexpr int RPI = 64 / LPR;      // rows per pass of the wave
    constexpr int IT = 32 / RPI;       // passes per strip
    const int g = lane >> 5, li = lane & 31;
    const int c8 = (lane % LPR) * 8, r_in = lane / LPR;
    const int nvalid = N - (col0 + c8);
    const bool ragged = (N & 7) != 0 && N - col0 < NJP * 32;  // wave-uniform
    float* const buf = (float*)lds;
    // NULL operands get empty ranges: their stores drop.
    auto rsrc = [&](char* p, int ld) { return p ? c_rsrc(p, M, N, ld, row0, col0, ES) : make_rsrc(nullptr, 0); };
    const __amdgpu_buffer_rsrc_t rc = rsrc(C, ldc), rg = rsrc(e.G, e.ldg), ru = rsrc(e.U, e.ldu);
    float bg[8], bu[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // columns past N: the last one's, which feeds nothing stored
        const int col = col0 + c8 + j < N ? col0 + c8 + j : N - 1;
        bg[j] = e.bias_g ? e.bias_g[col] : 0.0f;
        bu[j] = e.bias_u ? e.bias_u[col] : 0.0f;
    }
    auto at = [&](int r, int ld) { return nvalid > 0 ? (uint32_t)((r * ld + c8) * ES) : OOB_LANE; };
#pragma unroll 1
    for (int mi = 0; mi < MI; ++mi) {
        if (row0 + mi * 32 >= M) break;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int k = 0; k < MI; ++k) {
            if (k != mi) continue;
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    buf[(8 * (r >> 2) + 4 * g + (r & 3)) * P + nj * 32 + li] = acc[k][nj][r];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float vg[IT * 8], vu[IT * 8];
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const float* q = buf + (it * RPI + r_in) * P + c8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 x = *(const f32x4*)(q + 4 * h), y = *(const f32x4*)(q + NJP * 32 + 4 * h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    vg[it * 8 + 4 * h + j] = x[j] + bg[4 * h + j];
                    vu[it * 8 + 4 * h + j] = y[j] + bu[4 * h + j];
                }
            }
        }
        auto put = [&](__amdgpu_buffer_rsrc_t r, int ld, const float (&v)[IT * 8]) {
            Row8<OUT> o;
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = v[it * 8 + j];
                o.set(x);
                if (!ragged) o.store_whole(r, at(mi * 32 + it * RPI + r_in, ld));
                else o.store(r, at(mi * 32 + it * RPI + r_in, ld), nvalid);
            }
        };
        if (e.G) put(rg, e.ldg, vg);
        if (e.U) put(ru, e.ldu, vu);
        if (!C) continue;
        apply_act<OUT>(vg, e.act);
#pragma unroll
        for (int i = 0; i < IT * 8; ++i) vg[i] *= vu[i];
        put(rc, ldc, vg);
    }
}

template <int IN, int OUT, int TBM, int TBP, int S>
__global__ __launch_bounds__(256) void gated_kernel(GatedArgs a, int kchunk, int64_t zstride, GatedEpi e) {
    using T = TileG<IN, TBM, TBP, S>;
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
    {
        const int z = (int)blockIdx.y;
        const int kbeg = z * kchunk;
        a.A += (int64_t)kbeg * T::ES;
        a.Bg += (int64_t)kbeg * a.ldbg * T::ES;
        a.Bu += (int64_t)kbeg * a.ldbu * T::ES;
        if (e.G) e.G += z * zstride;
        if (e.U) e.U += z * zstride;
        a.K = (a.K - kbeg) < kchunk ? (a.K - kbeg) : kchunk;
    }
    int tm, tn;
    map_tile((int)blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * TBM, n0 = tn * TBP;
    const int rows_a = (a.M - m0) < TBM ? (a.M - m0) : TBM;
    const int cols_b = (a.N - n0) < TBP ? (a.N - n0) : TBP;
    f32x16 acc[T::MI][T::NJ];
    mainloop_g<IN, TBM, TBP, S>(a, m0, n0, rows_a, cols_b, smem, acc);
    __syncthreads();  // every wave is done with the operand ring
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    store_gated<OUT, T::MI, T::NJP>(acc, a.C, a.M, a.N, a.ldc, m0 + (wave >> 1) * (TBM / 2),
                                    n0 + (wave & 1) * (TBP / 2), lane, e, smem + wave * full_lds<T::NJ>);
}

// ------------------------------------------------------------------ small outputs
//
// As slicet.hip: a workgroup of four waves owns 32 MI rows of 32 columns of G and U, each wave
// takes an equal run of 128-byte K blocks (64 k, fp32 32) into its own LDS stages and holds the
// whole tile's sums for its k; the four are added in LDS in wave order.  A's rows lie in LDS
// K-contiguous (gemm16's swizzle), the weights' k-rows as in memory, read through the transpose
// read or, fp32, one value at a time (the two lane halves 4 k-rows apart meet in the same banks,
// which costs less than the matrix instructions they feed).  512^3 with nothing kept: fp32 8.0 us
// where split grid tiles take 20, bf16 4.2 where unsplit ones take 8.5.
template <int MI>
struct SliceG {
    static constexpr int W = 4;
    static constexpr int A_BLK = 128 * 32 * MI, W_BLK = 128 * 32;  // bytes of a block of A, of a weight
    static constexpr int STAGE = A_BLK + 2 * W_BLK;
    static constexpr int NA = A_BLK / 1024, NW = W_BLK / 1024;     // direct-to-LDS loads
    static constexpr int RED = W * MI * 2 * 16 * 64 * 4;
    static constexpr int LDS = 2 * W * STAGE > RED ? 2 * W * STAGE : RED;
};

template <int IN, int OUT, int MI>
__global__ __launch_bounds__(256) void gated_slice_kernel(GatedArgs a, GatedEpi e) {
    using T = SliceG<MI>;
    constexpr int W = T::W, ES = IN == IN_F32 ? 4 : 2, BK = 128 / ES, RB = 32 * ES;
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
    int tm, tn;
    map_tile((int)blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 5, li = lane & 31;
    const int m0 = tm * 32 * MI, n0 = tn * 32;
    const int rows_a = (a.M - m0) < 32 * MI ? (a.M - m0) : 32 * MI;
    const int cols = (a.N - n0) < 32 ? (a.N - n0) : 32;
    const int nblk = (a.K + BK - 1) / BK;
    const int kb0 = (int)((int64_t)wave * nblk / W);
    const int nb = (int)((int64_t)(wave + 1) * nblk / W) - kb0;

    f32x16 acc[2][MI];  // G's blocks, U's
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[u][mi][r] = 0.0f;

    char* const mine = smem + wave * 2 * T::STAGE;
    int va[T::NA], vw[2][T::NW];
#pragma unroll
    for (int j = 0; j < T::NA; ++j) {
        const int row = A16_RPB * j + lane / A16_CH;
        va[j] = row * a.lda * ES + (((lane % A16_CH) ^ a16_phi(row)) << 4);
    }
#pragma unroll
    for (int j = 0; j < T::NW; ++j) {
        const int q = 1024 * j + 16 * lane;  // k-row q / RB, byte q % RB of the row
        vw[0][j] = (q / RB) * a.ldbg * ES + q % RB;
        vw[1][j] = (q / RB) * a.ldbu * ES + q % RB;
    }
    auto load = [&](int i, int s) {
        const int k0 = (kb0 + i) * BK;
        const int krem = (a.K - k0) < BK ? (a.K - k0) : BK;
        char* st = mine + s * T::STAGE;
        const auto ra = make_rsrc(a.A + ((int64_t)m0 * a.lda + k0) * ES, ((int64_t)(rows_a - 1) * a.lda + krem) * ES);
#pragma unroll
        for (int j = 0; j < T::NA; ++j) dma16(ra, lds_addr(st + 1024 * j), va[j]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int ld = u ? a.ldbu : a.ldbg;
            const auto rw = make_rsrc((u ? a.Bu : a.Bg) + ((int64_t)k0 * ld + n0) * ES,
                                      ((int64_t)(krem - 1) * ld + cols) * ES);
#pragma unroll
            for (int j = 0; j < T::NW; ++j) dma16(rw, lds_addr(st + T::A_BLK + u * T::W_BLK + 1024 * j), vw[u][j]);
        }
    };
    // The transpose read's slot, as in slicet.hip.
    const int grp = lane >> 4;
    const int slot = ((8 * (grp >> 1) + ((lane >> 2) & 3)) * 32 + 16 * (grp & 1) + 4 * (lane & 3)) * 2;
    run_steps<1>(nb, load, [&](int i, int s, auto newer) {
        // This step's loads have landed; at most the newer step's are in flight.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(decltype(newer)::value * (T::NA + 2 * T::NW), 15));
        __builtin_amdgcn_sched_barrier(0);
        const char* st = mine + s * T::STAGE;
        u32x4 fa[MI][4], fw[2][4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int mi = 0; mi < MI; ++mi) fa[mi][h] = *(const u32x4*)(st + a16_off(mi * 32 + li, 2 * h + g));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const char* w = st + T::A_BLK + u * T::W_BLK;
                if constexpr (IN == IN_F32) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        fw[u][h][q] = *(const uint32_t*)(w + ((8 * h + 4 * g + q) * 32 + li) * 4);
                } else {
                    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const u32x2 p = __builtin_bit_cast(
                            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (lds_s16x4_t*)(w + slot + (16 * h + 4 * t) * 64)));
                        fw[u][h][2 * t] = p[0];
                        fw[u][h][2 * t + 1] = p[1];
                    }
                }
            }
        }
        // The reads are done before the slot's next loads are issued.
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        __builtin_amdgcn_sched_barrier(0);
        const int k0 = (kb0 + i) * BK;
        if (k0 + BK > a.K) {  // A's row padding (k-rows past K read zeros)
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int mi = 0; mi < MI; ++mi)
                    fa[mi][h] = mask_bytes(fa[mi][h], (a.K - k0) * ES - 16 * (2 * h + g));
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    if constexpr (IN == IN_F32) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[u][mi] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                as_float(fa[mi][h][q]), as_float(fw[u][h][q]), acc[u][mi], 0, 0, 0);
                    } else if constexpr (IN == IN_BF16) {
                        acc[u][mi] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            __builtin_bit_cast(bf16x8, fa[mi][h]), __builtin_bit_cast(bf16x8, fw[u][h]), acc[u][mi],
                            0, 0, 0);
                    } else {
                        acc[u][mi] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                            __builtin_bit_cast(f16x8, fa[mi][h]), __builtin_bit_cast(f16x8, fw[u][h]), acc[u][mi],
                            0, 0, 0);
                    }
                }
    });
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();  // every wave is done with its stages: the sums reuse them

    // Value idx = 16 mi + r of either product, wave w finishing idx in [w PER, w PER + PER).
    float* const red = (float*)smem;
    constexpr int NV = MI * 16, PER = NV / W;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i) red[((wave * 2 + u) * NV + i) * 64 + lane] = acc[u][i / 16][i % 16];
    __syncthreads();
    float v[2][PER];
    const int col = n0 + li;
    const bool in_n = col < a.N;
    const float bias[2] = {e.bias_g && in_n ? e.bias_g[col] : 0.0f, e.bias_u && in_n ? e.bias_u[col] : 0.0f};
    int row[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int idx = wave * PER + q;
        row[q] = m0 + (idx / 16) * 32 + 8 * ((idx % 16) >> 2) + 4 * g + (idx & 3);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float s = red[(u * NV + idx) * 64 + lane];
#pragma unroll
            for (int w = 1; w < W; ++w) s += red[((w * 2 + u) * NV + idx) * 64 + lane];
            v[u][q] = s + bias[u];
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        char* const to = u ? e.U : e.G;
        if (!to) continue;
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (in_n && row[q] < a.M) store_c<OUT>(to, (int64_t)row[q] * (u ? e.ldu : e.ldg) + col, v[u][q]);
    }
    apply_act<OUT>(v[0], e.act);
#pragma unroll
    for (int q = 0; q < PER; ++q)
        if (in_n && row[q] < a.M) store_c<OUT>(a.C, (int64_t)row[q] * a.ldc + col, v[0][q] * v[1][q]);
}

// Sums the splits' partial products in ascending order and finishes: four columns of one row
// per thread.  W[z]: M x 2 ldw, G's columns from 0 and U's from ldw.
template <int OUT>
__global__ __launch_bounds__(256) void gated_reduce_kernel(const float* __restrict__ W, int splits, int64_t zstride,
                                                           int ldw, char* __restrict__ C, int ldc, int M, int N,
                                                           GatedEpi e) {
    const int nq = ldw >> 2;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= (int64_t)M * nq) return;
    const int row = (int)(t / nq);
    const int col0 = (int)(t - (int64_t)row * nq) * 4;
    const float* p = W + (int64_t)row * 2 * ldw + col0;
    f32x4 g = *(const f32x4*)p, u = *(const f32x4*)(p + ldw);
#pragma unroll 4
    for (int z = 1; z < splits; ++z) {
        g += *(const f32x4*)(p + z * zstride);
        u += *(const f32x4*)(p + z * zstride + ldw);
    }
    float vg[4], vu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = col0 + j < N ? col0 + j : N - 1;
        vg[j] = g[j] + (e.bias_g ? e.bias_g[col] : 0.0f);
        vu[j] = u[j] + (e.bias_u ? e.bias_u[col] : 0.0f);
    }
    auto put = [&](char* to, int ld, const float (&v)[4]) {
        constexpr int ES = fmt_es<OUT>;
        char* const q = to + ((int64_t)row * ld + col0) * ES;
        if (col0 + 4 <= N) {  // an aligned 16- or 8-byte piece
            if constexpr (OUT == OUT_F32) {
                *(f32x4*)q = f32x4{v[0], v[1], v[2], v[3]};
            } else {
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                *(u32x2*)q = u32x2{pack16<OUT>(v[0], v[1]), pack16<OUT>(v[2], v[3])};
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col0 + j < N) store_c<OUT>(q, j, v[j]);
        }
    };
    if (e.G) put(e.G, e.ldg, vg);
    if (e.U) put(e.U, e.ldu, vu);
    apply_act<OUT>(vg, e.act);
#pragma unroll
    for (int j = 0; j < 4; ++j) vg[j] *= vu[j];
    put(C, ldc, vg);
}

// ------------------------------------------------------------------ launches

template <int IN, int OUT>
hipError_t go_gated(const GatedLaunch& L) {
    const void* fn = nullptr;
    if constexpr (IN != IN_F32) {
        if (L.tbm == 256 && L.tbp == 128) fn = (const void*)gated_kernel<IN, OUT, 256, 128, 2>;
    }
    if (L.tbm == 128 && L.tbp == 64)
        fn = L.stages == 4 ? (const void*)gated_kernel<IN, OUT, 128, 64, 4>
                           : (const void*)gated_kernel<IN, OUT, 128, 64, 2>;
    if (L.waves == 4 && L.tbp == 32)
        fn = L.tbm == 32   ? (const void*)gated_slice_kernel<IN, OUT, 1>
             : L.tbm == 64 ? (const void*)gated_slice_kernel<IN, OUT, 2>
                           : nullptr;
    if (!fn) return hipErrorInvalidValue;
    GatedArgs a{L.A, L.Bg, L.Bu, L.C, L.M, L.N, L.K, L.lda, L.ldbg, L.ldbu, L.ldc, L.tiles_m, L.tiles_n};
    if (L.waves > 0) {
        if (L.splits != 1 || !L.C) return hipErrorInvalidValue;
        GatedEpi e = L.e;
        void* args[] = {&a, &e};
        return hipLaunchKernel(fn, dim3((unsigned)(L.tiles_m * L.tiles_n)), dim3(256), args, 0, L.stream);
    }
    int kchunk = L.kchunk;
    int64_t zs = L.zstride;
    GatedEpi e = L.e;
    void* args[] = {&a, &kchunk, &zs, &e};
    return hipLaunchKernel(fn, dim3((unsigned)(L.tiles_m * L.tiles_n), (unsigned)L.splits), dim3(256), args, 0,
                           L.stream);
}

template <int OUT>
hipError_t go_reduce(const float* W, int splits, int64_t zstride, int ldw, char* C, int ldc, int M, int N,
                     const GatedEpi& epi, hipStream_t stream) {
    const int64_t blocks = ((int64_t)M * (ldw / 4) + 255) / 256;
    if (blocks <= 0) return hipSuccess;
    if (blocks >= (int64_t)1 << 23) return hipErrorInvalidValue;
    GatedEpi e = epi;
    void* args[] = {&W, &splits, &zstride, &ldw, &C, &ldc, &M, &N, &e};
    return hipLaunchKernel((const void*)gated_reduce_kernel<OUT>, dim3((unsigned)blocks), dim3(256), args, 0, stream);
}

}  // namespace

hipError_t launch_gated(const GatedLaunch& L) {
    if (L.in == IN_F32 && L.out == OUT_F32) return go_gated<IN_F32, OUT_F32>(L);
    if (L.in == IN_BF16 && L.out == OUT_BF16) return go_gated<IN_BF16, OUT_BF16>(L);
    if (L.in == IN_BF16 && L.out == OUT_F32) return go_gated<IN_BF16, OUT_F32>(L);
    if (L.in == IN_F16 && L.out == OUT_F16) return go_gated<IN_F16, OUT_F16>(L);
    if (L.in == IN_F16 && L.out == OUT_F32) return go_gated<IN_F16, OUT_F32>(L);
    return hipErrorInvalidValue;
}

hipError_t launch_gated_reduce(const float* W, int splits, int64_t zstride, int ldw, char* C, int ldc, int M, int N,
                               int out, const GatedEpi& e, hipStream_t stream) {
    if (ldw % 4 != 0 || splits < 1) return hipErrorInvalidValue;
    if (out == OUT_F32) return go_reduce<OUT_F32>(W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    if (out == OUT_BF16) return go_reduce<OUT_BF16>(W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    if (out == OUT_F16) return go_reduce<OUT_F16>(W, splits, zstride, ldw, C, ldc, M, N, e, stream);
    return hipErrorInvalidValue;
}

}  // namespace dgemm
