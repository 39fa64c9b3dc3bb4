// feedforward.hip -- the C ABI of a feed-forward block's operators beside linear.hip's: gated
// projections and their gradients (gemm_gated, gemm_gated_bwd), layer norms and theirs
// (layernorm, layernorm_bwd), products of 8-bit operands with a scale per block and the
// quantizer of those (gemm_f8_block, quant_f8_block).  Host code only: validation, plans and
// launches.

#include <algorithm>

#include "host.h"

namespace dgemm {
namespace {

// A matrix of block scales: value (i, b) at p[i * s_row + b * s_blk].
struct Scales {
    const float* p;
    int64_t rows, blocks, s_row, s_blk;
    int64_t extent() const { return rows > 0 && blocks > 0 ? (rows - 1) * s_row + (blocks - 1) * s_blk + 1 : 0; }
    Mat mat() const { return vec(p, extent()); }  // first to last value
};

// Strides, pointer and alignment; an output's values are apart from each other.
int check_scales(const Scales& s, bool output) {
    if (s.s_row < 0 || s.s_blk < 0) return DGEMM_ERR_LEADING_DIM;
    if (s.extent() == 0) return DGEMM_OK;
    if (!s.p) return DGEMM_ERR_INVALID_VALUE;
    if (check_vec(s.p, 4) != DGEMM_OK) return DGEMM_ERR_MISALIGNED;
    const bool by_row = (s.blocks == 1 || s.s_blk > 0) && (s.rows == 1 || s.s_row > (s.blocks - 1) * s.s_blk);
    const bool by_blk = (s.rows == 1 || s.s_row > 0) && (s.blocks == 1 || s.s_blk > (s.rows - 1) * s.s_row);
    if (output && !by_row && !by_blk) return DGEMM_ERR_LEADING_DIM;
    if (PANEL_ROWS * s.s_row * 4 >= DESC_LIMIT) return DGEMM_ERR_TOO_LARGE;
    return DGEMM_OK;
}

// Launch, first loads and last stores, which the grid kernels' estimate leaves out.
constexpr double GRID_US = 2.5;

// fp32 outputs and few rows: the widened products, whose sums are fp32.
int block_in(int of, int M) { return of == OUT_F32 || M <= SKINNY_M ? IN_F8W : IN_F8; }

// The tiles of blockf8.hip, in the terms of the other 8-bit products (the scaled additions cost some
// of the rate, and an underfilled chip does not run the small one faster); `each`: a scale per
// row of B.
TileCand block_tile(int i, bool each) {
    const double f = each ? 0.89 : 1.0;
    return i == 0 ? TileCand{256, 256, 0.87 * f, 0.0, 0.0, 0.87 * f, 0.6}
                  : TileCand{128, 128, 0.55 * f, 1.26, 1.35, 0.6 * f, 1.0};
}

// Tiles whose waves split K (32 x 32 with 8 waves, 64 x 64 with 4) by the time of a round of 256,
// grid tiles and K splits by the common estimate.  us, slices of 32 / of 64 / best grid plan:
// bf16 C, 64 x 4096 x 4096 5.8 / 12.0 / 14.5, 17 x 8192 x 1024 3.6 / 6.3 / 8.5, 300 x 1000 x 2000 8.5 /
// 9.4 / 13.3, 1000^3 13.1 / 9.2 / 10.2, 512 x 4096 x 4096 38.5 / 25.1 / 25.3, 700 x 5000 x 3000 67.7 / 45.1 /
// 26.6; fp32 C, 700 x 5000 x 3000 71 / 55 / 35.  bm = 0: none fits.
Plan plan_block(int of, int rows_b, int M, int N, int K, uint64_t ws) {
    const int in = block_in(of, M);
    if (M > 0 && M <= SKINNY_M && N > 0) return plan_skinny(in, LAY_NT, M, N, K, 0);
    const int nk = (int)ceil_div(std::max(K, 1), F8_BLOCK);
    const bool each = rows_b == 1;
    auto slices = [&](int t) {
        Plan p{t, t, 1, K, 0, 0};
        p.waves = t == 32 ? 8 : 4;
        return p;
    };
    const int tiles = in == IN_F8 ? 2 : 1;  // fp32 C: the small one
    int fm, fn, fs;
    if (forced_grid(fm, fn, fs) && fm == fn) {
        if (fm == 32 || fm == 64) return slices(fm);
        for (int i = 2 - tiles; i < 2; ++i)
            if (block_tile(i, each).bm == fm) {
                const Plan p = plan_pieces(block_tile(i, each), F8_BLOCK, M, N, K, fs, ws);
                if (p.splits > 0) return p;
            }
    }
    Plan best{};
    double best_us = -1.0;
    for (int t = 32; t <= 64; t += 32) {
        const int64_t n = ceil_div(M, t) * ceil_div(N, t);
        if (n > INT32_MAX) continue;
        const double wide = in == IN_F8 ? 1.0 : t == 32 ? 1.12 : 1.3;  // fp32 C, by the widened products
        const double round =
            (t == 32 ? 2.3 + 0.55 * (double)ceil_div(nk, 8) : 4.5 + 0.85 * (double)ceil_div(nk, 4)) * wide;
        const double us = 1.1 + (double)ceil_div(n, NUM_CU) * round;
        if (best_us < 0.0 || us < best_us) {
            best_us = us;
            best = slices(t);
        }
    }
    for (int s = 1; s <= MAX_SPLITS && s <= nk; ++s)
        for (int i = 2 - tiles; i < 2; ++i) {
            const TileCand t = block_tile(i, each);
            const Plan p = plan_pieces(t, F8_BLOCK, M, N, K, s, ws);
            if (p.splits != s) continue;
            const double us = estimate_us(in, out_esize(of), M, N, t, s, s == 1 ? nk : p.kchunk / F8_BLOCK, p.ldw) /
                                  (s > 1 ? SPLIT_MARGIN : 1.0) + GRID_US;
            if (best_us < 0.0 || us < best_us) {
                best_us = us;
                best = p;
            }
        }
    return best;
}

int run_block(int of, int M, int N, int K, const void* A, int lda, const void* B, int ldb, void* C, int ldc,
              const BlockScales& s, const EpiArgs& e, const Plan& p, void* ws, hipStream_t stream) {
    GemmLaunch L{};
    L.in = block_in(of, M);
    L.out = of;
    L.layout = LAY_NT;
    L.tbm = p.bm;
    L.tbn = p.bn;
    L.slice_waves = p.waves;
    L.splits = p.splits;
    L.kchunk = p.splits > 1 ? p.kchunk : std::max(K, 1);
    L.epi = EPI_FULL;
    L.A = (const char*)A;
    L.B = (const char*)B;
    L.C = (char*)C;
    L.M = M;
    L.N = N;
    L.K = K;
    L.lda = lda;
    L.ldb = ldb;
    L.ldc = ldc;
    L.tiles_m = (int)ceil_div(M, p.bm);
    L.tiles_n = (int)ceil_div(N, p.bn);
    L.e = e;
    L.stream = stream;
    if ((int64_t)L.tiles_m * L.tiles_n > INT32_MAX) return DGEMM_ERR_TOO_LARGE;
    if (p.kind == PLAN_SKINNY) return launched(launch_blockf8_skinny(L, s));
    if (p.splits == 1) return launched(launch_blockf8(L, s));
    L.out = OUT_F32;
    L.C = (char*)ws;
    L.ldc = p.ldw;
    L.c_zstride = (int64_t)M * p.ldw * 4;
    L.e = EpiArgs{};
    L.e.alpha = 1.0f;
    if (launch_blockf8(L, s) != hipSuccess) return DGEMM_ERR_LAUNCH;
    return launched(launch_splitk_reduce((const float*)ws, p.splits, (int64_t)M * p.ldw, p.ldw, (char*)C, ldc, M,
                                         N, of, EPI_FULL, e, stream));
}

// ------------------------------------------------------------- gated projections

// Tiles of gated.hip, their columns of G and U counted together: the estimates of the grid
// kernels with the same accumulators and steps.
constexpr TileCand TILES_G16[] = {{256, 256, 1.0, 0.0, 0.0, 1.0, 0.6}, {128, 128, 0.6, 1.26, 1.35, 0.8, 1.0}};
constexpr TileCand TILES_G32[] = {{128, 128, 0.85, 1.5, 1.5, 0.85, 1.0}};

struct GatedPlan {
    int bm, bn;     // bn: columns of G (and of U)
    int splits, kchunk, ldw, waves;
    int64_t ws_bytes;
    bool skinny;
};

// A plan at `splits` K pieces of whole steps of bk; splits = 0 if it does not fit.
GatedPlan gated_pieces(int bm, int bn, int bk, int M, int N, int K, int splits, uint64_t ws) {
    const Plan q = plan_pieces(TileCand{bm, bn, 1, 0, 0, 1, 1}, bk, M, N, K, splits, UINT64_MAX);
    GatedPlan p{bm, bn, q.splits, q.kchunk, q.ldw, 0, 2 * q.ws_bytes, false};
    if (p.splits > 1 && ((uint64_t)p.ws_bytes > ws || (int64_t)PANEL_ROWS * 2 * p.ldw * 4 >= DESC_LIMIT)) p.splits = 0;
    return p;
}

// At most SKINNY_M rows: as plan_skinny's strips of B stored along the output, of both weights,
// but never of 128 columns (two weights' loads are as wide as one's twice: 1 x 14336 x 4096 bf16, weights
// from the last-level cache, 32 / 64 / 128 columns 43.8 / 37.4 / 38.4 us), and split from the same K on
// in fp32.  From HBM, us, the fastest unsplit / this rule's plan (pieces):
//            bf16                  fp32
//    1 x  1024 x  1024    7.2 /  7.3 (1)     9.3 /  9.5 (1)
//    1 x   512 x  8192   54.9 / 12.7 (16)   66.2 / 16.4 (16)
//    1 x  1024 x  4096   30.0 / 11.3 (15)   34.4 / 14.9 (15)
//    1 x  4096 x  4096   32.8 / 19.5 (4)    38.0 / 32.7 (4)
//   16 x  4096 x  4096   35.4 / 20.7 (4)    42.2 / 33.9 (4)
//    1 x  4096 x 11008   79.9 / 39.3 (4)    96.9 / 72.0 (4)
//    1 x  8192 x  2048   21.0 / 21.7 (1)    25.8 / 25.9 (1)   (two pieces 19.0, 29.7)
//    1 x 11008 x  4096   37.5 / 37.6 (1)    73.3 / 73.6 (1)   (four pieces 38.6, 70.7)
//    1 x 14336 x  4096   47.3 / 47.9 (1)    86.0 / 85.8 (1)   (two pieces 51.5, 88.9)
GatedPlan plan_gated_skinny(int in, int M, int N, int K, uint64_t ws) {
    auto strips = [&](int cols, int waves, int splits) {  // splits = 0 if it does not fit
        GatedPlan p = gated_pieces(SKINNY_M, cols, 32, M, N, K, splits, UINT64_MAX);
        if (p.splits > 1 && p.kchunk % 64 == 0) {  // an odd number of steps, as plan_skinny's
            p.kchunk += 32;
            p.splits = (int)ceil_div(K, p.kchunk);
            p.ws_bytes = p.splits > 1 ? (int64_t)p.splits * M * 2 * p.ldw * 4 : 0;
        }
        if ((uint64_t)p.ws_bytes > ws) p.splits = 0;  // what the pieces need once they are final
        p.waves = waves;
        p.skinny = true;
        return p;
    };
    int fm, fn, fs;
    if (forced_grid(fm, fn, fs) && fm == SKINNY_M && (fn == 32 || fn == 64)) {
        const GatedPlan p = strips(fn, fn == 32 ? 16 : 8, fs);
        if (p.splits > 0) return p;
    }
    if (K >= 2048 && 2 * (int64_t)N <= 5 * (int64_t)K) {
        const int s = (int)std::min<int64_t>(std::min(MAX_SPLITS, K / 256), NUM_CU / ceil_div(N, 64));
        if (s >= 2) {
            const GatedPlan p = strips(64, 8, s);
            if (p.splits > 1) return p;
        }
    }
    return ceil_div(N, 32) > NUM_CU ? strips(64, 8, 1) : strips(32, 16, 1);
}

// bm = 0: none fits.
GatedPlan plan_gated(int in, int es_out, int M, int N, int K, uint64_t ws) {
    if (M > 0 && M <= SKINNY_M && N > 0) return plan_gated_skinny(in, M, N, K, ws);
    const TileCand* tiles = in == IN_F32 ? TILES_G32 : TILES_G16;
    const int n = in == IN_F32 ? 1 : 2, bk = in == IN_F32 ? 32 : 64;
    const int nk = (int)ceil_div(std::max(K, 1), bk);
    int fm, fn, fs;
    auto slices = [&](int bm) { return GatedPlan{bm, 32, 1, K, 0, 4, 0, false}; };
    if (forced_grid(fm, fn, fs) && fn == fm && (fm == 32 || fm == 64)) return slices(fm);
    if (forced_grid(fm, fn, fs))
        for (int i = 0; i < n; ++i)
            if (tiles[i].bm == fm && tiles[i].bn == fn) {
                const GatedPlan p = gated_pieces(fm, fn / 2, bk, M, N, K, fs, ws);
                if (p.splits > 0) return p;
            }
    GatedPlan best{};
    double best_us = -1.0;
    // Small outputs: a round of 256 tiles whose waves split K, by its blocks of 128 bytes per wave,
    // against the grid tiles.  Measured (us; 32 x 32 / 64 x 32 slices / best grid plan with a
    // workspace): bf16 512^3 4.2 / 5.3 / 8.5, 64 x 2048 x 1024 5.0 / 6.5 / 11.4, 512 x 1024 x 512
    // 7.1 / 5.4 / 8.6, 1024^3 20.9 / 12.5 / 12.0, 300 x 600 x 8192 35.0 / 37.5 / 22.9; fp32 512^3
    // 8.0 / 12.5 / 20.1, 64 x 4096 x 4096 42.9 / 69.8 / 69.4, 1024^3 47.5 / 41.9 / 46.4, 256 x 256 x
    // 4096 38.7 / 70.2 / 28.0.  Slices draw on HBM unevenly, 4.6 TB/s of the weights at most (bf16,
    // slices / grid: 64 x 14336 x 4096 50.7 / 41.8, 32 x 11008 x 4096 40.1 / 33.3), and a K split pays
    // SPLIT_US for its second launch beside the estimate (261 x 76 x 2325 7.2 / 12.1 in 8 pieces).
    constexpr double SPLIT_US = 2.0;
    const double weights_us = 2.0 * (double)K * N * in_esize(in) / 4.6e6;
    const double nb = (double)ceil_div(nk, 4);
    for (int t = 32; t <= 64; t += 32) {
        const int64_t n = ceil_div(M, t) * ceil_div(N, 32);
        if (n > INT32_MAX) continue;
        const double round = in == IN_F32 ? (t == 32 ? 1.8 + 1.27 * nb : 3.6 + 2.05 * nb)
                                          : (t == 32 ? 1.6 + 0.75 * nb : 2.6 + 0.9 * nb);
        const double us = std::max(1.1 + (double)ceil_div(n, NUM_CU) * round, weights_us);
        if (best_us < 0.0 || us < best_us) {
            best_us = us;
            best = slices(t);
        }
    }
    const int N2 = (int)std::min<int64_t>(2 * up(N, 32), INT32_MAX);
    for (int s = 1; s <= MAX_SPLITS && s <= nk; ++s)
        for (int i = 0; i < n; ++i) {
            const TileCand& t = tiles[i];
            const GatedPlan p = gated_pieces(t.bm, t.bn / 2, bk, M, N, K, s, ws);
            if (p.splits != s) continue;
            double us = estimate_us(in, es_out, M, N2, t, s, s == 1 ? nk : p.kchunk / bk, s == 1 ? 0 : 2 * p.ldw);
            us = us / (s > 1 ? SPLIT_MARGIN : 1.0) + GRID_US + (s > 1 ? SPLIT_US : 0.0);
            if (best_us < 0.0 || us < best_us) {
                best_us = us;
                best = p;
            }
        }
    return best;
}

int run_gated(int in, int of, int M, int N, int K, const void* A, int lda, const void* Bg, int ldbg, const void* Bu,
              int ldbu, void* C, int ldc, const GatedEpi& e, const GatedPlan& p, void* ws, hipStream_t stream) {
    GatedLaunch L{};
    L.in = in;
    L.out = of;
    L.tbm = p.bm;
    L.tbp = p.bn;
    L.A = (const char*)A;
    L.Bg = (const char*)Bg;
    L.Bu = (const char*)Bu;
    L.C = (char*)C;
    L.M = M;
    L.N = N;
    L.K = K;
    L.lda = lda;
    L.ldbg = ldbg;
    L.ldbu = ldbu;
    L.ldc = ldc;
    L.tiles_m = (int)ceil_div(M, p.bm);
    L.tiles_n = (int)ceil_div(N, p.bn);
    L.splits = p.splits;
    L.kchunk = p.splits > 1 ? p.kchunk : std::max(K, 1);
    L.waves = p.waves;
    L.e = e;
    L.stream = stream;
    const int64_t wgs = (int64_t)L.tiles_m * L.tiles_n * p.splits;
    if (wgs > INT32_MAX) return DGEMM_ERR_TOO_LARGE;
    // Alone on its CU the 128 x 64 tile has room for a ring of four stages (as gemm16's).
    L.stages = p.bm == 128 && wgs <= NUM_CU ? 4 : 2;
    const auto launch = p.skinny ? launch_gated_skinny : launch_gated;
    if (p.splits == 1) return launched(launch(L));
    L.out = OUT_F32;
    L.C = nullptr;
    L.zstride = (int64_t)M * 2 * p.ldw * 4;
    L.e = GatedEpi{};
    L.e.G = (char*)ws;
    L.e.U = (char*)ws + (int64_t)p.ldw * 4;
    L.e.ldg = L.e.ldu = 2 * p.ldw;
    if (launch(L) != hipSuccess) return DGEMM_ERR_LAUNCH;
    return launched(launch_gated_reduce((const float*)ws, p.splits, (int64_t)M * 2 * p.ldw, p.ldw, (char*)C, ldc, M, N,
                                        of, e, stream));
}

// The pieces of gemm_gated_bwd's workspace, in order: dG, dU, the column sums of the biases, an
// operand's transpose (fp32), then what fp32 products' plans may use.
struct GatedBwdParts {
    int lddz, ldp, chunks;
    int64_t dz, part, trans, required;  // dz: of one of the two
};

GatedBwdParts gated_bwd_parts(int in, int M, int N, int K, bool products, bool dbias) {
    GatedBwdParts b{};
    const int es = in_esize(in);
    b.lddz = (int)up(N, 16 / es);
    b.ldp = (int)up(N, 4);
    b.chunks = (int)ceil_div(M, act_grad_rows(M, N));
    b.dz = products ? up((int64_t)M * b.lddz * es, WS_ALIGN) : 0;
    b.part = dbias ? up((int64_t)b.chunks * 2 * b.ldp * 4, WS_ALIGN) : 0;
    if (products && es == 4 && M > SKINNY_M)
        b.trans = up(std::max((int64_t)N * up(K, 4), (int64_t)K * up(M, 4)) * 4, WS_ALIGN);
    b.required = 2 * b.dz + b.part + b.trans;
    return b;
}

// How the products of a gated layer's backward pass run: tile sizes of the input's gradient (nt)
// and of the weights' (tn), 0 where it is not wanted; slices: slicet.hip's tiles, else gemmt.hip's.
struct GatedBwdPlan {
    int nt, tn;  // 0: none fits
    bool nt_slices, tn_slices, together, tn_first, transposes;  // transposes: fp32 by the grid kernels
    // Grid tiles: nt's K steps in runs of `per`, with partial sums of pitch ldw; tn's rows likewise.
    int splits = 1, per = 0, ldw = 0, tn_splits = 1, tn_per = 0, tn_ldw = 0;
    int64_t ws_bytes = 0;  // of those
};

// M rows, K inputs, N gated outputs: nt has M x K outputs of 2 N terms, tn two of K x N of M.
GatedBwdPlan plan_gated_bwd(int in, int M, int N, int K, bool dA, bool dB, uint64_t ws) {
    const int f = in == IN_F32 ? IN_F32 : IN_BF16;
    const int kn = (int)std::min<int64_t>(2 * up(N, 64), INT32_MAX);
    GatedBwdPlan best{};
    double best_us = -1.0;
    auto consider = [&](double us, const GatedBwdPlan& p) {
        if (best_us >= 0.0 && us >= best_us) return;
        best_us = us;
        best = p;
    };
    auto nt_tiles = [&](int t) { return dA ? ceil_div(M, t) * ceil_div(K, t) : 0; };
    auto tn_tiles = [&](int t) { return dB ? 2 * ceil_div(K, t) * ceil_div(N, t) : 0; };
    int fm, fn, fs;
    const bool forced = forced_grid(fm, fn, fs) && fm == fn &&
                        (fm == 32 || fm == 64 || (f != IN_F32 && (fm == 128 || fm == 256)));
    auto allowed = [&](int t) { return !forced || t == fm; };
    // One product alone: us, tile and kind.
    struct Alone { double us; int tile; bool slices; };
    auto alone = [&](bool nt) {
        Alone a{-1.0, 0, false};
        for (int t = 32; t <= 64; t += 32) {
            const int64_t n = nt ? nt_tiles(t) : tn_tiles(t);
            if (!allowed(t) || n > INT32_MAX / 2) continue;
            const double us = pair_us(n, slice_tile_us(f, t, nt ? kn : M), 0, 0.0);
            if (a.us < 0.0 || us < a.us) a = Alone{us, t, true};
        }
        for (const TileCand& t : TILES_T) {
            const int64_t n = nt ? nt_tiles(t.bm) : tn_tiles(t.bm);
            if (f == IN_F32 || !allowed(t.bm) || n > INT32_MAX / 2) continue;
            bool first;
            const double us = pair_grid_us(t, in, n, nt ? kn : M, 0, 0, first);
            if (a.us < 0.0 || us < a.us) a = Alone{us, t.bm, false};
        }
        return a;
    };
    for (int a = 32; a <= 64; a += 32)
        for (int b = 32; b <= 64; b += 32) {
            if (((!dA || !dB) && a != b) || !allowed(a) || !allowed(b)) continue;
            const int64_t ta = nt_tiles(a), tb = tn_tiles(b);
            if (ta + tb > (forced ? (int64_t)INT32_MAX / 2 : f == IN_F32 ? PAIR_TILES_32 : PAIR_TILES_16)) continue;
            const double wa = slice_tile_us(f, a, kn), wb = slice_tile_us(f, b, M);
            const double fwd = pair_us(ta, wa, tb, wb), rev = pair_us(tb, wb, ta, wa);
            consider(std::min(fwd, rev), GatedBwdPlan{a, b, true, true, true, rev < fwd, false});
        }
    if (f != IN_F32)
        for (const TileCand& t : TILES_T) {
            const int64_t ta = nt_tiles(t.bm), tb = tn_tiles(t.bm);
            if (!allowed(t.bm) || ta + tb > INT32_MAX / 2) continue;
            // Up to 64 rows the weights' tiles are one step and their stores, which two workgroups
            // per CU overlap and one does not (4 x 2228 x 3330 bf16 23.2 us with 128 x 128, 28.5 with
            // 256 x 256, 16 x 4096 x 4096 38.3 and 45.0).
            if (M <= 64 && t.bm == 256 && !forced) continue;
            bool tn_first;
            // Three products on 128 x 128 tiles were slower than the estimate for two.
            const double f128 = t.bm == 128 ? 1.15 : 1.0;
            const double us = pair_grid_us(t, in, ta, kn, tb, M, tn_first) * f128;
            consider(us, GatedBwdPlan{t.bm, t.bm, false, false, true, tn_first, false});
            // dA's sums are twice as long as a plain layer's: where its tiles are few they are the
            // pass's longest, and in runs of their steps, to a workspace, fill the CUs that it leaves
            // idle.  The whole pass in us, bf16, M x N x K, whole / in runs:
            //    300 x 1500 x  900    43.0 /  21.9   (128 x 128, 5 runs)
            //    100 x 3000 x 4000    85.3 /  35.5   (128 x 128, 4)
            //   1000 x 2744 x 1032    93.7 /  50.4   (256 x 256, 6)
            //    600 x 8000 x 1000     189 /  67.4   (256 x 256, 8)
            //   2000 x 4000 x 2000     171 /   141   (256 x 256, 2)
            //   3000 x 6000 x 1500     285 /   260   (256 x 256, 2)
            // With these constants the plan chosen among 1 to 12 runs of either tile takes 3 % more
            // than the fastest on average over ten such layers, 14 % at most.
            // The weights' sums are as long as the batch, and a small layer's are split the same way,
            // alone or with dA's (us, dA's sums alone in runs / these too):
            //   4096 x  578 x  488    42.1 / 38.7   (128 x 128, 3 runs)
            //   4096 x 1226 x  276    51.1 / 42.8   (128 x 128, 3)
            //  16384 x  512 x  128    66.8 / 38.6   (128 x 128, 16 of the batch)
            const int steps = kn / 64, tn_steps = (int)ceil_div(M, 64);
            auto runs = [&](int sa, int sb) {
                GatedBwdPlan p{t.bm, t.bm, false, false, true, false, false};
                if (dA && sa > 1) {
                    p.per = (int)ceil_div(steps, sa);
                    p.splits = (int)ceil_div(steps, p.per);
                }
                if (dB && sb > 1) {
                    p.tn_per = (int)ceil_div(tn_steps, sb) * 64;
                    p.tn_splits = (int)ceil_div(M, p.tn_per);
                }
                p.ldw = (int)up(K, 4);
                p.tn_ldw = (int)up(N, 4);
                int64_t out = 0;
                if (p.splits > 1) p.ws_bytes = (int64_t)p.splits * M * p.ldw * 4, out = (int64_t)M * K * 2;
                if (p.tn_splits > 1) {
                    p.ws_bytes += (int64_t)p.tn_splits * 2 * K * p.tn_ldw * 4;
                    out += (int64_t)K * N * 4;
                }
                const int64_t na = ta * p.splits, nb = tb * p.tn_splits;
                if (p.ws_bytes == 0 || (uint64_t)p.ws_bytes > ws || na + nb > INT32_MAX / 2 ||
                    (int64_t)PANEL_ROWS * std::max(p.ldw, p.tn_ldw) * 4 >= DESC_LIMIT)
                    return;
                const double sum_us = 4.0 + (2.0 * (double)p.ws_bytes + (double)out) / 8e6;
                const int la = p.splits > 1 ? p.per * 64 : kn, lb = p.tn_splits > 1 ? p.tn_per : M;
                const double split_us = pair_grid_us(t, in, na, la, nb, lb, p.tn_first) * f128 + sum_us;
                consider(forced ? 0.0 : split_us, p);
            };
            if (forced) {
                if (fs > 1) runs(std::min(fs, steps), std::min(fs, tn_steps));
                continue;
            }
            for (int s = 2; s <= MAX_SPLITS && s <= steps && dA; ++s) runs(s, 1);
            // Both in runs of about the same length, while they fit the CUs at once.
            for (int s = 2; s <= MAX_SPLITS && s <= tn_steps && dB; ++s) {
                const int sa = (int)std::min<int64_t>(MAX_SPLITS, (int64_t)steps * s / std::max(tn_steps, 1));
                if (s > 2 && tb * s > 2 * NUM_CU) break;
                runs(sa, s);
                if (sa > 1) runs(1, s);
            }
        }
    if (f == IN_F32 && !forced && M > SKINNY_M) {
        double us = 0.0;
        if (dA)
            us += 2 * (PAIR_GAP_US + (double)K * N * 8.0 / 4e6 + PAIR_GAP_US +
                       plan_us(in, 4, make_plan(in, 4, M, K, N, ws, false), M, K, N));
        if (dB)
            us += PAIR_GAP_US + (double)K * M * 8.0 / 4e6 +
                  2 * (PAIR_GAP_US + plan_us(in, 4, make_plan(in, 4, K, N, M, ws, false), K, N, M));
        consider(us, GatedBwdPlan{0, 0, false, false, false, false, true});
    }
    if (dA && dB && !forced) {
        const Alone a = alone(true), b = alone(false);
        if (a.us >= 0.0 && b.us >= 0.0)
            consider(a.us + b.us + PAIR_GAP_US, GatedBwdPlan{a.tile, b.tile, a.slices, b.slices, false, false, false});
    }
    return best;
}

// Whether a backward pass of few rows is left to the kernels for few rows (skinny.hip): one launch
// for dA and one for each weight, against one launch, or two, by the plan above.  The whole pass in
// us, M x N x K, by them / by the plan:
//   bf16   1 x   64 x   64   12.9 /  6.4     fp32   1 x   64 x   64   14.6 /  8.3
//         16 x 1000 x 1000   24.5 / 15.5           16 x 1000 x 1000   31.0 / 26.5
//         10 x 5121 x   64   31.3 / 18.5           10 x 5121 x   64   43.5 / 58.3
//          4 x 2228 x 3330   27.9 / 23.9            4 x 2228 x 3330   42.4 / 96.0
//         16 x 4096 x 4096   54.7 / 40            16 x 4096 x 1024   60.0 / 55.5
//          8 x 8192 x 4096   70.9 / 66.5            8 x 8192 x 4096    177 /  298
// (16-bit, from the fourth row on, with dA's sums in runs.)  fp32 layers above the small ones all take
// the kernels for few rows, 16 x 4096 x 1024 among them: the plan is close there and far behind at more
// columns or terms.
bool few_rows(int in, int M, int N, int K, const GatedBwdPlan& p) {
    const bool small = N <= 1024 && (int64_t)N * K <= 1 << 20;
    return M <= SKINNY_M && (M == 0 || (!small && (in == IN_F32 || p.ws_bytes == 0)));
}

GemmLaunch bwd_launch(int in, int layout, int tile, bool slices, int M, int N, int K, const void* X, int ldx,
                      const void* Y, int ldy, void* C, int ldc, hipStream_t stream) {
    GemmLaunch L{};
    L.in = in;
    L.out = out_format(in, DGEMM_OUT_SAME);
    L.tbm = L.tbn = tile;
    L.layout = layout;
    L.slice_waves = slices ? 4 : 0;
    L.splits = 1;
    L.kchunk = K;
    L.epi = EPI_FULL;
    L.e.alpha = 1.0f;
    L.A = (const char*)X;
    L.B = (const char*)Y;
    L.C = (char*)C;
    L.M = M;
    L.N = N;
    L.K = K;
    L.lda = ldx;
    L.ldb = ldy;
    L.ldc = ldc;
    L.tiles_m = (int)ceil_div(M, tile);
    L.tiles_n = (int)ceil_div(N, tile);
    L.stream = stream;
    return L;
}

}  // namespace
}  // namespace dgemm

using namespace dgemm;

extern "C" {

int quant_f8_block(int in, int rows, int transpose, int M, int N, const void* X, int ldx, void* Q, int ldq,
                   float* scale, int scale_row, int scale_block, void* stream) {
    const int fmt = row_fmt(in);
    if (fmt < 0 || M < 0 || N < 0 || (transpose != 0 && transpose != 1) || (rows != 1 && rows != F8_BLOCK))
        return DGEMM_ERR_INVALID_VALUE;
    const int R = transpose ? N : M, C = transpose ? M : N;
    const Mat mX{X, M, N, ldx, out_esize(fmt)}, mQ{Q, R, C, ldq, 1};
    const Scales s{scale, ceil_div(R, rows), ceil_div(C, F8_BLOCK), scale_row, scale_block};
    int st;
    if ((st = check_mat(mX)) != DGEMM_OK || (st = check_mat(mQ)) != DGEMM_OK ||
        (st = check_scales(s, true)) != DGEMM_OK)
        return st;
    if (M == 0 || N == 0) return DGEMM_OK;
    if ((rows != 1 || transpose) && ceil_div(M, F8_BLOCK) * ceil_div(N, F8_BLOCK) >= (int64_t)1 << 23)
        return DGEMM_ERR_TOO_LARGE;
    const Mat ins[] = {mX}, outs[] = {mQ, s.mat()};
    if (any_overlap(outs, 2, ins, 1)) return DGEMM_ERR_ALIAS;
    if ((st = check_device()) != DGEMM_OK) return st;
    const QuantBlockArgs a{(const char*)X, (char*)Q, scale, M, N, ldx, ldq, scale_row, scale_block};
    return launched(launch_quant_block(a, fmt, rows, transpose, (hipStream_t)stream));
}

int gemm_f8_block(int out, int rows_b, int M, int N, int K, const void* A, int lda, const void* B, int ldb,
                  void* C, int ldc, const float* scale_a, int sa_row, int sa_block, const float* scale_b,
                  int sb_row, int sb_block, const float* bias, int act, const void* R, int ldr, void* workspace,
                  size_t workspace_bytes, void* stream) {
    const int of = row_fmt(out);
    if (of < 0 || M < 0 || N < 0 || K < 0 || !valid_act(act) || (workspace_bytes > 0 && !workspace) ||
        (rows_b != 1 && rows_b != F8_BLOCK))
        return DGEMM_ERR_INVALID_VALUE;
    const int eo = out_esize(of);
    const bool reads = M > 0 && N > 0;
    const Mat mA{A, reads ? M : 0, K, lda, 1}, mB{B, reads ? N : 0, K, ldb, 1}, mC{C, M, N, ldc, eo};
    const Mat mR{R, R ? M : 0, N, ldr, eo};
    const int64_t kb = ceil_div(K, F8_BLOCK);
    const Scales sa{scale_a, mA.rows, kb, sa_row, sa_block}, sb{scale_b, ceil_div(mB.rows, rows_b), kb, sb_row, sb_block};
    int st;
    if ((st = check_mat(mA)) != DGEMM_OK || (st = check_mat(mB)) != DGEMM_OK || (st = check_mat(mC)) != DGEMM_OK ||
        (R && (st = check_mat(mR)) != DGEMM_OK) || (st = check_scales(sa, false)) != DGEMM_OK ||
        (st = check_scales(sb, false)) != DGEMM_OK)
        return st;
    if (!reads) return DGEMM_OK;
    const Plan p = plan_block(of, rows_b, M, N, K, workspace ? workspace_bytes : 0);
    if (p.bm == 0) return DGEMM_ERR_TOO_LARGE;
    const Mat ws = bytes_of(workspace, p.ws_bytes);
    if (check_vec(bias, 4) != DGEMM_OK || check_vec(ws.p, 16) != DGEMM_OK) return DGEMM_ERR_MISALIGNED;
    // R may be C itself (each element is read before it is written), not overlap it in any other way.
    const bool in_place = R == C && (ldr == ldc || M == 1);
    const Mat none{nullptr, 0, 0, 0, 0};
    const Mat ins[] = {mA, mB, in_place ? none : mR, vec(bias, N), sa.mat(), sb.mat()}, outs[] = {mC, ws};
    if (any_overlap(outs, 2, ins, 6) || (in_place && any_overlap(&ws, 1, &mR, 1))) return DGEMM_ERR_ALIAS;
    if ((st = check_device()) != DGEMM_OK) return st;
    EpiArgs e{};
    e.alpha = 1.0f;
    e.bias = bias;
    e.act = act;
    e.res = (const char*)R;
    e.ldr = ldr;
    return run_block(of, M, N, K, A, lda, B, ldb, C, ldc,
                     BlockScales{scale_a, scale_b, sa_row, sa_block, sb_row, sb_block, rows_b}, e, p, workspace,
                     (hipStream_t)stream);
}

int gemm_f8_block_plan(int out, int rows_b, int M, int N, int K, size_t workspace_bytes, int* tile_rows,
                       int* tile_cols, int* splits, size_t* workspace_used) {
    const int of = row_fmt(out);
    if (of < 0 || M < 0 || N < 0 || K < 0 || (rows_b != 1 && rows_b != F8_BLOCK)) return DGEMM_ERR_INVALID_VALUE;
    if (ceil_div(M, 128) * ceil_div(N, 128) > INT32_MAX) return DGEMM_ERR_TOO_LARGE;
    const Plan p = plan_block(of, rows_b, M, N, K, workspace_bytes);
    return p.bm == 0 ? DGEMM_ERR_TOO_LARGE : report(p, tile_rows, tile_cols, splits, workspace_used);
}

int layernorm(int in, int out, int M, int N, const void* X, int ldx, const void* R, int ldr, void* S, int lds,
              const float* weight, const float* bias, float eps, void* Y, int ldy, float* scale, int scale_row,
              int scale_block, float* mean, float* rstd, void* stream) {
    const int fmt = row_fmt(in);
    if (fmt < 0 || M < 0 || N < 0 || !(eps >= 0.0f) || out < DGEMM_ROWS_SAME || out > DGEMM_ROWS_F8_BLOCK)
        return DGEMM_ERR_INVALID_VALUE;
    const bool f8 = out != DGEMM_ROWS_SAME, blocks = out == DGEMM_ROWS_F8_BLOCK;
    const int es = out_esize(fmt);
    const Mat mX{X, M, N, ldx, es}, mR{R, M, N, ldr, es}, mS{S, M, N, lds, es}, mY{Y, M, N, ldy, f8 ? 1 : es};
    const Scales sc{scale, M, blocks ? ceil_div(N, F8_BLOCK) : 1, blocks ? scale_row : 1, blocks ? scale_block : 1};
    int st;
    if ((st = check_mat(mX)) != DGEMM_OK || (st = check_mat(mY)) != DGEMM_OK) return st;
    if (R && (st = check_mat(mR)) != DGEMM_OK) return st;
    if (S && (st = check_mat(mS)) != DGEMM_OK) return st;
    if (M == 0 || N == 0) return DGEMM_OK;
    if (!weight || (!f8 && scale)) return DGEMM_ERR_INVALID_VALUE;
    if (N > ROW_MAX) return DGEMM_ERR_TOO_LARGE;
    if (f8 && (st = check_scales(sc, true)) != DGEMM_OK) return st;
    if (check_vec(weight, 16) != DGEMM_OK || check_vec(bias, 16) != DGEMM_OK || check_vec(mean, 4) != DGEMM_OK ||
        check_vec(rstd, 4) != DGEMM_OK)
        return DGEMM_ERR_MISALIGNED;
    // As rmsnorm: S and Y may each be X or R themselves and share nothing else with the inputs.
    const auto same = [&](const Mat& o, const Mat& i) {
        return o.p == i.p && o.es == i.es && (o.ld == i.ld || M == 1);
    };
    const Mat none{nullptr, 0, 0, 0, 0};
    const Mat outs[] = {mS, mY, f8 ? sc.mat() : none, vec(mean, M), vec(rstd, M)};
    if (any_overlap(outs, 5, nullptr, 0)) return DGEMM_ERR_ALIAS;
    for (int i = 0; i < 5; ++i) {
        const bool whole = i < 2;
        const Mat ins[] = {whole && same(outs[i], mX) ? none : mX, !R || (whole && same(outs[i], mR)) ? none : mR,
                           vec(weight, N), vec(bias, N)};
        if (any_overlap(&outs[i], 1, ins, 4)) return DGEMM_ERR_ALIAS;
    }
    if ((st = check_device()) != DGEMM_OK) return st;
    const RowArgs a{(const char*)X, (const char*)R, (char*)S, weight, (char*)Y, scale, rstd, eps, M, N,
                    ldx, ldr, lds, ldy, bias, mean, sc.s_row, sc.s_blk};
    return launched(launch_layernorm(a, fmt, out, (hipStream_t)stream));
}

int layernorm_bwd(int in, int M, int N, const void* dY, int lddy, const void* S, int lds, const float* weight,
                  const float* mean, const float* rstd, const void* dS, int ldds, void* dX, int lddx,
                  float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    const int fmt = row_fmt(in);
    if (fmt < 0 || M < 0 || N < 0 || (workspace_bytes > 0 && !workspace)) return DGEMM_ERR_INVALID_VALUE;
    const int es = out_esize(fmt);
    const Mat mdY{dY, M, N, lddy, es}, mS{S, M, N, lds, es}, mdS{dS, M, N, ldds, es}, mdX{dX, M, N, lddx, es};
    int st;
    if ((st = check_mat(mdY)) != DGEMM_OK || (st = check_mat(mS)) != DGEMM_OK ||
        (st = check_mat(mdX)) != DGEMM_OK)
        return st;
    if (dS && (st = check_mat(mdS)) != DGEMM_OK) return st;
    const bool sums = dweight || dbias;
    if (N == 0 || (M == 0 && !sums)) return DGEMM_OK;
    if (M > 0 && (!weight || !mean || !rstd)) return DGEMM_ERR_INVALID_VALUE;
    if (N > NORM_BWD_MAX) return DGEMM_ERR_TOO_LARGE;
    if (check_vec(weight, 16) != DGEMM_OK || check_vec(mean, 4) != DGEMM_OK || check_vec(rstd, 4) != DGEMM_OK ||
        check_vec(dweight, 4) != DGEMM_OK || check_vec(dbias, 4) != DGEMM_OK || check_vec(workspace, 16) != DGEMM_OK)
        return DGEMM_ERR_MISALIGNED;
    const int grid = layernorm_bwd_grid(M, N, fmt), ldp = (int)up(N, 4);
    size_t need = 0;
    if (sums) layernorm_bwd_workspace(M, N, &need);
    if (need > workspace_bytes) return DGEMM_ERR_WORKSPACE;
    // dX may be dY or dS itself (a row is read before it is written).
    const auto same = [&](const Mat& i) { return mdX.p == i.p && (mdX.ld == i.ld || M == 1); };
    const Mat none{nullptr, 0, 0, 0, 0};
    const Mat ws = bytes_of(workspace, need);
    const Mat in_x[] = {same(mdY) ? none : mdY, mS, dS ? (same(mdS) ? none : mdS) : none, vec(weight, N),
                        vec(mean, M), vec(rstd, M), vec(dweight, N), vec(dbias, N), ws};
    const Mat out_w[] = {vec(dweight, N), vec(dbias, N), ws};
    const Mat in_w[] = {mdY, mS, dS ? mdS : none, vec(weight, N), vec(mean, M), vec(rstd, M)};
    if (any_overlap(&mdX, 1, in_x, 9) || any_overlap(out_w, 3, in_w, 6)) return DGEMM_ERR_ALIAS;
    if ((st = check_device()) != DGEMM_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    float* const part = sums ? (float*)workspace : nullptr;
    const NormBwdArgs a{(const char*)dY, (const char*)S, (const char*)dS, weight, rstd, (char*)dX,
                        part, M, N, lddy, lds, ldds, lddx, ldp, mean};
    if (M > 0 && launch_layernorm_bwd(a, fmt, s) != hipSuccess) return DGEMM_ERR_LAUNCH;
    if (!sums) return DGEMM_OK;
    const int G = M > 0 ? grid : 0;
    return launched(launch_col_reduce2(ColReduceArgs{part, dweight, G, 2 * ldp, dweight ? N : 0},
                                       ColReduceArgs{part + ldp, dbias, G, 2 * ldp, dbias ? N : 0}, s));
}

int layernorm_bwd_workspace(int M, int N, size_t* required) {
    if (M < 0 || N < 0) return DGEMM_ERR_INVALID_VALUE;
    if (N > NORM_BWD_MAX) return DGEMM_ERR_TOO_LARGE;
    // The 16-bit types' count, the larger.
    if (required) *required = (size_t)layernorm_bwd_grid(M, N, OUT_BF16) * 2 * (size_t)up(N, 4) * 4;
    return DGEMM_OK;
}

int gemm_gated(int in, int out, int M, int N, int K, const void* A, int lda, const void* Bg, int ldbg, const void* Bu,
               int ldbu, void* C, int ldc, const float* bias_g, const float* bias_u, int act, void* G, int ldg,
               void* U, int ldu, void* workspace, size_t workspace_bytes, void* stream) {
    if (in < IN_F32 || in > IN_F16 || M < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    const int of = out_format(in, out);
    if (of < 0 || !valid_act(act) || (workspace_bytes > 0 && !workspace)) return DGEMM_ERR_INVALID_VALUE;
    const int eo = out_esize(of), es = in_esize(in);
    const bool reads = M > 0 && N > 0;
    const Mat mA{A, reads ? M : 0, K, lda, es}, mBg{Bg, reads ? K : 0, N, ldbg, es}, mBu{Bu, reads ? K : 0, N, ldbu, es};
    const Mat mC{C, M, N, ldc, eo}, mG{G, G ? M : 0, N, ldg, eo}, mU{U, U ? M : 0, N, ldu, eo};
    int st;
    if ((st = check_mat(mA)) != DGEMM_OK || (st = check_mat(mBg)) != DGEMM_OK || (st = check_mat(mBu)) != DGEMM_OK ||
        (st = check_mat(mC)) != DGEMM_OK || (G && (st = check_mat(mG)) != DGEMM_OK) ||
        (U && (st = check_mat(mU)) != DGEMM_OK))
        return st;
    if (!reads) return DGEMM_OK;
    const GatedPlan p = plan_gated(in, eo, M, N, K, workspace ? workspace_bytes : 0);
    if (p.bm == 0) return DGEMM_ERR_TOO_LARGE;
    const Mat ws = bytes_of(workspace, p.ws_bytes);
    if (check_vec(bias_g, 4) != DGEMM_OK || check_vec(bias_u, 4) != DGEMM_OK || check_vec(ws.p, 16) != DGEMM_OK)
        return DGEMM_ERR_MISALIGNED;
    const Mat ins[] = {mA, mBg, mBu, vec(bias_g, N), vec(bias_u, N)}, outs[] = {mC, mG, mU, ws};
    if (any_overlap(outs, 4, ins, 5)) return DGEMM_ERR_ALIAS;
    if ((st = check_device()) != DGEMM_OK) return st;
    return run_gated(in, of, M, N, K, A, lda, Bg, ldbg, Bu, ldbu, C, ldc,
                     GatedEpi{bias_g, bias_u, act, (char*)G, (char*)U, ldg, ldu}, p, workspace, (hipStream_t)stream);
}

int gemm_gated_plan(int in, int out, int M, int N, int K, size_t workspace_bytes, int* tile_rows, int* tile_cols,
                    int* splits, size_t* workspace_used) {
    if (in < IN_F32 || in > IN_F16 || M < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    const int of = out_format(in, out);
    if (of < 0) return DGEMM_ERR_INVALID_VALUE;
    if (ceil_div(M, 128) * ceil_div(N, 64) > INT32_MAX) return DGEMM_ERR_TOO_LARGE;
    const GatedPlan p = plan_gated(in, out_esize(of), M, N, K, workspace_bytes);
    if (p.bm == 0) return DGEMM_ERR_TOO_LARGE;
    Plan q{};
    q.bm = p.bm;
    q.bn = p.bn;
    q.splits = p.splits;
    q.ws_bytes = p.ws_bytes;
    return report(q, tile_rows, tile_cols, splits, workspace_used);
}

int gemm_gated_bwd(int in, int out, int M, int N, int K, const void* A, int lda, const void* Bg, int ldbg,
                   const void* Bu, int ldbu, const void* dC, int lddc, const void* G, int ldg, const void* U, int ldu,
                   int act, void* dA, int ldda, void* dBg, int lddbg, void* dBu, int lddbu, float* dbias_g,
                   float* dbias_u, void* workspace, size_t workspace_bytes, void* stream) {
    if (in < IN_F32 || in > IN_F16 || M < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    const int cf = out_format(in, out);
    if (cf < 0 || !valid_act(act) || (workspace_bytes > 0 && !workspace)) return DGEMM_ERR_INVALID_VALUE;
    const int es = in_esize(in), ec = out_esize(cf);
    const bool dB = dBg || dBu, bias = dbias_g || dbias_u;
    const Mat mA{A, dB ? M : 0, K, lda, es}, mBg{Bg, dA ? K : 0, N, ldbg, es}, mBu{Bu, dA ? K : 0, N, ldbu, es};
    const Mat mdC{dC, M, N, lddc, ec}, mG{G, M, N, ldg, ec}, mU{U, M, N, ldu, ec};
    const Mat mdA{dA, dA ? M : 0, K, ldda, es}, mdBg{dBg, dBg ? K : 0, N, lddbg, es}, mdBu{dBu, dBu ? K : 0, N, lddbu, es};
    int st;
    if (dB && (st = check_mat(mA)) != DGEMM_OK) return st;
    if (dA && ((st = check_mat(mBg)) != DGEMM_OK || (st = check_mat(mBu)) != DGEMM_OK)) return st;
    if ((st = check_mat(mdC)) != DGEMM_OK || (st = check_mat(mG)) != DGEMM_OK || (st = check_mat(mU)) != DGEMM_OK)
        return st;
    if ((dA && (st = check_mat(mdA)) != DGEMM_OK) || (dBg && (st = check_mat(mdBg)) != DGEMM_OK) ||
        (dBu && (st = check_mat(mdBu)) != DGEMM_OK))
        return st;
    if (check_vec(dbias_g, 4) != DGEMM_OK || check_vec(dbias_u, 4) != DGEMM_OK || check_vec(workspace, 16) != DGEMM_OK)
        return DGEMM_ERR_MISALIGNED;
    const GatedBwdParts b = gated_bwd_parts(in, M, N, K, dA || dB, bias);
    if ((uint64_t)b.required > workspace_bytes) return DGEMM_ERR_WORKSPACE;
    // The rows of A's transpose (fp32), for the weights' gradients, are as long as M.
    if (es == 4 && dB && M > SKINNY_M && (int64_t)PANEL_ROWS * up(M, 4) * 4 >= DESC_LIMIT) return DGEMM_ERR_TOO_LARGE;
    const Mat ws = bytes_of(workspace, (int64_t)std::min<uint64_t>(workspace_bytes, INT64_MAX));
    const Mat ins[] = {mA, mBg, mBu, mdC, mG, mU};
    const Mat outs[] = {mdA, mdBg, mdBu, vec(dbias_g, N), vec(dbias_u, N), ws};
    if (any_overlap(outs, 6, ins, 6)) return DGEMM_ERR_ALIAS;
    const bool want_a = dA && M > 0 && K > 0, want_b = dB && K > 0 && N > 0;
    const int64_t gemm_bytes = (int64_t)std::min<uint64_t>(workspace_bytes, INT64_MAX) - b.required;
    GatedBwdPlan p{};
    if (want_a || want_b) p = plan_gated_bwd(in, M, N, K, want_a, want_b, (uint64_t)gemm_bytes);
    const bool few = few_rows(in, M, N, K, p);
    if (!few && (want_a || want_b) && !p.transposes && p.nt == 0) return DGEMM_ERR_TOO_LARGE;
    if ((st = check_device()) != DGEMM_OK) return st;

    char* const w = (char*)workspace;
    char* const dG = w;
    char* const dU = w + b.dz;
    float* const part = (float*)(w + 2 * b.dz);
    float* const w_trans = (float*)(w + 2 * b.dz + b.part);
    char* const w_gemm = w + b.required;
    hipStream_t s = (hipStream_t)stream;
    if (M > 0 && N > 0 && (dA || dB || bias)) {
        const bool products = (dA || dB) && K > 0;
        const GatedGradArgs a{(const char*)dC, (const char*)G, (const char*)U, products ? dG : nullptr,
                              products ? dU : nullptr, bias ? part : nullptr, M, N, lddc, ldg, ldu, b.lddz, b.ldp,
                              act_grad_rows(M, N), act};
        if (launch_gated_grad(a, cf, out_format(in, DGEMM_OUT_SAME), s) != hipSuccess) return DGEMM_ERR_LAUNCH;
    }
    const int G2 = M > 0 ? b.chunks : 0;
    const ColReduceArgs sg{part, dbias_g, G2, 2 * b.ldp, dbias_g ? N : 0};
    const ColReduceArgs su{part + b.ldp, dbias_u, G2, 2 * b.ldp, dbias_u ? N : 0};
    void* const dW[2] = {dBg, dBu};
    const int lddw[2] = {lddbg, lddbu};
    char* const dz[2] = {dG, dU};

    if (few) {
        // Few rows: the weights once through registers for dA, rank-M updates for theirs.
        if (want_a) {
            const Plan q = plan_skinny(in, LAY_NT, M, K, (int)std::min<int64_t>(2 * (int64_t)N, INT32_MAX), 0);
            GemmLaunch L = bwd_launch(in, LAY_NT, q.bn, true, M, K, N, dG, b.lddz, Bg, ldbg, dA, ldda, s);
            L.tiles_m = 1;
            L.slice_waves = q.waves;
            if (launch_skinny_two(L, dU, (const char*)Bu, ldbu) != hipSuccess) return DGEMM_ERR_LAUNCH;
        }
        for (int i = 0; i < 2; ++i)
            if (want_b && dW[i]) {
                const GemmLaunch L = bwd_launch(in, LAY_TN, 32, true, K, N, M, A, lda, dz[i], b.lddz, dW[i], lddw[i], s);
                if (launch_skinny(L) != hipSuccess) return DGEMM_ERR_LAUNCH;
            }
        return launched(launch_col_reduce2(sg, su, s));
    }
    if (!want_a && !want_b) return launched(launch_col_reduce2(sg, su, s));
    if (!p.transposes) {
        GatedBwdLaunch L{};
        L.nt = bwd_launch(in, LAY_NT, p.nt, p.nt_slices, M, K, N, dG, b.lddz, Bg, ldbg, dA, ldda, s);
        for (int i = 0; i < 2; ++i) {
            L.tn[i] = bwd_launch(in, LAY_TN, p.tn, p.tn_slices, K, N, M, A, lda, dz[i], b.lddz, dW[i], lddw[i], s);
            if (!want_b || !dW[i]) L.tn[i].tiles_m = 0;
        }
        if (!want_a) L.nt.tiles_m = 0;
        L.A2 = dU;
        L.B2 = (const char*)Bu;
        L.ldb2 = ldbu;
        L.tn_first = p.tn_first;
        L.sums[0] = sg;
        L.sums[1] = su;
        L.nt.kchunk = 2 * (int)ceil_div(N, 64);
        if (p.ws_bytes > 0) {
            // Sums in runs go to the workspace, dA's first, and are added by one more launch.
            SplitSum sums[3];
            int count = 0;
            char* at = w_gemm;
            auto to_workspace = [&](GemmLaunch& g, int splits, int per, int ldw) {
                sums[count++] = SplitSum{(const float*)at, (int64_t)g.M * ldw, g.C, splits, ldw, g.ldc, g.M, g.N};
                g.splits = splits;
                g.kchunk = per;
                g.C = at;
                g.ldc = ldw;
                g.c_zstride = (int64_t)g.M * ldw * 4;
                at += splits * g.c_zstride;
            };
            if (p.splits > 1) to_workspace(L.nt, p.splits, p.per, p.ldw);
            for (GemmLaunch& g : L.tn) {
                if (p.tn_splits <= 1) continue;
                if (g.tiles_m) to_workspace(g, p.tn_splits, p.tn_per, p.tn_ldw);
                else g.splits = p.tn_splits, g.kchunk = p.tn_per, g.c_zstride = (int64_t)K * p.tn_ldw * 4;
            }
            if (launch_gemmt_gated(L) != hipSuccess) return DGEMM_ERR_LAUNCH;
            return launched(launch_splitk_reduce3(sums, count, out_format(in, DGEMM_OUT_SAME), s));
        }
        if (p.together) return launched((p.nt_slices ? launch_slicet_gated : launch_gemmt_gated)(L));
        // Apart: the input's gradient, then the weights' with the sums.
        GatedBwdLaunch first = L;
        first.tn[0] = first.tn[1] = L.nt;
        first.tn[0].tiles_m = first.tn[1].tiles_m = 0;
        first.sums[0].N = first.sums[1].N = 0;
        first.tn_first = false;
        if ((p.nt_slices ? launch_slicet_gated : launch_gemmt_gated)(first) != hipSuccess) return DGEMM_ERR_LAUNCH;
        L.nt = L.tn[0];
        L.nt.tiles_m = 0;
        L.tn_first = false;
        return launched((p.tn_slices ? launch_slicet_gated : launch_gemmt_gated)(L));
    }
    // fp32 of large layers: the grid kernels, which take A[M x K] B[K x N].
    if (launch_col_reduce2(sg, su, s) != hipSuccess) return DGEMM_ERR_LAUNCH;
    const void* const W[2] = {Bg, Bu};
    const int ldw[2] = {ldbg, ldbu};
    for (int i = 0; i < 2 && want_a; ++i) {
        const int ldt = (int)up(K, 4);
        if (N > 0 && launch_transpose32((const float*)W[i], ldw[i], K, N, w_trans, ldt, s) != hipSuccess)
            return DGEMM_ERR_LAUNCH;
        EpiArgs e{};
        e.alpha = 1.0f;
        e.beta = i ? 1.0f : 0.0f;
        st = run(in, OUT_F32, M, K, N, dz[i], b.lddz, w_trans, ldt, dA, ldda, e, i ? EPI_BASIC : EPI_NONE,
                 make_plan(in, 4, M, K, N, (uint64_t)gemm_bytes, false), w_gemm, s);
        if (st != DGEMM_OK) return st;
    }
    if (!want_b) return DGEMM_OK;
    const int ldt = (int)up(M, 4);
    if (launch_transpose32((const float*)A, lda, M, K, w_trans, ldt, s) != hipSuccess) return DGEMM_ERR_LAUNCH;
    for (int i = 0; i < 2; ++i) {
        if (!dW[i]) continue;
        EpiArgs e{};
        e.alpha = 1.0f;
        st = run(in, OUT_F32, K, N, M, w_trans, ldt, dz[i], b.lddz, dW[i], lddw[i], e, EPI_NONE,
                 make_plan(in, 4, K, N, M, (uint64_t)gemm_bytes, false), w_gemm, s);
        if (st != DGEMM_OK) return st;
    }
    return DGEMM_OK;
}

int gemm_gated_bwd_workspace(int in, int out, int M, int N, int K, size_t* required, size_t* best) {
    if (in < IN_F32 || in > IN_F16 || M < 0 || N < 0 || K < 0 || out_format(in, out) < 0)
        return DGEMM_ERR_INVALID_VALUE;
    const GatedBwdParts b = gated_bwd_parts(in, M, N, K, true, true);
    int64_t more = 0;
    const uint64_t any = (uint64_t)1 << 40;
    if (M > 0 && K > 0) {
        // One gradient alone is split more readily than both.
        for (int i = 0; i < 3; ++i) more = std::max(more, plan_gated_bwd(in, M, N, K, i < 2, i != 1, any).ws_bytes);
        if (in == IN_F32 && M > SKINNY_M) {
            more = std::max(more, make_plan(in, 4, M, K, N, any, false).ws_bytes);
            more = std::max(more, make_plan(in, 4, K, N, M, any, false).ws_bytes);
        }
    }
    if (required) *required = (size_t)b.required;
    if (best) *best = (size_t)(b.required + more);
    return DGEMM_OK;
}

}  // extern "C"
