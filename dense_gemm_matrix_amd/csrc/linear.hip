// linear.hip -- the C ABI of the linear layer's operators: products with the
// full epilogue and their gradients (gemm_act, gemm_act_bwd), 8-bit products
// (gemm_f8), norms and quantizers.  Host code only: validation, plans and
// launches; the kernels live in the files that dgemm_internal.h names.

#include <algorithm>
#include <cmath>

#include "dgemm.h"
#include "dgemm_internal.h"
#include "plan.h"

namespace dgemm {
namespace {

constexpr int64_t WS_ALIGN = 256;  // pieces of a workspace start on this

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// A row-major matrix operand of a call.
struct Mat {
    const void* p;
    int64_t rows, cols, ld, es;
    Span span() const { return matrix_span(p, rows, cols, ld, es); }
    bool empty() const { return rows <= 0 || cols <= 0; }
};

// Pitch, pointer, alignment and the 32-bit panel limit of one matrix.
int check_mat(const Mat& m) {
    if (m.ld < std::max<int64_t>(m.cols, 1)) return DGEMM_ERR_LEADING_DIM;
    if (!m.empty()) {
        if (!m.p) return DGEMM_ERR_INVALID_VALUE;
        if (((uintptr_t)m.p & 15) || (m.ld * m.es) % 16) return DGEMM_ERR_MISALIGNED;
    }
    if ((int64_t)PANEL_ROWS * m.ld * m.es >= DESC_LIMIT) return DGEMM_ERR_TOO_LARGE;
    return DGEMM_OK;
}

// An fp32 vector operand (NULL: absent).
Mat vec(const void* p, int64_t n) { return Mat{p, p ? 1 : 0, n, n, 4}; }

int check_vec(const void* p, int align) {
    return ((uintptr_t)p & (uintptr_t)(align - 1)) ? DGEMM_ERR_MISALIGNED : DGEMM_OK;
}

// Whether any of `outs` shares a byte with another of them or with any of `ins`.
bool any_overlap(const Mat* outs, int n_out, const Mat* ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        if (!outs[i].p) continue;
        for (int j = 0; j < n_in; ++j)
            if (ins[j].p && spans_overlap(outs[i].span(), ins[j].span())) return true;
        for (int j = 0; j < i; ++j)
            if (outs[j].p && spans_overlap(outs[i].span(), outs[j].span())) return true;
    }
    return false;
}

Mat bytes_of(void* p, int64_t n) { return Mat{p, n > 0 ? 1 : 0, n, n, 1}; }

bool valid_act(int act) { return act >= DGEMM_ACT_NONE && act <= DGEMM_ACT_SILU; }

// -------------------------------------------------------------------- plans

// Tiles of gemmt.hip: gemm16's constants, whose schedule and bytes per step it
// shares (an 8-bit step is 128 k in the same time).
constexpr TileCand TILES_T[] = {{256, 256, 1.0, 0.0, 0.0, 1.0, 0.6},
                                {128, 128, 0.6, 1.26, 1.35, 0.8, 1.0}};

int t_step(int in) { return in >= IN_F8 ? 128 : 64; }

// Plan of one tile at `splits` K pieces (1: unsplit); splits = 0 if it does not fit.
Plan plan_pieces(const TileCand& t, int bk, int M, int N, int K, int splits, uint64_t ws_avail) {
    Plan p{t.bm, t.bn, 1, K, 0, 0};
    if (splits <= 1 || K <= 0) return p;
    const int nk = (int)ceil_div(K, bk);
    const int steps = (int)ceil_div(nk, std::min(splits, nk));
    p.splits = (int)ceil_div(nk, steps);
    p.kchunk = steps * bk;
    if (p.splits == 1) { p.kchunk = K; return p; }
    p.ldw = (int)up(N, 4);
    p.ws_bytes = (int64_t)p.splits * M * p.ldw * 4;
    if ((uint64_t)p.ws_bytes > ws_avail || (int64_t)PANEL_ROWS * p.ldw * 4 >= DESC_LIMIT ||
        ceil_div(M, t.bm) * ceil_div(N, t.bn) * p.splits > INT32_MAX)
        p.splits = 0;
    return p;
}

// The transposed layouts' plan: the estimate's choice among the slice-K tiles
// (slicet.hip; slicek16's constants, an 8-bit block being 128 k), the two grid
// tiles and 1 to 16 splits, by the same terms and margin as the other plans.
Plan plan_t(int in, int layout, int es_out, int M, int N, int K, uint64_t ws_avail, double* us_out = nullptr) {
    const int bk = t_step(in);
    int fm, fn, fs;
    if (forced_grid(fm, fn, fs) && fm == fn && (fm == 32 || fm == 64)) {
        Plan p{fm, fm, 1, K, 0, 0};
        p.waves = fs == 1 ? 4 : fs;
        p.layout = layout;
        if (slice_waves_t(fm, p.waves) && ceil_div(M, fm) * ceil_div(N, fm) <= INT32_MAX) return p;
    }
    if (forced_grid(fm, fn, fs))
        for (const TileCand& t : TILES_T)
            if (t.bm == fm && t.bn == fn) {
                Plan p = plan_pieces(t, bk, M, N, K, fs, ws_avail);
                p.layout = layout;
                if (p.splits > 0) return p;
            }
    Plan best{};
    double best_us = -1.0;
    const int nk = (int)ceil_div(std::max(K, 1), bk);
    const bool slice = slice_plan_t(M, N, std::min(K, nk * 64), best, best_us);
    best.kchunk = K;
    for (const TileCand& t : TILES_T) {
        if (slice) break;  // as for A[M x K] B[K x N]: unsplit small outputs are the slice-K kernel's
        const double us = estimate_us(in, es_out, M, N, t, 1, nk, 0);
        if (best_us < 0.0 || us < best_us) {
            best_us = us;
            best = plan_pieces(t, bk, M, N, K, 1, 0);
        }
    }
    // Against a slice-K tile a split also pays its second launch's gap on a stream:
    // 27 x 165 with 3571 k in 8 bits took 9.1 us in 14 pieces, 5.0 in slices, where
    // the estimates are 5.2 and 7.3.
    const double margin = slice ? 0.65 : SPLIT_MARGIN;
    best_us *= margin;
    for (const TileCand& t : TILES_T)
        for (int s = 2; s <= MAX_SPLITS && s <= nk; ++s) {
            const Plan p = plan_pieces(t, bk, M, N, K, s, ws_avail);
            if (p.splits != s) continue;
            const double us = estimate_us(in, es_out, M, N, t, s, p.kchunk / bk, p.ldw);
            if (us < best_us) {
                best_us = us;
                best = p;
            }
        }
    best.layout = layout;
    if (us_out) *us_out = best.splits == 1 ? best_us / margin : best_us;
    return best;
}

// At most SKINNY_M rows.
//
// K-contiguous B: strips of 16 columns, never split (a strip of 16 outputs already
// reads whole lines).  16 waves while each strip has a CU to itself; of more strips
// a CU holds several, with 8 waves, or 4 where K is at most 16 steps of 128 bytes
// (e4m3 from HBM, 16 / 8 / 4 waves in us: 1 x 4096 x 4096 5.7 / 5.8 / -, 1 x 14336 x
// 4096 18.1 / 14.0 / 13.6, 1 x 8192 x 8192 17.7 / 15.2 / 15.7, 1 x 60000 x 2048
// - / 29.7 / 22.8).
//
// B stored along the output, unsplit: strips of 32 columns with 16 waves, one to a CU,
// or from more such strips than CUs on 64 with 8 waves (from HBM, us, 32 / 64: 1 x 8192 x
// 2048 11.8 / 12.2, 1 x 9216 x 2048 16.5 / 13.0, 1 x 12288 x 4096 35.0 / 25.2).
//
// Deep K leaves a wave of an unsplit strip many steps one after another, each a round
// of memory latency (1.6 us per 1024 k from HBM where the strips have a CU each), and
// half-line strips waste what HBM delivers.  Given a workspace, K is split over
// workgroups, for a second launch (2.5 us and the partial sums): from K = 2048 on (fp32,
// whose steps are longer, 1536), unless N is more than 2.5 K, where the strips alone keep
// HBM busy.  Strips of 64 columns, or 128 (16-bit) from N = 4096 on, up to 16 pieces of
// at least 256 k and up to 256 workgroups (a few more than that, and some CUs hold two:
// 1 x 5120 x 4096 in 6 / 8 pieces 13.8 / 17.3 us).  A piece has an odd number of 32-k
// steps: with an even one and a power-of-two pitch, all pieces start on the same memory
// channels (1 x 4096 x 14336 in 8 pieces of 56 steps 32.6 us, of 57 steps 24.0).
// The three thresholds are where both plans take the same time.  From a sweep of 18 K
// (512 to 28672), 19 N (100 to 28672) and 1, 4 and 16 rows, in us, B from HBM (enough
// weights in turn) / the same B again, from the last-level cache:
//                         unsplit        split
//    1 x  512 x  2048    9.3 /  4.5     7.6 /  6.2
//    1 x  512 x  4104   15.7 /  6.2     8.0 /  6.5
//   16 x 1024 x  3500   16.6 /  6.5     8.2 /  6.5
//    1 x 2048 x  2048    9.9 /  4.6     7.9 /  6.2
//    1 x 2048 x  4096   16.8 /  6.3     9.3 /  6.8
//    1 x 2048 x  8192   30.1 / 15.2    12.4 /  8.4
//   16 x 3000 x  5000   22.4 / 14.4    12.8 /  9.7
//    1 x 4096 x  2048   10.2 /  4.5     9.6 /  6.5
//    1 x 4096 x  4096   17.5 /  8.7    12.2 /  8.1
//   16 x 4096 x  4096   20.3 / 12.5    13.3 / 10.2
//    1 x 5120 x  5120   29.9 / 18.2    15.0 / 12.8
//    1 x 4096 x 14336   53.2 / 34.0    28.6 / 22.8
//    1 x 8192 x  4096   20.2 / 14.3    19.0 / 15.0
//   16 x 9216 x  4096   25.7 / 16.1    21.0 / 17.4
//   16 x 11008 x 8192   44.4 / 30.6    39.4 / 32.0
//    1 x 14336 x 8192   48.8 / 36.6    49.2 / 37.8
//    1 x 4096 x  1024    6.5 /  3.8     7.5 /  5.6   (unsplit)
//    1 x 11008 x 4096   20.3 / 15.6    21.1 / 18.5   (unsplit)
//   fp32, 16 x 1024 x 1536 11.7 / 8.6, 8.4 / 6.9; 1 x 4096 x 4096 23.2 / 15.8, 19.3 / 15.9;
//    1 x 5120 x 5120 33.5 / 20.8, 25.9 / 21.7; 16 x 8192 x 4096 33.9 / 23.9, 29.7 / 25.7
// Over the sweep (from HBM) the chosen plan takes 1 % more than the fastest one on average,
// 6 % at the 90th percentile, 23 % at most (16 x 28672 x 16384).
Plan plan_skinny(int in, int layout, int M, int N, int K, uint64_t ws_avail) {
    Plan p{SKINNY_M, 16, 1, K, 0, 0};
    p.waves = 16;
    p.kind = PLAN_SKINNY;
    if (layout == LAY_NT) {
        p.layout = LAY_NT;
        if (ceil_div(N, 16) > NUM_CU) p.waves = (int64_t)K * in_esize(in) <= 16 * 128 ? 4 : 8;
        return p;
    }
    auto strips = [&](int cols, int splits) {  // splits = 0 if it does not fit
        Plan q = plan_pieces(TileCand{SKINNY_M, cols, 1, 0, 0, 1, 1}, 32, M, N, K, splits, ws_avail);
        if (q.splits > 1 && q.kchunk % 64 == 0) {  // an odd number of steps
            q.kchunk += 32;
            q.splits = (int)ceil_div(K, q.kchunk);
            q.ws_bytes = (int64_t)q.splits * M * q.ldw * 4;
        }
        q.waves = cols == 32 ? 16 : 8;
        q.kind = PLAN_SKINNY;
        return q;
    };
    int fm, fn, fs;
    const bool f32 = in == IN_F32;
    if (forced_grid(fm, fn, fs) && fm == SKINNY_M && (fn == 32 || fn == 64 || (fn == 128 && !f32))) {
        const Plan q = strips(fn, fs);
        if (q.splits > 0) return q;
    }
    if (K >= (f32 ? 1536 : 2048) && 2 * (int64_t)N <= 5 * (int64_t)K) {
        const int cols = f32 || N < 4096 ? 64 : 128;
        const int s = (int)std::min<int64_t>(std::min(MAX_SPLITS, K / 256), NUM_CU / ceil_div(N, cols));
        if (s >= 2) {
            const Plan q = strips(cols, s);
            if (q.splits > 1) return q;
        }
    }
    return strips(ceil_div(N, 32) > NUM_CU ? 64 : 32, 1);
}

Plan plan_act(int in, int es_out, int M, int N, int K, uint64_t ws_avail) {
    if (in != IN_F32X3 && M > 0 && M <= SKINNY_M && N > 0)
        return plan_skinny(in, LAY_NN, M, N, K, ws_avail);
    return make_plan(in, es_out, M, N, K, ws_avail, false);
}

// fp32 outputs and few rows: the widened products, whose sums are fp32.
int f8_in(int of, int M) { return of == OUT_F32 || M <= SKINNY_M ? IN_F8W : IN_F8; }

Plan plan_f8(int of, int M, int N, int K, uint64_t ws_avail) {
    const int in = f8_in(of, M);
    if (M > 0 && M <= SKINNY_M && N > 0) return plan_skinny(in, LAY_NT, M, N, K, ws_avail);
    return plan_t(in, LAY_NT, out_esize(of), M, N, K, ws_avail);
}

int report(const Plan& p, int* tile_rows, int* tile_cols, int* splits, size_t* used) {
    if (tile_rows) *tile_rows = p.bm;
    if (tile_cols) *tile_cols = p.bn;
    if (splits) *splits = p.splits;
    if (used) *used = (size_t)p.ws_bytes;
    return DGEMM_OK;
}

// ------------------------------------------------- the forward products' call

struct Fwd {
    Mat A, B, C, R, Z, bias, sa, sb;
    int act;
};

int check_fwd(const Fwd& f, const Mat& ws) {
    if (f.R.p && check_mat(f.R) != DGEMM_OK) return check_mat(f.R);
    if (f.Z.p && check_mat(f.Z) != DGEMM_OK) return check_mat(f.Z);
    if (check_vec(f.bias.p, 4) != DGEMM_OK || check_vec(f.sa.p, 4) != DGEMM_OK ||
        check_vec(f.sb.p, 4) != DGEMM_OK || check_vec(ws.p, 16) != DGEMM_OK)
        return DGEMM_ERR_MISALIGNED;
    // R may be C itself (each element is read before it is written), not overlap
    // it in any other way.
    const bool in_place = f.R.p == f.C.p && (f.R.ld == f.C.ld || f.C.rows == 1);
    const Mat none{nullptr, 0, 0, 0, 0};
    const Mat ins[] = {f.A, f.B, in_place ? none : f.R, f.bias, f.sa, f.sb};
    const Mat outs[] = {f.C, f.Z, ws};
    if (any_overlap(outs, 3, ins, 6)) return DGEMM_ERR_ALIAS;
    return DGEMM_OK;
}

EpiArgs epi_of(const Fwd& f) {
    EpiArgs e{};
    e.alpha = 1.0f;
    e.bias = (const float*)f.bias.p;
    e.act = f.act;
    e.res = (const char*)f.R.p;
    e.pre = (char*)f.Z.p;
    e.ldr = (int)f.R.ld;
    e.ldz = (int)f.Z.ld;
    e.scale_a = (const float*)f.sa.p;
    e.scale_b = (const float*)f.sb.p;
    return e;
}

// ---------------------------------------------------------- the backward call

// The pieces of gemm_act_bwd's workspace, in order: dZ (unless dC serves), the
// column sums of dbias, an operand's transpose (fp32), then what the products'
// plans may use.
struct BwdParts {
    bool own_dz;
    int lddz, ldp, chunks, ldt;
    int64_t dz, part, trans, required;
};

BwdParts bwd_parts(int in, int cfmt, int M, int N, int K, int act, bool products, bool dbias) {
    BwdParts b{};
    const int es = in_esize(in);
    const int dfmt = out_format(in, DGEMM_OUT_SAME);
    b.own_dz = products && (act != DGEMM_ACT_NONE || cfmt != dfmt);
    b.lddz = (int)up(N, 16 / es);
    b.ldp = (int)up(N, 4);
    b.chunks = (int)ceil_div(M, act_grad_rows(M, N));
    b.dz = b.own_dz ? up((int64_t)M * b.lddz * es, WS_ALIGN) : 0;
    // One chunk's column sums are dbias itself.
    b.part = dbias && b.chunks != 1 ? up((int64_t)b.chunks * b.ldp * 4, WS_ALIGN) : 0;
    if (products && es == 4 && M > SKINNY_M)
        b.trans = up(std::max((int64_t)N * up(K, 4), (int64_t)K * up(M, 4)) * 4, WS_ALIGN);
    b.required = b.dz + b.part + b.trans;
    return b;
}

// The product of a backward pass over `rows` rows, M x N with K terms per sum.
// Few rows: B once through registers for dA, a rank-`rows` update for dB (fp32
// arithmetic for 3 x bf16 too).
Plan plan_bwd(int in, int layout, int rows, int M, int N, int K, uint64_t ws) {
    if (rows <= SKINNY_M && M > 0 && N > 0) {
        if (layout == LAY_NT) return plan_skinny(in, LAY_NT, M, N, K, 0);
        Plan p{32, 512, 1, K, 0, 0};
        p.kind = PLAN_SKINNY;
        p.layout = LAY_TN;
        return p;
    }
    if (in == IN_BF16 || in == IN_F16) return plan_t(in, layout, 2, M, N, K, ws);
    return make_plan(in, 4, M, N, K, ws, false);
}

int run_bwd_product(int in, int layout, int rows, int M, int N, int K, const void* X, int ldx, const void* Y,
                    int ldy, const Mat& out, char* ws, int64_t ws_bytes, hipStream_t stream) {
    if (out.empty()) return DGEMM_OK;
    const Plan p = plan_bwd(in, layout, rows, M, N, K, (uint64_t)ws_bytes);
    EpiArgs e{};
    e.alpha = 1.0f;
    // The kernels of transposed layouts store through the full epilogue's row segments.
    return run(p.kind == PLAN_SKINNY && in == IN_F32X3 ? IN_F32 : in, out_format(in, DGEMM_OUT_SAME), M,
               N, K, X, ldx, Y, ldy, (void*)out.p, (int)out.ld, e,
               p.layout != LAY_NN ? EPI_FULL : EPI_NONE, p, ws, stream);
}

constexpr double PAIR_GAP_US = 2.0;          // another launch
// Most tiles: more are the 16-bit grid's (1500^3: 45 us, together 50); fp32's
// grid kernels are slower than the pair's 64 x 64 tiles at many odd sizes
// (1500^3 181 / 155 us, 3500^3 1748 / 1487), so there the estimate decides.
constexpr int64_t PAIR_TILES_16 = 4 * NUM_CU, PAIR_TILES_32 = 32 * NUM_CU;

// A product of the backward pass by itself, M x N with K terms; in fp32 with the
// launch that transposes an operand.
double alone_us(int in, int layout, int M, int N, int K, uint64_t ws) {
    double us = 0.0;
    if (in_esize(in) == 2) {
        plan_t(in, layout, 2, M, N, K, ws, &us);
        return us;
    }
    const double transposed = (double)K * (layout == LAY_NT ? N : M) * 8.0 / 4e6;
    return PAIR_GAP_US + transposed + plan_us(in, 4, make_plan(in, 4, M, N, K, ws, false), M, N, K);
}

Plan slice4(int layout, int ts, int K) {
    Plan p{ts, ts, 1, K, 0, 0};
    p.waves = 4;
    p.layout = layout;
    return p;
}

// The plans of a small backward pass's two products in one launch of slice-K
// tiles (with its column sums): tile sizes, which product's workgroups come first,
// and whether it is worth it.
struct PairPlan {
    Plan nt, tn;
    bool use, tn_first;
};

// A CU holds one of these workgroups (128 KB of LDS), and each starts where one
// ended.  `ta` tiles of `wa` us, then `tb` of `wb`: after the first product
// ta % 256 CUs are one tile later than the others.
double pair_us(int64_t ta, double wa, int64_t tb, double wb) {
    const int64_t late = ta % NUM_CU, q = ta / NUM_CU;
    const double done = (double)ceil_div(ta, NUM_CU) * wa;
    int64_t left = tb;
    int64_t i = 0, j = 0;  // tiles so far on each early and each late CU
    double t = done;
    while (left > 0) {
        const double e = (double)q * wa + (double)(i + 1) * wb;
        const double l = (double)(q + 1) * wa + (double)(j + 1) * wb;
        const bool early = late == 0 || e <= l;
        left -= early ? NUM_CU - late : late;
        (early ? i : j) += 1;
        t = std::max(t, early ? e : l);
    }
    return t;
}

// `ta` grid tiles of ka terms and `tb` of kb, one workgroup of 256 x 256 per CU or
// two of 128 x 128, in estimate_us's terms.  256 x 256: the schedule above, faster
// where it leaves CUs idle (a half-filled chip clocks higher: a step 1.2 us, not
// 1.7).  128 x 128: the work at the rate of shared CUs, and a tail where the last
// round is not full, or the longest tile.  Within 15 % of 18 layers from 600 x 800 x 3000 to 5000^3.
double pair_grid_us(const TileCand& t, int in, int64_t ta, int ka, int64_t tb, int kb, bool& b_first) {
    const double step = step_us(in) * t.bm * t.bn / 65536.0 / t.eff;
    const double wa = (double)ceil_div(ka, t_step(in)) * step + 1.0;
    const double wb = (double)ceil_div(kb, t_step(in)) * step + 1.0;
    const double work = ((double)ta * wa + (double)tb * wb) / NUM_CU;
    b_first = wb > wa;
    if (t.pair2 > 0.0) {
        const double rounds = (double)(ta + tb) / (2 * NUM_CU);
        const double tail = (std::ceil(rounds) - rounds) * std::min(wa, wb);
        return std::max((work * 1.05 + tail) * t.pair2 / 2, std::max(wa, wb) * 1.05);
    }
    const double us = b_first ? pair_us(tb, wb, ta, wa) : pair_us(ta, wa, tb, wb);
    return us * (0.7 + 0.3 * work / us);
}

// One launch saves the other launches' time (2.4 us of host time each, 1.5 to 2 us
// of a graph) and fills the CUs that one product's tiles leave idle; the longer
// tiles go first.  The whole backward pass in us, M x N x K, apart / together:
//   bf16   256 x  256 x  256    14.9 /   8.2   (slice-K tiles)
//          917 x  415 x 1035    24.4 /  15.1   (slice-K)
//          600 x  800 x 3000    29.8 /  19.7   (128 x 128)
//         1024 x 2048 x 2048    43.8 /  33.2   (128 x 128)
//         2048 x 4096 x 4096     154 /   129   (256 x 256)
//         4096 x 4096 x 4096     251 /   241   (256 x 256)
//         5000 x 5000 x 5000     551 /   541   (256 x 256)
//   fp32   256^3 20.9 / 7.7, 917 x 415 x 1035 47.0 / 30.8, 1024^3 69 / 51
PairPlan plan_pair(int in, int M, int N, int K, bool dA, bool dB, bool sums, uint64_t ws) {
    PairPlan r{};
    const int f = in_esize(in) == 4 ? IN_F32 : IN_BF16;  // 3 x bf16 in fp32 arithmetic here
    int fm, fn, fs;
    const bool forced = forced_grid(fm, fn, fs);
    const bool tile = forced && fm == fn && (fm == 32 || fm == 64) && (fs == 1 || fs == 4);
    const bool grid = forced && fm == fn && (fm == 128 || fm == 256) && fs == 1 && f == IN_BF16 && dA && dB;
    if (forced && !tile && !grid) return r;
    double best = (double)((dA ? 1 : 0) + (dB ? 1 : 0) + (sums ? 1 : 0) - 1) * PAIR_GAP_US;
    if (dA) best += alone_us(in, LAY_NT, M, K, N, ws);
    if (dB) best += alone_us(in, LAY_TN, K, N, M, ws);
    for (int a = 32; a <= 64 && !grid; a += 32)
        for (int b = 32; b <= 64; b += 32) {
            if ((!dA && a > 32) || (!dB && b > 32) || (tile && ((dA && a != fm) || (dB && b != fm)))) continue;
            const int64_t ta = dA ? ceil_div(M, a) * ceil_div(K, a) : 0;
            const int64_t tb = dB ? ceil_div(K, b) * ceil_div(N, b) : 0;
            if (ta + tb > (tile ? (int64_t)INT32_MAX / 2 : f == IN_F32 ? PAIR_TILES_32 : PAIR_TILES_16)) continue;
            const double wa = slice_tile_us(f, a, N), wb = slice_tile_us(f, b, M);
            const double fwd = pair_us(ta, wa, tb, wb), rev = pair_us(tb, wb, ta, wa);
            if (!tile && std::min(fwd, rev) >= best) continue;
            best = std::min(fwd, rev);
            r.use = true;
            r.tn_first = rev < fwd;
            r.nt = slice4(LAY_NT, a, N);
            r.tn = slice4(LAY_TN, b, M);
        }
    if (f == IN_F32 || !dA || !dB || tile) return r;
    for (const TileCand& t : TILES_T) {
        if (grid && t.bm != fm) continue;
        const int64_t ta = ceil_div(M, t.bm) * ceil_div(K, t.bn), tb = ceil_div(K, t.bm) * ceil_div(N, t.bn);
        if (ta + tb > INT32_MAX / 2) continue;
        bool tn_first;
        const double us = pair_grid_us(t, in, ta, N, tb, M, tn_first);
        if (!grid && us >= best) continue;
        best = us;
        r.use = true;
        r.tn_first = tn_first;
        r.nt = Plan{t.bm, t.bn, 1, N, 0, 0};
        r.tn = Plan{t.bm, t.bn, 1, M, 0, 0};
        r.nt.layout = LAY_NT;
        r.tn.layout = LAY_TN;
    }
    return r;
}

GemmLaunch pair_launch(int in, const Plan& p, int M, int N, int K, const void* X, int ldx, const void* Y,
                        int ldy, void* C, int ldc, hipStream_t stream) {
    GemmLaunch L{};
    L.in = in == IN_F32X3 ? IN_F32 : in;
    L.out = out_format(in, DGEMM_OUT_SAME);
    L.tbm = p.bm;
    L.tbn = p.bn;
    L.layout = p.layout;
    L.slice_waves = p.waves;
    L.splits = 1;
    L.epi = EPI_FULL;
    L.A = (const char*)X;
    L.B = (const char*)Y;
    L.C = (char*)C;
    L.M = M;
    L.N = N;
    L.K = K;
    L.lda = ldx;
    L.ldb = ldy;
    L.ldc = ldc;
    L.tiles_m = (int)ceil_div(M, p.bm);
    L.tiles_n = (int)ceil_div(N, p.bn);
    L.stream = stream;
    return L;
}

int launched(hipError_t e) { return e == hipSuccess ? DGEMM_OK : DGEMM_ERR_LAUNCH; }

// Format codes DGEMM_IN_F32 / _BF16 / _F16 of an elementwise operator.
int row_fmt(int in) {
    return in == DGEMM_IN_F32 ? OUT_F32 : in == DGEMM_IN_BF16 ? OUT_BF16 : in == DGEMM_IN_F16 ? OUT_F16 : -1;
}

}  // namespace
}  // namespace dgemm

using namespace dgemm;

extern "C" {

int gemm_act(int in, int out, int M, int N, int K, const void* A, int lda, const void* B, int ldb,
             void* C, int ldc, const float* bias, int act, const void* R, int ldr, void* Z, int ldz,
             void* workspace, size_t workspace_bytes, void* stream) {
    if (in < IN_F32 || in > IN_F32X3) return DGEMM_ERR_INVALID_VALUE;
    const int of = out_format(in, out);
    if (of < 0 || !valid_act(act) || (workspace_bytes > 0 && !workspace)) return DGEMM_ERR_INVALID_VALUE;
    const int eo = out_esize(of), es = in_esize(in);
    int st = validate(M, N, K, A, lda, B, ldb, C, ldc, in, eo);
    if (st != DGEMM_OK) return st;
    if (M == 0 || N == 0) return DGEMM_OK;
    const Plan p = plan_act(in, eo, M, N, K, workspace ? workspace_bytes : 0);
    const Fwd f{{A, M, K, lda, es}, {B, K, N, ldb, es}, {C, M, N, ldc, eo}, {R, M, N, ldr, eo},
                {Z, M, N, ldz, eo}, vec(bias, N), vec(nullptr, 0), vec(nullptr, 0), act};
    st = check_fwd(f, bytes_of(workspace, p.ws_bytes));
    if (st != DGEMM_OK) return st;
    st = check_device();
    if (st != DGEMM_OK) return st;
    return run(in, of, M, N, K, A, lda, B, ldb, C, ldc, epi_of(f), EPI_FULL, p, workspace,
               (hipStream_t)stream);
}

int gemm_act_plan(int in, int out, int M, int N, int K, size_t workspace_bytes, int* tile_rows,
                  int* tile_cols, int* splits, size_t* workspace_used) {
    if (in < IN_F32 || in > IN_F32X3 || M < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    const int of = out_format(in, out);
    if (of < 0) return DGEMM_ERR_INVALID_VALUE;
    if (ceil_div(M, 128) * ceil_div(N, 128) > INT32_MAX) return DGEMM_ERR_TOO_LARGE;
    return report(plan_act(in, out_esize(of), M, N, K, workspace_bytes), tile_rows, tile_cols, splits,
                  workspace_used);
}

int gemm_act_bwd(int in, int out, int M, int N, int K, const void* A, int lda, const void* B, int ldb,
                 const void* dC, int lddc, const void* Z, int ldz, int act, void* dA, int ldda,
                 void* dB, int lddb, float* dbias, void* workspace, size_t workspace_bytes,
                 void* stream) {
    if (in < IN_F32 || in > IN_F32X3 || M < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    const int cf = out_format(in, out);
    if (cf < 0 || !valid_act(act) || (workspace_bytes > 0 && !workspace)) return DGEMM_ERR_INVALID_VALUE;
    const int es = in_esize(in), ec = out_esize(cf);
    const bool use_z = act != DGEMM_ACT_NONE;
    const Mat mA{A, dB ? M : 0, K, lda, es}, mB{B, dA ? K : 0, N, ldb, es}, mdC{dC, M, N, lddc, ec};
    const Mat mZ{use_z ? Z : nullptr, use_z ? M : 0, N, ldz, ec};
    const Mat mdA{dA, dA ? M : 0, K, ldda, es}, mdB{dB, dB ? K : 0, N, lddb, es};
    int st;
    if (dB && (st = check_mat(mA)) != DGEMM_OK) return st;
    if (dA && (st = check_mat(mB)) != DGEMM_OK) return st;
    if ((st = check_mat(mdC)) != DGEMM_OK) return st;
    if (use_z && (st = check_mat(mZ)) != DGEMM_OK) return st;
    if (dA && (st = check_mat(mdA)) != DGEMM_OK) return st;
    if (dB && (st = check_mat(mdB)) != DGEMM_OK) return st;
    if (check_vec(dbias, 4) != DGEMM_OK || check_vec(workspace, 16) != DGEMM_OK) return DGEMM_ERR_MISALIGNED;
    const BwdParts b = bwd_parts(in, cf, M, N, K, act, dA || dB, dbias != nullptr);
    if ((uint64_t)b.required > workspace_bytes) return DGEMM_ERR_WORKSPACE;
    // The products address the workspace's matrices in panels too.  dZ's rows are no longer
    // than dC's and those of B's transpose (fp32) no longer than dA's, which are checked; those
    // of A's transpose, for dB, are as long as M.
    if (es == 4 && dB && M > SKINNY_M && (int64_t)PANEL_ROWS * up(M, 4) * 4 >= DESC_LIMIT)
        return DGEMM_ERR_TOO_LARGE;
    const Mat ws = bytes_of(workspace, (int64_t)std::min<uint64_t>(workspace_bytes, INT64_MAX));
    const Mat ins[] = {mA, mB, mdC, mZ}, outs[] = {mdA, mdB, vec(dbias, N), ws};
    if (any_overlap(outs, 4, ins, 4)) return DGEMM_ERR_ALIAS;
    if ((st = check_device()) != DGEMM_OK) return st;

    char* const w = (char*)workspace;
    char* const w_part = w + b.dz;
    float* const w_trans = (float*)(w + b.dz + b.part);
    char* const w_gemm = w + b.required;
    const int64_t gemm_bytes = (int64_t)workspace_bytes - b.required;
    hipStream_t s = (hipStream_t)stream;
    const void* dz = dC;
    int lddz = lddc;
    if (b.own_dz) {
        dz = w;
        lddz = b.lddz;
    }
    if (M > 0 && N > 0 && (b.own_dz || dbias)) {
        const ActGradArgs a{(const char*)dC, (const char*)mZ.p, b.own_dz ? w : nullptr,
                            !dbias ? nullptr : b.chunks == 1 ? dbias : (float*)w_part, M, N, lddc, ldz, b.lddz, b.ldp,
                            act_grad_rows(M, N), act};
        if (launch_act_grad(a, cf, out_format(in, DGEMM_OUT_SAME), s) != hipSuccess)
            return DGEMM_ERR_LAUNCH;
    }
    ColReduceArgs sums{(const float*)w_part, dbias, b.chunks, b.ldp, dbias && b.chunks != 1 ? N : 0};
    if ((dA || dB) && M > SKINNY_M && N > 0 && K > 0) {
        // The products and the column sums in one launch where that is faster.
        const PairPlan p = plan_pair(in, M, N, K, dA, dB, sums.N > 0, (uint64_t)gemm_bytes);
        if (p.use) {
            GemmLaunch nt = pair_launch(in, p.nt, M, K, N, dz, lddz, B, ldb, dA, ldda, s);
            GemmLaunch tn = pair_launch(in, p.tn, K, N, M, A, lda, dz, lddz, dB, lddb, s);
            if (!dA) nt.tiles_m = 0;
            if (!dB) tn.tiles_m = 0;
            return launched((p.nt.waves > 0 ? launch_slicet_pair : launch_gemmt_pair)(nt, tn, p.tn_first, sums));
        }
    }
    if (sums.N > 0 && launch_col_reduce(sums, s) != hipSuccess) return DGEMM_ERR_LAUNCH;
    const bool f32 = es == 4 && M > SKINNY_M;  // the fp32 kernels take A[M x K] B[K x N] only
    if (dA) {
        const void* y = B;
        int ldy = ldb;
        if (f32 && !mB.empty() && M > 0) {
            ldy = (int)up(K, 4);
            if (launch_transpose32((const float*)B, ldb, K, N, w_trans, ldy, s) != hipSuccess)
                return DGEMM_ERR_LAUNCH;
            y = w_trans;
        }
        st = run_bwd_product(in, LAY_NT, M, M, K, N, dz, lddz, y, ldy, mdA, w_gemm, gemm_bytes, s);
        if (st != DGEMM_OK) return st;
    }
    if (dB) {
        const void* x = A;
        int ldx = lda;
        if (f32 && !mA.empty() && N > 0) {
            ldx = (int)up(M, 4);
            if (launch_transpose32((const float*)A, lda, M, K, w_trans, ldx, s) != hipSuccess)
                return DGEMM_ERR_LAUNCH;
            x = w_trans;
        }
        st = run_bwd_product(in, LAY_TN, M, K, N, M, x, ldx, dz, lddz, mdB, w_gemm, gemm_bytes, s);
        if (st != DGEMM_OK) return st;
    }
    return DGEMM_OK;
}

int gemm_act_bwd_workspace(int in, int out, int M, int N, int K, int act, size_t* required,
                           size_t* best) {
    if (in < IN_F32 || in > IN_F32X3 || M < 0 || N < 0 || K < 0 || !valid_act(act))
        return DGEMM_ERR_INVALID_VALUE;
    const int cf = out_format(in, out);
    if (cf < 0) return DGEMM_ERR_INVALID_VALUE;
    const BwdParts b = bwd_parts(in, cf, M, N, K, act, true, true);
    int64_t more = 0;
    const uint64_t any = (uint64_t)1 << 40;
    if (M > 0 && K > 0) more = std::max(more, plan_bwd(in, LAY_NT, M, M, K, N, any).ws_bytes);
    if (K > 0 && N > 0) more = std::max(more, plan_bwd(in, LAY_TN, M, K, N, M, any).ws_bytes);
    if (required) *required = (size_t)b.required;
    if (best) *best = (size_t)(b.required + more);
    return DGEMM_OK;
}

int gemm_f8(int out, int M, int N, int K, const void* A, int lda, const void* B, int ldb, void* C,
            int ldc, const float* scale_a, const float* scale_b, const float* bias, int act,
            const void* R, int ldr, void* workspace, size_t workspace_bytes, void* stream) {
    const int of = row_fmt(out);
    if (of < 0 || M < 0 || N < 0 || K < 0 || !valid_act(act) || (workspace_bytes > 0 && !workspace))
        return DGEMM_ERR_INVALID_VALUE;
    const int eo = out_esize(of);
    const bool reads = M > 0 && N > 0;
    const Fwd f{{A, reads ? M : 0, K, lda, 1}, {B, reads ? N : 0, K, ldb, 1}, {C, M, N, ldc, eo},
                {R, M, N, ldr, eo}, {nullptr, 0, 0, 0, eo}, vec(bias, N), vec(scale_a, M),
                vec(scale_b, N), act};
    int st;
    if ((st = check_mat(f.A)) != DGEMM_OK || (st = check_mat(f.B)) != DGEMM_OK ||
        (st = check_mat(f.C)) != DGEMM_OK)
        return st;
    if (!reads) return DGEMM_OK;
    if (!scale_a || !scale_b) return DGEMM_ERR_INVALID_VALUE;
    const Plan p = plan_f8(of, M, N, K, workspace ? workspace_bytes : 0);
    if ((st = check_fwd(f, bytes_of(workspace, p.ws_bytes))) != DGEMM_OK) return st;
    if ((st = check_device()) != DGEMM_OK) return st;
    return run(f8_in(of, M), of, M, N, K, A, lda, B, ldb, C, ldc, epi_of(f), EPI_FULL, p, workspace,
               (hipStream_t)stream);
}

int gemm_f8_plan(int out, int M, int N, int K, size_t workspace_bytes, int* tile_rows, int* tile_cols,
                 int* splits, size_t* workspace_used) {
    const int of = row_fmt(out);
    if (of < 0 || M < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    if (ceil_div(M, 128) * ceil_div(N, 128) > INT32_MAX) return DGEMM_ERR_TOO_LARGE;
    return report(plan_f8(of, M, N, K, workspace_bytes), tile_rows, tile_cols, splits,
                  workspace_used);
}

int rmsnorm(int in, int out, int M, int N, const void* X, int ldx, const void* R, int ldr, void* S,
            int lds, const float* weight, float eps, void* Y, int ldy, float* scale, float* rstd,
            void* stream) {
    const int fmt = row_fmt(in);
    if (fmt < 0 || M < 0 || N < 0 || !(eps >= 0.0f) || (out != DGEMM_ROWS_SAME && out != DGEMM_ROWS_F8))
        return DGEMM_ERR_INVALID_VALUE;
    const bool f8 = out == DGEMM_ROWS_F8;
    const int es = out_esize(fmt);
    const Mat mX{X, M, N, ldx, es}, mR{R, M, N, ldr, es}, mS{S, M, N, lds, es}, mY{Y, M, N, ldy, f8 ? 1 : es};
    int st;
    if ((st = check_mat(mX)) != DGEMM_OK || (st = check_mat(mY)) != DGEMM_OK) return st;
    if (R && (st = check_mat(mR)) != DGEMM_OK) return st;
    if (S && (st = check_mat(mS)) != DGEMM_OK) return st;
    if (M == 0 || N == 0) return DGEMM_OK;
    if (!weight || (f8 && !scale) || (!f8 && scale)) return DGEMM_ERR_INVALID_VALUE;
    if (N > ROW_MAX) return DGEMM_ERR_TOO_LARGE;
    if (check_vec(weight, 16) != DGEMM_OK || check_vec(scale, 4) != DGEMM_OK || check_vec(rstd, 4) != DGEMM_OK)
        return DGEMM_ERR_MISALIGNED;
    // S and Y may each be X or R themselves (a row is read before it is written;
    // for Y only in X's format), and share nothing else with the inputs.
    const auto same = [&](const Mat& o, const Mat& i) {
        return o.p == i.p && o.es == i.es && (o.ld == i.ld || M == 1);
    };
    const Mat none{nullptr, 0, 0, 0, 0};
    const Mat outs[] = {mS, mY, vec(scale, M), vec(rstd, M)};
    if (any_overlap(outs, 4, nullptr, 0)) return DGEMM_ERR_ALIAS;
    for (const Mat& o : outs) {
        const bool whole = o.p && o.cols == N && o.rows == M && (o.p == S || o.p == Y);
        const Mat ins[] = {whole && same(o, mX) ? none : mX, R ? (whole && same(o, mR) ? none : mR) : none,
                           vec(weight, N)};
        if (any_overlap(&o, 1, ins, 3)) return DGEMM_ERR_ALIAS;
    }
    if ((st = check_device()) != DGEMM_OK) return st;
    const RowArgs a{(const char*)X, (const char*)R, (char*)S, weight, (char*)Y, scale, rstd, eps, M, N,
                    ldx, ldr, lds, ldy};
    return launched(launch_rows(a, fmt, true, f8, (hipStream_t)stream));
}

int rmsnorm_bwd(int in, int M, int N, const void* dY, int lddy, const void* S, int lds,
                const float* weight, const float* rstd, const void* dS, int ldds, void* dX, int lddx,
                float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    const int fmt = row_fmt(in);
    if (fmt < 0 || M < 0 || N < 0 || (workspace_bytes > 0 && !workspace)) return DGEMM_ERR_INVALID_VALUE;
    const int es = out_esize(fmt);
    const Mat mdY{dY, M, N, lddy, es}, mS{S, M, N, lds, es}, mdS{dS, M, N, ldds, es}, mdX{dX, M, N, lddx, es};
    int st;
    if ((st = check_mat(mdY)) != DGEMM_OK || (st = check_mat(mS)) != DGEMM_OK ||
        (st = check_mat(mdX)) != DGEMM_OK)
        return st;
    if (dS && (st = check_mat(mdS)) != DGEMM_OK) return st;
    if (N == 0 || (M == 0 && !dweight)) return DGEMM_OK;
    if (M > 0 && (!weight || !rstd)) return DGEMM_ERR_INVALID_VALUE;
    if (N > NORM_BWD_MAX) return DGEMM_ERR_TOO_LARGE;
    if (check_vec(weight, 16) != DGEMM_OK || check_vec(rstd, 4) != DGEMM_OK ||
        check_vec(dweight, 4) != DGEMM_OK || check_vec(workspace, 16) != DGEMM_OK)
        return DGEMM_ERR_MISALIGNED;
    const int grid = norm_bwd_grid(M, N), ldp = (int)up(N, 4);
    const int64_t need = dweight ? (int64_t)grid * ldp * 4 : 0;
    if ((uint64_t)need > workspace_bytes) return DGEMM_ERR_WORKSPACE;
    // dX may be dY or dS itself (a row is read before it is written).
    const auto same = [&](const Mat& i) { return mdX.p == i.p && (mdX.ld == i.ld || M == 1); };
    const Mat none{nullptr, 0, 0, 0, 0};
    const Mat ws = bytes_of(workspace, need);
    const Mat out_x[] = {mdX}, in_x[] = {same(mdY) ? none : mdY, mS, dS ? (same(mdS) ? none : mdS) : none,
                                         vec(weight, N), vec(rstd, M), vec(dweight, N), ws};
    const Mat out_w[] = {vec(dweight, N), ws};
    const Mat in_w[] = {mdY, mS, dS ? mdS : none, vec(weight, N), vec(rstd, M)};
    if (any_overlap(out_x, 1, in_x, 7) || any_overlap(out_w, 2, in_w, 5)) return DGEMM_ERR_ALIAS;
    if ((st = check_device()) != DGEMM_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    const NormBwdArgs a{(const char*)dY, (const char*)S, (const char*)dS, weight, rstd, (char*)dX,
                        dweight ? (float*)workspace : nullptr, M, N, lddy, lds, ldds, lddx, ldp};
    if (M > 0 && launch_norm_bwd(a, fmt, s) != hipSuccess) return DGEMM_ERR_LAUNCH;
    if (dweight) return launched(launch_col_reduce(ColReduceArgs{(const float*)workspace, dweight, grid, ldp, N}, s));
    return DGEMM_OK;
}

int rmsnorm_bwd_workspace(int M, int N, size_t* required) {
    if (M < 0 || N < 0) return DGEMM_ERR_INVALID_VALUE;
    if (N > NORM_BWD_MAX) return DGEMM_ERR_TOO_LARGE;
    if (required) *required = (size_t)norm_bwd_grid(M, N) * (size_t)up(N, 4) * 4;
    return DGEMM_OK;
}

int quant_f8(int in, int transpose, int M, int N, const void* X, int ldx, void* Q, int ldq,
             float* scale, void* stream) {
    const int fmt = row_fmt(in);
    if (fmt < 0 || M < 0 || N < 0 || (transpose != 0 && transpose != 1)) return DGEMM_ERR_INVALID_VALUE;
    const Mat mX{X, M, N, ldx, out_esize(fmt)};
    const Mat mQ{Q, transpose ? N : M, transpose ? M : N, ldq, 1};
    int st;
    if ((st = check_mat(mX)) != DGEMM_OK || (st = check_mat(mQ)) != DGEMM_OK) return st;
    // Rows (columns) without elements still have a scale, that of an empty maximum.
    if ((transpose ? N : M) == 0) return DGEMM_OK;
    if (!scale) return DGEMM_ERR_INVALID_VALUE;
    if (!transpose && N > ROW_MAX) return DGEMM_ERR_TOO_LARGE;
    if (check_vec(scale, 4) != DGEMM_OK) return DGEMM_ERR_MISALIGNED;
    const Mat ins[] = {mX}, outs[] = {mQ, vec(scale, transpose ? N : M)};
    if (any_overlap(outs, 2, ins, 1)) return DGEMM_ERR_ALIAS;
    if ((st = check_device()) != DGEMM_OK) return st;
    RowArgs a{};
    a.X = (const char*)X;
    a.Y = (char*)Q;
    a.scale = scale;
    a.M = M;
    a.N = N;
    a.ldx = ldx;
    a.ldy = ldq;
    if (transpose) return launched(launch_quant_cols(a, fmt, (hipStream_t)stream));
    return launched(launch_rows(a, fmt, false, true, (hipStream_t)stream));
}

}  // extern "C"
