// feedforward.hip -- the C ABI of a feed-forward block's operators beside linear.hip's:
// layer norms and their gradients (layernorm, layernorm_bwd), products of 8-bit operands with
// a scale per block and the quantizer of those (gemm_f8_block, quant_f8_block).  Host code
// only: validation, plans and launches.

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

// fp32 outputs and few rows: the widened products, whose sums are fp32.
int block_in(int of, int M) { return of == OUT_F32 || M <= SKINNY_M ? IN_F8W : IN_F8; }

Plan plan_block(int of, int rows_b, int M, int N, int K, uint64_t ws) {
    const int in = block_in(of, M);
    if (M > 0 && M <= SKINNY_M && N > 0) return plan_skinny(in, LAY_NT, M, N, K, 0);
    return plan_t(in, LAY_NT, out_esize(of), M, N, K, ws, nullptr, in == IN_F8 && rows_b != 1);
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
    return report(plan_block(of, rows_b, M, N, K, workspace_bytes), tile_rows, tile_cols, splits, workspace_used);
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
    const int grid = norm_bwd_grid(M, N), ldp = (int)up(N, 4);
    const int64_t need = sums ? (int64_t)grid * 2 * ldp * 4 : 0;
    if ((uint64_t)need > workspace_bytes) return DGEMM_ERR_WORKSPACE;
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
    if (required) *required = (size_t)norm_bwd_grid(M, N) * 2 * (size_t)up(N, 4) * 4;
    return DGEMM_OK;
}

}  // extern "C"
