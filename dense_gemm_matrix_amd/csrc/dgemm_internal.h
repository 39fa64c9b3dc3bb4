// dgemm_internal.h -- what the library's translation units share: format
// codes, the workgroup -> tile map, the epilogue arguments, and one launch
// description per kernel family.  Host-visible; no device code.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace dgemm {

enum InFmt { IN_F32 = 0, IN_BF16 = 1, IN_F16 = 2, IN_F32X3 = 3,  // F32X3: fp32 via 3 x bf16
             // e4m3 (gemm_f8): on the 8-bit matrix instructions, and with the values
             // widened to bf16 for the fp32 accumulation of fp32 outputs
             IN_F8 = 4, IN_F8W = 5 };
enum OutFmt { OUT_F32 = 0, OUT_BF16 = 1, OUT_F16 = 2 };

constexpr int NTHREADS = 256;   // 4 waves: the fp32 kernels' workgroup
constexpr int GROUP_M = 4;      // tile rows per strip in the tile walk
constexpr int NUM_XCD = 8;      // XCDs that workgroups are dealt across
constexpr int NUM_CU = 256;     // compute units of an MI355X

inline int in_esize(int in) { return (in == IN_F32 || in == IN_F32X3) ? 4 : in >= IN_F8 ? 1 : 2; }
inline int out_esize(int out) { return out == OUT_F32 ? 4 : 2; }

// Workgroup -> output tile.  Step 1: workgroups are dealt to XCDs in turn, so
// wg % 8 is its XCD; give XCD x the contiguous run of tile indices
// [start_x, start_x + count_x), runs sized as evenly as possible.  Step 2: walk
// tile indices in strips GROUP_M tile-rows high, column by column, so a run of
// ~32 tiles covers a compact block (4 x 8 at 4096 x 4096).  Both steps are
// bijections for any tile counts (the last strip may be shorter).
__host__ __device__ inline void map_tile(int wg, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int ntiles = tiles_m * tiles_n;
    const int x = wg % NUM_XCD;
    const int local = wg / NUM_XCD;
    const int q = ntiles / NUM_XCD;
    const int r = ntiles % NUM_XCD;
    const int t = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + local;
    const int per_strip = GROUP_M * tiles_n;
    const int strip = t / per_strip;
    const int first_m = strip * GROUP_M;
    const int rows_in_strip = (tiles_m - first_m) < GROUP_M ? (tiles_m - first_m) : GROUP_M;
    const int rem = t - strip * per_strip;
    tm = first_m + rem % rows_in_strip;
    tn = rem / rows_in_strip;
}

// Epilogue levels of the GEMM kernels.
//   EPI_BASIC (gemm_ex): C := relu(alpha * acc + beta * C_old + bias[col]).
//     C_old is read only when beta != 0; bias may be NULL; relu != 0 clamps
//     negatives to 0.
//   EPI_FULL (gemm_act, gemm_f8): z := acc * scale_a[row] * scale_b[col] +
//     bias[col]; Z := z; C := act(z) + R.  The scales, bias, Z and R may be
//     NULL; Z and R have C's format.
enum EpiLevel { EPI_NONE = 0, EPI_BASIC = 1, EPI_FULL = 2 };

struct EpiArgs {
    float alpha;
    float beta;
    const float* bias;
    int relu;
    // EPI_FULL only
    int act;               // a dgemm_act code
    const char* res;       // R, row pitch ldr
    char* pre;             // Z, row pitch ldz
    int ldr, ldz;
    const float* scale_a;  // both or neither
    const float* scale_b;
};

// dgemm_act codes, for the device code.
enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// How the operands lie in memory: A[M x K] B[K x N]; A[M x K] B[N x K] (both
// K-contiguous); A[K x M] B[K x N].
enum Layout { LAY_NN = 0, LAY_NT = 1, LAY_TN = 2 };

// Column sums: out[n] = sum over g < G of part[g * ldp + n], n < N.
struct ColReduceArgs {
    const float* part;
    float* out;
    int G, ldp, N;
};
inline int col_reduce_blocks(int N) { return (N + 15) / 16; }

// One GEMM launch.  The grid is (tiles_m * tiles_n, splits): workgroup
// (x, z) computes tile map_tile(x) over k in [z * kchunk, min(K, (z + 1) *
// kchunk)) and writes it at C + z * c_zstride bytes.  Unsplit launches have
// splits = 1 and kchunk = K.
struct GemmLaunch {
    int in, out, tbm, tbn;
    int layout;  // a Layout; the transposed ones are gemmt.hip's
    int stages;  // LDS stages of the 16-bit kernel's 128 x 128 tile (2, or 4 alone on a CU)
    int slice_waves;  // waves per workgroup of a slice-K launch (0: a grid launch)
    int epi;     // the EpiLevel at which the kernel applies `e` (only with splits == 1)
    const char* A;
    const char* B;
    char* C;
    int M, N, K, lda, ldb, ldc;
    int tiles_m, tiles_n, splits, kchunk;
    int64_t c_zstride;
    EpiArgs e;
    hipStream_t stream;
};

// ------------------------------------------------------------------ Stream-K
//
// The nine-levels tutorial's section 2.9 names Stream-K as the refinement of
// Split-K that gives every thread block the same amount of work.  Here, for
// grids of at most one 256 x 256 tile per CU (the 16-bit kernel's tile), a
// persistent grid of G workgroups (G a multiple of the 8 XCDs, one per CU):
// the tiles map_tile gives XCD x (tile walk positions x + 8 u, u < n_x) are
// laid end to end as W = n_x nk iterations (one iteration = one 64-k step of
// one tile), and XCD x's R = G / 8 workgroups (b = x + 8 j, rank j) take
// consecutive runs of equal length: rank j covers [floor(j W / R),
// floor((j + 1) W / R)).  The host keeps n_x <= R (so a run is at most nk
// iterations long and touches at most two tiles) and W >= R (so no run is
// empty).
//
// A rank computes the pieces of its run (one or two: the k range it holds of
// each tile it touches) into fp32 partial-tile slots, then publishes them with
// one flag.  Each tile is then reduced by all of its contributors together:
// the tile's 64 blocks of 32 x 32 outputs are dealt out in equal runs, and the
// i-th of its n contributors sums its blocks' partials in contributor order
// (k order), applies the epilogue and stores them.  Every output is so added
// in one fixed order whatever the timing: a deterministic fix-up with no
// atomic arithmetic, whose reads are shared evenly by the workgroups of the
// tile.  All contributors of a tile are on one XCD, so partial sums meet in
// that XCD's L2.
//
// Waits are bounded: a reducer waits for a contributor's flag at most
// wait_ticks (wall-clock ticks); a piece that has not appeared by then (its
// rank has not started, for instance because the grid is not co-resident) the
// reducer computes itself, into that rank's slot, with the same code on the
// same data: the bits the contributor writes, so a late contributor
// overwrites them with themselves.  No wait can therefore hang the kernel, and
// the output never depends on which path ran.  A flag holds the launch's
// 64-bit epoch (a new value per launch from the host), so flags left by
// earlier launches in the workspace are never taken for this launch's.
//
// part: 2 G fp32 tiles of 256 KiB (slots 2 b and 2 b + 1: workgroup b's first
// and second piece); flags: G 64-bit words.
struct SkSched {
    int tiles_m, tiles_n;
    int nk;         // 64-k steps per tile
    char* part;
    unsigned long long* flags;
    unsigned long long epoch;
    long long wait_ticks;
};

constexpr int SK_TILE = 256;    // the Stream-K macro-tile, square
constexpr int SK_BK = 64;       // k per iteration
constexpr int SK_BLOCKS = 64;   // 32 x 32 output blocks per tile

// Rank j of XCD x and its run [s0, s1) of the XCD's W iterations.
struct SkRun {
    int x, j, R, nk, W, s0, s1;
    int u0;        // the tile of the first piece (of the XCD's list)
    int npieces;   // 1 or 2 (the second: tile u0 + 1)
    __host__ __device__ int start(int r) const { return (int)((int64_t)r * W / R); }
    __host__ __device__ int pos(int u) const { return x + NUM_XCD * u; }  // tile walk position
    __host__ __device__ int rank_of(int it) const {  // the rank whose run holds iteration it
        return (int)((((int64_t)it + 1) * R - 1) / W);
    }
    __host__ __device__ int first(int u) const { return rank_of(u * nk); }
    __host__ __device__ int last(int u) const { return rank_of((u + 1) * nk - 1); }
    // Slot of rank p's piece of tile u.
    __host__ __device__ int slot(int p, int u) const {
        return 2 * (x + NUM_XCD * p) + (start(p) / nk == u ? 0 : 1);
    }
    // Rank p's k range [kb, ke) of tile u, in iterations of the tile.
    __host__ __device__ void piece(int p, int u, int& kb, int& ke) const {
        const int t0 = u * nk;
        const int a = start(p), b = start(p + 1);
        kb = (a > t0 ? a : t0) - t0;
        ke = (b < t0 + nk ? b : t0 + nk) - t0;
    }
};

__host__ __device__ inline SkRun sk_run(const SkSched& sk, int b, int G) {
    SkRun r;
    r.x = b % NUM_XCD;
    r.j = b / NUM_XCD;
    r.R = G / NUM_XCD;
    r.nk = sk.nk;
    const int tiles = sk.tiles_m * sk.tiles_n;
    const int nx = tiles > r.x ? (tiles - r.x + NUM_XCD - 1) / NUM_XCD : 0;
    r.W = nx * sk.nk;
    r.s0 = r.start(r.j);
    r.s1 = r.start(r.j + 1);
    r.u0 = r.W > 0 ? r.s0 / sk.nk : 0;
    r.npieces = r.W == 0 ? 0 : (r.s1 > (r.u0 + 1) * sk.nk ? 2 : 1);
    return r;
}

// Blocks [lo, hi) of tile u that rank j reduces: its share among the tile's
// contributors first(u) .. last(u).
__host__ __device__ inline void sk_share(const SkRun& r, int u, int& lo, int& hi) {
    const int f = r.first(u), n = r.last(u) - f + 1, i = r.j - f;
    lo = SK_BLOCKS * i / n;
    hi = SK_BLOCKS * (i + 1) / n;
}

// Workspace of a Stream-K launch of `grid` workgroups: 2 grid partial tiles,
// then one 64-bit flag per workgroup.
constexpr int64_t sk_ws_bytes(int grid) {
    return (int64_t)2 * grid * SK_TILE * SK_TILE * 4 + (int64_t)grid * 8;
}

// Per kernel family; each returns hipErrorInvalidValue for a combination it
// has no instantiation for.
hipError_t launch_gemm16(const GemmLaunch& L);  // IN_BF16, IN_F16
// The Stream-K launch: L as for launch_gemm16 with tbm = tbn = 256 and
// splits = 1; `grid` workgroups, a multiple of NUM_XCD.
hipError_t launch_gemm16_sk(const GemmLaunch& L, const SkSched& s, int grid);
hipError_t launch_gemm32(const GemmLaunch& L);  // IN_F32, IN_F32X3
hipError_t launch_gemmt(const GemmLaunch& L);   // LAY_NT, LAY_TN: 16-bit; LAY_NT: IN_F8, IN_F8W
hipError_t launch_slicet(const GemmLaunch& L);  // as launch_gemmt with slice_waves > 0
// A LAY_NT and a LAY_TN launch of 4-wave slice-K tiles (16-bit or fp32; tiles_m = 0:
// none) and (if r.N > 0) column sums, in one kernel, the TN tiles first if tn_first: the backward pass of a small
// layer.
hipError_t launch_slicet_pair(const GemmLaunch& nt, const GemmLaunch& tn, bool tn_first,
                              const ColReduceArgs& r);
// The same of 16-bit grid tiles, 128 x 128 or 256 x 256 for both.
hipError_t launch_gemmt_pair(const GemmLaunch& nt, const GemmLaunch& tn, bool tn_first,
                             const ColReduceArgs& r);
// The products of a gated layer's backward pass and its column sums in one kernel: nt (LAY_NT) is
// nt.A nt.B^T + A2 B2^T (A2 with nt.A's row pitch), tn the weights' gradients (LAY_TN); tiles_m = 0
// or N = 0: none.  One tile size for all (launch_gemmt_gated, 16-bit) or one for nt and one for
// tn (launch_slicet_gated, 4 waves); the TN tiles first if tn_first.  launch_gemmt_gated: nt's K
// steps (of 64, of both pairs) in nt.splits runs of nt.kchunk steps, their fp32 sums at nt.C + z
// nt.c_zstride; tn's rows of the batch in tn[0].splits runs of tn[0].kchunk, as far apart at both C.
struct GatedBwdLaunch {
    GemmLaunch nt, tn[2];
    const char* A2;
    const char* B2;
    int ldb2;
    bool tn_first;
    ColReduceArgs sums[2];
};
hipError_t launch_gemmt_gated(const GatedBwdLaunch& L);
hipError_t launch_slicet_gated(const GatedBwdLaunch& L);
hipError_t launch_slicek16(const GemmLaunch& L);  // IN_BF16, IN_F16 with slice_waves > 0

// Products of at most SKINNY_M rows (skinny.hip): LAY_NN of 16-bit and fp32
// operands, LAY_NT of those and IN_F8W, and the rank-K update LAY_TN with at most
// SKINNY_M terms (K) per sum.  L.tbn names the strip of columns per workgroup,
// L.slice_waves the waves that share a strip's K; splits (LAY_NN only), kchunk and
// the partials' C as for a grid launch.
constexpr int SKINNY_M = 16;
hipError_t launch_skinny(const GemmLaunch& L);
// C = A B^T + A2 B2^T of few rows (A2 with A's row pitch), LAY_NT of 16-bit and fp32 operands.
hipError_t launch_skinny_two(const GemmLaunch& L, const char* A2, const char* B2, int ldb2);

// Products of e4m3 operands with a scale per block (blockf8.hip): A[M x K] B[N x K]^T, block b
// of K being [F8_BLOCK b, F8_BLOCK (b + 1)), row i of A scaled by sa[i sa_row + b sa_blk], row j
// of B by sb[(j / rows_b) sb_row + b sb_blk], rows_b 1 or F8_BLOCK.  g describes the launch as
// for launch_gemmt / launch_slicet / launch_skinny (in: IN_F8, or IN_F8W for the widened
// products); a split's kchunk is a multiple of F8_BLOCK.
struct BlockScales {
    const float* sa;
    const float* sb;
    int sa_row, sa_blk, sb_row, sb_blk, rows_b;
};
hipError_t launch_blockf8(const GemmLaunch& g, const BlockScales& s);
hipError_t launch_blockf8_skinny(const GemmLaunch& g, const BlockScales& s);

// Gated projections (gated.hip, skinny.hip): C := act(G) U, G := A Bg + bias_g, U := A Bu + bias_u.
// biases, G and U may be NULL, and C for a split's partial products.
struct GatedEpi {
    const float* bias_g;
    const float* bias_u;
    int act;
    char* G;
    char* U;
    int ldg, ldu;
};
// tbm x tbp tiles (tbp columns of G and of U); split z, of kchunk k, writes G and U at z zstride
// bytes.  waves = 4: a tile's K split over its waves (32 x 32, 64 x 32; unsplit).  Few rows: strips
// of tbp columns, `waves` waves each (launch_gated_skinny).
struct GatedLaunch {
    int in, out, tbm, tbp, stages, waves;
    const char* A;
    const char* Bg;
    const char* Bu;
    char* C;
    int M, N, K, lda, ldbg, ldbu, ldc, tiles_m, tiles_n, splits, kchunk;
    int64_t zstride;
    GatedEpi e;
    hipStream_t stream;
};
hipError_t launch_gated(const GatedLaunch& L);
hipError_t launch_gated_skinny(const GatedLaunch& L);
// W[z]: M x 2 ldw fp32 partial products of G and, from column ldw on, of U.
hipError_t launch_gated_reduce(const float* W, int splits, int64_t zstride, int ldw, char* C, int ldc, int M, int N,
                               int out, const GatedEpi& e, hipStream_t stream);

// Split-K reduction: C[i][j] = epilogue(sum_{z < splits} W[z][i][j]) with W
// fp32, row pitch ldw (a multiple of 4) and split stride zstride elements.
hipError_t launch_splitk_reduce(const float* W, int splits, int64_t zstride, int ldw, char* C,
                                int ldc, int M, int N, int out, int epi, const EpiArgs& e,
                                hipStream_t stream);

// C [M x N] (16-bit) = the sum of `splits` fp32 matrices of pitch ldw, zstride floats apart; up to
// three such sums in one launch.
struct SplitSum {
    const float* W;
    int64_t zstride;
    char* C;
    int splits, ldw, ldc, M, N;
};
hipError_t launch_splitk_reduce3(const SplitSum* sums, int count, int out, hipStream_t stream);

// ------------------------------------------- norms, quantizers, activations

constexpr int ROW_MAX = 32768;       // longest row of the norm and the row quantizer
constexpr int NORM_BWD_MAX = 16384;  // of the norm's backward pass

// Output rows (dgemm_rows): X's format, e4m3 with a scale per row, or per block of
// F8_BLOCK columns.
enum Rows { ROWS_SAME = 0, ROWS_F8 = 1, ROWS_F8_BLOCK = 2 };
constexpr int F8_BLOCK = 128;

// A pass over the rows of X (norm.hip, layernorm.hip).  R, S, rstd may be NULL; Y is in X's
// format, or e4m3 with `scale` (per row; per column for launch_quant_cols,
// which writes Y transposed and uses X, Y and scale only; per row and block, at row *
// s_row + block * s_blk).  Layer norm also: bias, mean (each may be NULL).
struct RowArgs {
    const char* X;
    const char* R;
    char* S;
    const float* weight;
    char* Y;
    float* scale;
    float* rstd;
    float eps;
    int M, N, ldx, ldr, lds, ldy;
    const float* bias;
    float* mean;
    int64_t s_row, s_blk;
};
hipError_t launch_rows(const RowArgs& a, int fmt, bool norm, int rows, hipStream_t stream);
hipError_t launch_layernorm(const RowArgs& a, int fmt, int rows, hipStream_t stream);
hipError_t launch_quant_cols(const RowArgs& a, int fmt, hipStream_t stream);

// The norm's backward pass; part: norm_bwd_grid(M, N) rows of ldp fp32 partial
// sums of dweight, or NULL.
struct NormBwdArgs {
    const char* dY;
    const char* S;
    const char* dS;
    const float* weight;
    const float* rstd;
    char* dX;
    float* part;
    int M, N, lddy, lds, ldds, lddx, ldp;
    const float* mean;  // layer norm, whose partial sums are two rows of ldp each: dweight's, dbias'
};
int norm_bwd_grid(int M, int N);
int layernorm_bwd_grid(int M, int N, int fmt);
hipError_t launch_norm_bwd(const NormBwdArgs& a, int fmt, hipStream_t stream);
hipError_t launch_layernorm_bwd(const NormBwdArgs& a, int fmt, hipStream_t stream);

// X or its transpose in 8 bits with a scale per block of `rows` x F8_BLOCK (quantblock.hip):
// block (i, b) of Q at scale[i s_row + b s_blk].
struct QuantBlockArgs {
    const char* X;
    char* Q;
    float* scale;
    int M, N, ldx, ldq;
    int64_t s_row, s_blk;
};
hipError_t launch_quant_block(const QuantBlockArgs& a, int fmt, int rows, bool transpose, hipStream_t stream);

// dZ = dC act'(Z) (actgrad.hip).  Z NULL: dZ = dC.  dZ may be NULL; part: one row
// of ldp fp32 column sums per rows_per rows, or NULL.
struct ActGradArgs {
    const char* dC;
    const char* Z;
    char* dZ;
    float* part;
    int M, N, lddc, ldz, lddz, ldp, rows_per, act;
};
// The gated layer's: dG = dC U act'(G), dU = dC act(G); part: two rows of ldp sums per rows_per
// rows, dG's and dU's, or NULL.
struct GatedGradArgs {
    const char* dC;
    const char* G;
    const char* U;
    char* dG;
    char* dU;
    float* part;
    int M, N, lddc, ldg, ldu, lddz, ldp, rows_per, act;
};
hipError_t launch_gated_grad(const GatedGradArgs& a, int cf, int df, hipStream_t stream);
int act_grad_rows(int M, int N);
hipError_t launch_act_grad(const ActGradArgs& a, int cf, int df, hipStream_t stream);
hipError_t launch_col_reduce(const ColReduceArgs& a, hipStream_t stream);
// Two of them in one launch (N = 0: none).
hipError_t launch_col_reduce2(const ColReduceArgs& a, const ColReduceArgs& b, hipStream_t stream);
hipError_t launch_transpose32(const float* X, int ldx, int M, int N, float* Y, int ldy,
                              hipStream_t stream);

}  // namespace dgemm
