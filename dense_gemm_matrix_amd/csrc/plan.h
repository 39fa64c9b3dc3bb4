// plan.h -- host code shared by the entry points (dgemm.hip, linear.hip):
// operand checks, the launch plan and its estimate, and the launch of a plan.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "dgemm_internal.h"

namespace dgemm {

constexpr int64_t DESC_LIMIT = (int64_t)1 << 31;  // 32-bit buffer offsets
constexpr int PANEL_ROWS = 256;                   // rows of A one descriptor spans

int check_device();  // DGEMM_OK on a gfx950, else DGEMM_ERR_DEVICE

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The bytes a row-major operand occupies: `rows` rows of `row_bytes` each,
// `pitch` bytes apart.  A contiguous range is one row.
struct Span {
    uintptr_t base;
    int64_t rows, row_bytes, pitch;
};

Span matrix_span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize);
bool spans_overlap(Span x, Span y);

// The checks that every product's A, B and C share (in: a dgemm_in code).
int validate(int M, int N, int K, const void* A, int lda, const void* B, int ldb, const void* C,
             int ldc, int in, int es_out);

constexpr int MAX_SPLITS = 16;
constexpr double SPLIT_MARGIN = 0.9;      // a split plan must be predicted 10% faster

// pair = 0: one workgroup per CU.  fp32 has the 128 x 128 tile only: in a
// sweep of forced plans 256 x 256 was slower at every shape (4096^3: 1049 us
// against 1002 us), and the cost model never chose it; eff stays relative to
// a 256 x 256 workgroup so that step_us keeps one meaning.
// `pair2`: the pair factor of grids of two or more rounds of pairs; `last`: the
// cost of a last, partly filled round at zero fill (1: whole rounds).
struct TileCand { int bm, bn; double eff, pair, pair2, eff1, last; };

enum PlanKind { PLAN_GRID = 0, PLAN_STREAM_K = 1, PLAN_SKINNY = 2 };

struct Plan {
    int bm, bn;
    int splits, kchunk;   // kchunk: K per split (a multiple of the K step)
    int ldw;              // row pitch of the fp32 partials, in elements
    int64_t ws_bytes;     // workspace the plan uses (0 when unsplit)
    int kind = PLAN_GRID;
    int waves = 0;        // slice-K and skinny plans: waves per workgroup (0: a grid plan)
    int layout = LAY_NN;  // the operands' Layout
};

// Microseconds per K step of one 256 x 256 workgroup.
double step_us(int in);
// Estimated time of a grid plan of tile t (dgemm.hip explains the terms).
double estimate_us(int in, int es_out, int M, int N, const TileCand& t, int splits,
                   int steps_per_split, int ldw);
// The tile and split count forced by dgemm_set_plan_override, if a grid plan is.
bool forced_grid(int& bm, int& bn, int& splits);
// The 16-bit slice-K plan for an M x N output with K terms and its estimate; false
// where the output is too large for one.  slice_waves_t: whether the kernels have
// tile ts with `waves` waves.
bool slice_plan_t(int M, int N, int K, Plan& p, double& us);
bool slice_waves_t(int ts, int waves);
// Time of one 4-wave slice-K tile of K terms on a CU, workgroup after workgroup
// (in: IN_BF16 for both 16-bit formats, IN_F32).
double slice_tile_us(int in, int ts, int K);
// Estimated time of plan p of A[M x K] B[K x N].
double plan_us(int in, int es_out, const Plan& p, int M, int N, int K);
Plan make_plan(int in, int es_out, int M, int N, int K, uint64_t ws_avail, bool allow_sk);

// Validated arguments and a plan -> its launches, with epilogue e at level epi.
int run(int in, int outfmt, int M, int N, int K, const void* A, int lda, const void* B, int ldb,
        void* C, int ldc, const EpiArgs& e, int epi, const Plan& p, void* ws, hipStream_t stream);
int out_format(int in, int out);

}  // namespace dgemm
