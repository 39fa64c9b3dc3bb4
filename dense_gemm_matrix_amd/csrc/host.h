// host.h -- argument checks that the entry points of linear.hip and feedforward.hip share.
#pragma once

#include <algorithm>

#include "dgemm.h"
#include "dgemm_internal.h"
#include "plan.h"

namespace dgemm {

constexpr int64_t WS_ALIGN = 256;  // pieces of a workspace start on this

inline int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// A row-major matrix operand of a call.
struct Mat {
    const void* p;
    int64_t rows, cols, ld, es;
    Span span() const { return matrix_span(p, rows, cols, ld, es); }
    bool empty() const { return rows <= 0 || cols <= 0; }
};

// Pitch, pointer, alignment and the 32-bit panel limit of one matrix.
inline int check_mat(const Mat& m) {
    if (m.ld < std::max<int64_t>(m.cols, 1)) return DGEMM_ERR_LEADING_DIM;
    if (!m.empty()) {
        if (!m.p) return DGEMM_ERR_INVALID_VALUE;
        if (((uintptr_t)m.p & 15) || (m.ld * m.es) % 16) return DGEMM_ERR_MISALIGNED;
    }
    if ((int64_t)PANEL_ROWS * m.ld * m.es >= DESC_LIMIT) return DGEMM_ERR_TOO_LARGE;
    return DGEMM_OK;
}

// An fp32 vector operand (NULL: absent).
inline Mat vec(const void* p, int64_t n) { return Mat{p, p ? 1 : 0, n, n, 4}; }

inline int check_vec(const void* p, int align) {
    return ((uintptr_t)p & (uintptr_t)(align - 1)) ? DGEMM_ERR_MISALIGNED : DGEMM_OK;
}

// Whether any of `outs` shares a byte with another of them or with any of `ins`.
inline bool any_overlap(const Mat* outs, int n_out, const Mat* ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        if (!outs[i].p) continue;
        for (int j = 0; j < n_in; ++j)
            if (ins[j].p && spans_overlap(outs[i].span(), ins[j].span())) return true;
        for (int j = 0; j < i; ++j)
            if (outs[j].p && spans_overlap(outs[i].span(), outs[j].span())) return true;
    }
    return false;
}

inline Mat bytes_of(void* p, int64_t n) { return Mat{p, n > 0 ? 1 : 0, n, n, 1}; }

inline bool valid_act(int act) { return act >= DGEMM_ACT_NONE && act <= DGEMM_ACT_SILU; }

inline int launched(hipError_t e) { return e == hipSuccess ? DGEMM_OK : DGEMM_ERR_LAUNCH; }

// Format codes DGEMM_IN_F32 / _BF16 / _F16 of an elementwise operator.
inline int row_fmt(int in) {
    return in == DGEMM_IN_F32 ? OUT_F32 : in == DGEMM_IN_BF16 ? OUT_BF16 : in == DGEMM_IN_F16 ? OUT_F16 : -1;
}

// A plan for a gemm_*_plan query.
inline int report(const Plan& p, int* tile_rows, int* tile_cols, int* splits, size_t* used) {
    if (tile_rows) *tile_rows = p.bm;
    if (tile_cols) *tile_cols = p.bn;
    if (splits) *splits = p.splits;
    if (used) *used = (size_t)p.ws_bytes;
    return DGEMM_OK;
}

}  // namespace dgemm
