// stage16.h -- LDS layouts of the matrix kernels' operand stages, shared by
// gemm16.hip and gemmt.hip: rows of 128 bytes for operands stored K-contiguous,
// and k-rows for operands stored along the output's rows or columns.
#pragma once

#include "kern_common.h"

namespace dgemm {

constexpr int BKA = 64;                        // K per A slab
constexpr int A16_CH = BKA / 8;                // 16-byte chunks per A row
constexpr int A16_ROW = BKA * 2;               // bytes per staged A row
constexpr int A16_RPB = 1024 / A16_ROW;        // A rows per 1 KiB load block

// Byte offset of chunk c (0..7) of A row r in a slab.  ds_read_b128 serves
// groups of 4 consecutive lanes from a 64-byte window of banks (measured on
// gfx950 with SQ_LDS_BANK_CONFLICT), and the 4 lanes of a group read 4
// consecutive rows at one chunk: a16_phi gives those rows 4 distinct slots.
__device__ __forceinline__ int a16_phi(int row) { return (row ^ (row >> 2)) & (A16_CH - 1); }
__device__ __forceinline__ int a16_off(int row, int chunk) {
    return row * A16_ROW + ((chunk ^ a16_phi(row)) << 4);
}
// Byte offset of chunk c of B row k in a stage with row pitch `row_bytes` (a
// multiple of 256).  ds_read_b64_tr_b16 serves 32 lanes from a 256-byte
// window (measured), and those 32 lanes read 4 consecutive k rows x 64 bytes;
// the XOR puts the four rows' pieces in distinct quarters of the window.
__device__ __forceinline__ int b16_swz(int k) { return ((k & 3) << 1) ^ ((k & 1) << 3); }
__device__ __forceinline__ int b16_off(int k, int chunk, int row_bytes) {
    return k * row_bytes + ((chunk ^ b16_swz(k)) << 4);
}

}  // namespace dgemm
