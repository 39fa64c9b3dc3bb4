// kern_common.h -- device helpers shared by the GEMM kernels: vector types,
// buffer resources, the direct-to-LDS load, wait counts and the epilogue.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dgemm_internal.h"

namespace dgemm {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4_t;

constexpr uint32_t BUF_WORD3 = 0x00020000u;  // raw buffer: 32-bit data format, no swizzle

// A raw buffer resource covering [base, base + bytes), the range rounded up to
// 16 bytes.  The buffer unit range-checks whole dwords, so a range ending in
// the middle of a dword (an odd count of 16-bit elements) would return the
// last element as zero.  Rounding up is safe: bases and row pitches are 16-byte
// aligned, so the extra bytes share a 16-byte chunk (hence a page) with the
// last element; they are masked (A's K tail) or feed only unstored outputs
// (B's columns past N).  bytes <= 0 gives an empty range.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const char* base, int64_t bytes) {
    const int64_t rounded = bytes > 0 ? (bytes + 15) & ~(int64_t)15 : 0;
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)rounded, (int)BUF_WORD3);
}

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int voffset) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, voffset, 0, 0);
}

// Reinterpret a 32-bit word as fp32.  The word is taken by value: clang's
// __builtin_bit_cast applied directly to an ext-vector element subscript
// (v[e]) reads element 0 whatever e is, so callers pass v[e] through here.
__device__ __forceinline__ float as_float(uint32_t w) { return __builtin_bit_cast(float, w); }

// LDS byte address of a pointer into a __shared__ array.
__device__ __forceinline__ uint32_t lds_addr(const char* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// One direct-to-LDS 16-byte-per-lane buffer load: lane l's 16 bytes from
// rsrc + voffset land at LDS byte lds + 16 l.  Issued as inline assembly so that
// the compiler does not guard every later LDS read with a wait for ALL such
// loads (it cannot tell which LDS bytes they write); the kernel waits for them
// explicitly with s_waitcnt vmcnt before the barrier that publishes a stage.
// An LDS DMA needs one wait state after the SALU write of M0 that it reads
// (the compiler keeps one instruction between them for its own LDS DMA), hence
// the s_nop.
// M0 is reserved to the compiler, which warns about the clobber; nothing else
// in these kernels uses M0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds, int voffset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voffset), "s"(rsrc)
                 : "memory", "m0");
}
// The same of 4 bytes per lane: lane l's land at LDS byte lds + 4 l.
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds, int voffset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voffset), "s"(rsrc)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// s_waitcnt immediate: wait until at most vm vector-memory and lgkm LDS/scalar
// operations of this wave are outstanding.
constexpr int waitcnt_imm(int vm, int lgkm) {
    return (vm & 0xf) | ((vm >> 4) << 14) | (0x7 << 4) | ((lgkm & 0xf) << 8);
}

template <int OUT>
__device__ __forceinline__ float load_c(const char* C, int64_t idx) {
    if (OUT == OUT_F32) return *reinterpret_cast<const float*>(C + idx * 4);
    if (OUT == OUT_BF16) return (float)*reinterpret_cast<const __bf16*>(C + idx * 2);
    return (float)*reinterpret_cast<const _Float16*>(C + idx * 2);
}

template <int OUT>
__device__ __forceinline__ void store_c(char* C, int64_t idx, float v) {
    if (OUT == OUT_F32) {
        *reinterpret_cast<float*>(C + idx * 4) = v;
    } else if (OUT == OUT_BF16) {
        *reinterpret_cast<__bf16*>(C + idx * 2) = (__bf16)v;      // round to nearest even
    } else {
        *reinterpret_cast<_Float16*>(C + idx * 2) = (_Float16)v;  // round to nearest even
    }
}

// The fused epilogue on one fp32 sum s: alpha * s + beta * C_old + bias, then
// the optional ReLU (a NaN passes through), in fp32, before the one rounding
// to C's format.  C_old is the element at byte address p.
template <int OUT>
__device__ __forceinline__ float epilogue_at(float s, const char* p, float bias, const EpiArgs& e) {
    float v = e.alpha * s;
    if (e.beta != 0.0f) v += e.beta * load_c<OUT>(p, 0);
    v += bias;
    if (e.relu && v < 0.0f) v = 0.0f;
    return v;
}

// The same for element idx of C.
template <int OUT>
__device__ __forceinline__ float epilogue(float s, const char* C, int64_t idx, float bias,
                                          const EpiArgs& e) {
    return epilogue_at<OUT>(s, C + idx * (OUT == OUT_F32 ? 4 : 2), bias, e);
}

// Epilogue of the GEMM kernels.  32x32 accumulator layout: lane (g, li) holds
// column li and, in register r, row 8 * (r / 4) + 4 * g + r % 4 of its block.
//
// Every tile takes one branch-free path: a buffer resource over C from the
// wave's corner (row0, col0) to the end of C's valid region, stores at 32-bit
// byte offsets = a per-lane part + a wave-uniform part.  Elements past the last
// row fall outside the resource's range, and lanes whose column is past N get
// an offset beyond any range (OOB_LANE): the buffer unit drops those stores
// (and returns zeros for those loads), so nothing outside M x N is written and
// no element needs a test.  Offsets stay below 2^31 because a 256-row panel of
// C is under 2 GiB (the ABI's precondition) and a range is at most 2^31 - 16
// bytes.
constexpr uint32_t OOB_LANE = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t c_rsrc(char* C, int M, int N, int ldc, int row0,
                                                         int col0, int es) {
    char* base = C + ((int64_t)row0 * ldc + col0) * es;
    int64_t rem = ((int64_t)(M - 1 - row0) * ldc + (N - col0)) * es;
    if (rem > 0x7ffffff0) rem = 0x7ffffff0;
    return make_rsrc(base, rem);
}

template <int OUT>
__device__ __forceinline__ float load_c_at(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (OUT == OUT_F32)
        return as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
    const uint32_t h = __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
    if constexpr (OUT == OUT_BF16) return as_float(h << 16);
    return (float)__builtin_bit_cast(_Float16, (unsigned short)h);
}

// The fused epilogue on one fp32 sum s read through the C resource.
template <int OUT>
__device__ __forceinline__ float epilogue_rs(float s, __amdgpu_buffer_rsrc_t r, uint32_t off,
                                             float bias, const EpiArgs& e) {
    float v = e.alpha * s;
    if (e.beta != 0.0f) v += e.beta * load_c_at<OUT>(r, off);
    v += bias;
    if (e.relu && v < 0.0f) v = 0.0f;
    return v;
}

// Two fp32 values rounded to nearest even in C's 16-bit format, `lo` in the
// low half of the word.
template <int OUT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {lo, hi};
    if constexpr (OUT == OUT_BF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// Eight e4m3 values (two words) as bf16, exactly: the four significant bits and
// exponents down to 2^-9 fit.
__device__ __forceinline__ bf16x8 widen_f8(uint32_t lo, uint32_t hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// DPP quad permutation [1, 0, 3, 2]: lane l reads lane l ^ 1.
constexpr int DPP_QUAD_XOR1 = 1 | (0 << 2) | (3 << 4) | (2 << 6);

__device__ __forceinline__ uint32_t swap_adjacent_lanes(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, DPP_QUAD_XOR1, 0xf, 0xf, false);
}

// One store per element: fp32 C, or 16-bit C when a tile's column edge falls
// between the two columns of a lane pair (N odd).
template <int OUT, int MI, int NJ, int EPI>
__device__ __forceinline__ void store_elems(const f32x16 (&acc)[MI][NJ], __amdgpu_buffer_rsrc_t r,
                                           int N, int ldc, int col0, int g, int li,
                                           const EpiArgs& e) {
    constexpr int ES = OUT == OUT_F32 ? 4 : 2;
#pragma unroll
    for (int nj = 0; nj < NJ; ++nj) {
        const int col = col0 + nj * 32 + li;
        const uint32_t lane = col < N ? (uint32_t)((4 * g * ldc + nj * 32 + li) * ES) : OOB_LANE;
        float bias = 0.0f;
        if (EPI && e.bias && col < N) bias = e.bias[col];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
            for (int rr = 0; rr < 16; ++rr) {
                const uint32_t off = lane + (uint32_t)((mi * 32 + 8 * (rr >> 2) + (rr & 3)) * ldc * ES);
                float v = acc[mi][nj][rr];
                if constexpr (EPI) v = epilogue_rs<OUT>(v, r, off, bias, e);
                if constexpr (OUT == OUT_F32) {
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, (int)off, 0, 0);
                } else {
                    const uint32_t p = pack16<OUT>(v, 0.0f);
                    __builtin_amdgcn_raw_buffer_store_b16((unsigned short)p, r, (int)off, 0, 0);
                }
            }
        }
    }
}

// 16-bit C with both columns of every lane pair inside or both outside: an
// even lane l and lane l + 1 hold columns c and c + 1, and registers r and
// r + 1 (r even) rows R and R + 1.  Each lane rounds its two values into one
// word; one exchange between the two lanes then gives the even lane row R,
// columns c .. c + 1, and the odd lane row R + 1, the same columns: one 4-byte
// store where the per-element form needs two 2-byte ones, and each half-wave
// store writes two 64-byte row pieces instead of one.  The epilogue and the
// rounding act on each value before the exchange, so the stored values are
// those of store_elems.  Needs every lane of the wave active.
template <int OUT, int MI, int NJ, int EPI>
__device__ __forceinline__ void store_pairs16(const f32x16 (&acc)[MI][NJ], __amdgpu_buffer_rsrc_t r,
                                              int N, int ldc, int col0, int g, int li,
                                              const EpiArgs& e) {
    const int odd = li & 1;
    // v_perm_b32 takes bytes 0-3 from its second source and 4-7 from its first:
    // the even lane keeps its low half (row R) and takes the neighbour's; the odd
    // lane takes the neighbour's high half (row R + 1) and keeps its own.
    const uint32_t sel = odd ? 0x03020706u : 0x05040100u;
#pragma unroll
    for (int nj = 0; nj < NJ; ++nj) {
        const int col = col0 + nj * 32 + li;
        const uint32_t own = col < N ? (uint32_t)((4 * g * ldc + nj * 32 + li) * 2) : OOB_LANE;
        const uint32_t word = col - odd < N ? (uint32_t)(((4 * g + odd) * ldc + nj * 32 + li - odd) * 2)
                                            : OOB_LANE;
        float bias = 0.0f;
        if (EPI && e.bias && col < N) bias = e.bias[col];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
            for (int rr = 0; rr < 16; rr += 2) {
                const uint32_t rows = (uint32_t)((mi * 32 + 8 * (rr >> 2) + (rr & 3)) * ldc * 2);
                float v0 = acc[mi][nj][rr];
                float v1 = acc[mi][nj][rr + 1];
                if constexpr (EPI) {
                    v0 = epilogue_rs<OUT>(v0, r, own + rows, bias, e);
                    v1 = epilogue_rs<OUT>(v1, r, own + rows + (uint32_t)(ldc * 2), bias, e);
                }
                const uint32_t p = pack16<OUT>(v0, v1);
                const uint32_t w = __builtin_amdgcn_perm(swap_adjacent_lanes(p), p, sel);
                __builtin_amdgcn_raw_buffer_store_b32(w, r, (int)(word + rows), 0, 0);
            }
        }
    }
}

// PAIRS (16-bit C): the launch's N is even, so no lane pair straddles the
// column edge and every tile takes store_pairs16; with N odd the kernel is
// instantiated with store_elems instead (deciding inside the kernel costs
// registers on every tile).
template <int OUT, int MI, int NJ, int EPI, bool PAIRS>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[MI][NJ], char* C, int M, int N,
                                           int ldc, int row0, int col0, int g, int li,
                                           const EpiArgs& e) {
    if (row0 >= M || col0 >= N) return;  // this wave's part of the tile lies outside C
    constexpr int ES = OUT == OUT_F32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t r = c_rsrc(C, M, N, ldc, row0, col0, ES);
    if constexpr (OUT != OUT_F32 && PAIRS)
        store_pairs16<OUT, MI, NJ, EPI>(acc, r, N, ldc, col0, g, li, e);
    else
        store_elems<OUT, MI, NJ, EPI>(acc, r, N, ldc, col0, g, li, e);
}

// Zero the bytes of a 16-byte piece at and past `valid` (<= 0: all of them).
__device__ __forceinline__ u32x4 mask_bytes(u32x4 v, int valid) {
    u32x4 out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int n = valid - 4 * w;  // bytes of this word to keep
        out[w] = n >= 4 ? v[w] : n <= 0 ? 0u : v[w] & (0xffffffffu >> (32 - 8 * n));
    }
    return out;
}

// A wave's n steps in chunks of D: the next chunk's loads are issued before the
// current one is used, so D to 2 D steps are in flight, and the last chunk loads
// only the steps there are (a load past the end costs as much issue as a real
// one).  load(i, slot) and use(i, slot, newer): step i in slot `slot`, a constant
// once unrolled; newer (an integral_constant) steps have surely been loaded after
// the chunk, for a use that waits for its own loads by count.
template <int D, class Load, class Use>
__device__ __forceinline__ void run_steps(int n, Load load, Use use) {
    const int full = n > 0 ? n / D : 0, rem = n > 0 ? n - full * D : 0;
    auto rest = [&](int base) {  // the last chunk's loads, into slots base ..
#pragma unroll
        for (int s = 0; s < D - 1; ++s)
            if (s < rem) load(full * D + s, base + s);
    };
    using None = std::integral_constant<int, 0>;
    using Next = std::integral_constant<int, D>;
    auto use_rest = [&](int base) {
#pragma unroll
        for (int s = 0; s < D - 1; ++s)
            if (s < rem) use(full * D + s, base + s, None{});
    };
    if (full == 0) {
        rest(0);
        use_rest(0);
        return;
    }
#pragma unroll
    for (int s = 0; s < D; ++s) load(s, s);
    int c = 0;
    for (; c + 2 < full; c += 2) {
#pragma unroll
        for (int s = 0; s < D; ++s) load((c + 1) * D + s, D + s);
#pragma unroll
        for (int s = 0; s < D; ++s) use(c * D + s, s, Next{});
#pragma unroll
        for (int s = 0; s < D; ++s) load((c + 2) * D + s, s);
#pragma unroll
        for (int s = 0; s < D; ++s) use((c + 1) * D + s, D + s, Next{});
    }
    if (c + 1 < full) {
#pragma unroll
        for (int s = 0; s < D; ++s) load((c + 1) * D + s, D + s);
#pragma unroll
        for (int s = 0; s < D; ++s) use(c * D + s, s, Next{});
        rest(0);
#pragma unroll
        for (int s = 0; s < D; ++s) use((c + 1) * D + s, D + s, None{});
        use_rest(0);
    } else {
        rest(D);
#pragma unroll
        for (int s = 0; s < D; ++s) use(c * D + s, s, None{});
        use_rest(D);
    }
}

// ------------------------------------------------------- the full epilogue
//
// z := acc * scale_a[row] * scale_b[col] + bias[col];  Z := z;  C := act(z) + R.
//
// GELU and its tanh form, with Phi the normal distribution's integral:
//   gelu(z) = z Phi(z) = z (1 + erf(z / sqrt 2)) / 2
//   gelu_tanh(z) = z (1 + tanh(t)) / 2 = z / (1 + exp(-2 t)),
//     t = sqrt(2 / pi) (z + 0.044715 z^3)
// so gelu_tanh and silu(z) = z / (1 + exp(-z)) are one form z / (1 + exp(-p)), with
// p = 2 t or z, evaluated with the hardware's exp2 and reciprocal (1 ulp each).  As p
// falls, exp overflows to infinity and its reciprocal to 0: the limit -0.  Infinite z
// gives infinity or, at -infinity, NaN (-inf * 0), as the formula itself does in
// floating point; a NaN stays a NaN.  silu's p is z itself, not a cubic with a zero
// coefficient: 0 * inf would make a NaN of silu(+inf).
constexpr float LOG2E = 1.4426950408889634f;
constexpr float SQRT_2_PI = 0.7978845608028654f;
constexpr float GELU_C = 0.044715f;
constexpr float GELU_A = 2.0f * SQRT_2_PI;           // 2 t = z (GELU_A + GELU_B z^2)
constexpr float GELU_B = 2.0f * SQRT_2_PI * GELU_C;

__device__ __forceinline__ float sigmoid(float p) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * p));
}
__device__ __forceinline__ float gelu_2t(float z) { return z * (GELU_A + GELU_B * z * z); }

// Phi(z), the normal distribution's integral, and exp(-z^2 / 2) for its derivative, in
// two forms without branches for a whole tile's epilogue (the library's erff branches on |x|, per value).  A NaN makes the
// product z Phi(z) a NaN in both.
//
// For 16-bit outputs, Abramowitz and Stegun's 7.1.26: for x >= 0, erfc(x) =
// (a1 t + .. + a5 t^5) exp(-x^2) within 1.5e-7, t = 1 / (1 + 0.3275911 x).  In fp32
// z Phi(z) is off by at most 3.1e-7 of |z| (near 0), a thousandth of an fp16 half
// step; far below 0, where it vanishes against |z|, by 7e-7 of itself at -1, 5e-4 at -4
// and 1 % at -8.
//
// For fp32 outputs, about twice the operations, within 1.7 half steps of |z| and, to
// where exp(-z^2 / 2) leaves the normal range (z = -13), 7 half steps of z Phi(z):
//   |z| < 1: 1/2 + z P(z^2), a series of the odd part;
//   else for x = |z|: Phi(-x) = exp(-x^2 / 2) r Q(r), r = 1 / (x + 3), where r Q(r) is the
//   integral's ratio to exp(-x^2 / 2), smooth and near 0.4 / x far out.
// P's and Q's coefficients are least-squares fits of the largest relative error (7e-10 on
// z^2 <= 1, 1.3e-8 on 1 <= x <= 14.5).  The exponent's rounding, half a step of x^2 / 2, would
// be 4e-6 of the exponential at x = 10: it is carried along (x^2 and its product with
// log2(e) / 2 each as a sum of two floats).  fp32 4096^3 977 us with the short form, 981
// with this; bf16 operands and fp32 C, 4096 x 4096 x 1024: 50.9 and 58.6.
template <int OUT>
__device__ __forceinline__ float normal_cdf(float z, float& exp_half) {
    if constexpr (OUT != OUT_F32) {
        const float x = __builtin_fabsf(z) * 0.7071067811865476f;
        const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * x);
        const float p =
            t * (0.254829592f +
                 t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
        const float q = 0.5f * p * __builtin_amdgcn_exp2f(-LOG2E * x * x);
        exp_half = __builtin_amdgcn_exp2f(-0.5f * LOG2E * z * z);
        return z < 0.0f ? q : 1.0f - q;
    } else {
        constexpr float C = 0.7213475204444817f, C_LO = 9.62981495e-9f;  // log2(e) / 2 as C + C_LO
        const float a = __builtin_fabsf(z);
        const float x = a > 20.0f ? 20.0f : a;
        const float h = x * x, h_lo = __builtin_fmaf(x, x, -h);
        const float y = -C * h;
        float y_lo = __builtin_fmaf(-C, h, -y);
        y_lo = __builtin_fmaf(-C_LO, h, y_lo);
        y_lo = __builtin_fmaf(-C, h_lo, y_lo);
        const float e = __builtin_amdgcn_exp2f(y);
        exp_half = __builtin_fmaf(e, y_lo * 0.6931471805599453f, e);
        const float r = __builtin_amdgcn_rcpf(x + 3.0f);
        float q = 286.15369f;
        q = __builtin_fmaf(q, r, -291.42086f);
        q = __builtin_fmaf(q, r, 70.1957199f);
        q = __builtin_fmaf(q, r, 3.02561309f);
        q = __builtin_fmaf(q, r, 7.94888492f);
        q = __builtin_fmaf(q, r, 3.15222491f);
        q = __builtin_fmaf(q, r, 1.19792494f);
        q = __builtin_fmaf(q, r, 0.398929489f);
        q *= exp_half * r;
        const float far = z < 0.0f ? q : 1.0f - q;
        float s = -7.654207365703769e-06f;  // (x = |z| where it is used)
        s = __builtin_fmaf(s, h, 0.00011348637053743005f);
        s = __builtin_fmaf(s, h, -0.0011863299878314137f);
        s = __builtin_fmaf(s, h, 0.009973322972655296f);
        s = __builtin_fmaf(s, h, -0.06649035960435867f);
        s = __builtin_fmaf(s, h, 0.3989422917366028f);
        return a < 1.0f ? __builtin_fmaf(z, s, 0.5f) : far;
    }
}

// act applied to NE values of an output in format OUT; `act` is wave-uniform, so one
// branch serves them all.
template <int OUT, int NE>
__device__ __forceinline__ void apply_act(float (&v)[NE], int act) {
    if (act == ACT_SILU) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] *= sigmoid(v[i]);
    } else if (act == ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] *= sigmoid(gelu_2t(v[i]));
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            float e;
            v[i] *= normal_cdf<OUT>(v[i], e);
        }
    } else if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
    }
}

template <int FMT>
constexpr int fmt_es = FMT == OUT_F32 ? 4 : 2;

// Eight consecutive elements of one row, in its storage format, moved through
// a buffer resource in 16-byte pieces.  Only the first `nvalid` of them belong
// to the row: the others load as 0 (the 16 bytes that hold the row's last
// element are inside the resource, bases and pitches being multiples of 16) and
// are not stored.  `off` is a byte offset, OOB_LANE where nvalid <= 0 would
// leave it inside the resource.
template <int FMT>
struct Row8 {
    u32x4 w[FMT == OUT_F32 ? 2 : 1];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off, int nvalid) {
        load_whole(r, off);
        if (nvalid < 8) mask(nvalid);
    }
    // All eight, or none (`off` outside the resource).
    __device__ __forceinline__ void load_whole(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        w[0] = load16(r, (int)off);
        if constexpr (FMT == OUT_F32) w[1] = load16(r, (int)(off + 16));
    }
    __device__ __forceinline__ void store_whole(__amdgpu_buffer_rsrc_t r, uint32_t off) const {
        __builtin_amdgcn_raw_buffer_store_b128(w[0], r, (int)off, 0, 0);
        if constexpr (FMT == OUT_F32)
            __builtin_amdgcn_raw_buffer_store_b128(w[1], r, (int)(off + 16), 0, 0);
    }
    // The same from a plain 16-byte aligned address (lanes on different rows).
    __device__ __forceinline__ void load_from(const char* p, int nvalid) {
        w[0] = nvalid > 0 ? *(const u32x4*)p : u32x4{0u, 0u, 0u, 0u};
        if constexpr (FMT == OUT_F32)
            w[1] = nvalid > 4 ? *(const u32x4*)(p + 16) : u32x4{0u, 0u, 0u, 0u};
        if (nvalid < 8) mask(nvalid);
    }
    __device__ __forceinline__ void mask(int nvalid) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (FMT == OUT_F32)
                w[j >> 2][j & 3] = j < nvalid ? w[j >> 2][j & 3] : 0u;
            else
                w[0][j >> 1] &= j < nvalid ? 0xffffffffu : (j & 1) ? 0x0000ffffu : 0xffff0000u;
        }
    }
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, int nvalid) const {
        constexpr int ES = fmt_es<FMT>;
        if (nvalid >= 8) {
            store_whole(r, off);
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                const uint32_t o = j < nvalid ? off + j * ES : OOB_LANE;
                if constexpr (FMT == OUT_F32)
                    __builtin_amdgcn_raw_buffer_store_b32(w[j >> 2][j & 3], r, (int)o, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b16(
                        (unsigned short)(w[0][j >> 1] >> (16 * (j & 1))), r, (int)o, 0, 0);
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (FMT == OUT_F32) {
                v[j] = as_float(w[j >> 2][j & 3]);
            } else {
                const uint32_t h = w[0][j >> 1] >> (16 * (j & 1)) & 0xffffu;
                if constexpr (FMT == OUT_BF16) v[j] = as_float(h << 16);
                else v[j] = (float)__builtin_bit_cast(_Float16, (unsigned short)h);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        if constexpr (FMT == OUT_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j >> 2][j & 3] = __builtin_bit_cast(uint32_t, v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[0][j] = pack16<FMT>(v[2 * j], v[2 * j + 1]);
        }
    }
};

// LDS bytes store_tile_full needs per wave: 32 rows of the wave's NJ * 32
// columns, the pitch padded by 8 floats so that the two lane groups, whose
// rows are 4 apart, write to different halves of the 64 banks (4 pitches are
// 32 modulo 64 floats) and rows stay 16-byte aligned.
template <int NJ>
constexpr int full_pitch = NJ * 32 + 8;
template <int NJ>
constexpr int full_lds = 32 * full_pitch<NJ> * 4;

// The full epilogue of one wave's MI x NJ blocks.  The accumulator layout has
// one column per lane, which would read R and write C and Z two bytes at a
// time; instead each 32-row strip goes through the wave's own LDS region (free
// after the K loop; the caller has a barrier before) and comes back eight
// consecutive columns per lane, so R, Z and C move in 16-byte pieces of whole
// row segments.  With one wave per SIMD nothing else hides a wait, so a strip is
// straight code: all its LDS reads, then the arithmetic with one branch per
// strip (none per value), then the stores; R of the next strip is loaded as
// soon as this one's is used.  The strips themselves are a loop (only the
// accumulators' copy to LDS is written out per strip), which keeps the code in
// the instruction cache.
// TR: the accumulators are blocks of 16 x 16, twice as many each way, and hold the transpose:
// row lane % 16 and, in register r, column 4 (lane / 16) + r of their block.
template <int OUT, int MI, int NJ, bool TR = false, class Acc>
__device__ __forceinline__ void store_tile_full(const Acc& acc, char* C, int M, int N,
                                                int ldc, int row0, int col0, int lane,
                                                const EpiArgs& e, char* lds) {
    if (row0 >= M || col0 >= N) return;  // this wave's part of the tile lies outside C
    constexpr int ES = fmt_es<OUT>;
    constexpr int P = full_pitch<NJ>;
    constexpr int LPR = NJ * 4;        // lanes per row
    constexpr int RPI = 64 / LPR;      // rows per pass of the wave
    constexpr int IT = 32 / RPI;       // passes per strip
    const int g = lane >> 5, li = lane & 31;
    const int c8 = (lane % LPR) * 8, r_in = lane / LPR;
    const int nvalid = N - (col0 + c8);
    // Wave-uniform: whether the last column falls inside some lane's eight.
    const bool ragged = (N & 7) != 0 && N - col0 < NJ * 32;
    float* const buf = (float*)lds;
    const __amdgpu_buffer_rsrc_t rc = c_rsrc(C, M, N, ldc, row0, col0, ES);
    // NULL operands get empty ranges: their loads give zeros, their stores drop.
    const __amdgpu_buffer_rsrc_t rr =
        e.res ? c_rsrc((char*)e.res, M, N, e.ldr, row0, col0, ES) : make_rsrc(C, 0);
    const __amdgpu_buffer_rsrc_t rz =
        e.pre ? c_rsrc(e.pre, M, N, e.ldz, row0, col0, ES) : make_rsrc(C, 0);
    // Columns and rows past the edges read the last one's values: in bounds, and
    // what they feed is not stored.
    float bias[8], sb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int col = col0 + c8 + j < N ? col0 + c8 + j : N - 1;
        bias[j] = e.bias ? e.bias[col] : 0.0f;
        sb[j] = e.scale_b ? e.scale_b[col] : 1.0f;
    }
    // Byte offset of this lane's eight columns in row `r` of the wave's rows.
    auto at = [&](int r, int ld) {
        return nvalid > 0 ? (uint32_t)((r * ld + c8) * ES) : OOB_LANE;
    };
    Row8<OUT> res[IT];
    if (e.res) {
#pragma unroll
        for (int it = 0; it < IT; ++it) res[it].load_whole(rr, at(it * RPI + r_in, e.ldr));
    }
#pragma unroll 1
    for (int mi = 0; mi < MI; ++mi) {
        if (row0 + mi * 32 >= M) break;
        // This lane's values of the strip to LDS (after the previous strip's reads).
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int k = 0; k < MI; ++k) {
            if (k != mi) continue;
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj) {
                if constexpr (TR) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *(f32x4*)(buf + (16 * (q >> 1) + (lane & 15)) * P + nj * 32 +
                                  16 * (q & 1) + 4 * (lane >> 4)) =
                            acc[2 * k + (q >> 1)][2 * nj + (q & 1)];
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        buf[(8 * (r >> 2) + 4 * g + (r & 3)) * P + nj * 32 + li] = acc[k][nj][r];
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float v[IT * 8];
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const float* p = buf + (it * RPI + r_in) * P + c8;
            const f32x4 lo = *(const f32x4*)p, hi = *(const f32x4*)(p + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[it * 8 + j] = lo[j];
                v[it * 8 + 4 + j] = hi[j];
            }
        }
        if (e.scale_a) {
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int row = row0 + mi * 32 + it * RPI + r_in;
                const float sa = e.scale_a[row < M ? row : M - 1];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[it * 8 + j] = v[it * 8 + j] * sa * sb[j];
            }
        }
#pragma unroll
        for (int i = 0; i < IT * 8; ++i) v[i] += bias[i & 7];
        // Rows it of the strip, from v, to an output.
        auto put = [&](__amdgpu_buffer_rsrc_t r, int ld) {
            Row8<OUT> o;
            if (!ragged) {
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = v[it * 8 + j];
                    o.set(x);
                    o.store_whole(r, at(mi * 32 + it * RPI + r_in, ld));
                }
            } else {
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = v[it * 8 + j];
                    o.set(x);
                    o.store(r, at(mi * 32 + it * RPI + r_in, ld), nvalid);
                }
            }
        };
        if (e.pre) put(rz, e.ldz);
        apply_act<OUT>(v, e.act);
        if (e.res) {
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                float x[8];
                res[it].get(x);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[it * 8 + j] += x[j];
                // past the tile's last strip: rows of other tiles, or outside R
                res[it].load_whole(rr, at((mi + 1) * 32 + it * RPI + r_in, e.ldr));
            }
        }
        put(rc, ldc);
    }
}

// The full epilogue on NE fp32 sums v[i] of C's elements (row[i], col[i]),
// through plain pointers, for kernels that finish few elements per lane;
// elements outside M x N are skipped.  R is read before anything is stored.
template <int OUT, int NE>
__device__ __forceinline__ void finish_full(float (&v)[NE], const int (&row)[NE],
                                            const int (&col)[NE], char* C, int M, int N, int ldc,
                                            const EpiArgs& e) {
    float res[NE];
    bool in[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        in[i] = row[i] < M && col[i] < N;
        res[i] = e.res && in[i] ? load_c<OUT>(e.res, (int64_t)row[i] * e.ldr + col[i]) : 0.0f;
        if (e.scale_a && in[i]) v[i] = v[i] * e.scale_a[row[i]] * e.scale_b[col[i]];
        if (e.bias && in[i]) v[i] += e.bias[col[i]];
    }
    if (e.pre) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (in[i]) store_c<OUT>(e.pre, (int64_t)row[i] * e.ldz + col[i], v[i]);
    }
    apply_act<OUT>(v, e.act);
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (in[i]) store_c<OUT>(C, (int64_t)row[i] * ldc + col[i], e.res ? v[i] + res[i] : v[i]);
}

// ------------------------------------------------------------- column sums
//
// out[n] = sum over g < G of part[g][n], in a fixed order, by a workgroup of 256
// threads per 16 columns: 16 threads per column take every sixteenth row, sixteen
// loads in flight, then LDS adds the sixteen.  (64 columns per workgroup left most
// CUs idle: 256 x 4096 5.5 us.)
constexpr int COL_REDUCE_LDS = 256;  // floats

__device__ __forceinline__ void col_reduce(int block, const ColReduceArgs& a, float* lds) {
    const int c = (int)threadIdx.x & 15, q = (int)threadIdx.x >> 4;
    const int col = block * 16 + c;
    float v = 0.0f;
    if (col < a.N) {
        const float* p = a.part + col;
        for (int g = q; g < a.G; g += 16 * 16) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {  // rows past G: the last one's value, not added
                const int r = g + 16 * i < a.G ? g + 16 * i : a.G - 1;
                x[i] = p[(int64_t)r * a.ldp];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v += g + 16 * i < a.G ? x[i] : 0.0f;
        }
    }
    lds[threadIdx.x] = v;
    __syncthreads();
    if (q == 0 && col < a.N) {
#pragma unroll
        for (int i = 1; i < 16; ++i) v += lds[i * 16 + c];
        a.out[col] = v;
    }
}

}  // namespace dgemm
