// delta_common.h -- what the block kernels of the gated delta rule share
// (k_delta_prep.hip, k_delta_fwd.hip, k_delta_bwd.hip).
//
// Products run on v_mfma_f32_32x32x16_f16 with operands that are sums of two fp16
// numbers, hi + lo, under a power of two that brings the largest magnitude of
// the operand's row, column or tile to [2^13, 2^14): 22 bits of every value, and an
// absolute error of 2^-28 of the largest for small ones.  hi hi + hi lo + lo hi then
// has the accuracy of an fp32 product (what is left out is 2^-22 of it) at three
// times the cost of an fp16 one and a fifth of the fp32 matrix rate's.  bf16
// queries, keys, values and upstream gradients fit one fp16 number exactly (8 bits).
//
// A "page" is the 1 KB that one wave holds as an operand of one product: lane l
// has row l%32 (of A, or column of B) and 8 of 16 places of the contraction.
// Place s of half h = l/32 of page m is element page_at(m, h, s): the order in which a
// 32x32 result lies in registers, so that registers 8 m' .. 8 m'+7 of a result
// are, converted, page 2 block + m' of an operand of the next product.  Chains of
// products stay in registers; no transposition, no LDS.
#pragma once

#include "delta_internal.h"
#include "seq_common.h"

namespace convfwd {

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef float acc_t __attribute__((ext_vector_type(16)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kBlock = 64;                    // tokens
constexpr int kPage = 64;                     // uint4s of a page

__host__ __device__ constexpr int page_at(int m, int h, int s) { return 16 * m + (s < 4 ? 4 * h + s : 4 + 4 * h + s); }

// Row, within 32, of register i of a result; its column is the lane modulo 32.
__device__ __forceinline__ constexpr int acc_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

__device__ __forceinline__ acc_t mfma(h8_t a, h8_t b, acc_t c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ acc_t zeros() {
    acc_t z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// The power of two that brings a (>= 0) to [2^13, 2^14), at most 2^most; infinities get the smallest.
__device__ __forceinline__ float pow2_scale(float a, int most = 113) {
    const int e = (int)(__float_as_uint(a) >> 23) & 255;
    return __uint_as_float((uint32_t)min(267 - e, 127 + most) << 23);
}
// 1/s of a power of two.
__device__ __forceinline__ float pow2_inv(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Eight values as hi + lo.
struct Pair {
    h8_t hi, lo;
};
template <typename F> __device__ __forceinline__ Pair split8(F value) {
    Pair p;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = value(j);
        p.hi[j] = (_Float16)x;
        p.lo[j] = (_Float16)(x - (float)p.hi[j]);
    }
    return p;
}

__device__ __forceinline__ float max_abs(const acc_t &v, float m = 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}
// Over the two halves of a wave: the whole of a column of a result.
__device__ __forceinline__ float max_halves(float m) { return fmaxf(m, __shfl_xor(m, 32)); }

// Rows record of a block and value head: 64 floats each, then scalars.  The first four fill a page.
enum { kRowBEK, kRowBeta, kRowFK, kRowEQ, kRowE, kRowF, kRowKK, kRowKQ, kRowSizeK, kRowSizeQ, kRowG /* doubles */, kRowG2, kRowCount };
enum { kGamma = 64 * kRowCount, kInvT, kInvP };
constexpr int kRowsFloats = 64 * kRowCount + 64;

// Pages of T, TT, P, PT (64x64, lower triangular): 6 of 8, hi and lo.  T and P: lane = row i, places = columns j; page of
// block ib, m: ib 0 has m = 0, 1.  TT and PT: lane = column j, places = rows i; block 1 has m = 2, 3.
__host__ __device__ constexpr int low_page(int ib, int m) { return ib ? 2 + m : m; }
__host__ __device__ constexpr int high_page(int jb, int m) { return jb ? 2 + m : m; }
constexpr int kTriPages = 6;

// Where the parts of the workspace lie.  Counts are pages.
struct DeltaWs {
    uint4 *qk;               // per block and key head: K, KT, Q, QT (backward only), each `parts` times
    uint4 *tri;              // per block and value head, forward: T hi, T lo, P hi, P lo; backward: T, TT, PT, hi and lo
    float *rows;             // per block and value head: kRowsFloats
    float *ends;             // backward: gradients of the states behind the blocks, dk x dv padded to 32s
    int qk_pages, tri_pages;
    int per;                 // blocks of each of equal sequences
    int64_t blocks;
};

// The parts in `base`; returns the bytes they take.
int64_t delta_layout(const Seq &s, const Delta &d, bool bf16, bool bwd, void *base, DeltaWs &ws);
void launch_delta_prep(const Seq &s, const Delta &d, bool bf16, bool bwd, const DeltaWs &ws, const DeltaIn &in, hipStream_t st);

// First block number of sequence b, and block n's place.
__device__ __forceinline__ int64_t first_block(const Seq &s, int per, int b, int64_t first) {
    return s.off ? first / kBlock + b : (int64_t)b * per;
}
__device__ __forceinline__ Block find_block(const Seq &s, int per, int64_t n) {
    if (s.off) return packed_block(s, kBlock, n);
    Block t;
    t.b = (int)(n / per);
    t.k = (int)(n % per);
    return t;
}

}  // namespace convfwd
