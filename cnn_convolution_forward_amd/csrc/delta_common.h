// delta_common.h -- what the block kernels of the gated delta rule share
// (k_delta_prep.hip, k_delta_fwd.hip, k_delta_bwd.hip).
//
// Products run on v_mfma_f32_32x32x16_f16 with operands that are sums of two fp16
// numbers, hi + lo, under a power of two that brings the largest magnitude of the
// operand's row or column to [2^13, 2^14): 22 bits of a value down to 2^-16 of that largest,
// and an absolute error of 2^-38 of it below (half of fp16's smallest step; measured).  What shares a power of two is what one
// result is summed from, so that nothing takes the bits of results that do not depend on it: rows of q, k, T, P, and of the products
// in the gradients; columns of a state, and of values by 32 tokens.  (The gradients of q and k take one for all of a state.)
// An infinity has hi = inf and lo = NaN, and the rest of its row or column nothing.  hi hi + hi lo + lo hi then
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
#include "mfma_common.h"
#include "seq_common.h"

namespace convfwd {

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef float acc_t __attribute__((ext_vector_type(16)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kBlock = 64;                    // tokens
constexpr double kLog2eD = 1.4426950408889634074;

// exp of a difference of cumulative log decays, both times log2(e).
__device__ __forceinline__ float decay_of(double gi, double gj) { return __builtin_amdgcn_exp2f((float)(gi - gj)); }
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

// The power of two that brings a (>= 0) to [2^13, 2^14), at most 2^113, so that its inverse is a normal number; infinities get the
// smallest.  What such an inverse is multiplied with may be small, or large, too: the sum meets it first where it is below 1.
__device__ __forceinline__ float pow2_scale(float a) {
    const int e = (int)(__float_as_uint(a) >> 23) & 255;
    return __uint_as_float((uint32_t)min(267 - e, 240) << 23);
}
// 1/s of a power of two.
__device__ __forceinline__ float pow2_inv(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Eight values times a power of two as hi + lo, or as hi alone.  hi is hidden from the optimiser, which would
// make it a second time from the values where lo needs it.
struct Pair {
    h8_t hi, lo;
};
template <typename F> __device__ __forceinline__ h8_t half8(float scale, F value) {
    h8_t v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (_Float16)(value(j) * scale);
    return v;
}
template <typename F> __device__ __forceinline__ Pair split8(float scale, F value) {
    typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
    Pair p;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        h2_t h = {(_Float16)(value(j) * scale), (_Float16)(value(j + 1) * scale)};
        asm("" : "+v"(h));
        p.hi[j] = h[0], p.hi[j + 1] = h[1];
        p.lo[j] = (_Float16)fmaf(value(j), scale, -(float)h[0]);
        p.lo[j + 1] = (_Float16)fmaf(value(j + 1), scale, -(float)h[1]);
    }
    return p;
}

// Four values of one column of LDS, from four rows.  Of 16 lanes, p is row lane/4 % 4, columns 4 (lane % 4) .. + 3, and lane i gets
// column i: a transposed page from an upright one.
__device__ __forceinline__ h4_t read_columns(const _Float16 *p) {
    typedef short s4_t __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4_t lds_s4_t;
    return __builtin_bit_cast(h4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t *)p));
}

__device__ __forceinline__ float max_abs(const acc_t &v, float m = 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}
// Over the two halves of a wave: the whole of a column of a result.
__device__ __forceinline__ float max_halves(float m) { return fmaxf(m, __shfl_xor(m, 32)); }

// Rows record of a block and value head: 64 floats each, then a scalar.  The first four fill a page.  kRowInv*: what the power of
// two of each row of T, P and, backward, T^T and P^T has to be made good with.  Rows have their own, as they belong to tokens:
// queries and keys far larger than another token's, or infinite, cost that one nothing.
enum { kRowEK, kRowInvT, kRowFK, kRowEQ, kRowInvP, kForwardRows,
       kRowEZ = 0 /* E K beta InvTT, of Z in dS */, kRowInvPT = 1, kRowBeta = 4, kRowEKBack, kRowE, kRowF, kRowKK, kRowKQ, kRowSizeK, kRowSizeQ,
       kRowInvTBack, kRowInvTT, kRowG /* doubles, times log2(e) */, kRowG2, kRowCount };
enum { kGamma = 64 * kRowCount };
constexpr int kRowsFloats = 64 * kRowCount + 64;
static_assert(kRowG % 2 == 0 && (int)kForwardRows <= (int)kRowCount, "doubles are aligned");

// Pages of T, TT, P, PT (64x64, lower triangular): 6 of 8, hi and lo.  T and P: lane = row i, places = columns j; page of
// block ib, m: ib 0 has m = 0, 1.  TT and PT: lane = column j, places = rows i; block 1 has m = 2, 3.
__host__ __device__ constexpr int low_page(int ib, int m) { return ib ? 2 + m : m; }
__host__ __device__ constexpr int high_page(int jb, int m) { return jb ? 2 + m : m; }
constexpr int kTriPages = 6;

// Where the parts of the workspace lie.  Counts are pages.
struct DeltaWs {
    uint4 *qk;               // per block and key head: K, Q, or backward K, KT, Q, QT, each `parts` times
    uint4 *tri;              // per block and value head, forward: T hi, T lo, P hi, P lo; backward: T, TT, PT, hi and lo
    float *rows;             // per block and value head: kRowsFloats
    float *ends;             // backward: gradients of the states behind the blocks, dk x dv padded to 32s
    float *sums;             // per segment and value head: what it makes of a state, an offset dk x dv and a matrix dk x dk,
                             // transposed, both padded to 32s
    int segments, seg_blocks;
    int qk_pages, tri_pages;
    int per;                 // blocks of each of equal sequences
    int64_t blocks;
};

// The parts in `base`; returns the bytes they take.
int64_t delta_layout(const Seq &s, const Delta &d, bool bf16, bool bwd, void *base, DeltaWs &ws);
// fill: rows of the outputs that no sequence holds.
void launch_delta_prep(const Seq &s, const Delta &d, bool bf16, bool bwd, const DeltaWs &ws, const DeltaIn &in, const Fill &fill, hipStream_t st);
struct FillRows {
    RowsOut o;
    int cols, esize;
};
inline Fill delta_fill(const Seq &s, std::initializer_list<FillRows> outs) {
    Fill f = {};
    if (!s.fill || s.rows == 0) return f;
    for (const FillRows &r : outs) {
        f.p[f.n] = (uint16_t *)r.o.p, f.ld[f.n] = r.o.ld * (r.esize / 2), f.units[f.n] = r.cols * (r.esize / 2);
        ++f.n;
    }
    f.blocks = (int)std::min<int64_t>((s.rows + 255) / 256, 1024);
    return f;
}

// The joining of segments; `back`: of gradients, from the last segment to the first.
hipError_t launch_delta_join(const Seq &s, const Delta &d, const DeltaWs &ws, bool back, hipStream_t st);

// Waves of a workgroup share the pages in LDS; fewer to a workgroup where that leaves compute units empty.
inline int waves_of(int64_t chains, int slices) {
    int waves = slices < 4 ? slices : 4;
    while (waves > 1 && chains * ((slices + waves - 1) / waves) < 256) waves = (waves + 1) / 2;
    return waves;
}

// First block number of sequence b, and block n's place.
__device__ __forceinline__ int64_t first_block(const Seq &s, int per, int b, int64_t first) {
    return s.off ? first / kBlock + b : (int64_t)b * per;
}
// First segment number of sequence b; numbers are unique, as those of blocks are.
__device__ __forceinline__ int64_t first_segment(const Seq &s, const DeltaWs &ws, int b, int64_t first) {
    return s.off ? first / ((int64_t)kBlock * ws.seg_blocks) + b : (int64_t)b * ws.segments;
}
__device__ __forceinline__ Block find_block(const Seq &s, int per, int64_t n) {
    if (s.off) return packed_block(s, kBlock, n);
    Block t;
    t.b = (int)(n / per);
    t.k = (int)(n % per);
    return t;
}

// ---- memory ----

// Pages from global memory to LDS, asynchronously: four to a workgroup's wave in turn.  The instruction takes the
// LDS address from M0 (one wait state after it is written) and adds its offset on both sides; five states cover a base
// that a vector instruction wrote just before, which the compiler does not look for here.  In assembly because the
// compiler, which cannot tell one buffer from the other, waits for all such loads before any
// read of LDS.  They have no output registers; wait_copies is their wait.  M0 is named as written, which the compiler
// warns about, as it never keeps a value there.
__device__ __forceinline__ void copy4(const uint4 *src, uint32_t dst, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2\n\tglobal_load_lds_dwordx4 %1, %2 offset:1024\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:2*1024\n\tglobal_load_lds_dwordx4 %1, %2 offset:3*1024"
                 :
                 : "s"(dst), "v"(at), "s"(src)
                 : "memory", "m0");
}
__device__ __forceinline__ void copy1(const uint4 *src, uint32_t dst, uint32_t at) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(dst), "v"(at), "s"(src) : "memory", "m0");
}
template <int PAGES> __device__ __forceinline__ void copy_pages(const void *from, uint32_t dst, int wave, int waves, int lane) {
    const uint4 *src = (const uint4 *)from;
    for (int i = 4 * wave; i < PAGES; i += 4 * waves) {
        if (PAGES % 4 == 0 || i + 4 <= PAGES) {
            copy4(src + i * kPage, dst + i * 1024, 16 * lane);
        } else {
            for (int j = i; j < PAGES; ++j) copy1(src + j * kPage, dst + j * 1024, 16 * lane);
        }
    }
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p;
}

// Buffers of one block's rows, and of one head's state: offsets at or past `bytes` load zeros and store nothing, so rows
// past the sequence's end, columns past the head and the padding of a state need no branch.  Sizes stay below 2^30 (delta_api.cpp).
template <typename T> __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const T *p, int n, int64_t ld, int cols) {
    return make_rsrc(p, (uint32_t)(((n - 1) * ld + cols) * sizeof(T)));
}
__device__ __forceinline__ float load_at(__amdgpu_buffer_rsrc_t r, uint32_t off) { return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0)); }
__device__ __forceinline__ void store_at(__amdgpu_buffer_rsrc_t r, uint32_t off, float v) { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)off, 0, 0); }

// A column of a block's rows, in the order of a result's registers: token 32 (i / 16) + acc_row(i % 16, half).  at: the
// column's bytes, or kOob for none.
// As loaded: 16 bits are not packed, which would wait for the load.
template <typename T> struct Column {
    uint32_t v[32];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t ld, int half) {
        const uint32_t base = at + 4 * half * ld;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int off = (int)(base + (32 * (i >> 4) + acc_row(i & 15, 0)) * ld);
            if constexpr (sizeof(T) == 2) v[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
            else v[i] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
        }
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(sizeof(T) == 2 ? v[i] << 16 : v[i]); }
};

// Of tokens 32 t .. 32 t + 31.
template <typename T> __device__ __forceinline__ float max_column(const Column<T> &c, int t) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(c.get(16 * t + i)));
    return m;
}

// A state's columns (dim_k x dim_v, dim_v apart) to and from a result's registers.
template <int DKB> __device__ __forceinline__ void load_state(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t ld, int half, acc_t (&S)[DKB]) {
    const uint32_t base = at + 4 * half * ld;
#pragma unroll
    for (int i = 0; i < 16 * DKB; ++i) {
        S[i >> 4][i & 15] = load_at(r, base + (32 * (i >> 4) + acc_row(i & 15, 0)) * ld);
    }
}
template <int DKB> __device__ __forceinline__ void store_state(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t ld, int half, const acc_t (&S)[DKB]) {
    const uint32_t base = at + 4 * half * ld;
#pragma unroll
    for (int i = 0; i < 16 * DKB; ++i) store_at(r, base + (32 * (i >> 4) + acc_row(i & 15, 0)) * ld, S[i >> 4][i & 15]);
}

// What a segment makes of a state: 32 columns of the offset, or (from slice `slices` on) of the matrix, as rows of its transpose.
template <int DKB> __device__ __forceinline__ void store_sum(float *sums, int slices, int slice, int lane, const acc_t (&S)[DKB]) {
    const int half = lane >> 5, col = lane & 31, offset = 32 * DKB * 32 * slices;
    if (slice < slices) {
        store_state<DKB>(make_rsrc(sums, 4 * offset), 4 * (32 * slice + col), 128 * slices, half, S);
    } else if (slice < slices + DKB) {
        float *p = sums + offset + (32 * (slice - slices) + col) * 32 * DKB + 4 * half;
#pragma unroll
        for (int i = 0; i < 4 * DKB; ++i) {
            const float f[4] = {S[i >> 2][4 * (i & 3)], S[i >> 2][4 * (i & 3) + 1], S[i >> 2][4 * (i & 3) + 2], S[i >> 2][4 * (i & 3) + 3]};
            store_f32(p + 8 * i, f);
        }
    }
}

// Four neighbouring columns of a row where all four are the head's, of which `left` are; else zeros.  The address need only
// be aligned to an element.
template <typename T> __device__ __forceinline__ f4_t load4(__amdgpu_buffer_rsrc_t r, uint32_t off, int left) {
    f4_t f;
    const int o = left >= 4 ? (int)off : (int)kOob;
    if constexpr (sizeof(T) == 2) {
        typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
        const u2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, 0);
        f[0] = __uint_as_float(v[0] << 16), f[1] = __uint_as_float(v[0] & 0xffff0000u);
        f[2] = __uint_as_float(v[1] << 16), f[3] = __uint_as_float(v[1] & 0xffff0000u);
    } else {
        const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(v[j]);
    }
    return f;
}
// The last columns of a head whose width is no multiple of four, one by one (a wide load that passes the buffer's end is dropped
// whole); zeros where `left` is 4 or more, or none.
template <typename T> __device__ __forceinline__ f4_t load_rest(__amdgpu_buffer_rsrc_t r, uint32_t off, int left) {
    f4_t f = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int e = left < 4 && left > j ? (int)off + j * (int)sizeof(T) : (int)kOob;
        if constexpr (sizeof(T) == 2) f[j] = __uint_as_float((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, e, 0, 0) << 16);
        else f[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, e, 0, 0));
    }
    return f;
}
__device__ __forceinline__ void store_wide(__amdgpu_buffer_rsrc_t r, int off, const float (&f)[4], uint16_t *) {
    typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
    const u2_t v = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
    __builtin_amdgcn_raw_buffer_store_b64(v, r, off, 0, 0);
}
__device__ __forceinline__ void store_wide(__amdgpu_buffer_rsrc_t r, int off, const float (&f)[4], float *) {
    const u32x4_t v = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 0);
}
// The same for storing.  ragged: the width of heads is no multiple of four.
template <typename T> __device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t r, uint32_t off, int left, bool ragged, const float (&f)[4], T *kind) {
    store_wide(r, left >= 4 ? (int)off : (int)kOob, f, kind);
    if (ragged) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int o = left < 4 && left > j ? (int)off + j * (int)sizeof(T) : (int)kOob;
            if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(to_bf16(f[j]), r, o, 0, 0);
            else store_at(r, o, f[j]);
        }
    }
}

}  // namespace convfwd
