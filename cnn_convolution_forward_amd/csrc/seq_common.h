// seq_common.h -- what the kernels over sequences of tokens share: where a
// sequence's rows are, and loads and stores of VEC adjacent channels.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "seq_internal.h"

// A product and a sum are one operation only where the code says fmaf: whole and ragged runs, compiled
// apart, then give the same bits.
#pragma clang fp contract(off)

namespace convfwd {

// First row and length of sequence b.  Offsets come from device memory that
// the host has not seen, so they are clamped here: every row read or written
// is one of the tensor's.
__device__ __forceinline__ void seq_range(const Seq &s, int b, int64_t &first, int &len) {
    if (!s.off) {
        first = (int64_t)b * s.T;
        len = s.T;
        return;
    }
    const int64_t o0 = min(max((int64_t)s.off[b], (int64_t)0), s.rows);
    const int64_t o1 = min(max((int64_t)s.off[b + 1], o0), s.rows);
    first = o0;
    len = (int)min(o1 - o0, (int64_t)s.T);
}

// VEC adjacent channels as fp32.  T is uint16_t (bf16 bits) or float.  The
// address need only be aligned to an element: rows of odd width and column
// slices are read and written with the same wide accesses as aligned ones.
template <typename T, int VEC> struct Pack;
template <> struct Pack<uint16_t, 1> { typedef uint16_t type; };
template <> struct Pack<uint16_t, 2> { typedef uint32_t type; };
template <> struct Pack<uint16_t, 4> { typedef uint2 type; };
template <> struct Pack<uint16_t, 8> { typedef uint4 type; };
template <> struct Pack<float, 1> { typedef float type; };
template <> struct Pack<float, 2> { typedef float2 type; };
template <> struct Pack<float, 4> { typedef float4 type; };

template <typename T, int VEC>
__device__ __forceinline__ typename Pack<T, VEC>::type load_pack(const T *p) {
    typename Pack<T, VEC>::type v;
    __builtin_memcpy(&v, p, sizeof(v));
    return v;
}
// The same for data that a kernel reads once, with the non-temporal hint: at 8 x 2048 x 2048 bf16 the
// recurrence's backward pass takes 123 us without and 107 us with it, the causal convolution at 8 x 4096 x
// 4096 120 and 89 us.  Only for rows that start on a line: where rows share lines, these are fetched
// twice (5003 x 999 fp32, convolution backward: 21.2 us without, 24.1 us with it).  Stores with the hint are
// for the recurrence: at the end of a kernel what is dirty in the caches has to leave them before the
// next one starts (4 x 1024 x 2048 forward 23.4 us without, 21.4 us with it; backward at 8 x 4096 x 4096
// 409 and 387 us, at 8 x 2048 x 2048 107 and 109 us).  The causal convolution is slower with them (88.7 and
// 107 us at 8 x 4096 x 4096).
template <typename T, int VEC>
__device__ __forceinline__ typename Pack<T, VEC>::type load_once(const T *p) {
    typedef typename Pack<T, VEC>::type V;
    if constexpr (sizeof(V) < 4) {
        return load_pack<T, VEC>(p);
    } else {
        typedef uint32_t W __attribute__((ext_vector_type(sizeof(V) / 4), aligned(sizeof(T))));
        const W w = __builtin_nontemporal_load(reinterpret_cast<const W *>(p));
        V v;
        __builtin_memcpy(&v, &w, sizeof(v));
        return v;
    }
}
inline bool read_once(const void *p, int64_t ld, size_t esize) { return (uintptr_t)p % 64 == 0 && ld * (int64_t)esize % 64 == 0; }
template <bool ONCE = false, typename T, typename V> __device__ __forceinline__ void store_pack(T *p, const V &v) {
    if constexpr (ONCE && sizeof(V) >= 4) {
        typedef uint32_t W __attribute__((ext_vector_type(sizeof(V) / 4), aligned(sizeof(T))));
        W w;
        __builtin_memcpy(&w, &v, sizeof(v));
        __builtin_nontemporal_store(w, reinterpret_cast<W *>(p));
    } else {
        __builtin_memcpy(p, &v, sizeof(v));
    }
}

// bf16 bits to fp32 is a shift; fp32 to bf16 rounds to nearest even (a NaN
// stays a NaN) with the conversion instruction.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

template <int VEC> __device__ __forceinline__ void unpack(const uint32_t *u, float *f) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_f32(uint16_t v, float (&f)[1]) { f[0] = __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void to_f32(uint32_t v, float (&f)[2]) { unpack<2>(&v, f); }
__device__ __forceinline__ void to_f32(uint2 v, float (&f)[4]) {
    const uint32_t u[2] = {v.x, v.y};
    unpack<4>(u, f);
}
__device__ __forceinline__ void to_f32(uint4 v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    unpack<8>(u, f);
}
__device__ __forceinline__ void to_f32(float v, float (&f)[1]) { f[0] = v; }
__device__ __forceinline__ void to_f32(float2 v, float (&f)[2]) { f[0] = v.x, f[1] = v.y; }
__device__ __forceinline__ void to_f32(float4 v, float (&f)[4]) { f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w; }

template <typename T, int VEC> __device__ __forceinline__ void load_f32(const T *p, float (&f)[VEC]) {
    to_f32(load_pack<T, VEC>(p), f);
}

template <bool ONCE = false> __device__ __forceinline__ void store_f32(uint16_t *p, const float (&f)[1]) { *p = to_bf16(f[0]); }
template <bool ONCE = false> __device__ __forceinline__ void store_f32(uint16_t *p, const float (&f)[2]) {
    store_pack<ONCE>(p, pack_bf16(f[0], f[1]));
}
template <bool ONCE = false> __device__ __forceinline__ void store_f32(uint16_t *p, const float (&f)[4]) {
    store_pack<ONCE>(p, make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])));
}
template <bool ONCE = false> __device__ __forceinline__ void store_f32(uint16_t *p, const float (&f)[8]) {
    store_pack<ONCE>(p, make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
}
template <bool ONCE = false, int VEC> __device__ __forceinline__ void store_f32(float *p, const float (&f)[VEC]) {
    store_pack<ONCE>(p, f);
}

// Blocks of `tokens` tokens, numbered through the batch.  Equal sequences have
// per = ceil(T/tokens) (at least one) each, and so have packed ones if that is
// one.  Longer packed ones take the numbers from first/tokens + b on: distinct,
// and at most rows/tokens + B of them, whatever the lengths; a few stay unused.
struct Block {
    int b, k;               // sequence, and block in it: negative or past its end for an unused number
};
__host__ __device__ __forceinline__ int64_t block_count(const Seq &s, int tokens, int per) {
    return s.off && per > 1 ? s.rows / tokens + s.B : (int64_t)s.B * per;
}
// The block of number n; all lanes of a wave together.  64 starts are looked at in one load, so that 64
// sequences take one round and 4096 two.  Offsets that descend lead to some sequence, and to a block that
// the tensor could have, or to an unused number.
__device__ __forceinline__ Block packed_block(const Seq &s, int tokens, int64_t n) {
    const auto start = [&](int b) { return min(max((int64_t)s.off[b], (int64_t)0), s.rows) / tokens + b; };
    Block t;
    t.b = 0;
    for (int left = s.B; left > 1;) {                   // the last of `left` sequences from t.b on that starts at or before n
        const int step = (left + 63) / 64, i = t.b + (int)(threadIdx.x & 63) * step;
        const uint64_t on = __ballot(i < t.b + left && start(min(i, s.B - 1)) <= n);
        const int j = on ? 63 - __builtin_clzll(on) : 0;
        t.b += j * step;
        left = min(step, left - j * step);
    }
    const int64_t k = n - start(t.b);
    t.k = k >= 0 && k <= s.rows / tokens ? (int)k : -1;
    return t;
}

// Rows of up to three outputs that no sequence holds, to be set to zero: 64 rows to a wave, `blocks`
// workgroups for all of them (0: nothing is filled).  Rows are counted in units of two bytes.
struct Fill {
    uint16_t *p[3];
    int64_t ld[3];
    int n, units, blocks;
};
template <typename T> Fill fill_of(const Seq &s, int waves, std::initializer_list<T *> out, std::initializer_list<int64_t> ld) {
    constexpr int e = sizeof(T) / 2;
    Fill f = {};
    if (!s.fill || s.rows == 0) return f;
    for (T *o : out) f.p[f.n++] = (uint16_t *)o;
    int i = 0;
    for (int64_t l : ld) f.ld[i++] = l * e;
    f.units = s.C * e;
    f.blocks = (int)std::min<int64_t>((s.rows + 64 * waves - 1) / (64 * waves), 1024);
    return f;
}
// Worker `k` of n workgroups.  Each lane finds out about one row, by bisection of the offsets.
__device__ __forceinline__ void fill_rows(const Seq &s, const Fill &f, int64_t k, int64_t n) {
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    for (int64_t r0 = (k * waves + (threadIdx.x >> 6)) * 64; r0 < s.rows; r0 += n * waves * 64) {
        const int64_t r = r0 + lane;
        int lo = 0, hi = s.B;                           // sequences from lo on start behind row r
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (min(max((int64_t)s.off[mid], (int64_t)0), s.rows) <= r) lo = mid + 1;
            else hi = mid;
        }
        bool held = false;
        if (lo > 0) {
            int64_t first;
            int len;
            seq_range(s, lo - 1, first, len);
            held = r < first + len;
        }
        for (uint64_t open = __ballot(!held && r < s.rows); open; open &= open - 1) {
            const int64_t row = r0 + __builtin_ctzll(open);
            for (int o = 0; o < f.n; ++o) {
                uint16_t *p = f.p[o] + row * f.ld[o];
                for (int c = 8 * lane; c < f.units; c += 8 * 64) {
                    if (c + 8 <= f.units) {
                        store_pack(p + c, make_uint4(0, 0, 0, 0));
                    } else {
                        for (int q = c; q < f.units; ++q) p[q] = 0;
                    }
                }
            }
        }
    }
}

constexpr float kLog2e = 1.44269504088896340736f;

// 1/(1 + exp(-v)): 0 where that is no normal number (the reciprocal flushes, exp(-v) = inf
// gives 0); NaN stays NaN.
__device__ __forceinline__ float sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

}  // namespace convfwd
