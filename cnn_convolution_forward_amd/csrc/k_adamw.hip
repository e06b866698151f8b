// k_adamw.hip -- the AdamW step over many tensors at once (conv_adamw_step),
// moments in fp32 or in 8-bit codes with a scale per 256 elements.
//
// A pass over memory: per element p (read, written), the gradient (read), both
// moments (read, written) and the bf16 copy (written): 30 bytes with fp32
// gradients and moments, 18 with 8-bit moments.  HBM is the bound.
//
// One launch takes up to kMaxTensors tensors, whose pointers travel in the
// kernel's arguments: nothing is copied to the device and nothing has to be
// kept between calls.  Blocks of kChunk elements are numbered through all of
// its tensors; a workgroup finds its tensor by looking at all first numbers.
//
// Measured: 26 M parameters in 60 tensors with fp32 moments 129.1 us, 6.0 TB/s (a
// large copy reaches 5.2); 60 M in 120 with 8-bit moments, their values read back
// too, 319 us, 4.5 TB/s (219 us for the step alone, its vector instructions taking
// about as long as its bytes); 20 000 in 14 6.6 us, mostly the launch.  One element
// per load took 163.5, 661.9 and 8.0 us.
#include "optim_internal.h"
#include "seq_common.h"

namespace convfwd {
namespace {

constexpr int kThreads = 256;
constexpr int kQ = 256;                    // elements per 8-bit block: one wave, four each
constexpr int kChunk = 4096;               // elements per workgroup

struct Table {
    AdamwHyper h;
    int count, pad;
    AdamwTensor t[kMaxTensors];
};
static_assert(sizeof(Table) <= 4096, "kernel arguments");

// 32 bits per element from the tensor's key (seed, step and its place in the list), by two rounds of
// xor-shift and odd multiplication; shifts and multipliers are published ones (C. Wellons, "Prospecting for
// Hash Functions", 2018), found there by search for the least bias.
constexpr uint32_t kPlace = 0x9e3779b1u;       // z = key + place in the tensor * kPlace
__device__ __forceinline__ uint32_t random_bits(uint32_t z) {
    z = (z ^ (z >> 15)) * 0x2c1b3c6du;
    z = (z ^ (z >> 12)) * 0x297a2d39u;
    return z ^ (z >> 15);
}

// The tensor that a block belongs to: each lane looks at one entry (kMaxTensors <= 64), so this is
// one load and not a chain of them.
__device__ __forceinline__ const AdamwTensor &find(const Table &tb, uint32_t blk) {
    const int lane = threadIdx.x & 63;
    const uint32_t first = tb.t[min(lane, tb.count - 1)].first;
    const uint64_t on = __ballot(lane < tb.count && first <= blk);
    return tb.t[63 - __builtin_clzll(on)];
}

// Four adjacent elements at any element-aligned address: tensors may be slices
// that start anywhere, and a load of 4 to 16 bytes need not be aligned.
struct __attribute__((packed, aligned(4))) F4 { float f[4]; };
struct __attribute__((packed, aligned(2))) H4 { uint16_t h[4]; };
struct __attribute__((packed, aligned(1))) B4 { uint32_t b; };

template <bool BF16> struct Grad { typedef F4 type; typedef float elem; };
template <> struct Grad<true> { typedef H4 type; typedef uint16_t elem; };
__device__ __forceinline__ float value(const F4 &g, int e) { return g.f[e]; }
__device__ __forceinline__ float value(const H4 &g, int e) { return __uint_as_float((uint32_t)g.h[e] << 16); }

// Parameters, gradients and moments pass by once a step: non-temporal accesses, as a stream through the
// caches only displaces (26 M parameters: 152.6 us without the hints, 135.2 us with them).  The bf16 copy
// goes plainly beside fp32 moments (128 us) and as a stream beside 8-bit ones (60 M parameters with the
// values, before the roots were corrected: 293 us, 316 us plainly).
template <typename V, typename E> __device__ __forceinline__ V load_stream(const E *p) {
    typedef uint32_t W __attribute__((ext_vector_type(sizeof(V) / 4), aligned(sizeof(E))));
    const W w = __builtin_nontemporal_load(reinterpret_cast<const W *>(p));
    V v;
    __builtin_memcpy(&v, &w, sizeof(v));
    return v;
}
template <typename V, typename E> __device__ __forceinline__ void store_stream(E *p, const V &v) {
    typedef uint32_t W __attribute__((ext_vector_type(sizeof(V) / 4), aligned(sizeof(E))));
    W w;
    __builtin_memcpy(&w, &v, sizeof(v));
    __builtin_nontemporal_store(w, reinterpret_cast<W *>(p));
}

// Elements i .. i+3 of p, or what there is of them (n: the tensor's length; FULL: all are there).
template <bool FULL, typename V, typename E> __device__ __forceinline__ V load4(const E *p, int64_t i, int64_t n) {
    if (FULL || i + 4 <= n) return load_stream<V>(p + i);
    V v = {};
    E *o = reinterpret_cast<E *>(&v);
    for (int e = 0; e < 3; ++e)
        if (i + e < n) o[e] = p[i + e];
    return v;
}
template <bool FULL, bool STREAM = true, typename V, typename E>
__device__ __forceinline__ void store4(E *p, int64_t i, int64_t n, const V &v) {
    if (FULL || i + 4 <= n) {
        if (STREAM)
            store_stream(p + i, v);
        else
            *reinterpret_cast<V *>(p + i) = v;
        return;
    }
    const E *o = reinterpret_cast<const E *>(&v);
    for (int e = 0; e < 3; ++e)
        if (i + e < n) p[i + e] = o[e];
}
__device__ __forceinline__ H4 to_copy(const F4 &p) {
    const uint2 u = make_uint2(pack_bf16(p.f[0], p.f[1]), pack_bf16(p.f[2], p.f[3]));
    return __builtin_bit_cast(H4, u);
}

// The new moments, each operation rounded by itself (seq_common.h switches
// contraction off): what is encoded in 8 bits does not depend on the compiler.
__device__ __forceinline__ void moments(const AdamwHyper &h, float g, float &m, float &v) {
    const float m1 = m * h.b1, m2 = g * h.ob1;
    m = m1 + m2;
    const float g2 = g * g;
    const float v1 = v * h.b2, v2 = g2 * h.ob2;
    v = v1 + v2;
}

// The division and the root are the hardware's, good to a unit in the last place: their error is the
// step's, about 1e-7 of a change that is itself a small part of p.
__device__ __forceinline__ float update(const AdamwHyper &h, float keep, float p, float m, float v) {
    return p * keep - h.lr_c1 * m * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v) * h.inv_sqrt_c2 + h.eps);
}

constexpr int kUnits = kChunk / (4 * kThreads);     // groups of four elements per thread, all loaded first

template <bool BF16, bool FULL> __device__ __forceinline__ void adamw32_chunk(const Table &tb, const AdamwTensor &t) {
    typedef typename Grad<BF16>::type G;
    const float gs = tb.h.grad_scale ? *tb.h.grad_scale : 1.f;
    const int64_t i0 = (int64_t)(blockIdx.x - t.first) * kChunk + 4 * threadIdx.x, n = t.n;
    float *const tp = t.p, *const tm = (float *)t.m, *const tv = (float *)t.v;
    const auto *const tg = (const typename Grad<BF16>::elem *)t.g;
    F4 p[kUnits], m[kUnits], v[kUnits];
    G g[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int64_t i = i0 + u * 4 * kThreads;
        if (FULL || i < n) {
            g[u] = load4<FULL, G>(tg, i, n);
            m[u] = load4<FULL, F4>(tm, i, n);
            v[u] = load4<FULL, F4>(tv, i, n);
            p[u] = load4<FULL, F4>(tp, i, n);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int64_t i = i0 + u * 4 * kThreads;
        if (FULL || i < n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                moments(tb.h, value(g[u], e) * gs, m[u].f[e], v[u].f[e]);
                p[u].f[e] = update(tb.h, t.keep, p[u].f[e], m[u].f[e], v[u].f[e]);
            }
            store4<FULL>(tm, i, n, m[u]);
            store4<FULL>(tv, i, n, v[u]);
            store4<FULL>(tp, i, n, p[u]);
            if (t.copy) store4<FULL, false>(t.copy, i, n, to_copy(p[u]));
        }
    }
}

// Values of the codes: m = s (q/127)^2 with q's sign, v = s (q/255)^4.
__device__ __forceinline__ float decode_m(float q, float s) {
    const float u = q * (1.f / 127.f), w = u * fabsf(u);
    return w * s;
}
__device__ __forceinline__ float decode_v(float q, float s) {
    const float u = q * (1.f / 255.f), w = u * u, z = w * w;
    return z * s;
}

// The correctly rounded square root of y in [0, 1], from the hardware's s, which is a unit in the last
// place off at most.  The midpoint to the neighbour below, s', squares to s s' and a quarter of a unit's
// square: y <= s s' puts the root nearer to s' (and the like above): Tuckerman's rounding test
// (R. Agarwal et al., IBM J. Res. Dev. 30, 1986), with the products' exact residuals.  Below 2^-100 it may
// miss: the code is 0 there anyway.  Without the correction one element in some ten million takes another code
// than the same operations give elsewhere.  It costs 13 us of 321; before codes were packed as they are now it
// cost 17 of 326, and the library's own root 35.
__device__ __forceinline__ float exact_root(float y) {
    const float s = __builtin_amdgcn_sqrtf(y);
    const float below = __int_as_float(__float_as_int(s) - 1), above = __int_as_float(__float_as_int(s) + 1);
    const float r = fmaf(-below, s, y) <= 0.f ? below : s;
    return fmaf(-above, s, y) > 0.f ? above : r;
}

// The lower one of the two codes around x in [0, s], inv = 1/s.
template <bool SECOND> __device__ __forceinline__ float lower_code(float x, float inv) {
    const float top = SECOND ? 255.f : 127.f;
    float root = exact_root(x * inv);
    if (SECOND) root = exact_root(root);
    return fminf(floorf(root * top), top - 1.f);
}

// The code of x: the lower one or the one above, that with probability
// (x - below)/(above - below).
template <bool SECOND> __device__ __forceinline__ float encode(float x, float s, float low, uint32_t bits16) {
    const float v0 = SECOND ? decode_v(low, s) : decode_m(low, s);
    const float v1 = SECOND ? decode_v(low + 1.f, s) : decode_m(low + 1.f, s);
    const float rnd = (float)bits16 * 0x1p-16f, d = v1 - v0, a = rnd * d, e = x - v0;
    return a < e ? low + 1.f : low;
}

// The largest of a wave's non-negative values, as their bits (which order alike; a NaN is above all and
// so reaches the scale): four steps within rows of 16 lanes, then one value of each row.
template <int CTRL> __device__ __forceinline__ uint32_t max_with(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_max(float f) {
    uint32_t v = __float_as_uint(f);
    v = max_with<0xb1>(v);      // lanes 1 0 3 2
    v = max_with<0x4e>(v);      // lanes 2 3 0 1
    v = max_with<0x141>(v);     // half rows mirrored
    v = max_with<0x140>(v);     // rows mirrored
    const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
    const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
    return __uint_as_float(max(a, b));
}
// 1/s, one Newton step after the hardware's; 0 for s = 0.  The hardware's is 0 where 1/s is below the normal
// numbers (s > 2^126): there it is taken of s/16, and the result, two to three bits shorter, is still a place
// within 2^-20 of x/s.
__device__ __forceinline__ float inverse(float s) {
    const float f = s > 0x1p125f ? 0x1p-4f : 1.f, t = s * f, r = __builtin_amdgcn_rcpf(t);
    return s > 0.f ? fmaf(r, fmaf(-t, r, 1.f), r) * f : 0.f;
}
__device__ __forceinline__ float larger(float f, float g) {
    return __uint_as_float(max(__float_as_uint(f), __float_as_uint(g) & 0x7fffffffu));
}

__device__ __forceinline__ float signed_code(uint32_t q, int e) { return (float)(int8_t)(q >> (8 * e)); }
__device__ __forceinline__ float plain_code(uint32_t q, int e) { return (float)(uint8_t)(q >> (8 * e)); }

constexpr int kBlocks = kChunk / kQ / (kThreads / 64);     // 8-bit blocks per wave, all loaded first

template <bool BF16, bool FULL> __device__ __forceinline__ void adamw8_chunk(const Table &tb, const AdamwTensor &t) {
    typedef typename Grad<BF16>::type G;
    const float gs = tb.h.grad_scale ? *tb.h.grad_scale : 1.f;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n = t.n, blk0 = (int64_t)(blockIdx.x - t.first) * (kChunk / kQ) + w * kBlocks;
    float *const tp = t.p;
    uint8_t *const tm = (uint8_t *)t.m, *const tv = (uint8_t *)t.v;
    const auto *const tg = (const typename Grad<BF16>::elem *)t.g;
    F4 p[kBlocks];
    B4 qm[kBlocks], qv[kBlocks];
    G g[kBlocks];
    float ms[kBlocks], vs[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
        const int64_t i = (blk0 + u) * kQ + 4 * lane;
        if (FULL || (blk0 + u) * kQ < n) {
            ms[u] = t.m_scale[blk0 + u];
            vs[u] = t.v_scale[blk0 + u];
            g[u] = load4<FULL, G>(tg, i, n);
            qm[u] = load4<FULL, B4>(tm, i, n);
            qv[u] = load4<FULL, B4>(tv, i, n);
            p[u] = load4<FULL, F4>(tp, i, n);
        }
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
        const int64_t blk = blk0 + u, i = blk * kQ + 4 * lane;
        if (!FULL && blk * kQ >= n) break;
        float m[4], v[4], mmax = 0.f, vmax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float q = signed_code(qm[u].b, e);
            m[e] = decode_m(q, ms[u]);
            v[e] = decode_v(plain_code(qv[u].b, e), vs[u]);
            moments(tb.h, value(g[u], e) * gs, m[e], v[e]);
            p[u].f[e] = update(tb.h, t.keep, p[u].f[e], m[e], v[e]);
            // past the tensor's end there are zeros, which move no maximum (but 0 * NaN must not)
            if (FULL || i + e < n) mmax = larger(mmax, m[e]), vmax = larger(vmax, v[e]);
        }
        store4<FULL>(tp, i, n, p[u]);
        if (t.copy) store4<FULL>(t.copy, i, n, to_copy(p[u]));
        float sm = wave_max(mmax), sv = wave_max(vmax);
        if (sm < 0x1p-126f) sm = 0.f;
        if (sv < 0x1p-126f) sv = 0.f;
        const float im = inverse(sm), iv = inverse(sv), tiny = sv > 0.f ? 0.f : INFINITY;    // what a code 0 is for
        B4 om = {0}, ov = {0};
        const uint32_t place = t.key + ((uint32_t)i) * kPlace;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t z = random_bits(place + e * kPlace);
            const float am = fabsf(m[e]);
            const float cm = encode<false>(am, sm, lower_code<false>(am, im), z & 0xffffu);
            float cv = encode<true>(v[e], sv, lower_code<true>(v[e], iv), z >> 16);
            cv = v[e] > tiny ? fmaxf(cv, 1.f) : cv;
            om.b = __builtin_amdgcn_cvt_pk_u8_f32(m[e] < 0.f && cm > 0.f ? 256.f - cm : cm, e, om.b);      // two's complement
            ov.b = __builtin_amdgcn_cvt_pk_u8_f32(cv, e, ov.b);
        }
        store4<FULL>(tm, i, n, om);
        store4<FULL>(tv, i, n, ov);
        if (lane == 0) {
            t.m_scale[blk] = sm;
            t.v_scale[blk] = sv;
        }
    }
}

// p holds the output for m, copy (as float*) the one for v.
template <bool FULL> __device__ __forceinline__ void values_chunk(const AdamwTensor &t) {
    const int64_t i0 = (int64_t)(blockIdx.x - t.first) * kChunk + 4 * threadIdx.x, n = t.n;
    B4 qm[kUnits], qv[kUnits];
    float ms[kUnits], vs[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int64_t i = i0 + u * 4 * kThreads;
        if (FULL || i < n) {
            qm[u] = load4<FULL, B4>((const uint8_t *)t.m, i, n);
            qv[u] = load4<FULL, B4>((const uint8_t *)t.v, i, n);
            ms[u] = t.m_scale[i / kQ];
            vs[u] = t.v_scale[i / kQ];
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int64_t i = i0 + u * 4 * kThreads;
        if (FULL || i < n) {
            F4 m, v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float q = signed_code(qm[u].b, e);
                m.f[e] = decode_m(q, ms[u]);
                v.f[e] = decode_v(plain_code(qv[u].b, e), vs[u]);
            }
            store4<FULL>(t.p, i, n, m);
            store4<FULL>((float *)t.copy, i, n, v);
        }
    }
}

// Whether all elements of this workgroup's chunk are there: uniform, so that only a tensor's last chunk
// pays for the checks.
__device__ __forceinline__ bool whole(const AdamwTensor &t) { return (int64_t)(blockIdx.x - t.first + 1) * kChunk <= t.n; }

template <bool BF16> __global__ __launch_bounds__(kThreads) void adamw32_kernel(Table tb) {
    const AdamwTensor &t = find(tb, blockIdx.x);
    if (whole(t)) adamw32_chunk<BF16, true>(tb, t);
    else adamw32_chunk<BF16, false>(tb, t);
}
template <bool BF16> __global__ __launch_bounds__(kThreads) void adamw8_kernel(Table tb) {
    const AdamwTensor &t = find(tb, blockIdx.x);
    if (whole(t)) adamw8_chunk<BF16, true>(tb, t);
    else adamw8_chunk<BF16, false>(tb, t);
}
__global__ __launch_bounds__(kThreads) void values_kernel(Table tb) {
    const AdamwTensor &t = find(tb, blockIdx.x);
    if (whole(t)) values_chunk<true>(t);
    else values_chunk<false>(t);
}

}  // namespace

int64_t adamw_blocks(int64_t n) { return (n + kChunk - 1) / kChunk; }

hipError_t launch_adamw(const AdamwHyper &h, const AdamwTensor *t, int count, int mode, bool grad_bf16, hipStream_t st) {
    Table tb;
    tb.h = h;
    tb.pad = 0;
    for (int at = 0; at < count; at += kMaxTensors) {
        tb.count = count - at < kMaxTensors ? count - at : kMaxTensors;
        uint32_t blocks = 0;
        for (int i = 0; i < tb.count; ++i) {
            tb.t[i] = t[at + i];
            tb.t[i].first = blocks;
            blocks += (uint32_t)adamw_blocks(t[at + i].n);
        }
        if (mode == kAdamwValues)
            values_kernel<<<blocks, kThreads, 0, st>>>(tb);
        else if (mode == kAdamw8 && grad_bf16)
            adamw8_kernel<true><<<blocks, kThreads, 0, st>>>(tb);
        else if (mode == kAdamw8)
            adamw8_kernel<false><<<blocks, kThreads, 0, st>>>(tb);
        else if (grad_bf16)
            adamw32_kernel<true><<<blocks, kThreads, 0, st>>>(tb);
        else
            adamw32_kernel<false><<<blocks, kThreads, 0, st>>>(tb);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace convfwd
