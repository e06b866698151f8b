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
// its tensors; a workgroup finds its tensor by bisection over their first
// numbers (uniform: scalar loads).
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

// z = step and seed for the tensor; 32 bits per element, by two rounds of
// xor-shift and odd multiplication.
__device__ __forceinline__ uint32_t random_bits(uint32_t key, uint32_t i) {
    uint32_t z = key + i * 0x9e3779b1u;
    z = (z ^ (z >> 15)) * 0x2c1b3c6du;
    z = (z ^ (z >> 12)) * 0x297a2d39u;
    return z ^ (z >> 15);
}

__device__ __forceinline__ const AdamwTensor &find(const Table &tb, uint32_t blk) {
    int lo = 0, hi = tb.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tb.t[mid].first <= blk) lo = mid; else hi = mid - 1;
    }
    return tb.t[lo];
}

template <bool BF16> __device__ __forceinline__ float grad_at(const void *g, int64_t i) {
    float f[1];
    if (BF16) to_f32(((const uint16_t *)g)[i], f);
    else f[0] = ((const float *)g)[i];
    return f[0];
}

// The new moments, each operation rounded by itself: the values that are
// encoded in 8 bits do not depend on how the compiler contracts them.
__device__ __forceinline__ void moments(const AdamwHyper &h, float g, float &m, float &v) {
#pragma clang fp contract(off)
    const float m1 = m * h.b1, m2 = g * h.ob1;
    m = m1 + m2;
    const float g2 = g * g;
    const float v1 = v * h.b2, v2 = g2 * h.ob2;
    v = v1 + v2;
}

__device__ __forceinline__ float update(const AdamwHyper &h, float keep, float p, float m, float v) {
    return p * keep - h.lr_c1 * m / (sqrtf(v) * h.inv_sqrt_c2 + h.eps);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void adamw32_kernel(Table tb) {
    const AdamwTensor &t = find(tb, blockIdx.x);
    const float gs = tb.h.grad_scale ? *tb.h.grad_scale : 1.f;
    const int64_t i0 = (int64_t)(blockIdx.x - t.first) * kChunk;
    for (int e = threadIdx.x; e < kChunk; e += kThreads) {
        const int64_t i = i0 + e;
        if (i >= t.n) break;
        float m = ((float *)t.m)[i], v = ((float *)t.v)[i];
        moments(tb.h, grad_at<BF16>(t.g, i) * gs, m, v);
        const float p = update(tb.h, t.keep, t.p[i], m, v);
        ((float *)t.m)[i] = m;
        ((float *)t.v)[i] = v;
        t.p[i] = p;
        if (t.copy) t.copy[i] = to_bf16(p);
    }
}

// Values of the codes: m = s (q/127)^2 with q's sign, v = s (q/255)^4.
__device__ __forceinline__ float decode_m(float q, float s) {
#pragma clang fp contract(off)
    const float u = q * (1.f / 127.f), w = u * u;
    return w * s;
}
__device__ __forceinline__ float decode_v(float q, float s) {
#pragma clang fp contract(off)
    const float u = q * (1.f / 255.f), w = u * u, z = w * w;
    return z * s;
}

// The code of x in [0, s]: the one below or the one above, the upper with
// probability (x - below)/(above - below).
template <bool SECOND> __device__ __forceinline__ float encode(float x, float s, float inv, uint32_t bits16) {
#pragma clang fp contract(off)
    const float top = SECOND ? 255.f : 127.f;
    float root = sqrtf(x * inv);
    if (SECOND) root = sqrtf(root);
    const float low = fminf(floorf(root * top), top - 1.f);
    const float v0 = SECOND ? decode_v(low, s) : decode_m(low, s);
    const float v1 = SECOND ? decode_v(low + 1.f, s) : decode_m(low + 1.f, s);
    const float rnd = (float)bits16 * 0x1p-16f, d = v1 - v0, a = rnd * d, e = x - v0;
    float q = low + (a < e ? 1.f : 0.f);
    if (SECOND && q == 0.f && x > 0.f && s > 0.f) q = 1.f;
    return q;
}

// The largest over a wave; NaN wins, so that it reaches the scale.
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float u = __shfl_xor(v, o);
        v = (u > v || u != u) ? u : v;
    }
    return v;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(Table tb) {
    const AdamwTensor &t = find(tb, blockIdx.x);
    const float gs = tb.h.grad_scale ? *tb.h.grad_scale : 1.f;
    const int lane = threadIdx.x & 63;
    for (int q = threadIdx.x >> 6; q < kChunk / kQ; q += kThreads / 64) {
        const int64_t i0 = (int64_t)(blockIdx.x - t.first) * kChunk + q * kQ;
        if (i0 >= t.n) break;
        const int64_t blk = i0 / kQ;
        const float ms = t.m_scale[blk], vs = t.v_scale[blk];
        float m[4], v[4], mmax = 0.f, vmax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = i0 + 4 * lane + e;
            m[e] = v[e] = 0.f;
            if (i < t.n) {
                const float qm = (float)((const int8_t *)t.m)[i], qv = (float)((const uint8_t *)t.v)[i];
                m[e] = copysignf(decode_m(fabsf(qm), ms), qm);
                v[e] = decode_v(qv, vs);
                moments(tb.h, grad_at<BF16>(t.g, i) * gs, m[e], v[e]);
                const float p = update(tb.h, t.keep, t.p[i], m[e], v[e]);
                t.p[i] = p;
                if (t.copy) t.copy[i] = to_bf16(p);
            }
            const float am = fabsf(m[e]);
            mmax = (am > mmax || am != am) ? am : mmax;
            vmax = (v[e] > vmax || v[e] != v[e]) ? v[e] : vmax;
        }
        float sm = wave_max(mmax), sv = wave_max(vmax);
        if (sm < 0x1p-126f) sm = 0.f;
        if (sv < 0x1p-126f) sv = 0.f;
        const float im = sm > 0.f ? 1.f / sm : 0.f, iv = sv > 0.f ? 1.f / sv : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = i0 + 4 * lane + e;
            if (i < t.n) {
                const uint32_t z = random_bits(t.key, (uint32_t)i);
                const float cm = encode<false>(fabsf(m[e]), sm, im, z & 0xffffu), cv = encode<true>(v[e], sv, iv, z >> 16);
                ((int8_t *)t.m)[i] = (int8_t)(int)copysignf(cm, m[e]);
                ((uint8_t *)t.v)[i] = (uint8_t)(int)cv;
            }
        }
        if (lane == 0) {
            t.m_scale[blk] = sm;
            t.v_scale[blk] = sv;
        }
    }
}

// p holds the output for m, copy (as float*) the one for v.
__global__ __launch_bounds__(kThreads) void values_kernel(Table tb) {
    const AdamwTensor &t = find(tb, blockIdx.x);
    const int64_t i0 = (int64_t)(blockIdx.x - t.first) * kChunk;
    for (int e = threadIdx.x; e < kChunk; e += kThreads) {
        const int64_t i = i0 + e;
        if (i >= t.n) break;
        const float qm = (float)((const int8_t *)t.m)[i], qv = (float)((const uint8_t *)t.v)[i];
        t.p[i] = copysignf(decode_m(fabsf(qm), t.m_scale[i / kQ]), qm);
        ((float *)t.copy)[i] = decode_v(qv, t.v_scale[i / kQ]);
    }
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
