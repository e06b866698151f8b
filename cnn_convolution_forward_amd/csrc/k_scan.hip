// k_scan.hip -- the gated linear recurrence over tokens: forward, backward and
// the single-token step (conv_scan_*).
#include "conv_fwd.h"
#include "scan_math.h"

namespace convfwd {
namespace {

constexpr int kThreads = 64;
constexpr int kBlock = CONV_SCAN_BLOCK;

template <typename T>
__global__ __launch_bounds__(kThreads) void scan_fwd_kernel(Seq s, float scale, const T *__restrict__ x, int64_t ldx,
                                                            const T *__restrict__ gate, int64_t ldg,
                                                            const T *__restrict__ inp, int64_t ldi,
                                                            const float *__restrict__ decay, const float *__restrict__ h0,
                                                            T *__restrict__ y, int64_t ldy, float *__restrict__ hT,
                                                            float *__restrict__ states) {
    const int b = blockIdx.y, c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= s.C) return;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const float k = scan_rate(scale, decay[c]);
    const int64_t nb = (s.T + kBlock - 1) / kBlock;
    float h = h0 ? h0[(int64_t)b * s.C + c] : 0.f;
    for (int t = 0; t < len; ++t) {
        if (states && t % kBlock == 0) states[(b * nb + t / kBlock) * s.C + c] = h;
        const int64_t row = first + t;
        float xv[1], gv[1], iv[1];
        load_f32<T, 1>(x + row * ldx + c, xv);
        load_f32<T, 1>(gate + row * ldg + c, gv);
        load_f32<T, 1>(inp + row * ldi + c, iv);
        const ScanGates g(k, gv[0], iv[0]);
        h = fmaf(g.a, h, g.m * g.s * xv[0]);
        const float o[1] = {h};
        store_f32(y + row * ldy + c, o);
    }
    if (hT) hT[(int64_t)b * s.C + c] = h;
}

// One sequence and channel per thread, the 64-token blocks backwards: h is run
// forward through a block from its saved state and kept, then dh backwards.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_bwd_kernel(
    Seq s, float scale, const T *__restrict__ x, int64_t ldx, const T *__restrict__ gate, int64_t ldg,
    const T *__restrict__ inp, int64_t ldi, const float *__restrict__ decay, const float *__restrict__ states,
    const T *__restrict__ dy, int64_t lddy, const float *__restrict__ dhT, T *__restrict__ dx, int64_t lddx,
    T *__restrict__ dgate, int64_t lddg, T *__restrict__ dinp, int64_t lddi, float *__restrict__ part,
    float *__restrict__ dh0) {
    __shared__ float before[kBlock][kThreads];
    const int b = blockIdx.y, c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= s.C) return;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const float k = scan_rate(scale, decay[c]);
    const int64_t nb = (s.T + kBlock - 1) / kBlock;
    float e = dhT ? dhT[(int64_t)b * s.C + c] : 0.f, dk = 0.f;
    for (int blk = (len + kBlock - 1) / kBlock - 1; blk >= 0; --blk) {
        const int t0 = blk * kBlock, t1 = min(t0 + kBlock, len);
        float h = states[(b * nb + blk) * s.C + c];
        float xv[1], gv[1], iv[1], dv[1];
        for (int t = t0; t < t1; ++t) {
            const int64_t row = first + t;
            before[t - t0][threadIdx.x] = h;
            load_f32<T, 1>(x + row * ldx + c, xv);
            load_f32<T, 1>(gate + row * ldg + c, gv);
            load_f32<T, 1>(inp + row * ldi + c, iv);
            const ScanGates g(k, gv[0], iv[0]);
            h = fmaf(g.a, h, g.m * g.s * xv[0]);
        }
        for (int t = t1 - 1; t >= t0; --t) {
            const int64_t row = first + t;
            load_f32<T, 1>(x + row * ldx + c, xv);
            load_f32<T, 1>(gate + row * ldg + c, gv);
            load_f32<T, 1>(inp + row * ldi + c, iv);
            load_f32<T, 1>(dy + row * lddy + c, dv);
            const ScanGates g(k, gv[0], iv[0]);
            const float dh = dv[0] + e, dms = dh * g.m * g.s;
            const float dla = dh * g.a * (before[t - t0][threadIdx.x] - g.s * xv[0] * g.a * g.im);
            const float rdla = g.r * dla;
            const float o0[1] = {dms}, o1[1] = {-k * rdla * (1.f - g.r)}, o2[1] = {dms * xv[0] * (1.f - g.s)};
            store_f32(dx + row * lddx + c, o0);
            store_f32(dgate + row * lddg + c, o1);
            store_f32(dinp + row * lddi + c, o2);
            dk += rdla;
            e = g.a * dh;
        }
    }
    part[(int64_t)b * s.C + c] = dk;
    if (dh0) dh0[(int64_t)b * s.C + c] = e;
}

// ddecay[c] = -scale sigmoid(decay) * sum of the partial sums, in order.
__global__ __launch_bounds__(256) void scan_reduce_kernel(const float *__restrict__ part, int64_t n, int C, float scale,
                                                          const float *__restrict__ decay, float *__restrict__ ddecay) {
    __shared__ float red[4][64];
    const int cl = threadIdx.x & 63, q = threadIdx.x >> 6, c = blockIdx.x * 64 + cl;
    float v = 0.f;
    if (c < C)
        for (int64_t i = q; i < n; i += 4) v += part[i * C + c];
    red[q][cl] = v;
    __syncthreads();
    if (q == 0 && c < C)
        ddecay[c] = -scale * sigmoid(decay[c]) * ((red[0][cl] + red[1][cl]) + (red[2][cl] + red[3][cl]));
}

template <typename T>
__global__ __launch_bounds__(256) void scan_step_kernel(int B, int C, float scale, const T *__restrict__ x, int64_t ldx,
                                                        const T *__restrict__ gate, int64_t ldg,
                                                        const T *__restrict__ inp, int64_t ldi,
                                                        const float *__restrict__ decay, float *__restrict__ h,
                                                        T *__restrict__ y, int64_t ldy) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)B * C) return;
    const int b = (int)(i / C), c = (int)(i % C);
    float xv[1], gv[1], iv[1];
    load_f32<T, 1>(x + b * ldx + c, xv);
    load_f32<T, 1>(gate + b * ldg + c, gv);
    load_f32<T, 1>(inp + b * ldi + c, iv);
    const ScanGates g(scan_rate(scale, decay[c]), gv[0], iv[0]);
    const float o[1] = {fmaf(g.a, h[i], g.m * g.s * xv[0])};
    h[i] = o[0];
    store_f32(y + b * ldy + c, o);
}

}  // namespace

size_t scan_fwd_workspace(const Seq &s) { return 0; }
size_t scan_bwd_workspace(const Seq &s) { return (size_t)s.B * s.C * sizeof(float); }

hipError_t launch_scan_fwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate,
                           int64_t ldg, const void *inp, int64_t ldi, const float *decay, const float *h0, void *y,
                           int64_t ldy, float *hT, float *states, void *ws, hipStream_t st) {
    const dim3 grid((s.C + kThreads - 1) / kThreads, s.B);
    if (bf16)
        scan_fwd_kernel<uint16_t><<<grid, kThreads, 0, st>>>(s, scale, (const uint16_t *)x, ldx, (const uint16_t *)gate, ldg,
                                                             (const uint16_t *)inp, ldi, decay, h0, (uint16_t *)y, ldy, hT, states);
    else
        scan_fwd_kernel<float><<<grid, kThreads, 0, st>>>(s, scale, (const float *)x, ldx, (const float *)gate, ldg,
                                                          (const float *)inp, ldi, decay, h0, (float *)y, ldy, hT, states);
    return hipGetLastError();
}

hipError_t launch_scan_bwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                           const void *inp, int64_t ldi, const float *decay, const float *states, const void *dy, int64_t lddy,
                           const float *dhT, void *dx, int64_t lddx, void *dgate, int64_t lddg, void *dinp, int64_t lddi,
                           float *ddecay, float *dh0, void *ws, hipStream_t st) {
    const dim3 grid((s.C + kThreads - 1) / kThreads, s.B);
    float *part = (float *)ws;
    if (bf16) {
        typedef uint16_t T;
        scan_bwd_kernel<T><<<grid, kThreads, 0, st>>>(s, scale, (const T *)x, ldx, (const T *)gate, ldg, (const T *)inp, ldi, decay,
                                                      states, (const T *)dy, lddy, dhT, (T *)dx, lddx, (T *)dgate, lddg,
                                                      (T *)dinp, lddi, part, dh0);
    } else {
        typedef float T;
        scan_bwd_kernel<T><<<grid, kThreads, 0, st>>>(s, scale, (const T *)x, ldx, (const T *)gate, ldg, (const T *)inp, ldi, decay,
                                                      states, (const T *)dy, lddy, dhT, (T *)dx, lddx, (T *)dgate, lddg,
                                                      (T *)dinp, lddi, part, dh0);
    }
    scan_reduce_kernel<<<(s.C + 63) / 64, 256, 0, st>>>(part, s.B, s.C, scale, decay, ddecay);
    return hipGetLastError();
}

hipError_t launch_scan_step(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                            const void *inp, int64_t ldi, const float *decay, float *h, void *y, int64_t ldy, hipStream_t st) {
    const unsigned grid = (unsigned)(((int64_t)s.B * s.C + 255) / 256);
    if (bf16)
        scan_step_kernel<uint16_t><<<grid, 256, 0, st>>>(s.B, s.C, scale, (const uint16_t *)x, ldx, (const uint16_t *)gate, ldg,
                                                         (const uint16_t *)inp, ldi, decay, h, (uint16_t *)y, ldy);
    else
        scan_step_kernel<float><<<grid, 256, 0, st>>>(s.B, s.C, scale, (const float *)x, ldx, (const float *)gate, ldg,
                                                      (const float *)inp, ldi, decay, h, (float *)y, ldy);
    return hipGetLastError();
}

}  // namespace convfwd
