// k_norm.hip -- layer normalisation over the channels of each row, forward and
// backward (conv_norm_fwd, conv_norm_bwd).
//
//   y  = (x - mean) rstd w + b,   mean = sum x / C,   rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   dx = rstd (w dy - sum(w dy) / C - xh sum(w dy xh) / C),   xh = (x - mean) rstd
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// A dozen operations for four to six bytes: HBM is the bound, so each row is
// read once and held in registers between its sums and its result.  G threads
// share a row: 16 (four rows to a wave, no barrier), 64, or a whole workgroup of
// 256 to 1024 with its sums joined in LDS; the fewest with which a thread holds at
// most 32 channels (16 where it has 128 registers).  A thread keeps its channels, their weights, bias and sums
// of gradients in registers while its group walks through rows; the next row is
// loaded before the present one's sums.  Rows too wide for that, of more than 16384 channels, are read again.
//
// bf16, forward and backward: 16384 x 2048 25 us (5.4 TB/s) and 39 us (5.1), 4096 x 8192 26 (5.2) and
// 50 (4.0; with 256 threads to a row 59), 2048 x 16384 32 (4.2) and 71 (2.9: one workgroup to a compute unit, whose
// barriers nothing hides).  Rows that are read again, by single elements and with sums in memory: 2048 x 20480 81 and 324 us.
//
// The variance is a second sum over the registers, of squared distances from the
// mean: no cancellation.  Sums over rows: each workgroup adds its own rows, and a
// second kernel adds the workgroups' in a fixed order.
#include "seq_common.h"

namespace convfwd {
namespace {

constexpr int kThreads = 256;                          // of a workgroup, but for rows that take more
constexpr int kWide = 1024;                             // for rows that no workgroup holds
constexpr int threads_of(int G) { return G > kThreads ? G : kThreads; }
// Workgroups that walk through the rows; the numbers are the best of those tried at the sizes given.  Backward, each has a row of partial sums: 256 of them are enough to fill the chip
// with wide rows (16384 x 2048 bf16: 39.4 us, with 512 43.8), narrow ones have shorter sums and want more waves (131072 x 128:
// 24.2 us with 512, 31.2 with 256).  Forward: 25.4 us at 768, 27.2 at 1024, 66 with a workgroup for every four rows.
constexpr int kMaxForward = 768;
constexpr int max_backward(int G) { return G == 16 ? 512 : 256; }

template <int G> __device__ __forceinline__ float group_sum(float v, float *red, int &phase) {
#pragma unroll
    for (int m = (G < 64 ? G : 64) / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (G > 64) {
        // two buffers in turn: a wave that is a sum ahead writes the other one
        float *r = red + (phase ^= 1) * (G / 64);
        if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
        __syncthreads();
        v = r[0];
#pragma unroll
        for (int i = 1; i < G / 64; ++i) v += r[i];
    }
    return v;
}

// NV packs of VEC channels: pack i of thread li is at channel (i G + li) VEC.  Channels past C are zeros.
template <typename T, int VEC, int NV, int G, bool ONCE> struct RowRegs {
    typename Pack<T, VEC>::type v[NV];
    __device__ __forceinline__ void load(const T *p, int li, int C) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * G + li) * VEC;
            if (c + VEC <= C) {
                v[i] = ONCE ? load_once<T, VEC>(p + c) : load_pack<T, VEC>(p + c);
            } else {
                T t[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) t[j] = c + j < C ? p[c + j] : T(0);
                __builtin_memcpy(&v[i], t, sizeof(v[i]));
            }
        }
    }
    __device__ __forceinline__ void get(float (&f)[NV][VEC]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) to_f32(v[i], f[i]);
    }
};

template <typename T, int VEC, int NV, int G>
__device__ __forceinline__ void store_row(T *p, int li, int C, const float (&f)[NV][VEC]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * G + li) * VEC;
        if (c + VEC <= C) {
            store_f32(p + c, f[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float e[1] = {f[i][j]};
                if (c + j < C) store_f32(p + c + j, e);
            }
        }
    }
}

template <int VEC, int NV, int G>
__device__ __forceinline__ void load_param(const float *p, float other, int li, int C, float (&f)[NV][VEC]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * G + li) * VEC;
        if (p && c + VEC <= C) {
#pragma unroll
            for (int j = 0; j < VEC; j += 4) {
                float t[4];
                load_f32<float, 4>(p + c + j, t);
#pragma unroll
                for (int q = 0; q < 4; ++q) f[i][j + q] = t[q];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[i][j] = p && c + j < C ? p[c + j] : other;
        }
    }
}

template <typename T, int VEC, int NV, int G, bool ONCE>
__global__ __launch_bounds__(threads_of(G)) void norm_fwd_kernel(int64_t rows, int C, float eps, const T *__restrict__ x,
                                                            int64_t ldx, const float *__restrict__ w,
                                                            const float *__restrict__ b, T *__restrict__ y, int64_t ldy,
                                                            float *__restrict__ mean, float *__restrict__ rstd) {
    constexpr int kRows = threads_of(G) / G;
    __shared__ float red[2 * (G > 64 ? G / 64 : 1)];
    int phase = 0;
    const int li = threadIdx.x % G;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    float wf[NV][VEC], bf[NV][VEC];
    RowRegs<T, VEC, NV, G, ONCE> next;
    if (r < rows) next.load(x + r * ldx, li, C);
    load_param<VEC, NV, G>(w, 1.f, li, C, wf);
    load_param<VEC, NV, G>(b, 0.f, li, C, bf);
    const float inv = 1.f / (float)C;
    for (; r < rows; r += step) {
        const RowRegs<T, VEC, NV, G, ONCE> now = next;
        if (r + step < rows) next.load(x + (r + step) * ldx, li, C);
        float f[NV][VEC];
        now.get(f);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) s += f[i][j];
        const float m = group_sum<G>(s, red, phase) * inv;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const bool on = NV * G * VEC == C || (i * G + li) * VEC + j < C;
                f[i][j] = on ? f[i][j] - m : 0.f;
                s = fmaf(f[i][j], f[i][j], s);
            }
        const float k = 1.f / sqrtf(group_sum<G>(s, red, phase) * inv + eps);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[i][j] = fmaf(f[i][j] * k, wf[i][j], bf[i][j]);
        store_row<T, VEC, NV, G>(y + r * ldy, li, C, f);
        if (li == 0) {
            if (mean) mean[r] = m;
            if (rstd) rstd[r] = k;
        }
    }
}

// Rows wider than the registers: one workgroup to a row, which is read three times, mostly from the cache.
template <typename T>
__global__ __launch_bounds__(kWide) void norm_fwd_wide_kernel(int64_t rows, int C, float eps, const T *__restrict__ x,
                                                                 int64_t ldx, const float *__restrict__ w,
                                                                 const float *__restrict__ b, T *__restrict__ y,
                                                                 int64_t ldy, float *__restrict__ mean,
                                                                 float *__restrict__ rstd) {
    __shared__ float red[2 * kWide / 64];
    int phase = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *p = x + r * ldx;
        float f[1], s = 0.f;
        for (int c = threadIdx.x; c < C; c += kWide) load_f32<T, 1>(p + c, f), s += f[0];
        const float m = group_sum<kWide>(s, red, phase) / (float)C;
        s = 0.f;
        for (int c = threadIdx.x; c < C; c += kWide) load_f32<T, 1>(p + c, f), s = fmaf(f[0] - m, f[0] - m, s);
        const float k = 1.f / sqrtf(group_sum<kWide>(s, red, phase) / (float)C + eps);
        for (int c = threadIdx.x; c < C; c += kWide) {
            load_f32<T, 1>(p + c, f);
            const float o[1] = {fmaf((f[0] - m) * k, w ? w[c] : 1.f, b ? b[c] : 0.f)};
            store_f32(y + r * ldy + c, o);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[r] = m;
            if (rstd) rstd[r] = k;
        }
    }
}

// part: per workgroup C sums of dy xh, then C sums of dy; NULL: not wanted.
template <typename T, int VEC, int NV, int G, bool ONCE>
__global__ __launch_bounds__(threads_of(G)) void norm_bwd_kernel(int64_t rows, int C, const T *__restrict__ x, int64_t ldx,
                                                            const float *__restrict__ w, const float *__restrict__ mean,
                                                            const float *__restrict__ rstd, const T *__restrict__ dy,
                                                            int64_t lddy, T *__restrict__ dx, int64_t lddx,
                                                            float *__restrict__ part) {
    constexpr int kRows = threads_of(G) / G, kWidth = G * VEC * NV;
    __shared__ float red[2 * (G > 64 ? G / 64 : 1)];
    __shared__ float sums[kRows > 1 ? kRows * kWidth : 1];
    int phase = 0;
    const int li = threadIdx.x % G, gi = threadIdx.x / G;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t r = (int64_t)blockIdx.x * kRows + gi;
    float wf[NV][VEC], dw[NV][VEC], db[NV][VEC];
    RowRegs<T, VEC, NV, G, ONCE> nx, ny;
    float nm = 0.f, nk = 0.f;
    if (r < rows) {
        nx.load(x + r * ldx, li, C);
        ny.load(dy + r * lddy, li, C);
        nm = mean[r], nk = rstd[r];
    }
    // 1024 threads have 128 registers each: weights are read again for each row, from the cache
    constexpr bool kHold = G < 1024;
    if constexpr (kHold) load_param<VEC, NV, G>(w, 1.f, li, C, wf);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.f;
    const float inv = 1.f / (float)C;
    for (; r < rows; r += step) {
        const RowRegs<T, VEC, NV, G, ONCE> cx = nx, cy = ny;
        const float m = nm, k = nk;
        if (r + step < rows) {
            nx.load(x + (r + step) * ldx, li, C);
            ny.load(dy + (r + step) * lddy, li, C);
            nm = mean[r + step], nk = rstd[r + step];
        }
        float f[NV][VEC], g[NV][VEC], s0 = 0.f, s1 = 0.f;
        cx.get(f);
        cy.get(g);
        if constexpr (!kHold) {
            asm volatile("" : "+s"(w));                                  // in the loop
            load_param<VEC, NV, G>(w, 1.f, li, C, wf);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const bool on = NV * G * VEC == C || (i * G + li) * VEC + j < C;
                f[i][j] = on ? (f[i][j] - m) * k : 0.f;
                dw[i][j] = fmaf(g[i][j], f[i][j], dw[i][j]);
                db[i][j] += g[i][j];
                g[i][j] *= wf[i][j];
                s0 += g[i][j];
                s1 = fmaf(g[i][j], f[i][j], s1);
            }
        s0 = group_sum<G>(s0, red, phase) * inv;
        s1 = group_sum<G>(s1, red, phase) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[i][j] = k * (g[i][j] - s0 - f[i][j] * s1);
        store_row<T, VEC, NV, G>(dx + r * lddx, li, C, f);
    }
    if (!part) return;
    float *out = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if constexpr (kRows > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) sums[gi * kWidth + (i * G + li) * VEC + j] = q ? db[i][j] : dw[i][j];
            __syncthreads();
            for (int c = threadIdx.x; c < C; c += kThreads) {       // kRows > 1: kThreads of them
                float s = sums[c];
#pragma unroll
                for (int i = 1; i < kRows; ++i) s += sums[i * kWidth + c];
                out[q * C + c] = s;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int c = (i * G + li) * VEC + j;
                    if (c < C) out[q * C + c] = q ? db[i][j] : dw[i][j];
                }
        }
    }
}

// One workgroup to a block of rows: a channel's sums are kept in memory, by the thread that owns it.
template <typename T>
__global__ __launch_bounds__(kWide) void norm_bwd_wide_kernel(int64_t rows, int C, const T *__restrict__ x, int64_t ldx,
                                                                 const float *__restrict__ w, const float *__restrict__ mean,
                                                                 const float *__restrict__ rstd, const T *__restrict__ dy,
                                                                 int64_t lddy, T *__restrict__ dx, int64_t lddx,
                                                                 float *__restrict__ part) {
    __shared__ float red[2 * kWide / 64];
    int phase = 0;
    float *out = part ? part + (int64_t)blockIdx.x * 2 * C : nullptr;
    bool first = true;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, first = false) {
        const float m = mean[r], k = rstd[r];
        float f[1], g[1], s0 = 0.f, s1 = 0.f;
        for (int c = threadIdx.x; c < C; c += kWide) {
            load_f32<T, 1>(x + r * ldx + c, f);
            load_f32<T, 1>(dy + r * lddy + c, g);
            const float h = (f[0] - m) * k;
            if (out) {
                out[c] = fmaf(g[0], h, first ? 0.f : out[c]);
                out[C + c] = g[0] + (first ? 0.f : out[C + c]);
            }
            g[0] *= w ? w[c] : 1.f;
            s0 += g[0];
            s1 = fmaf(g[0], h, s1);
        }
        s0 = group_sum<kWide>(s0, red, phase) / (float)C;
        s1 = group_sum<kWide>(s1, red, phase) / (float)C;
        for (int c = threadIdx.x; c < C; c += kWide) {
            load_f32<T, 1>(x + r * ldx + c, f);
            load_f32<T, 1>(dy + r * lddy + c, g);
            const float h = (f[0] - m) * k;
            const float o[1] = {k * (g[0] * (w ? w[c] : 1.f) - s0 - h * s1)};
            store_f32(dx + r * lddx + c, o);
        }
    }
}

// dw and db from the workgroups' sums: 32 columns to a workgroup, 32 threads to a column.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float *__restrict__ part, int blocks, int C,
                                                        float *__restrict__ dw, float *__restrict__ db) {
    __shared__ float sums[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < 2 * C) {
#pragma unroll 4
        for (int i = y; i < blocks; i += 32) s += part[(int64_t)i * 2 * C + c];
    }
    sums[y][x] = s;
    __syncthreads();
    if (y || c >= 2 * C) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) s += sums[i][x];
    float *out = c < C ? dw : db;
    if (out) out[c < C ? c : c - C] = s;
}

// Threads to a row, and packs to a thread; G = 0: a row does not fit.  From 513 packs on the two directions differ: forward
// 4096 x 8192 bf16 takes 26 us with 256 threads and 32 with 512, backward, with four times the registers, 59 and 50.
struct Split {
    int G, NV;
};
Split split_of(int C, bool bf16, bool bwd) {
    const int n = (C + (bf16 ? 8 : 4) - 1) / (bf16 ? 8 : 4);       // packs
    if (n <= 16) return {16, 1};
    if (n <= 32) return {16, 2};
    if (n <= 64) return {64, 1};
    if (n <= 128) return {64, 2};
    if (n <= 256) return {64, 4};
    if (n <= 512) return {256, 2};
    if (n <= 1024) return bwd ? Split{512, 2} : Split{256, 4};
    if (n <= 2048) return bwd && !bf16 ? Split{512, 4} : Split{1024, 2};
    if (n <= 4096 && !bf16) return {1024, 4};
    return {0, 0};
}

template <bool BWD, typename F> hipError_t pick(int C, bool bf16, F f) {
    const Split s = split_of(C, bf16, BWD);
#define F32(g, n) \
    if (s.G == g && s.NV == n && !bf16) return f((float *)0, std::integral_constant<int, g>(), std::integral_constant<int, n>())
#define CASE(g, n) \
    F32(g, n);     \
    if (s.G == g && s.NV == n) return f((uint16_t *)0, std::integral_constant<int, g>(), std::integral_constant<int, n>())
    CASE(16, 1);
    CASE(16, 2);
    CASE(64, 1);
    CASE(64, 2);
    CASE(64, 4);
    CASE(256, 2);
    if constexpr (BWD) {
        CASE(512, 2);
        F32(512, 4);
    } else {
        CASE(256, 4);
        F32(1024, 2);
    }
    if (s.G == 1024 && s.NV == 2) return f((uint16_t *)0, std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
    F32(1024, 4);
    CASE(0, 0);
#undef CASE
#undef F32
    return hipErrorInvalidValue;
}

int blocks_of(int64_t rows, int G, int most) {
    const int64_t per = G ? threads_of(G) / G : 1;
    return (int)std::min<int64_t>((rows + per - 1) / per, most);
}
int blocks_bwd(int64_t rows, int C, bool bf16) {
    const int G = split_of(C, bf16, true).G;
    return blocks_of(rows, G, max_backward(G));
}

}  // namespace

hipError_t launch_norm_fwd(int64_t rows, int C, bool bf16, float eps, const void *x, int64_t ldx, const float *w, const float *b,
                           void *y, int64_t ldy, float *mean, float *rstd, hipStream_t st) {
    if (rows == 0) return hipSuccess;
    return pick<false>(C, bf16, [&](auto *t, auto g, auto n) {
        typedef std::remove_pointer_t<decltype(t)> T;
        constexpr int G = decltype(g)::value, NV = decltype(n)::value, VEC = sizeof(T) == 2 ? 8 : 4;
        const int blocks = blocks_of(rows, G, kMaxForward);
        if constexpr (G)
            (read_once(x, ldx, sizeof(T)) ? norm_fwd_kernel<T, VEC, NV, G, true> : norm_fwd_kernel<T, VEC, NV, G, false>)<<<blocks, threads_of(G), 0, st>>>(
                rows, C, eps, (const T *)x, ldx, w, b, (T *)y, ldy, mean, rstd);
        else
            norm_fwd_wide_kernel<T><<<blocks, kWide, 0, st>>>(rows, C, eps, (const T *)x, ldx, w, b, (T *)y, ldy, mean, rstd);
        return hipGetLastError();
    });
}

int64_t norm_bwd_workspace_floats(int64_t rows, int C, bool bf16) { return 2 * (int64_t)C * blocks_bwd(rows, C, bf16); }

hipError_t launch_norm_bwd(int64_t rows, int C, bool bf16, const void *x, int64_t ldx, const float *w, const float *mean,
                           const float *rstd, const void *dy, int64_t lddy, void *dx, int64_t lddx, float *dw, float *db,
                           float *part, hipStream_t st) {
    const int blocks = blocks_bwd(rows, C, bf16);
    if (!dw && !db) part = nullptr;
    hipError_t e = hipSuccess;
    if (rows > 0)
        e = pick<true>(C, bf16, [&](auto *t, auto g, auto n) {
            typedef std::remove_pointer_t<decltype(t)> T;
            constexpr int G = decltype(g)::value, NV = decltype(n)::value, VEC = sizeof(T) == 2 ? 8 : 4;
            if constexpr (G)
                (read_once(x, ldx, sizeof(T)) && read_once(dy, lddy, sizeof(T)) ? norm_bwd_kernel<T, VEC, NV, G, true>
                                                                          : norm_bwd_kernel<T, VEC, NV, G, false>)<<<blocks, threads_of(G), 0, st>>>(
                rows, C, (const T *)x, ldx, w, mean, rstd, (const T *)dy, lddy, (T *)dx, lddx, part);
            else
                norm_bwd_wide_kernel<T><<<blocks, kWide, 0, st>>>(rows, C, (const T *)x, ldx, w, mean, rstd, (const T *)dy, lddy,
                                                                     (T *)dx, lddx, part);
            return hipGetLastError();
        });
    if (e != hipSuccess || (!dw && !db)) return e;
    norm_sum_kernel<<<(2 * C + 31) / 32, 1024, 0, st>>>(part, blocks, C, dw, db);
    return hipGetLastError();
}

}  // namespace convfwd
